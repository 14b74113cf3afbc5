"""Performance cases of the serving round's operators.

Three operators that a speculative decode round runs beside the draft step and
the verification:

* ``logits``  -- target (or draft) logits to the probability rows that
  verification reads: repetition, frequency and presence penalties over the
  request's tokens, sparse biases, a grammar's bit mask, temperature, softmax;
* ``int4``    -- a few tokens' activations times a weight matrix held in 4 bits
  with one scale (and zero point) per group of weights;
* ``prefix``  -- attention of a batch's new tokens over a prompt prefix that all
  requests share and over each request's own cache.

``run`` computes a case in plain torch operations (fp32) unless ``own`` is set,
in which case it calls the library.  ``exact`` is the same in 64 bits, written
apart from it.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _logits_case(R, L, V, dtype, hist, bias, mask, pen=True, greedy=False, **kw):
    return dict(op="logits", R=R, L=L, V=V, dtype=dtype, hist=hist, bias=bias, mask=mask, pen=pen, greedy=greedy, **kw)


def _int4_case(R, N, K, group, zero, **kw):
    return dict(op="int4", R=R, N=N, K=K, group=group, zero=zero, **kw)


def _prefix_case(R, L, Hq, Hkv, hd, P, T, **kw):
    return dict(op="prefix", R=R, L=L, Hq=Hq, Hkv=Hkv, hd=hd, P=P, T=T, **kw)


def listed():
    return [
        # one request sampling its next token: launch latency counts
        _logits_case(1, 1, 32000, "f32", 64, 0, False, name="logits_one_token"),
        # a ragged vocabulary (rows that start on odd addresses), short histories, some biases
        _logits_case(7, 4, 32003, "f32", 300, 17, True, name="logits_odd_vocab"),
        # one draft step of 32 requests under a grammar, greedy requests among them
        _logits_case(32, 1, 129280, "f32", 1024, 8, True, greedy=True, name="logits_draft_r32"),
        # the verification of 64 requests with four drafts each, bf16 logits of the target's head
        _logits_case(64, 5, 129280, "bf16", 2048, 64, True, name="logits_verify_r64_l5"),
        # one token through a gate or up projection of the mid-sized module
        _int4_case(1, 2816, 1024, 64, False, name="int4_mid_gate_r1"),
        # odd sizes: few tokens, ragged rows and a ragged last group
        _int4_case(5, 1003, 2848, 128, True, name="int4_ragged_r5"),
        # one token through the large module's gate projection, zero points
        _int4_case(1, 18432, 7168, 128, True, name="int4_wide_gate_r1"),
        # the draft batch of 32 requests through the down projection (long reduction)
        _int4_case(32, 7168, 18432, 128, False, name="int4_wide_down_r32"),
        # a handful of chat requests on a short system prompt
        _prefix_case(4, 1, 16, 16, 64, 300, 64, name="prefix_short_prompt"),
        # the draft step's attention at the large module's width on an 8192-token prompt
        _prefix_case(32, 1, 56, 56, 128, 8192, 256, name="prefix_draft_r32"),
        # verification of four drafts (five new tokens) of 32 requests with grouped heads
        _prefix_case(32, 5, 32, 8, 128, 8192, 512, name="prefix_verify_r32_l5"),
        # few requests on a long shared document
        _prefix_case(6, 1, 64, 8, 128, 65000, 100, name="prefix_long_document"),
    ]


def _logu(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(("logits", "int4", "prefix"))
        if op == "logits":
            R, L = _logu(rng, 1, 64), rng.choice((1, 1, 2, 3, 4, 5, 8))
            c = _logits_case(R, L, _logu(rng, 1000, 129280), rng.choice(("f32", "bf16")), _logu(rng, 1, 4096),
                             rng.choice((0, 1, 16, 100)), rng.random() < 0.6, pen=rng.random() < 0.8,
                             greedy=rng.random() < 0.3)
            if R * L * c["V"] <= 64 * 5 * 129280:
                return c
        elif op == "int4":
            group = rng.choice((32, 64, 128))
            c = _int4_case(rng.choice((1, 2, 3, 4, 7, 8, 13, 16, 24, 32)), _logu(rng, 200, 18432),
                           32 * _logu(rng, 8, 576), group, rng.random() < 0.5)
            if c["N"] * c["K"] <= 18432 * 7168:
                return c
        else:
            Hkv = rng.choice((1, 2, 4, 8, 16, 32, 56))
            G = rng.choice((1, 1, 2, 4, 8))
            L = rng.choice((1, 1, 2, 4, 5))
            c = _prefix_case(_logu(rng, 1, 48), L, Hkv * G, Hkv, rng.choice((64, 128)), _logu(rng, 40, 65000),
                             _logu(rng, L, 1024))
            w, top = work(c), work(_prefix_case(32, 5, 32, 8, 128, 8192, 512))
            if c["Hq"] <= 64 and w["flops"] <= top["flops"] and w["bytes"] <= 3 * top["bytes"] and \
                    c["R"] * L * c["Hq"] * (c["P"] + c["T"]) <= 32 * 5 * 32 * 8704:
                return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _ctx_lens(case):
    """Tokens in each request's own cache, its new tokens included: spread over
    [L, T] by a low-discrepancy sequence."""
    L, T = case["L"], case["T"]
    return [L + int((T - L) * ((0.5 + 0.6180339887 * (r + 1)) % 1.0) + 0.5) for r in range(case["R"])]


def _zipf_cdf(V, dev):
    w = torch.arange(1, V + 1, dtype=torch.float64, device=dev).pow(-1.1).cumsum(0)
    return w / w[-1]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 17)

    def normal(shape, std, dtype):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    s = {"case": case}
    R = case["R"]
    if case["op"] == "logits":
        L, V, H = case["L"], case["V"], case["hist"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        rank = torch.log(torch.arange(1, V + 1, device=dev, dtype=torch.float32))
        s["logits"] = (normal((R, L, V), 2.0, torch.float32) - 1.1 * rank).to(dt)
        cdf = _zipf_cdf(V, dev)

        def tokens(shape):
            u = torch.rand(shape, generator=g, device=dev, dtype=torch.float64)
            return torch.searchsorted(cdf, u).clamp(max=V - 1).to(torch.int32)

        def uniform(lo, hi):
            return torch.rand(R, generator=g, device=dev) * (hi - lo) + lo

        s["hist"] = tokens((R, H))
        s["hist_len"] = torch.randint((H + 1) // 2, H + 1, (R,), generator=g, device=dev, dtype=torch.int32)
        s["prompt_len"] = (s["hist_len"] * torch.rand(R, generator=g, device=dev)).to(torch.int32)
        s["draft"] = tokens((R, L - 1)) if L > 1 else None
        s["temperature"] = uniform(0.6, 1.2)
        if case["greedy"]:
            s["temperature"][::3] = 0.0
        s["repetition"] = uniform(1.0, 1.3) if case["pen"] else None
        s["frequency"] = uniform(0.0, 0.5) if case["pen"] else None
        s["presence"] = uniform(-0.2, 0.6) if case["pen"] else None
        nb = case["bias"]
        s["bias_ids"] = s["bias"] = s["mask"] = None
        if nb:
            # distinct ids per request, the last ones unused (-1) in every other request
            step = max(1, V // nb)
            first = torch.randint(0, step, (R, 1), generator=g, device=dev)
            ids = (first + step * torch.arange(nb, device=dev)).to(torch.int32)
            ids[::2, nb - nb // 4:] = -1
            s["bias_ids"] = ids.contiguous()
            s["bias"] = normal((R, nb), 3.0, torch.float32)
        if case["mask"]:
            # a grammar allows few tokens in some states and most in others
            share = torch.rand((R, L, 1), generator=g, device=dev) ** 3
            words = -(-V // 32)
            bits = (torch.rand((R, L, words * 32), generator=g, device=dev) < share.clamp(min=0.001)).view(R, L, words, 32)
            bits[..., 0, 0] = True
            weight = (torch.ones(32, dtype=torch.int64, device=dev) << torch.arange(32, device=dev))
            m = (bits.to(torch.int64) * weight).sum(-1)
            s["mask"] = torch.where(m >= 1 << 31, m - (1 << 32), m).to(torch.int32)
    elif case["op"] == "int4":
        N, K, G = case["N"], case["K"], case["group"]
        s["x"] = normal((R, K), 1.0, torch.bfloat16)
        s["q"] = torch.randint(0, 256, (N, K // 2), generator=g, device=dev, dtype=torch.uint8)
        groups = -(-K // G)
        s["scale"] = ((torch.rand((N, groups), generator=g, device=dev) + 0.5) * 0.003).to(torch.bfloat16)
        s["zero"] = torch.randint(5, 11, (N, groups), generator=g, device=dev, dtype=torch.uint8) if case["zero"] else None
    else:
        L, Hq, Hkv, hd, P, T = (case[k] for k in ("L", "Hq", "Hkv", "hd", "P", "T"))
        s["q"] = normal((R, L, Hq, hd), 1.5, torch.bfloat16)
        s["prefix_k"] = normal((P, Hkv, hd), 1.0, torch.bfloat16)
        s["prefix_v"] = normal((P, Hkv, hd), 1.0, torch.bfloat16)
        s["kv_k"] = normal((R, T, Hkv, hd), 1.0, torch.bfloat16)
        s["kv_v"] = normal((R, T, Hkv, hd), 1.0, torch.bfloat16)
        s["ctx_len"] = torch.tensor(_ctx_lens(case), dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_logits(s):
    x = s["logits"].float()
    R, L, V = x.shape
    dev = x.device
    hist, draft = s["hist"].long(), s["draft"]
    at = torch.arange(hist.shape[1], device=dev)[None]
    valid = at < s["hist_len"][:, None]
    made = (valid & (at >= s["prompt_len"][:, None])).float()
    if s["repetition"] is not None:
        seen = torch.zeros((R, V), device=dev).scatter_add(1, hist, valid.float())
        n = torch.zeros((R, V), device=dev).scatter_add(1, hist, made)[:, None].repeat(1, L, 1)
        if draft is not None:
            before = torch.ones((L, L - 1), device=dev).tril(-1)
            n.scatter_add_(2, draft.long()[:, None].expand(R, L, L - 1), before.expand(R, L, L - 1))
        rep = s["repetition"][:, None, None]
        x = torch.where((seen[:, None] > 0) | (n > 0), torch.where(x > 0, x / rep, x * rep), x)
        x = x - (s["frequency"][:, None, None] * n + s["presence"][:, None, None] * (n > 0))
    if s["bias_ids"] is not None:
        ids = s["bias_ids"].long()
        dense = torch.zeros((R, V + 1), device=dev).scatter(1, torch.where(ids < 0, V, ids), s["bias"])
        x = x + dense[:, None, :V]
    if s["mask"] is not None:
        bits = (s["mask"][..., None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
        x = x.masked_fill(bits.reshape(R, L, -1)[..., :V] == 0, -math.inf)
    m = x.amax(-1, keepdim=True)
    t = s["temperature"][:, None, None]
    e = torch.exp((x - m) / torch.where(t > 0, t, 1.0))
    p = e / e.sum(-1, keepdim=True)
    v = torch.arange(V, device=dev)
    best = torch.where(x == m, v, V).amin(-1, keepdim=True)
    p = torch.where(t > 0, p, (v == best).float())
    return {"p": p, "status": torch.zeros((R, L), dtype=torch.int32, device=dev)}


def _plain_int4(s):
    q, K, G = s["q"], s["case"]["K"], s["case"]["group"]
    codes = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], K).float()
    zero = 8.0 if s["zero"] is None else s["zero"].float().repeat_interleave(G, 1)[:, :K]
    w = (codes - zero) * s["scale"].float().repeat_interleave(G, 1)[:, :K]
    return s["x"].float() @ w.t()


def _plain_prefix(s):
    c = s["case"]
    R, L, Hq, Hkv, hd, P, T = (c[k] for k in ("R", "L", "Hq", "Hkv", "hd", "P", "T"))
    dev = s["q"].device
    q = s["q"].float().view(R, L, Hkv, Hq // Hkv, hd) / math.sqrt(hd)
    sp = torch.einsum("rlhgd,phd->rlhgp", q, s["prefix_k"].float())
    so = torch.einsum("rlhgd,rthd->rlhgt", q, s["kv_k"].float())
    last = s["ctx_len"][:, None] - L + torch.arange(L, device=dev)  # each new token sees itself and what is before it
    see = torch.arange(T, device=dev) <= last[..., None]
    so = so.masked_fill(~see[:, :, None, None], -math.inf)
    m = torch.maximum(sp.amax(-1), so.amax(-1))[..., None]
    sp, so = torch.exp(sp - m), torch.exp(so - m)
    l = sp.sum(-1) + so.sum(-1)
    o = torch.einsum("rlhgp,phd->rlhgd", sp, s["prefix_v"].float()) + \
        torch.einsum("rlhgt,rthd->rlhgd", so, s["kv_v"].float())
    o = o / l[..., None]
    return {"o": o.reshape(R, L, Hq, hd).to(torch.bfloat16), "lse": (m[..., 0] + torch.log(l)).reshape(R, L, Hq)}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"logits": _plain_logits, "int4": _plain_int4, "prefix": _plain_prefix}[op](s)
    from deepseek_sequential_mtp_gb300 import lib
    if op == "logits":
        return lib.logits_probs(s["logits"], temperature=s["temperature"], hist=s["hist"], hist_len=s["hist_len"],
                                prompt_len=s["prompt_len"], draft=s["draft"], repetition=s["repetition"],
                                frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"],
                                bias=s["bias"], mask=s["mask"])
    if op == "int4":
        return lib.gemm_int4w(s["x"], s["q"], s["scale"], s["zero"], group=s["case"]["group"])
    return lib.prefix_attention(s["q"], s["prefix_k"], s["prefix_v"], s["kv_k"], s["kv_v"], s["ctx_len"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    R = case["R"]
    if case["op"] == "logits":
        rows, V = R * case["L"], case["V"]
        size = 4 if case["dtype"] == "f32" else 2
        b = rows * V * (size + 4) + (rows * 4 * -(-V // 32) if case["mask"] else 0)
        b += 4 * R * case["hist"] * (1 if case["pen"] else 0) + 8 * R * case["bias"]
        return {"bytes": b, "flops": 4 * rows * V}
    if case["op"] == "int4":
        N, K = case["N"], case["K"]
        b = N * K // 2 + N * -(-K // case["group"]) * (3 if case["zero"] else 2) + 2 * R * K + 4 * R * N
        return {"bytes": b, "flops": 2 * R * N * K}
    L, Hq, Hkv, hd, P = (case[k] for k in ("L", "Hq", "Hkv", "hd", "P"))
    ctx = _ctx_lens(case)
    b = 4 * hd * Hkv * (P + sum(ctx)) + R * L * Hq * (4 * hd + 4)
    pairs = R * L * P + sum(L * c - L * (L - 1) // 2 for c in ctx)
    return {"bytes": b, "flops": 4 * hd * Hq * pairs}


# ---------------------------------------------------------------------------
# the same in 64 bits
# ---------------------------------------------------------------------------
def _exact_logits(s):
    f = lambda k: None if s[k] is None else s[k].detach().cpu().double().numpy()  # noqa: E731
    i = lambda k: None if s[k] is None else s[k].detach().cpu().numpy()  # noqa: E731
    z_all = f("logits")
    R, L, V = z_all.shape
    hist, hist_len, prompt_len, draft = i("hist"), i("hist_len"), i("prompt_len"), i("draft")
    rep, freq, pres, temp = f("repetition"), f("frequency"), f("presence"), f("temperature")
    ids, bias, mask = i("bias_ids"), f("bias"), i("mask")
    for r in range(R):
        tokens = hist[r, :hist_len[r]]
        for j in range(L):
            z = z_all[r, j]
            made = tokens[prompt_len[r]:] if draft is None else np.concatenate([tokens[prompt_len[r]:], draft[r, :j]])
            if rep is not None:
                u = np.unique(np.concatenate([tokens, made]))
                z[u] = np.where(z[u] > 0, z[u] / rep[r], z[u] * rep[r])
                u, n = np.unique(made, return_counts=True)
                z[u] -= freq[r] * n + pres[r]
            if ids is not None:
                for v, b in zip(ids[r], bias[r]):
                    if v >= 0:
                        z[v] += b
            if mask is not None:
                ok = np.unpackbits(mask[r, j].view(np.uint8), bitorder="little")[:V].astype(bool)
                z[~ok] = -np.inf
            if temp[r] == 0:
                best = int(np.argmax(z))
                z[:] = 0.0
                z[best] = 1.0
            else:
                np.exp((z - z.max()) / temp[r], out=z)
                z /= z.sum()
    return {"p": z_all, "status": None}


def _exact_int4(s):
    x, q, sc, G = s["x"].double(), s["q"], s["scale"].double(), s["case"]["group"]
    R, K = x.shape
    parts = []
    for k0 in range(0, K, G):  # out = sum over groups of scale * (x . codes - zero * sum x)
        xg, qg = x[:, k0:k0 + G], q[:, k0 // 2:(k0 + G) // 2]
        low, high = (qg % 16).double(), torch.div(qg, 16, rounding_mode="floor").double()
        z = 8.0 if s["zero"] is None else s["zero"][:, k0 // G].double()
        dot = xg[:, 0::2] @ low.t() + xg[:, 1::2] @ high.t() - xg.sum(1, keepdim=True) * z
        parts.append(dot * sc[:, k0 // G])
        if len(parts) == 16:
            parts = [sum(parts)]
    return sum(parts).cpu().numpy()


def _exact_prefix(s):
    c = s["case"]
    R, L, Hq, Hkv, hd = (c[k] for k in ("R", "L", "Hq", "Hkv", "hd"))
    G = Hq // Hkv
    q, pk, pv = s["q"].double(), s["prefix_k"].double(), s["prefix_v"].double()
    o = torch.empty((R, L, Hq, hd), dtype=torch.float64, device=q.device)
    lse = torch.empty((R, L, Hq), dtype=torch.float64, device=q.device)
    for r, n in enumerate(_ctx_lens(c)):
        for i in range(L):
            own_rows = n - L + i + 1
            k = torch.cat([pk, s["kv_k"][r, :own_rows].double()]).transpose(0, 1)  # [Hkv, keys, hd]
            v = torch.cat([pv, s["kv_v"][r, :own_rows].double()]).transpose(0, 1)
            z = torch.bmm(q[r, i].view(Hkv, G, hd), k.transpose(1, 2)) * hd ** -0.5
            lse[r, i] = torch.logsumexp(z, -1).reshape(Hq)
            o[r, i] = torch.bmm(torch.softmax(z, -1), v).reshape(Hq, hd)
    return {"o": o.cpu().numpy(), "lse": lse.cpu().numpy()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"logits": _exact_logits, "int4": _exact_int4, "prefix": _exact_prefix}[case["op"]](s)
