"""mtp_logits_probs on the GPU against the fp64 oracle.

Tolerance of an entry (derived, not fitted; u = 2^-24 is half a step of fp32):
the shaped logit z takes at most 4 rounded operations on values up to Z =
max |intermediate|, so z and the maximum are each off by 4 u Z; t = (z - m) / T
adds a rounding each for the difference, 1/T, the product and the factor
log2 e with its own rounding (5 u |t|), twice where the slice's maximum is
moved to the row's; the exponentials are good to 2^-22 (three of them), the
sum over up to 64 values per thread and a tree, the division and the product
to 80 u.  Together p is off by a factor of at most
  u (8 Z / T + 10 |t| + 80 + 12),
beside values below 2^-126 that flush to zero."""
import numpy as np
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib, synth
from oracle import logits as ol
from oracle import verify as ov

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _inputs(R, L, V, dtype, H, nb, masked, seed, scale=3.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal((R, L, V)) * scale).astype(np.float32)).to(dtype)
    a = {"logits": x}
    a["hist"] = torch.from_numpy(rng.integers(-2, max(2, min(V, 60)) + 2, (R, H)).astype(np.int32))
    a["hist_len"] = torch.from_numpy(rng.integers(0, H + 1, R).astype(np.int32))
    a["prompt_len"] = torch.from_numpy(rng.integers(0, H + 1, R).astype(np.int32))
    if L > 1:
        a["draft"] = torch.from_numpy(rng.integers(0, min(V, 20), (R, L - 1)).astype(np.int32))
    for k, lo, hi in (("temperature", 0.4, 1.5), ("repetition", 0.8, 1.6), ("frequency", -0.3, 0.6),
                      ("presence", -0.5, 0.8)):
        a[k] = torch.from_numpy(rng.uniform(lo, hi, R).astype(np.float32))
    if nb:
        a["bias_ids"] = torch.from_numpy(rng.integers(-2, V + 2, (R, nb)).astype(np.int32))
        a["bias"] = torch.from_numpy(rng.standard_normal((R, nb)).astype(np.float32) * 2)
    if masked:
        a["mask"] = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (R, L, -(-V // 32))).astype(np.int32))
    return a


def _oracle(a):
    x = a["logits"].double().numpy()
    R, L, V = x.shape
    g = lambda k, r, d: d if a.get(k) is None else float(a[k][r])  # noqa: E731
    p, st = np.zeros((R, L, V)), np.zeros((R, L), dtype=np.int32)
    for r in range(R):
        h = a["hist"][r, :int(a["hist_len"][r])].tolist() if a.get("hist") is not None else []
        n = int(a["prompt_len"][r]) if a.get("prompt_len") is not None else 0
        biases = list(zip(a["bias_ids"][r].tolist(), a["bias"][r].tolist())) if a.get("bias_ids") is not None else ()
        for j in range(L):
            made = h[n:] + (a["draft"][r, :j].tolist() if a.get("draft") is not None else [])
            allowed = ol.unpack_mask(a["mask"][r, j].numpy(), V) if a.get("mask") is not None else None
            p[r, j], st[r, j] = ol.row(x[r, j], h[:n], made, g("repetition", r, 1.0), g("frequency", r, 0.0),
                                       g("presence", r, 0.0), biases, allowed, g("temperature", r, 1.0))
    return p, st


def _run(a, **kw):
    got = lib.logits_probs(**{k: (v.cuda() if torch.is_tensor(v) else v) for k, v in a.items()}, **kw)
    torch.cuda.synchronize()
    return got["p"].cpu().double().numpy(), got["status"].cpu().numpy()


def _check(a, got):
    p, st = got
    rp, rst = _oracle(a)
    np.testing.assert_array_equal(st, rst)
    x = a["logits"].double().numpy()
    Z = np.abs(np.where(np.isfinite(x), x, 0)).max() * 1.7 + 12.0  # repetition <= 1.6, penalties and biases < 12
    T = a["temperature"].double().numpy()[:, None, None] if a.get("temperature") is not None else np.ones((1, 1, 1))
    T = np.where(T > 0, T, 1.0)
    with np.errstate(divide="ignore"):
        t = -np.log(np.maximum(rp, 1e-300))  # |t| <= -log p since the sum is at least 1
    np.testing.assert_array_less(np.abs(p - rp), U * (8 * Z / T + 10 * t + 92) * rp + 1.2e-38 + 1e-300)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,L,V,H,nb,masked", [
    (1, 1, 1, 1, 0, False), (3, 2, 31, 7, 3, True), (2, 1, 64, 0, 1, True), (2, 3, 2049, 40, 5, True),
    (5, 2, 3000, 100, 40, True), (4, 1, 4096, 700, 0, False), (1, 5, 16385, 64, 100, True), (70, 1, 2500, 9, 2, False),
    (2, 2, 33001, 300, 4, True), (160, 1, 16400, 30, 0, True)])
def test_rows(dtype, R, L, V, H, nb, masked):
    """Every cluster size and vector count for few and many rows, aligned and
    ragged vocabularies, ids outside the vocabulary, repeated biases."""
    a = _inputs(R, L, V, dtype, H, nb, masked, R + 10 * L + V)
    _check(a, _run(a))


@pytest.mark.parametrize("V", [129280, 262145, 524288])
def test_large_vocabularies(V):
    a = _inputs(2, 2, V, torch.float32, 50, 3, True, V)
    for k in ("hist", "draft"):
        a[k] = (a[k].long() * (V // 70)).clamp(-1, V - 1).to(torch.int32)
    p, st = _run(a)
    assert (st == 0).all()
    _check({**{k: v[:1] for k, v in a.items()}}, (p[:1], st[:1]))


def test_defaults_are_a_softmax_and_rows_a_distance_apart():
    V = 1003
    wide = torch.randn(3, 2, 1100, generator=torch.Generator().manual_seed(0)) * 4
    a = {"logits": wide[..., :V]}
    got = lib.logits_probs(wide.cuda()[..., :V])
    _check(a, (got["p"].cpu().double().numpy(), got["status"].cpu().numpy()))


def test_in_place_and_given_outputs():
    a = _inputs(6, 2, 5000, torch.float32, 20, 2, True, 4)
    dev = {k: v.cuda() for k, v in a.items()}
    want = lib.logits_probs(**dev)
    out = {"p": dev["logits"], "status": torch.empty(6, 2, dtype=torch.int32, device="cuda")}
    got = lib.logits_probs(**dev, out=out)
    assert got["p"].data_ptr() == dev["logits"].data_ptr()
    assert torch.equal(got["p"], want["p"]) and torch.equal(got["status"], want["status"])


def test_greedy_takes_the_lowest_of_equal_maxima():
    """Maxima in other slices of the row's cluster, and rows masked down to one token."""
    V = 40000
    x = torch.zeros(3, 1, V)
    x[0, 0, [39999, 25000, 25001]] = 5.0
    x[1, 0, 7] = -1.0
    mask = torch.full((3, 1, V // 32), -1, dtype=torch.int32)
    mask[2] = 0
    mask[2, 0, 1234] = 1 << 5
    a = {"logits": x, "temperature": torch.zeros(3), "mask": mask}
    p, st = _run(a)
    assert (st == 0).all() and p.sum() == 3
    assert p[0, 0, 25000] == 1 and p[1, 0, 0] == 1 and p[2, 0, 1234 * 32 + 5] == 1


def test_rows_without_an_answer():
    """Nothing allowed, only -inf allowed, NaN or +inf allowed or masked, bad
    parameters, the type's lowest value, overflow of a penalised logit."""
    V, low = 5000, torch.finfo(torch.float32).min
    x = torch.randn(10, 1, V, generator=torch.Generator().manual_seed(1))
    mask = torch.full((10, 1, 157), -1, dtype=torch.int32)
    mask[0] = 0                       # nothing allowed
    x[1] = -np.inf                    # only -inf
    x[2, 0, 4999] = np.nan            # allowed NaN, in the last slice
    x[3, 0, 0] = np.inf               # allowed +inf
    x[4, 0, 64:96] = np.nan           # masked NaN
    x[4, 0, 96:128] = np.inf
    mask[4, 0, 2:4] = 0
    x[5] = low                        # all at the lowest value: uniform
    x[6, 0, 1:] = low                 # the lowest value beside a real one
    x[9] = low
    rep = torch.ones(10)
    rep[9] = 4.0                      # lowest * 4 = -inf, for every token (hist holds them all)
    temp = torch.ones(10)
    temp[7] = -1.0
    temp[8] = float("nan")
    hist = torch.arange(V, dtype=torch.int32).repeat(10, 1)
    hl = torch.zeros(10, dtype=torch.int32)
    hl[9] = V
    a = {"logits": x, "mask": mask, "repetition": rep, "temperature": temp, "hist": hist, "hist_len": hl,
         "prompt_len": torch.zeros(10, dtype=torch.int32)}
    p, st = _run(a)
    assert st[:, 0].tolist() == [1, 1, 2, 2, 0, 0, 0, 3, 3, 1]
    assert (p[st[:, 0] != 0] == 0).all()
    np.testing.assert_allclose(p[5], 1 / V, rtol=92 * U)
    assert p[6, 0, 0] == 1 and (p[4, 0, 64:128] == 0).all()
    keep = {k: v[4:5] for k, v in a.items()}
    _check(keep, (p[4:5], st[4:5]))


def test_same_bits_every_time_and_from_a_graph():
    """Counts and biases are collected by atomics; the result does not depend on
    their order.  A captured call replayed on new inputs equals a direct one."""
    a = {k: v.cuda() for k, v in _inputs(9, 3, 30000, torch.bfloat16, 2000, 300, True, 8).items()}
    a["hist"] %= 40
    b = {k: v.cuda() for k, v in _inputs(9, 3, 30000, torch.bfloat16, 2000, 300, True, 9).items()}
    want = lib.logits_probs(**a)["p"]
    for _ in range(20):
        assert torch.equal(lib.logits_probs(**a)["p"], want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lib.logits_probs(**a, stream=side)
    side.synchronize()
    assert torch.equal(got["p"], want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = lib.logits_probs(**a)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["p"], want)
    want_b = lib.logits_probs(**b)["p"]
    for k in a:
        a[k].copy_(b[k])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["p"], want_b)


def test_rows_feed_verification():
    """Target logits under a grammar -> p -> spec_verify: accepted drafts and the
    drawn token follow the verify oracle on the kernel's own rows, and no
    emitted token is one that the grammar forbids."""
    R, gamma, V = 24, 3, 4000
    c = synth.make_verify_inputs(synth.VerifyConfig(name="v", R=R, gamma=gamma, V=V), 5)
    a = _inputs(R, gamma + 1, V, torch.float32, 60, 4, False, 6)
    a["logits"] = torch.log(c["p"]).clamp(min=-80)
    a["draft"] = c["draft"]
    words = np.random.default_rng(3).integers(-2 ** 31, 2 ** 31, (R, gamma + 1, V // 32)).astype(np.int32)
    a["mask"] = torch.from_numpy(words | (words >> 1))
    dev = {k: v.cuda() for k, v in a.items()}
    rows = lib.logits_probs(**dev)
    out = lib.spec_verify(rows["p"], c["q"].cuda(), dev["draft"], 77, 1)
    lib.check_errors()
    ref = ov.spec_verify(rows["p"].cpu().numpy(), c["q"].numpy(), c["draft"].numpy(), 77, 1)
    keep = ref["margin"] > 1e-6
    for k, kr in (("accepted", "accepted"), ("next_token", "token"), ("n_emit", "n_emit"), ("status", "status")):
        np.testing.assert_array_equal(out[k].cpu().numpy()[keep], ref[kr][keep])
    acc, nxt = out["accepted"].cpu().numpy(), out["next_token"].cpu().numpy()
    assert (out["status"].cpu().numpy() == 0).all()
    for r in range(R):
        for j, v in enumerate(c["draft"][r, :acc[r]].tolist() + [int(nxt[r])]):
            assert (int(a["mask"][r, j, v >> 5]) >> (v & 31)) & 1


def test_refusals():
    x = torch.zeros(2, 2, 100, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    for kw in (dict(temperature=f(3)), dict(hist=i(2, 5), hist_len=i(3)), dict(hist_len=i(2)), dict(draft=i(2, 2)),
               dict(bias_ids=i(2, 3)), dict(bias_ids=i(2, 3), bias=f(2, 4)), dict(mask=i(2, 2, 3)),
               dict(temperature=f(2).double()), dict(temperature=torch.ones(2)),
               dict(hist=i(2, 10)[:, ::2]), dict(bias_ids=i(2, 4096), bias=f(2, 4096))):
        with pytest.raises(lib.MtpError):
            lib.logits_probs(x, **kw)
    for bad in (x[0], x.half(), x.transpose(1, 2), x.cpu(), torch.zeros(1, 1, 524289, device="cuda"),
                torch.zeros(3, 2, 100, device="cuda")[:, :, ::2]):
        with pytest.raises(lib.MtpError):
            lib.logits_probs(bad)
    assert lib.logits_probs(torch.zeros(0, 1, 5, device="cuda"))["p"].shape == (0, 1, 5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,L,V", [(130, 4, 5000), (125, 5, 4099), (4, 128, 9000)])
def test_more_rows_than_the_few_row_form_takes(dtype, R, L, V):
    """More CTAs than three per SM: whole batches and a last one, 16-byte rows and
    odd ones, greedy rows and rows in place among them."""
    a = _inputs(R, L, V, dtype, 90, 7, True, R + V)
    a["temperature"][::9] = 0.0
    _check(a, _run(a))
    if dtype == torch.float32:
        d = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in a.items()}
        want = lib.logits_probs(**d)
        out = {"p": d["logits"], "status": torch.empty((R, L), dtype=torch.int32, device="cuda")}
        got = lib.logits_probs(**d, out=out)
        assert torch.equal(got["p"], want["p"]) and torch.equal(got["status"], want["status"])
