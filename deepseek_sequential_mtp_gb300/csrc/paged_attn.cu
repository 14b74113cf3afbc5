// Attention of a batch's new tokens over a paged key/value cache of bf16, or of
// e4m3 codes with a power of two per 16 rows and head.
//
// o = softmax(scale q K^T) V for every (request, token, head) in parts of
// (reference m, sum l, output o) each, joined at the end:
// o = sum 2^(m_p - M) o_p / sum 2^(m_p - M) l_p.
//
// With s_j the score (in powers of two) of key j and 2^(E_j) the scale of its value's
// block, the weight that meets the code of the value is w_j = 2^(s_j + E_j - m), m the running maximum of
// s_j + E_j: the scales cost an addition, and the products take the codes as they are.  The sum
// takes w_j 2^(-E_j).
//
// Short tables and few items: a CTA per item, one launch (paged_item_kernel: loads that wait for one another).  Else three kernels, by
// what bounds each: 8 bits on tcgen05 (paged_cols_kernel: HBM, 32 requests of 56 heads and 6500 keys
// on average 441 us, 6.3 TB/s of codes; with 20 rows per key head the softmax of a block, 120 us where the bytes take
// 60), bf16 on mma.sync from a ring of 16 keys per warp (paged_rows_kernel: launch and first loads for
// small caches, HBM for large ones), many rows as gathered bf16 rows through the attention over own caches
// (below), whose products are the bound.
#include <cuda.h>

#include <algorithm>

#include "attn_steps.cuh"
#include "gemm_tc.cuh"
#include "mbarrier.cuh"
#include "paged.cuh"
#include "prefix_attn.cuh"
#include "tcgen05.cuh"

MTP_DEFINE_ERROR_WORD(mtp_take_errors_paged_attn)

namespace mtp {
namespace {

constexpr int kTileRows = 16;  // rows of a warp (M of mma.m16n8k16)

// x 2^(2 e), f = 2^e: references of blocks whose scales are far apart differ by more than a float's exponent holds
__device__ __forceinline__ float scale_twice(float x, float f) { return x * f * f; }

// What a launch works on.  An item is a (request, key head, tile of rows); a step
// is `keys` keys of an item.  The steps of all items are dealt to the workers (groups of warps, or
// CTAs) in equal contiguous ranges; a worker's range within an item (a segment) leaves `parts`
// records for each row.
struct Shape {
  int R, L, H, Hkv, G, rows, tiles, tile_rows, rec_rows, causal;  // rows: L G of a (request, key head)
  int keys, parts;  // keys of a step, records of a segment
  int cap, per_page, n_pages, table_len, workers, least;
  const int32_t *ctx_len, *n_new, *table;
  const uint8_t *ks, *vs;
  const __nv_bfloat16* q;
  long long q_r, q_l, q_h;

  __device__ __forceinline__ int ctx(int r) const { return min(max(ctx_len[r], 0), cap); }
  __device__ __forceinline__ int fresh(int r) const { return n_new ? min(max(n_new[r], 0), L) : L; }
  __device__ __forceinline__ int steps(int r) const { return fresh(r) > 0 ? (ctx(r) + keys - 1) / keys : 0; }
  __device__ __forceinline__ int items() const { return Hkv * tiles; }
  // rows j < sees(i, ..) are seen by token i
  __device__ __forceinline__ int sees(int i, int ctx, int fresh) const {
    return i >= fresh ? 0 : max(causal ? ctx - (fresh - 1 - i) : ctx, 0);
  }
};

// The same value in every lane, known as such to the compiler: branches on it keep a warp together (a shuffle within a branch
// that may part the warp took 230 cycles instead of 36).
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ long long uniform(long long v) { return __shfl_sync(0xffffffffu, v, 0); }

// steps of requests before r (all of them for r = R), by a whole warp
__device__ __forceinline__ long long steps_before(const Shape& sh, int r, int lane) {
  long long sum = 0;
  for (int i = lane; i < r; i += 32) sum += sh.steps(i);
  return uniform(warp_total(sum)) * sh.items();
}
// worker k of n takes steps [k total / n, (k + 1) total / n), at least `least` of them where there are so many
struct Deal {
  long long total;
  int n;
  __device__ __forceinline__ Deal(long long total_, int least, int workers) : total(total_) {
    const long long most = quotient(total + least - 1, least);
    n = static_cast<int>(min(most, static_cast<long long>(workers)));
  }
  __device__ __forceinline__ long long start(int k) const { return k * total / n; }
  __device__ __forceinline__ int owner(long long pos) const { return static_cast<int>(quotient((pos + 1) * n - 1, total)); }
};

// a place in the order of steps, the same in every lane
struct Cursor {
  int r, item, step, steps, ctx, fresh;
  long long left;  // of the worker's range
  __device__ __forceinline__ void request(const Shape& sh) {
    ctx = uniform(sh.ctx(r));
    fresh = uniform(sh.fresh(r));
    steps = fresh > 0 ? (ctx + sh.keys - 1) / sh.keys : 0;
  }
  __device__ __forceinline__ void begin(const Shape& sh, long long from, long long to, int lane) {
    left = to - from;
    long long start = 0;
    r = 0;
    for (int base = 0; base < sh.R; base += 32) {
      const long long c = base + lane < sh.R ? static_cast<long long>(sh.steps(base + lane)) * sh.items() : 0;
      long long incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const unsigned over = __ballot_sync(0xffffffffu, start + incl > from);
      if (over) {
        const int src = __ffs(over) - 1;
        r = base + src;
        start += __shfl_sync(0xffffffffu, incl - c, src);
        break;
      }
      start += __shfl_sync(0xffffffffu, incl, 31);
    }
    r = uniform(r);
    request(sh);
    const long long in = from - uniform(start);
    item = static_cast<int>(quotient(in, steps));
    step = static_cast<int>(in - static_cast<long long>(item) * steps);
  }
  __device__ __forceinline__ void next(const Shape& sh) {
    --left;
    if (++step < steps || left == 0) return;
    step = 0;
    if (++item < sh.items()) return;
    item = 0;
    do {
      ++r;
      request(sh);
    } while (steps == 0);  // left > 0: there is another
  }
};

struct PagedMaps {
  CUtensorMap k, v;
};

// ---------------------------------------------------------------------------
// bf16: rows along mma.sync's M
// ---------------------------------------------------------------------------
// kGroup warps with 16 rows each share a ring of steps of 16 keys.
template <int HD, int kGroup>
struct Cfg {
  static constexpr int kWarps = 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPieces = HD / 64;               // of 128 bytes per row
  static constexpr int kTileBytes = 16 * HD * 2;        // keys, or values
  static constexpr int kBoxBytes = 16 * 128;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = kGroup * 24 * 1024 / kStageBytes;
  static constexpr int kRings = kWarps / kGroup;
  static constexpr int kLag = kGroup > 1 ? 1 : 0;       // steps after which a stage is filled again
  static constexpr int kOffBar = kRings * kStages * kStageBytes;  // full and empty per stage
  static constexpr int kOffMeta = kOffBar + 16 * kRings * kStages;
  static constexpr int kSmemBytes = kOffMeta + 4 * kRings * kStages + 16;
};

// address of 16-byte chunk c of row `row` of a tile that TMA wrote with the 128-byte swizzle
__device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int row, int c) {
  return tile + (c >> 3) * (16 * 128) + row * 128 + (((c ^ row) & 7) << 4);
}

// 16 rows of a warp: queries, and a part (reference, sum, output) of their own.
template <int HD>
struct Rows {
  uint32_t q[HD / 16][4];
  float mx[2], sum[2], o[HD / 8][4];
  int see[2];
  bool flag;
};

template <int HD>
__device__ __forceinline__ void load_rows(Rows<HD>& w, const Shape& sh, int r, int head, int row0, int ctx, int fresh, int lane) {
  const int g = lane >> 2, t = lane & 3;
  w.flag = false;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = row0 + 8 * e + g, i = row / sh.G;
    const bool is = row < sh.rows;
    w.see[e] = is ? sh.sees(i, ctx, fresh) : 0;
    w.mx[e] = -INFINITY;
    w.sum[e] = 0.f;
    const __nv_bfloat16* q = sh.q + r * sh.q_r + i * sh.q_l + (head * sh.G + row - i * sh.G) * sh.q_h;
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
      w.q[k][e] = is ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * t) : 0;
      w.q[k][2 + e] = is ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8 + 2 * t) : 0;
    }
  }
#pragma unroll
  for (int n = 0; n < HD / 8; ++n) w.o[n][0] = w.o[n][1] = w.o[n][2] = w.o[n][3] = 0.f;
}

// 16 keys from key0 on, `left` of them up to the end of the request's rows (0: a bad page).
// kEdge: some row does not see all of them.
template <int HD, bool kEdge>
__device__ __forceinline__ void step_rows(Rows<HD>& w, uint32_t k_at, uint32_t v_at, int key0, int left, float scale_log2, int lane) {
  const int t = lane & 3;
  float sc[2][4] = {};
#pragma unroll
  for (int k = 0; k < HD / 16; ++k) {
    uint32_t f[4];
    ldsm_x4(chunk_at(k_at, (lane & 7) + 8 * (lane >> 4), 2 * k + ((lane >> 3) & 1)), f);
    mma_16816(sc[0], w.q[k], f[0], f[1]);
    mma_16816(sc[1], w.q[k], f[2], f[3]);
  }
  uint32_t pa[2][4];
  float alpha[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float v[2][2], top = -INFINITY;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[n][i] = sc[n][2 * e + i] * scale_log2;
        if (kEdge && (key0 + 8 * n + 2 * t + i >= w.see[e] || left <= 0)) v[n][i] = -INFINITY;
        top = fmaxf(top, v[n][i]);
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float now = top > w.mx[e] + kStaleMaxLog2 ? top : w.mx[e];
    const float neg = now == -INFINITY ? 0.f : -now;
    alpha[e] = now == w.mx[e] ? 1.f : ex2(w.mx[e] + neg);
    w.mx[e] = now;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      v[n][0] = ex2(v[n][0] + neg), v[n][1] = ex2(v[n][1] + neg);
      pa[0][e + 2 * n] = pack2_bf16(v[n][0], v[n][1]);
      const float2 f = unpack2_bf16(pa[0][e + 2 * n]);
      pa[1][e + 2 * n] = pack2_bf16(v[n][0] - f.x, v[n][1] - f.y);
    }
    w.sum[e] = fmaf(w.sum[e], alpha[e], (v[0][0] + v[0][1]) + (v[1][0] + v[1][1]));
  }
  if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
    for (int n = 0; n < HD / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) w.o[n][i] *= alpha[i >> 1];
  }
#pragma unroll
  for (int c2 = 0; c2 < HD / 16; ++c2) {
    uint32_t f[4];
    ldsm_x4_t(chunk_at(v_at, lane & 15, 2 * c2 + (lane >> 4)), f);
    if constexpr (kEdge) {
      // values past the end and of bad pages are not looked at, and what is not finite is taken out for rows that do not
      // see it (the join puts it back for those that do)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 8 * (i & 1) + 2 * t;
        uint32_t x = f[i] & ((key < left ? 0xffffu : 0u) | (key + 1 < left ? 0xffff0000u : 0u));
        const uint32_t odd = ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        w.flag |= odd != 0;
        f[i] = x & ~((odd >> 15) * 0xffffu);
      }
    }
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
      mma_16816(w.o[2 * c2 + ch], pa[0], f[2 * ch], f[2 * ch + 1]);
      mma_16816(w.o[2 * c2 + ch], pa[1], f[2 * ch], f[2 * ch + 1]);
    }
  }
}

template <int HD>
__device__ __forceinline__ void store_rows(Rows<HD>& w, const Shape& sh, long long rec, int row0, float2* rec_ml, float* rec_o, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const bool any = __any_sync(0xffffffffu, w.flag);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    w.sum[e] += __shfl_xor_sync(0xffffffffu, w.sum[e], 1);
    w.sum[e] += __shfl_xor_sync(0xffffffffu, w.sum[e], 2);
    const int row = 8 * e + g;
    if (row0 + row >= sh.rows) continue;
    const float l = w.see[e] > 0 ? w.sum[e] : 0.f;
    if (t == 0) rec_ml[rec + row] = make_float2(l == 0.f ? -INFINITY : w.mx[e], any ? -l : l);
    if (l == 0.f) continue;  // a part without a key is not read
    float* to = rec_o + (rec + row) * HD;
#pragma unroll
    for (int n = 0; n < HD / 8; ++n) *reinterpret_cast<float2*>(to + 8 * n + 2 * t) = make_float2(w.o[n][2 * e], w.o[n][2 * e + 1]);
  }
}

// A group of kGroup warps has 16 rows each and a ring, which its first warp fills with TMA boxes
// of 16 keys; the warps wait for nothing but the copies, and the first for the others when it fills a
// stage again.
template <int HD, int kGroup>
__global__ void __launch_bounds__(Cfg<HD, kGroup>::kThreads, 1)
paged_rows_kernel(const __grid_constant__ PagedMaps maps, const Shape sh, float scale_log2, float2* __restrict__ rec_ml,
                  float* __restrict__ rec_o) {
  using C = Cfg<HD, kGroup>;
  pdl_trigger();  // the joining kernel may start its setup
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t s0 = smem_u32(smem);
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31, ring_id = warp / kGroup, in_group = warp % kGroup;
  if (s0 & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(&g_mtp_error_word, MTP_DEVERR_TIMEOUT);
    return;
  }
  const uint32_t ring = s0 + ring_id * C::kStages * C::kStageBytes, full = s0 + C::kOffBar + 16 * ring_id * C::kStages;
  const uint32_t empty = full + 8 * C::kStages;
  int* bad_page = reinterpret_cast<int*>(smem + C::kOffMeta) + ring_id * C::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMeta + 4 * C::kRings * C::kStages);
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 2 * C::kRings * C::kStages; ++i) mbar_init(s0 + C::kOffBar + 8 * i, i / C::kStages % 2 ? kGroup : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  const Deal deal(steps_before(sh, sh.R, lane), sh.least, sh.workers);
  const int worker = ring_id * gridDim.x + blockIdx.x;
  if (worker >= deal.n) return;
  auto wwait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_phase(bar, parity, abort_flag, &g_mtp_error_word));
  };
  const long long from = deal.start(worker), to = deal.start(worker + 1);
  Cursor in;  // what is asked for
  in.begin(sh, from, to, lane);
  Cursor at = in;  // what is worked on

  int have_r = -1, have_base = -1, page = -1;  // pages of 32 blocks of 16 keys, one per lane
  uint32_t asked = 0;
  auto ask = [&]() {
    if (kGroup > 1 && asked >= C::kStages && !wwait(empty + 8 * (asked % C::kStages), (asked / C::kStages - 1) & 1)) return false;
    const int base = in.step & ~31;
    if (in.r != have_r || base != have_base) {
      const int b = base + lane;
      page = -1;
      if (16ll * b < in.ctx) {
        page = sh.table[static_cast<long long>(in.r) * sh.table_len + b / sh.per_page];
        if (page < 0 || page >= sh.n_pages) {
          atomicOr(&g_mtp_error_word, MTP_DEVERR_PAGE_RANGE);
          page = -1;
        }
      }
      have_r = in.r, have_base = base;
    }
    const int id = __shfl_sync(0xffffffffu, page, in.step & 31);
    const uint32_t slot = asked % C::kStages, bar = full + 8 * slot, to_k = ring + slot * C::kStageBytes;
    if (lane == 0) {
      bad_page[slot] = id < 0;
      mbar_expect_tx(bar, id < 0 ? 0 : C::kStageBytes);
    }
    __syncwarp();
    if (id >= 0 && lane < 2 * C::kPieces) {
      const int piece = lane % C::kPieces, v = lane / C::kPieces;
      tma_tile_4d(to_k + v * C::kTileBytes + piece * C::kBoxBytes, v ? &maps.v : &maps.k, 0, piece, in.step % sh.per_page * 16,
                  id * sh.Hkv + in.item / sh.tiles, bar);
    }
    ++asked;
    in.next(sh);
    return true;
  };
  bool ok = true;
  if (in_group == 0)
    while (ok && asked < C::kStages && in.left > 0) ok = ask();

  Rows<HD> w;
  bool begins = true;
  for (uint32_t done = 0; ok && at.left > 0;) {
    const int head = at.item / sh.tiles, row0 = ((at.item - head * sh.tiles) * kGroup + in_group) * kTileRows;
    if (begins) load_rows<HD>(w, sh, at.r, head, row0, at.ctx, at.fresh, lane);
    begins = false;
    const uint32_t slot = done % C::kStages, k_at = ring + slot * C::kStageBytes, v_at = k_at + C::kTileBytes;
    if (!wwait(full + 8 * slot, (done / C::kStages) & 1)) break;
    const bool bad = bad_page[slot];
    const int key0 = at.step * 16;
    if (row0 < sh.rows) {
      if (key0 + 16 > at.ctx - (sh.causal ? at.fresh - 1 : 0) || bad)
        step_rows<HD, true>(w, k_at, v_at, key0, bad ? 0 : at.ctx - key0, scale_log2, lane);
      else
        step_rows<HD, false>(w, k_at, v_at, key0, at.ctx - key0, scale_log2, lane);
    }
    __syncwarp();
    if (kGroup > 1 && lane == 0) mbar_arrive1(empty + 8 * slot);
    ++done;
    if (in_group == 0 && in.left > 0 && done > C::kLag) ok = ask();
    if (at.step + 1 == at.steps || at.left == 1) {
      const long long rec = (static_cast<long long>(at.r) * sh.items() + at.item + worker) * sh.rec_rows + in_group * kTileRows;
      store_rows<HD>(w, sh, rec, row0, rec_ml, rec_o, lane);
      begins = true;
    }
    at.next(sh);
  }
  // no copy may still be landing when the warp leaves (matters only after an abort)
  if (in_group == 0)
    for (uint32_t x = asked > C::kStages ? asked - C::kStages : 0; x < asked; ++x)
      wait_drain(full + 8 * (x % C::kStages), (x / C::kStages) & 1, kWaitLimitCycles);
}

// ---------------------------------------------------------------------------
// 8 bits: keys along TMEM's lanes
// ---------------------------------------------------------------------------
// The products are taken as S^T = K Q^T (128 keys by the rows) and O^T = V^T P^T (hd by the rows), so that the
// cache's codes are the operands with M = 128, as TMA brings them, and the few rows are N.
// kind::f8f6f4 takes codes on both sides: a query row is 2^up (hi + lo), two products
// into one sum; a weight w <= 448 is a + 2^-4 b + 2^-9 c in columns and accumulators of their own (fp16's
// precision, and off by 2^-26 of the largest weight at the most).  A thread has a key, whose
// block's scales are numbers of its own, and goes over the rows.
//   two or three groups of four warps: softmax of every second or third block, each with a reference, a sum and an
//                 output of its own (parts)
//   load warp     loads keys and values
//   product warp  issues every product: scores as many blocks ahead of the outputs as there are groups
//   query warp    turns a segment's queries into codes, a segment ahead
//   page warp     walks ahead and looks up the blocks' pages and exponents
constexpr int kCols = 128;                 // keys of a block
// A weight is 2^7 at the reference and at most 448; the codes' least step is 2^-18.  Weights below half of it leave the outputs, not
// the sums: n keys share less than n 2^-26 of the largest that way.  (2^4 and 4.8 bits of slack: references are raised more seldom, 117
// us instead of 120 for 5 tokens of 64 requests and 438 instead of 441 for one of 32, but weights end at 2^-23: 11000 keys at 2^-23.7
// of the largest had no share in the outputs.)
constexpr float kTopLog2 = 7.0f;
constexpr float kSlackLog2 = 1.8f;
// kMax: rows that a tile may have; the launch's, a multiple of 8, are a number of its own (loops over them are
// not unrolled: unrolled ones were bound by the fetching of instructions, 1130 us instead of 895 for 1024 tokens of two prompts).
template <int HD, int kMax>
struct Wide {
  static constexpr int kW = kMax <= 24 ? 3 : 2;  // groups of softmax warps (of many rows TMEM holds no more than two's outputs)
  static constexpr int kLoadWarp = 4 * kW, kMmaWarp = kLoadWarp + 1, kQWarp = kLoadWarp + 2, kMetaWarp = kLoadWarp + 3;
  static constexpr int kThreads = 32 * (4 * kW + 4);
  static constexpr int kTileBytes = kCols * HD;
  static constexpr int kKStages = HD == 64 ? 8 : kMax <= 24 ? 5 : 4, kVStages = HD == 64 ? 8 : kMax <= 16 ? 7 : 6;
  static constexpr int kSCols = (kMax + 15) / 16 * 16, kOCols = (3 * kMax + 15) / 16 * 16;  // of a group
  static constexpr int kPBytes = kOCols * kCols;
  static constexpr int kQBytes = 2 * kMax * HD;
  static constexpr int kRing = 16;                 // blocks that are looked up ahead
  static constexpr int kOffV = kKStages * kTileBytes;
  static constexpr int kOffP = kOffV + kVStages * kTileBytes;
  static constexpr int kOffQ = kOffP + kW * kPBytes;
  static constexpr int kOffRow = kOffQ + 2 * kQBytes;           // per queries' buffer: scale, keys seen of each row
  static constexpr int kOffMax = kOffRow + 2 * kMax * 8;        // per group: see below
  static constexpr int kGroupBytes = kMax * 4 * 5 + 128 * 8 + 32;
  static constexpr int kOffMeta = kOffMax + kW * kGroupBytes;          // per block of the ring: exponents, pages of 8 blocks of 16 keys
  static constexpr int kOffBar = kOffMeta + kRing * 48;
  // k, v full, empty per stage; meta full, empty; q full, empty; s full, s free, p full, pv done per group; drain
  static constexpr int kNumBars = 2 * (kKStages + kVStages + kRing) + 4 + 4 * kW + 1;
  static constexpr int kSmemBytes = kOffBar + 8 * kNumBars + 16;
  // TMEM: scores of the groups, outputs, sums
  static constexpr uint32_t kColO = kW * kSCols, kColL = kColO + kW * kOCols, kUsed = kColL + kW * kMax;
  static constexpr uint32_t kTmemCols = kUsed <= 256 ? 256 : 512;
  static_assert(kUsed <= 512 && kSmemBytes <= 232448, "what an SM has");
};

// shared-memory descriptor: version 1; layout 2 and 4 are the 128- and the 64-byte swizzle, 0 none
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(layout) << 61);
}
// kind::f8f6f4, e4m3 by e4m3 to fp32; MN-major flags of A and B
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}
// called by a converged warp; one lane, always the same, issues
__device__ __forceinline__ void umma_e4m3_warp(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_tile_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
#define MTP_R8(r) "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
// 8 columns of this thread's lane from one place or three, and to one
__device__ __forceinline__ void tmem_ld8(uint32_t a, float (&x)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : MTP_R8(r)
      : "r"(a)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld8x3(uint32_t a, uint32_t b, uint32_t c, float (&x)[8], float (&y)[8], float (&z)[8]) {
  uint32_t r[8], s[8], t[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%24];\n"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%25];\n"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%26];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : MTP_R8(r), MTP_R8(s), MTP_R8(t)
      : "r"(a), "r"(b), "r"(c)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i]), y[i] = __uint_as_float(s[i]), z[i] = __uint_as_float(t[i]);
}
#undef MTP_R8
__device__ __forceinline__ void tmem_st8_nowait(uint32_t a, const float (&x)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(a), "r"(__float_as_uint(x[0])),
               "r"(__float_as_uint(x[1])), "r"(__float_as_uint(x[2])), "r"(__float_as_uint(x[3])), "r"(__float_as_uint(x[4])),
               "r"(__float_as_uint(x[5])), "r"(__float_as_uint(x[6])), "r"(__float_as_uint(x[7]))
               : "memory");
}
// barriers of a group's four warps, each converged first: a warp that comes apart into its threads (as after a wait of each of
// them) stays so through a barrier that counts threads, and what follows is then issued for each part (the shuffles below: 270
// cycles a row)
__device__ __forceinline__ void group_sync(int group) {
  __syncwarp();
  asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(1 + group) : "memory");
}
__device__ __forceinline__ bool group_any(int group, bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %2, 0;\n barrier.cta.red.or.pred.aligned q, %1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(r)
               : "r"(1 + group), "r"(static_cast<uint32_t>(v))
               : "memory");
  return uniform(static_cast<int>(r)) != 0;
}
// two fp16 values to two codes, and 2^up times what the codes leave of them (exact)
__device__ __forceinline__ uint32_t take_codes(__half2& v, __half2 up) {
  uint16_t c;
  uint32_t back;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(*reinterpret_cast<const uint32_t*>(&v)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(c));
  v = __hmul2(__hsub2(v, *reinterpret_cast<const __half2*>(&back)), up);
  return c;
}
__device__ __forceinline__ uint32_t to_codes(__half2 v) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(*reinterpret_cast<const uint32_t*>(&v)));
  return c;
}

template <int HD, int kMax>
__global__ void __launch_bounds__(Wide<HD, kMax>::kThreads, 1)
paged_cols_kernel(const __grid_constant__ PagedMaps maps, const Shape sh, int box, float scale_log2, float2* __restrict__ rec_ml,
                  float* __restrict__ rec_o) {
  using C = Wide<HD, kMax>;
  const int NR = sh.tile_rows;  // rows of a tile, a multiple of 8
  pdl_trigger();  // the joining kernel may start its setup
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t s0 = smem_u32(smem), bar0 = s0 + C::kOffBar;
  if (s0 & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(&g_mtp_error_word, MTP_DEVERR_TIMEOUT);
    return;
  }
  auto k_full = [&](uint32_t g) { return bar0 + 8u * (g % C::kKStages); };
  auto k_empty = [&](uint32_t g) { return bar0 + 8u * (C::kKStages + g % C::kKStages); };
  const uint32_t barv = bar0 + 16u * C::kKStages;
  auto v_full = [&](uint32_t g) { return barv + 8u * (g % C::kVStages); };
  auto v_empty = [&](uint32_t g) { return barv + 8u * (C::kVStages + g % C::kVStages); };
  const uint32_t barm = barv + 16u * C::kVStages;
  auto m_full = [&](uint32_t g) { return barm + 8u * (g % C::kRing); };
  auto m_empty = [&](uint32_t g) { return barm + 8u * (C::kRing + g % C::kRing); };
  const uint32_t barq = barm + 16u * C::kRing;
  auto q_full = [&](uint32_t i) { return barq + 8u * (i & 1); };
  auto q_empty = [&](uint32_t i) { return barq + 16u + 8u * (i & 1); };
  auto s_full = [&](uint32_t x) { return barq + 32u + 8u * x; };
  auto s_free = [&](uint32_t x) { return barq + 32u + 8u * (C::kW + x); };
  auto p_full = [&](uint32_t x) { return barq + 32u + 8u * (2 * C::kW + x); };
  auto pv_done = [&](uint32_t x) { return barq + 32u + 8u * (3 * C::kW + x); };
  const uint32_t drain = barq + 32u + 32u * C::kW;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 8 * C::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // of block g: 8 exponents of keys, values (0: no rows), 8 pages
  auto meta = [&](uint32_t g) { return reinterpret_cast<uint16_t*>(smem + C::kOffMeta + g % C::kRing * 48); };
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < C::kKStages; ++i) mbar_init(k_full(i), 1), mbar_init(k_empty(i), 1);
    for (uint32_t i = 0; i < C::kVStages; ++i) mbar_init(v_full(i), 1), mbar_init(v_empty(i), 1);
    for (uint32_t i = 0; i < C::kRing; ++i) mbar_init(m_full(i), 1), mbar_init(m_empty(i), 5);  // the loader, a group's warps
    for (uint32_t x = 0; x < 2; ++x) mbar_init(q_full(x), 1), mbar_init(q_empty(x), 1 + 4 * C::kW);
    for (uint32_t x = 0; x < C::kW; ++x) {
      mbar_init(s_full(x), 1);
      mbar_init(s_free(x), 128);
      mbar_init(p_full(x), 128);
      mbar_init(pv_done(x), 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == C::kMmaWarp) tmem_alloc_cols(smem_u32(tmem_slot), C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_phase(bar, parity, abort_flag, &g_mtp_error_word); };
  auto wwait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };

  const Deal deal(steps_before(sh, sh.R, lane), sh.least, sh.workers);
  const int worker = static_cast<int>(blockIdx.x);
  Cursor at;
  at.left = 0;
  if (worker < deal.n) at.begin(sh, deal.start(worker), deal.start(worker + 1), lane);
  // blocks of the segment that starts at the cursor
  auto segment = [&]() { return static_cast<int>(min(static_cast<long long>(at.steps - at.step), at.left)); };
  auto skip = [&](int n) {  // to the next segment
    at.left -= n - 1;
    at.step += n - 1;
    at.next(sh);
  };

  if (warp == C::kMetaWarp) {
    // 8 lanes per block, four blocks at a time
    for (uint32_t g0 = 0; at.left > 0; g0 += 4) {
      int r = 0, head = 0, step = 0, ctx = 0;
      uint32_t n = 0;
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        if (at.left == 0) break;
        if (static_cast<uint32_t>(lane >> 3) == i) r = at.r, head = at.item / sh.tiles, step = at.step, ctx = at.ctx;
        ++n;
        at.next(sh);
      }
      const bool is = static_cast<uint32_t>(lane >> 3) < n;
      const int b = 8 * step + (lane & 7);
      int page = -1;
      uint32_t exps = 0;
      if (is && 16ll * b < ctx) {
        page = sh.table[static_cast<long long>(r) * sh.table_len + b / sh.per_page];
        if (page < 0 || page >= sh.n_pages) {
          atomicOr(&g_mtp_error_word, MTP_DEVERR_PAGE_RANGE);
          page = -1;
        } else {
          const long long s = (static_cast<long long>(page) * sh.Hkv + head) * sh.per_page + b % sh.per_page;
          exps = max(static_cast<uint32_t>(sh.ks[s]), 1u) | max(static_cast<uint32_t>(sh.vs[s]), 1u) << 8;
        }
      }
      bool ok = true;
      for (uint32_t i = 0; i < n && ok; ++i)
        if (g0 + i >= C::kRing) ok = wwait(m_empty(g0 + i), ((g0 + i) / C::kRing - 1) & 1);
      if (!ok) break;
      if (is) {
        uint16_t* m = meta(g0 + (lane >> 3));
        m[lane & 7] = static_cast<uint16_t>(exps);
        reinterpret_cast<int*>(m + 8)[lane & 7] = page;
      }
      __syncwarp();
      if (is && (lane & 7) == 0) mbar_arrive1(m_full(g0 + (lane >> 3)));
    }
  } else if (warp == C::kLoadWarp) {
    uint32_t g = 0;
    const int boxes = kCols / box, per_box = box / 16;
    const int i = lane & 15;  // a lane per box of keys, 16 lanes on one per box of values
    for (; at.left > 0; ++g) {
      if (!wwait(m_full(g), (g / C::kRing) & 1)) break;
      const int id = i < boxes ? reinterpret_cast<const int*>(meta(g) + 8)[i * per_box] : -1;
      __syncwarp();
      if (lane == 0) mbar_arrive1(m_empty(g));
      const uint32_t n = __popc(__ballot_sync(0xffffffffu, id >= 0 && lane < 16));
      const int row = (at.step * (kCols / 16) + i * per_box) % sh.per_page * 16, head = at.item / sh.tiles;
      if (g >= C::kKStages && !wwait(k_empty(g), (g / C::kKStages - 1) & 1)) break;
      if (lane == 0) mbar_expect_tx(k_full(g), n * box * HD);
      __syncwarp();
      if (id >= 0 && lane < 16)
        tma_tile_3d(s0 + g % C::kKStages * C::kTileBytes + i * box * HD, &maps.k, 0, row, id * sh.Hkv + head, k_full(g));
      const bool free = g < C::kVStages || wwait(v_empty(g), (g / C::kVStages - 1) & 1);
      if (lane == 0) mbar_expect_tx(v_full(g), free ? n * box * HD : 0);
      __syncwarp();
      if (id >= 0 && lane >= 16 && free)
        tma_tile_3d(s0 + C::kOffV + g % C::kVStages * C::kTileBytes + i * box * HD, &maps.v, 0, row, id * sh.Hkv + head, v_full(g));
      at.next(sh);
    }
    // no copy may still be landing when the CTA leaves (matters only after an abort)
    for (uint32_t y = g > C::kKStages ? g - C::kKStages : 0; y < g; ++y) wait_drain(k_full(y), (y / C::kKStages) & 1, kWaitLimitCycles);
    for (uint32_t y = g > C::kVStages ? g - C::kVStages : 0; y < g; ++y) wait_drain(v_full(y), (y / C::kVStages) & 1, kWaitLimitCycles);
  } else if (warp == C::kMmaWarp) {
    // (the columns are a multiple of 16; those beyond the rows hold anything)
    const uint32_t idesc_s = idesc_e4m3(kCols, (NR + 15) / 16 * 16, false, false), idesc_o = idesc_e4m3(128, (3 * NR + 15) / 16 * 16, true, true);
    constexpr uint32_t kLayout = HD == 128 ? 2 : 4;
    uint32_t g = 0, b = 0, seg = 0;  // next block for scores, for outputs; segment of the former
    int n = 0, j = 0;                // blocks of the segment, next one
    uint32_t firsts = 0;             // a bit per block under way: whether it is its group's first of a segment
    // whichever is ready: the scores of block g, as far ahead as there are groups, or the outputs of block b
    auto ready = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test_wait(bar, parity)); };
    long long since = cycles_now();
    for (uint32_t spins = 0; at.left > 0 || b < g; ++spins) {
      if (at.left > 0 && g - b <= C::kW) {
        const uint32_t x = g % C::kW, k_at = s0 + g % C::kKStages * C::kTileBytes, q_at = s0 + C::kOffQ + (seg & 1) * C::kQBytes;
        if (ready(k_full(g), (g / C::kKStages) & 1) && (g < C::kW || ready(s_free(x), (g / C::kW - 1) & 1)) &&
            (j > 0 || ready(q_full(seg), (seg >> 1) & 1))) {
          if (j == 0) n = segment();
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 2 * HD / 32; ++k) {
            const int kk = k % (HD / 32);
            umma_e4m3_warp(tmem + x * C::kSCols, smem_desc(k_at + 32 * kk, 16, 8 * HD, kLayout),
                           smem_desc(q_at + (k == kk ? 0 : NR * HD) + 32 * kk, 16, 8 * HD, kLayout), idesc_s, k > 0);
          }
          umma_commit_warp(s_full(x));
          umma_commit_warp(k_empty(g));
          if (j + 1 == n) umma_commit_warp(q_empty(seg));
          firsts = (firsts & ~(1u << (g & 7))) | (j < C::kW ? 1u << (g & 7) : 0u);
          ++g;
          if (++j == n) {
            j = 0;
            ++seg;
            skip(n);
          }
          spins = 0;
        }
      }
      if (b < g) {
        const uint32_t x = b % C::kW, v_at = s0 + C::kOffV + b % C::kVStages * C::kTileBytes, p_at = s0 + C::kOffP + x * C::kPBytes;
        if (ready(p_full(x), (b / C::kW) & 1) && ready(v_full(b), (b / C::kVStages) & 1)) {
          tc_fence_after();
          const bool first = firsts >> (b & 7) & 1;
#pragma unroll
          for (int k = 0; k < kCols / 32; ++k)
            umma_e4m3_warp(tmem + C::kColO + x * C::kOCols, smem_desc(v_at + 32 * HD * k, 0, 8 * HD, kLayout), smem_desc(p_at + 512 * k, 128, 2048, 0),
                           idesc_o, k > 0 || !first);
          umma_commit_warp(pv_done(x));
          umma_commit_warp(v_empty(b));
          ++b;
          spins = 0;
        }
      }
      if (spins == 0) since = cycles_now();
      if ((spins & 31u) == 31u) {
        if (*abort_flag) break;
        if (cycles_now() - since > kWaitLimitCycles) {
          *abort_flag = 1;
          atomicOr(&g_mtp_error_word, MTP_DEVERR_TIMEOUT);
          break;
        }
      }
    }
    umma_commit_warp(drain);  // no product may be under way when the CTA leaves (matters only after an abort)
    wait_drain(drain, 0, kWaitLimitCycles);
  } else if (warp == C::kQWarp) {
    for (uint32_t seg = 0; at.left > 0; ++seg) {
      if (seg >= 2 && !wwait(q_empty(seg), ((seg >> 1) - 1) & 1)) break;
      const int head = at.item / sh.tiles, row0 = (at.item - head * sh.tiles) * NR, nr = min(sh.rows - row0, NR);
      uint8_t* q_at = smem + C::kOffQ + (seg & 1) * C::kQBytes;
      float* scales = reinterpret_cast<float*>(smem + C::kOffRow) + (seg & 1) * 2 * kMax;
      int* sees = reinterpret_cast<int*>(scales + kMax);
      // one, two or four lanes per row, each with a part of it, read twice (a whole warp per row and shuffles for its maximum: 20
      // rows took 20 us)
      const int per = nr <= 8 ? 4 : nr <= 16 ? 2 : 1, chunks = HD / 16 / per, c0 = lane % per * chunks;
#pragma unroll 1
      for (int base = 0; base < nr; base += 32 / per) {
        const int n = base + lane / per, row = row0 + min(n, nr - 1), i = row / sh.G;
        const uint4* from = reinterpret_cast<const uint4*>(sh.q + at.r * sh.q_r + i * sh.q_l + (head * sh.G + row - i * sh.G) * sh.q_h) + 2 * c0;
        uint32_t top = 0;  // magnitudes are ordered as integers: what is not finite is the largest
#pragma unroll 4
        for (int c = 0; c < 2 * chunks; ++c) {
          const uint4 v = from[c];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(w[e] << 16 & 0x7fff0000u, w[e] & 0x7fff0000u));
        }
        if (per > 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        if (per > 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (n >= nr) continue;
        const bool odd = top >= 0x7f800000u;                                // NaN for every score of the row
        const int up = min(7 - (static_cast<int>(top >> 23) - 127), 100);  // to [2^7, 2^8)
        const float f = power_of_two(up);
        if (c0 == 0) {
          scales[n] = scale_log2 * power_of_two(-up);
          sees[n] = sh.sees(i, at.ctx, at.fresh);
        }
        const __half2 one = __float2half2_rn(1.f);
#pragma unroll 2
        for (int c = 0; c < chunks; ++c) {
          const uint4 v[2] = {from[2 * c], from[2 * c + 1]};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4& w = v[e / 2];
            const float2 x = unpack2_bf16(e & 1 ? w.z : w.x), y = unpack2_bf16(e & 1 ? w.w : w.y);
            __half2 a = __floats2half2_rn(x.x * f, x.y * f), b = __floats2half2_rn(y.x * f, y.y * f);
            hi[e] = take_codes(a, one) | take_codes(b, one) << 16;
            lo[e] = to_codes(a) | to_codes(b) << 16;
            if (odd) hi[e] = 0x7f7f7f7fu;
          }
          // rows of HD bytes, swizzled over their width: 16-byte chunk c0 + c
          auto put = [&](int to, const uint32_t (&w)[4]) {
            const int at_c = HD == 128 ? ((c0 + c) ^ to) & 7 : ((c0 + c) ^ (to >> 1)) & 3;
            *reinterpret_cast<uint4*>(q_at + to * HD + at_c * 16) = make_uint4(w[0], w[1], w[2], w[3]);
          };
          put(n, hi);
          put(NR + n, lo);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive1(q_full(seg));
      skip(segment());
    }
  } else {
    // Softmax.  After an abort everything runs on (the waits return at once), so that the groups'
    // barriers meet.
    constexpr int kPitch = 68;  // of a row's 64 numbers
    const int x = warp >> 2, j = threadIdx.x & 127, w4 = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(w4 * 32) << 16);
    const uint32_t s_at = lanes + x * C::kSCols, o_at = lanes + C::kColO + x * C::kOCols, l_at = lanes + C::kColL + x * kMax;
    const uint32_t every = (1u << (NR / 8)) - 1;  // chunks of 8 rows
    // of the group: a row's scale and what is added to its scores (7 - reference); what its weights shrink by; its largest exponent
    // over the top (0: none); parts' maxima or sums; a second factor for references that values' scales put further apart than a
    // float's exponent holds; chunks over the top in three turns; rows without a reference, and whether any has a second factor
    float2* rows = reinterpret_cast<float2*>(smem + C::kOffMax + x * C::kGroupBytes);
    float* shift = reinterpret_cast<float*>(rows + kMax);
    int* largest = reinterpret_cast<int*>(shift + kMax);
    float* parts = reinterpret_cast<float*>(largest + kMax);
    float* rest = parts + 256;
    uint32_t* need = reinterpret_cast<uint32_t*>(rest + kMax);
    uint32_t* unset = need + 3;
    uint8_t* p_group = smem + C::kOffP + x * C::kPBytes;
    uint8_t* p_to = p_group + (j >> 3) * 128 + (j & 7) * 16;
    if (j < 3) need[j] = 0;
    if (j < kMax) largest[j] = 0;
    uint32_t g = 0, third = 0;
    for (uint32_t seg = 0; at.left > 0; ++seg) {
      const int n_blocks = segment();
      const int head = at.item / sh.tiles, row0 = (at.item - head * sh.tiles) * NR, nr = min(sh.rows - row0, NR);
      const float* scales = reinterpret_cast<const float*>(smem + C::kOffRow) + (seg & 1) * 2 * kMax;
      const int* sees = reinterpret_cast<const int*>(scales + kMax);
      const uint32_t g0 = g;
      const uint32_t skipped = (x + C::kW - g0 % C::kW) % C::kW;
      const int mine = (n_blocks - static_cast<int>(skipped) + C::kW - 1) / C::kW;  // the group's blocks of the segment
      wwait(q_full(seg), (seg >> 1) & 1);
      if (w4 < 2) {
        const bool live = j < nr && sees[min(j, nr - 1)] > 0;
        if (j < NR) rows[j] = j < nr ? make_float2(scales[j], 0.f) : make_float2(0.f, -1e30f);  // (columns without a row: no weights)
        const uint32_t bits = __ballot_sync(0xffffffffu, live);
        if (lane == 0) unset[w4] = bits;
      }
      group_sync(x);
      uint32_t forced = every;  // chunks with rows without a reference
      bool flag = false;
      g += skipped;
#pragma unroll 1
      for (int k = 0; k < mine; ++k, g += C::kW) {
        const bool begun = k > 0;
        const uint32_t turn = g / C::kW;
        const int key0 = (at.step + static_cast<int>(g - g0)) * kCols;
        wwait(m_full(g), (g / C::kRing) & 1);
        const uint4 all = *reinterpret_cast<const uint4*>(meta(g));
        const uint32_t m = meta(g)[j >> 4];
        __syncwarp();
        if (lane == 0) mbar_arrive1(m_empty(g));
        const uint32_t halves[4] = {all.x, all.y, all.z, all.w};
        bool edge = key0 + kCols > at.ctx - (sh.causal ? at.fresh - 1 : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) edge |= (halves[i] & 0xffffu) == 0 || halves[i] >> 16 == 0;
        edge = uniform(static_cast<int>(edge)) != 0;
        const int away = min(max(static_cast<int>(m >> 8) - 127, -100), 100);
        const float kf = power_of_two(static_cast<int>(m & 0xff) - 127), d = static_cast<float>(away), up = power_of_two(away);
        const int seen_at = m == 0 ? 0x7fffffff : key0 + j;  // rows that see more than that see the key
        // exponents of the weights of rows c .. c + 7, but for d, the exponent of the value's scale
        auto exponents = [&](int c, float (&z)[8]) {
          tmem_ld8(s_at + c, z);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float4 rc = *reinterpret_cast<const float4*>(rows + c + i);
            z[i] = fmaf(z[i] * kf, rc.x, rc.y);
            z[i + 1] = fmaf(z[i + 1] * kf, rc.z, rc.w);
          }
          if (edge) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (seen_at >= sees[c + i]) z[i] = -INFINITY;
          }
        };
        wwait(s_full(x), turn & 1);
        tc_fence_after();
        uint32_t over = 0;
#pragma unroll 1
        for (int c = 0; c < NR; c += 8) {
          float z[8];
          exponents(c, z);
          const float most = fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
          if (most + d > kTopLog2 + kSlackLog2 && begun) {  // (positive floats are ordered as integers)
            over |= 1u << (c / 8);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (z[i] + d > kTopLog2 + kSlackLog2) atomicMax(largest + c + i, __float_as_int(z[i] + d));
          }
        }
        if (over) atomicOr(need + third, over);
        if (turn > 0) wwait(pv_done(x), (turn - 1) & 1);  // the weights' buffer, and the output
        const uint32_t next_third = third == 2 ? 0 : third + 1;
        if (j == 0) need[next_third] = 0;  // (last looked at two barriers ago)
        group_sync(x);
        const uint32_t which = static_cast<uint32_t>(uniform(static_cast<int>(need[third] | forced)));
        third = next_third;
        if (which) {
          // Rows of these chunks whose scores are over the top, or that have no reference yet, get one.
          if (forced) {
            // maxima of two lanes together, then of 64 numbers a row by way of the weights' buffer
            float* put = reinterpret_cast<float*>(p_group);
#pragma unroll 1
            for (int c = 0; c < NR; c += 8) {
              if (!(forced >> (c / 8) & 1)) continue;
              float z[8];
              exponents(c, z);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float s = fmaxf(z[i] + d, __shfl_xor_sync(0xffffffffu, z[i] + d, 16));
                if (lane < 16) put[(c + i) * kPitch + w4 * 16 + lane] = s;
              }
            }
            group_sync(x);
            for (int i = j; i < NR * 4; i += 128) {
              if (!(forced >> (i / 32) & 1)) continue;
              const float4* from = reinterpret_cast<const float4*>(put + i / 4 * kPitch) + i % 4;
              float top = -INFINITY;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 v = from[4 * e];
                top = fmaxf(top, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
              }
              parts[i % 4 * NR + i / 4] = top;
            }
            group_sync(x);
          }
          if (w4 < 2) {
            bool bare = false;
            float by = 0.f;
            if (j < nr) {
              bare = unset[w4] >> lane & 1;
              float top = -INFINITY;
              if (bare) {
                top = fmaxf(fmaxf(parts[j], parts[NR + j]), fmaxf(parts[2 * NR + j], parts[3 * NR + j]));
              } else if (largest[j] != 0) {
                top = __int_as_float(largest[j]);
              }
              largest[j] = 0;
              if (top > -INFINITY) {
                const float was = rows[j].y, now = was + (kTopLog2 - top);
                rows[j].y = now;
                by = bare ? 0.f : now - was;  // (a row without a reference has nothing to shrink; `now` is rounded)
                bare = false;
              }
            }
            if (j < NR) shift[j] = ex2(fmaxf(by, -120.f)), rest[j] = ex2(fminf(by + 120.f, 0.f));
            __syncwarp();
            const uint32_t far = __ballot_sync(0xffffffffu, by < -120.f);
            const uint32_t bits = __ballot_sync(0xffffffffu, bare);
            if (lane == 0) unset[w4] = bits, unset[2 + w4] = far;
          }
          group_sync(x);
          forced = 0;
          const int to = uniform(static_cast<int>(unset[2] | unset[3])) != 0 ? 2 * NR : NR;  // far apart: `rest` after `shift`
#pragma unroll 1
          for (int c2 = 0; c2 < to; c2 += 8) {
            const int c = c2 < NR ? c2 : c2 - NR;
            if (unset[c / 32] >> (c % 32) & 0xffu) forced |= 1u << (c / 8);
            if (!begun || !(which >> (c / 8) & 1)) continue;
            float f[8], l[8];
            const float* sc = c2 < NR ? shift : rest;
            *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(sc + c);
            *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(sc + c + 4);
            tc_fence_after();
            float o0[8], o1[8], o2[8];
            tmem_ld8(l_at + c, l);
            tmem_ld8x3(o_at + c, o_at + NR + c, o_at + 2 * NR + c, o0, o1, o2);
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] *= f[i], o0[i] *= f[i], o1[i] *= f[i], o2[i] *= f[i];
            tmem_st8_nowait(l_at + c, l);
            tmem_st8_nowait(o_at + c, o0);
            tmem_st8_nowait(o_at + NR + c, o1);
            tmem_st8_nowait(o_at + 2 * NR + c, o2);
            tmem_wait_st();
          }
          forced = static_cast<uint32_t>(uniform(static_cast<int>(forced)));
          tc_fence_before();
        }
        // weights
#pragma unroll 1
        for (int c = 0; c < NR; c += 8) {
          float z[8], l[8];
          if (begun) {
            tmem_ld8(l_at + c, l);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] = 0.f;
          }
          exponents(c, z);
          uint32_t code[3][2];
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            uint32_t part[3][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int n = i + 2 * h;
              const float w0 = ex2(z[n]), w1 = ex2(z[n + 1]);
              l[n] += w0;
              l[n + 1] += w1;
              __half2 v = __floats2half2_rn(w0 * up, w1 * up);
              part[0][h] = take_codes(v, __float2half2_rn(16.f));
              part[1][h] = take_codes(v, __float2half2_rn(32.f));
              part[2][h] = to_codes(v);
            }
#pragma unroll
            for (int p = 0; p < 3; ++p) code[p][i / 4] = part[p][0] | part[p][1] << 16;
          }
          tmem_st8_nowait(l_at + c, l);
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            const int n = p * NR + c;
            *reinterpret_cast<uint2*>(p_to + n / 16 * (16 * kCols) + n % 16) = make_uint2(code[p][0], code[p][1]);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive1(s_free(x));
        if (edge) {
          // values past the end and of bad pages are not looked at, and NaN is taken out for rows that do not see it
          // (the join puts it back for those that do)
          wwait(v_full(g), (g / C::kVStages) & 1);
          uint4* row = reinterpret_cast<uint4*>(smem + C::kOffV + g % C::kVStages * C::kTileBytes + j * HD);
          const bool past = key0 + j >= at.ctx || m == 0;
#pragma unroll 1
          for (int i = 0; i < HD / 16; ++i) {
            uint4 v = past ? make_uint4(0, 0, 0, 0) : row[i];
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
            bool any = past;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t nan = ((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              if (nan) {
                any = flag = true;
                w[e] &= ~((nan >> 7) * 0xffu);
              }
            }
            if (any) row[i] = v;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive1(p_full(x));
      }
      // the group's part
      const long long rec = ((static_cast<long long>(at.r) * sh.items() + at.item + worker) * C::kW + x) * sh.rec_rows;
      const bool any = group_any(x, flag);
      if (mine > 0) {
        wwait(pv_done(x), (g / C::kW - 1) & 1);  // of the group's last block
        tc_fence_after();
        // sums of a row over the threads: two lanes together, then 64 numbers a row by way of the weights' buffer
        float* put = reinterpret_cast<float*>(p_group);
#pragma unroll 1
        for (int c = 0; c < NR; c += 8) {
          float l[8];
          tmem_ld8(l_at + c, l);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float s = l[i] + __shfl_xor_sync(0xffffffffu, l[i], 16);
            if (lane < 16) put[(c + i) * kPitch + w4 * 16 + lane] = s;
          }
        }
        group_sync(x);
        for (int i = j; i < NR * 4; i += 128) {
          const float4* from = reinterpret_cast<const float4*>(put + i / 4 * kPitch) + i % 4;
          const float4 a = from[0], b = from[4], c = from[8], e = from[12];
          parts[i % 4 * NR + i / 4] = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w)) + (((c.x + c.y) + (c.z + c.w)) + ((e.x + e.y) + (e.z + e.w)));
        }
        group_sync(x);
#pragma unroll 1
        for (int c = 0; c < nr; c += 8) {
          float o0[8], o1[8], o2[8];
          tmem_ld8x3(o_at + c, o_at + NR + c, o_at + 2 * NR + c, o0, o1, o2);
          if (j < HD) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c + i < nr) rec_o[(rec + c + i) * HD + j] = fmaf(o2[i], 0x1p-9f, fmaf(o1[i], 0x1p-4f, o0[i]));
          }
        }
        tc_fence_before();
      }
      if (j < nr) {
        float sum = 0.f;
        if (mine > 0 && sees[j] > 0) sum = (parts[j] + parts[NR + j]) + (parts[2 * NR + j] + parts[3 * NR + j]);
        rec_ml[rec + j] = make_float2(sum == 0.f ? -INFINITY : -rows[j].y, any ? -sum : sum);
      }
      group_sync(x);  // what is shared within the group is used again
      if (lane == 0) mbar_arrive1(q_empty(seg));
      g = g0 + n_blocks;
      skip(n_blocks);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMmaWarp) tmem_free_cols(tmem, C::kTmemCols);
}

// Values that are not finite back into kD elements of an output, from d0 on: those of the keys that the kernels take them out of, as far
// as the row sees them.
template <bool kF8, int kD>
__device__ __forceinline__ void put_back(const Shape& sh, const mtp_paged_cache& c, int r, int head, int ctx, int fresh, int see, int d0, float (&o)[kD]) {
  const int j0 = max((ctx - (sh.causal ? fresh - 1 : 0)) / sh.keys * sh.keys, 0);
  for (int j = j0; j < see; ++j) {
    const int page = sh.table[static_cast<long long>(r) * sh.table_len + j / c.page];
    if (page < 0 || page >= sh.n_pages) continue;
    const size_t v_at = ((static_cast<size_t>(page) * sh.Hkv + head) * c.page + j % c.page) * c.head_dim + d0;
#pragma unroll
    for (int d = 0; d < kD; ++d) {
      if constexpr (kF8) {
        if ((static_cast<const uint8_t*>(c.v)[v_at + d] & 0x7f) == 0x7f) o[d] = NAN;
      } else {
        const float x = __bfloat162float(static_cast<const __nv_bfloat16*>(c.v)[v_at + d]);
        if (!(fabsf(x) < INFINITY)) o[d] += x;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Short caches: a CTA per item
// ---------------------------------------------------------------------------
// Where a table holds few rows, the time is launches and loads that wait for one another: a CTA has 16 rows of a (request, key
// head) and all keys, every eighth step of 16 a warp's, as bf16 (exactly, also of 8 bits); their parts are joined in shared
// memory, so that there is one launch, no record and no workspace.
template <int HD>
struct Item {
  static constexpr int kWarps = 8, kThreads = 32 * kWarps;
  static constexpr int kTileBytes = 16 * HD * 2;
  static constexpr int kWarpBytes = 2 * kTileBytes;  // keys and values of a step; then the warp's output, 16 x HD floats
  static constexpr int kOffMl = kWarps * kWarpBytes;
  static constexpr int kSmemBytes = kOffMl + kWarps * 16 * 8;
};
template <int HD, bool kF8>
__global__ void __launch_bounds__(Item<HD>::kThreads, 1)
paged_item_kernel(const Shape sh, const mtp_paged_cache c, float scale_log2, __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  using C = Item<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int rest = blockIdx.x / sh.tiles, tile = blockIdx.x - rest * sh.tiles, r = rest / sh.Hkv, head = rest - r * sh.Hkv;
  const int ctx = uniform(sh.ctx(r)), fresh = uniform(sh.fresh(r)), steps = uniform(sh.steps(r));
  const int mine = (steps - warp + C::kWarps - 1) / C::kWarps;  // this warp's steps, 32 at the most
  int page = -1;
  if (lane < mine) {
    page = sh.table[static_cast<long long>(r) * sh.table_len + (warp + C::kWarps * lane) / sh.per_page];
    if (page < 0 || page >= sh.n_pages) {
      atomicOr(&g_mtp_error_word, MTP_DEVERR_PAGE_RANGE);
      page = -1;
    }
  }
  Rows<HD> w;
  load_rows<HD>(w, sh, r, head, tile * kTileRows, ctx, fresh, lane);
  constexpr int kLoads = kF8 ? HD / 32 : HD / 16;  // 16 bytes of keys, and of values, per lane
  uint4 kr[kLoads], vr[kLoads];
  float ks = 0.f, vs = 0.f;
  int id = -1;
  auto fetch = [&](int i) {
    id = __shfl_sync(0xffffffffu, page, i & 31);
    if (i >= mine || id < 0) return;
    const int block = (warp + C::kWarps * i) % sh.per_page;
    const long long b = (static_cast<long long>(id) * sh.Hkv + head) * sh.per_page + block;
    const uint4* k = reinterpret_cast<const uint4*>(c.k) + b * (kLoads * 32) + lane;
    const uint4* v = reinterpret_cast<const uint4*>(c.v) + b * (kLoads * 32) + lane;
#pragma unroll
    for (int e = 0; e < kLoads; ++e) kr[e] = k[32 * e], vr[e] = v[32 * e];
    if constexpr (kF8) {
      ks = power_of_two(max(static_cast<int>(sh.ks[b]), 1) - 127);
      vs = power_of_two(max(static_cast<int>(sh.vs[b]), 1) - 127);
    }
  };
  uint8_t* mem = smem + warp * C::kWarpBytes;
  const uint32_t k_at = smem_u32(mem), v_at = k_at + C::kTileBytes;
  auto put = [&](uint8_t* to, const uint4 (&x)[kLoads], float f) {
#pragma unroll
    for (int e = 0; e < kLoads; ++e) {
      const int n = 32 * e + lane;
      if constexpr (kF8) {
        const int row = n / (HD / 16), ch = n % (HD / 16) * 2;
        const uint32_t words[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t h[2];
          asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, u;\n}\n"
              : "=r"(h[0]), "=r"(h[1])
              : "r"(words[i]));
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&h[g]));
            y[2 * i + g] = pack2_bf16(z.x * f, z.y * f);
          }
        }
        *reinterpret_cast<uint4*>(to + chunk_at(0, row, ch)) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(to + chunk_at(0, row, ch + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
      } else {
        *reinterpret_cast<uint4*>(to + chunk_at(0, n / (HD / 8), n % (HD / 8))) = x[e];
      }
    }
  };
  fetch(0);
#pragma unroll 1
  for (int i = 0; i < mine; ++i) {
    const bool is = id >= 0;  // (a bad page is not looked at)
    if (is) {
      put(mem, kr, ks);
      put(mem + C::kTileBytes, vr, vs);
    }
    __syncwarp();
    fetch(i + 1);
    const int key0 = 16 * (warp + C::kWarps * i);
    if (is) {
      if (key0 + 16 > ctx - (sh.causal ? fresh - 1 : 0))
        step_rows<HD, true>(w, k_at, v_at, key0, ctx - key0, scale_log2, lane);
      else
        step_rows<HD, false>(w, k_at, v_at, key0, ctx - key0, scale_log2, lane);
    }
    __syncwarp();
  }
  // the warps' parts
  const int g = lane >> 2, t = lane & 3;
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    w.sum[e] += __shfl_xor_sync(0xffffffffu, w.sum[e], 1);
    w.sum[e] += __shfl_xor_sync(0xffffffffu, w.sum[e], 2);
    const float l = w.see[e] > 0 ? w.sum[e] : 0.f;
    if (t == 0) ml[warp * 16 + 8 * e + g] = make_float2(l == 0.f ? -INFINITY : w.mx[e], l);
    float* to = reinterpret_cast<float*>(mem) + (8 * e + g) * HD;
#pragma unroll
    for (int n = 0; n < HD / 8; ++n) *reinterpret_cast<float2*>(to + 8 * n + 2 * t) = make_float2(w.o[n][2 * e], w.o[n][2 * e + 1]);
  }
  const bool any = __syncthreads_or(w.flag) != 0;
  constexpr int kD = HD / 16;  // elements of a thread
  const int in = threadIdx.x / 16, row = tile * kTileRows + in, d0 = threadIdx.x % 16 * kD;
  if (row >= sh.rows) return;
  float M = -INFINITY, L = 0.f, o[kD];
#pragma unroll
  for (int d = 0; d < kD; ++d) o[d] = 0.f;
#pragma unroll
  for (int x = 0; x < C::kWarps; ++x) M = fmaxf(M, ml[x * 16 + in].x);
#pragma unroll 1
  for (int x = 0; x < C::kWarps; ++x) {
    const float2 part = ml[x * 16 + in];
    if (part.y == 0.f) continue;
    const float f = ex2(part.x - M);
    L = fmaf(f, part.y, L);
    const float4* from = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + x * C::kWarpBytes) + in * HD + d0);
#pragma unroll
    for (int d = 0; d < kD; d += 4) {
      const float4 v = from[d / 4];
      o[d] = fmaf(f, v.x, o[d]), o[d + 1] = fmaf(f, v.y, o[d + 1]), o[d + 2] = fmaf(f, v.z, o[d + 2]), o[d + 3] = fmaf(f, v.w, o[d + 3]);
    }
  }
  const int i = row / sh.G, h = head * sh.G + row - i * sh.G;
  if (any) put_back<kF8, kD>(sh, c, r, head, ctx, fresh, sh.sees(i, ctx, fresh), d0, o);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const long long to_row = (static_cast<long long>(r) * sh.L + i) * sh.H + h;
  uint32_t y[kD / 2];
#pragma unroll
  for (int d = 0; d < kD; d += 2) y[d / 2] = pack2_bf16(o[d] * inv, o[d + 1] * inv);
  if constexpr (kD == 8)
    *reinterpret_cast<uint4*>(out + to_row * HD + d0) = make_uint4(y[0], y[1], y[2], y[3]);
  else
    *reinterpret_cast<uint2*>(out + to_row * HD + d0) = make_uint2(y[0], y[1]);
  if (lse && d0 == 0) lse[to_row] = L == 0.f ? -INFINITY : M * kLn2 + logf(L);
}

// Joins the records of one (request, token, head): by a warp, or with kSplit by a CTA, each warp every fourth record.
// Which records there are follows from the lengths alone and is worked out under the kernel before.
constexpr int kJoinWarps = 4;
constexpr int kSplitRows = 8;  // up to this many rows per SM have a CTA each
template <int HD, bool kF8, bool kSplit>
__global__ void __launch_bounds__(32 * kJoinWarps)
paged_join_kernel(const Shape sh, const mtp_paged_cache c, const float2* __restrict__ rec_ml, const float* __restrict__ rec_o,
                  __nv_bfloat16* __restrict__ out, float* __restrict__ lse, float* __restrict__ rec, long long rec_stride) {
  constexpr int kD = HD / 32;
  __shared__ float shared[kSplit ? kJoinWarps : 1][HD];
  const int lane = threadIdx.x & 31, warp = uniform(static_cast<int>(threadIdx.x >> 5));
  const int row = kSplit ? blockIdx.x : blockIdx.x * kJoinWarps + warp;  // (2^24 at the most)
  if (row >= sh.R * sh.L * sh.H) return;
  const int i0 = row / sh.H, h = row - i0 * sh.H, r = i0 / sh.L, i = i0 - r * sh.L;
  const int head = h / sh.G, in_rows = i * sh.G + h - head * sh.G, tile = in_rows / sh.tile_rows;
  const int ctx = sh.ctx(r), fresh = sh.fresh(r), steps = sh.steps(r), see = sh.sees(i, ctx, fresh);
  long long total = 0, before = 0;
  for (int k = lane; k < sh.R; k += 32) {
    const int n = sh.steps(k);
    total += n;
    before += k < r ? n : 0;
  }
  total = uniform(warp_total(total)) * sh.items();
  before = uniform(warp_total(before)) * sh.items();
  int n = 0;
  long long rec0 = 0;
  if (see > 0 && steps > 0) {
    const Deal deal(total, sh.least, sh.workers);
    const int item = head * sh.tiles + tile;
    const long long begin = before + static_cast<long long>(item) * steps;
    const int w0 = deal.owner(begin), w1 = deal.owner(begin + steps - 1);
    rec0 = (static_cast<long long>(r) * sh.items() + item + w0) * sh.parts * sh.rec_rows + in_rows % sh.tile_rows;
    n = (w1 - w0 + 1) * sh.parts;
  }
  n = uniform(n);
  float M = -INFINITY, L = 0.f, o[kD];
#pragma unroll
  for (int d = 0; d < kD; ++d) o[d] = 0.f;
  bool flag = false;
  pdl_wait();  // the records
  for (int k = lane; k < n; k += 32) M = fmaxf(M, rec_ml[rec0 + static_cast<long long>(k) * sh.rec_rows].x);
  M = warp_max(M);
  for (int base = 0; base < n; base += 32) {
    float w = 0.f;
    if (base + lane < n) {
      const float2 ml = rec_ml[rec0 + static_cast<long long>(base + lane) * sh.rec_rows];
      flag |= __float_as_int(ml.y) < 0;
      if (ml.y != 0.f) {
        w = ex2(0.5f * (ml.x - M));
        L += scale_twice(fabsf(ml.y), w);
      }
    }
    const int m = min(32, n - base);
    constexpr int kAhead = 4, kStep = kSplit ? kJoinWarps : 1;
    for (int k = kSplit ? warp : 0; k < m; k += kAhead * kStep) {
      float x[kAhead][kD], wk[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int at = k + a * kStep;
        wk[a] = __shfl_sync(0xffffffffu, w, min(at, 31));
        if (at >= m) wk[a] = 0.f;
#pragma unroll
        for (int d = 0; d < kD; ++d) x[a][d] = 0.f;
        if (wk[a] != 0.f) {  // (a part without a key holds nothing)
          const float* from = rec_o + (rec0 + static_cast<long long>(base + at) * sh.rec_rows) * HD + lane * kD;
          if constexpr (kD == 4)
            *reinterpret_cast<float4*>(x[a]) = *reinterpret_cast<const float4*>(from);
          else
            *reinterpret_cast<float2*>(x[a]) = *reinterpret_cast<const float2*>(from);
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
#pragma unroll
        for (int d = 0; d < kD; ++d) o[d] += scale_twice(x[a][d], wk[a]);
    }
  }
  L = warp_sum(L);
  if constexpr (kSplit) {
#pragma unroll
    for (int d = 0; d < kD; ++d) shared[warp][lane * kD + d] = o[d];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int d = 0; d < kD; ++d) {
      const int at = lane * kD + d;
      o[d] = (shared[0][at] + shared[1][at]) + (shared[2][at] + shared[3][at]);
    }
  }
  if (__any_sync(0xffffffffu, flag)) put_back<kF8, kD>(sh, c, r, head, ctx, fresh, see, lane * kD, o);
  if (rec) {
    float* to = rec + static_cast<long long>(row) * rec_stride;
    if (lane == 0) {
      to[0] = M * kLn2;
      to[1] = L;
    }
#pragma unroll
    for (int d = 0; d < kD; ++d) to[2 + lane * kD + d] = o[d];
    return;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  __nv_bfloat16* to = out + static_cast<long long>(row) * HD + lane * kD;
  if constexpr (kD == 4)
    *reinterpret_cast<uint2*>(to) = make_uint2(pack2_bf16(o[0] * inv, o[1] * inv), pack2_bf16(o[2] * inv, o[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(to) = pack2_bf16(o[0] * inv, o[1] * inv);
  if (lse && lane == 0) lse[row] = L == 0.f ? -INFINITY : M * kLn2 + logf(L);
}

struct Layout {
  size_t ml, o, total;
};
// warps of 16 rows that share a ring (bf16); rows of a tile (8 bits): as few tiles as 48 rows each make, and then as few
// rows
int group_of(int rows) { return rows <= kTileRows ? 1 : rows <= 2 * kTileRows ? 2 : rows <= 4 * kTileRows ? 4 : 8; }
int cols_of(int rows) {
  const int tiles = (rows + 47) / 48;
  return ((rows + tiles - 1) / tiles + 7) / 8 * 8;
}
Shape shape_of(int R, int L, int H, const mtp_paged_cache& c) {
  Shape s{};
  s.R = R, s.L = L, s.H = H, s.Hkv = c.n_kv_heads, s.G = H / c.n_kv_heads;
  s.rows = L * s.G;
  const bool f8 = c.dtype == MTP_E4M3;
  s.tile_rows = f8 ? cols_of(s.rows) : kTileRows * group_of(s.rows);
  s.tiles = (s.rows + s.tile_rows - 1) / s.tile_rows;
  s.rec_rows = std::min(s.rows, s.tile_rows);
  s.keys = f8 ? kCols : 16;
  s.least = f8 ? 1 : 4;
  s.parts = !f8 ? 1 : s.tile_rows <= 24 ? 3 : 2;  // (Wide::kW)
  s.cap = c.table_len * c.page;
  s.per_page = c.page / 16;
  s.n_pages = c.n_pages;
  s.table_len = c.table_len;
  s.workers = f8 ? sm_count_current() : sm_count_current() * (8 / group_of(s.rows));
  return s;
}
Layout layout_of(const Shape& s, int hd) {
  const size_t recs = (static_cast<size_t>(s.R) * s.Hkv * s.tiles + s.workers) * s.parts * s.rec_rows;
  Layout l;
  l.ml = 0;
  l.o = (recs * sizeof(float2) + 255) / 256 * 256;
  l.total = l.o + recs * hd * sizeof(float);
  return l;
}

bool cache_map(CUtensorMap* m, const void* p, const mtp_paged_cache& c, int box) {
  const uint64_t heads = static_cast<uint64_t>(c.n_pages) * c.n_kv_heads;
  if (c.dtype == MTP_E4M3) return tensor_map_rows(m, p, c.head_dim, c.page, heads, box);
  const uint64_t row = 2 * static_cast<uint64_t>(c.head_dim);
  const uint64_t dims[4] = {64, row / 128, static_cast<uint64_t>(c.page), heads};
  const uint64_t strides[3] = {128, row, c.page * row};
  const uint32_t boxes[4] = {64, 1, 16, 1};
  return tensor_map_bf16_4d(m, p, dims, strides, boxes);
}

template <int HD, int kGroup>
mtp_status rows_launch(const PagedMaps& maps, const PagedAttn& p, const Shape& s, float2* ml, float* o, cudaStream_t st) {
  using C = Cfg<HD, kGroup>;
  static PerDevice attr;
  if (!smem_limit(attr, paged_rows_kernel<HD, kGroup>, C::kSmemBytes)) return MTP_ERR_CUDA;
  paged_rows_kernel<HD, kGroup><<<sm_count_current(), C::kThreads, C::kSmemBytes, st>>>(maps, s, p.scale * kLog2e, ml, o);
  return MTP_OK;
}
template <int HD, int kMax>
mtp_status cols_launch(const PagedMaps& maps, const PagedAttn& p, const Shape& s, int box, float2* ml, float* o, cudaStream_t st) {
  using C = Wide<HD, kMax>;
  static PerDevice attr;
  if (!smem_limit(attr, paged_cols_kernel<HD, kMax>, C::kSmemBytes)) return MTP_ERR_CUDA;
  paged_cols_kernel<HD, kMax><<<sm_count_current(), C::kThreads, C::kSmemBytes, st>>>(maps, s, box, p.scale * kLog2e, ml, o);
  return MTP_OK;
}
template <int HD, bool kF8>
mtp_status launch(const PagedAttn& p, const Shape& s, const Layout& l, uint8_t* ws, cudaStream_t st) {
  PagedMaps maps;
  const int box = p.c.page % 128 == 0 ? 128 : p.c.page % 64 == 0 ? 64 : p.c.page % 32 == 0 ? 32 : 16;
  if (!cache_map(&maps.k, p.c.k, p.c, box) || !cache_map(&maps.v, p.c.v, p.c, box)) return MTP_ERR_CUDA;
  float2* ml = reinterpret_cast<float2*>(ws + l.ml);
  float* o = reinterpret_cast<float*>(ws + l.o);
  mtp_status status;
  if constexpr (kF8) {
    status = s.tile_rows <= 16   ? cols_launch<HD, 16>(maps, p, s, box, ml, o, st)
             : s.tile_rows <= 24 ? cols_launch<HD, 24>(maps, p, s, box, ml, o, st)
                                 : cols_launch<HD, 48>(maps, p, s, box, ml, o, st);
  } else {
    const int group = group_of(s.rows);
    status = group == 1   ? rows_launch<HD, 1>(maps, p, s, ml, o, st)
             : group == 2 ? rows_launch<HD, 2>(maps, p, s, ml, o, st)
             : group == 4 ? rows_launch<HD, 4>(maps, p, s, ml, o, st)
                          : rows_launch<HD, 8>(maps, p, s, ml, o, st);
  }
  if (status != MTP_OK) return status;
  MTP_LAUNCH_CHECK();
  note_launch();
  const long long rows = static_cast<long long>(s.R) * s.L * s.H;
  const bool split = rows <= static_cast<long long>(kSplitRows) * sm_count_current();
  const dim3 grid(static_cast<unsigned>(split ? rows : (rows + kJoinWarps - 1) / kJoinWarps));
  MTP_CUDA_TRY(launch_pdl(split ? paged_join_kernel<HD, kF8, true> : paged_join_kernel<HD, kF8, false>, grid, dim3(32 * kJoinWarps), 0, st,
                          s, p.c, ml, o, p.o, p.lse, p.rec, p.rec_stride));
  note_launch();
  return MTP_OK;
}

}  // namespace

namespace {

// Many rows: the requests' rows are gathered as dense bf16 rows, exactly, and go through the attention over own caches
// (prefix_attn.cu), whose 128 rows share a block of keys.  Gathered, and in brackets tile by tile by the kernels above, us of a call out
// of a cold cache, hd 128, 8 key heads:
//   two requests of 8000 rows, 4 heads per key head    8 bits       bf16
//     1024 tokens (4096 rows per key head)             381 (882)    387 (2204)
//     256, 64                                          127 (236), 62 (82)    131 (538), 68 (142)
//     32, 16 (128, 64 rows)                            56 (58), 52 (38)      59 (80), 55 (52)
//   4096 rows each, 8 heads per key head
//     8 tokens (64 rows) of 8, 32, 64 requests         82 (55), 258 (154), 487 (284)    91 (88), 303 (315), 578 (619)
//     12 tokens                                        84 (68), 264 (200), 502 (371)    94 (140), 309 (522), 588 (1026)
//     16 tokens                                        86 (91), 274 (279), 514 (532)    95 (144), 315 (531), 601 (1049)
// So bf16 gains from 64 rows on, 8 bits from 128; between the two 8 bits pay up to 1.7 times here, for weights of 2^-15 instead of
// 2^-11.  Only where the copy is at most 4 GB.
constexpr int kDenseRows = 64;
constexpr unsigned long long kDenseMost = 1ull << 32;

struct Dense {
  bool use;
  long long T;
  size_t k, v, ctx, ws, total;
};
Dense dense_of(int R, int L, int H, const mtp_paged_cache& c) {
  Dense d{};
  if (static_cast<long long>(L) * (H / c.n_kv_heads) < kDenseRows) return d;
  d.T = static_cast<long long>(c.table_len) * c.page + L;  // (a request may sit out up to L tokens, see kv_dense_launch)
  const unsigned long long one = 2ull * R * d.T * c.n_kv_heads * c.head_dim;
  if (d.T > 0x7FFFFFFFll || 2 * one > kDenseMost || !prefix_attn_sizes_ok(R, L, H, c.n_kv_heads, c.head_dim, 0, static_cast<int>(d.T))) return d;
  d.use = true;
  const auto up = [](unsigned long long n) { return (n + 255) / 256 * 256; };
  d.k = 0;
  d.v = up(one);
  d.ctx = d.v + up(one);
  d.ws = d.ctx + up(4ull * R);
  d.total = d.ws + prefix_attn_workspace_bytes(R, L, H, c.n_kv_heads, c.head_dim, 0, static_cast<int>(d.T));
  return d;
}

// zeros for the tokens from n_new[r] on, 8 elements per thread
__global__ void __launch_bounds__(256) paged_hide_kernel(int L, int H, int hd, long long n, const int32_t* __restrict__ n_new,
                                                         __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= n) return;
  const int per = hd / 8;
  const long long row = at / per;
  const int i = static_cast<int>(row / H % L), r = static_cast<int>(row / H / L);
  if (i < n_new[r]) return;
  *reinterpret_cast<uint4*>(out + at * 8) = make_uint4(0, 0, 0, 0);
  if (lse && at % per == 0) lse[row] = -INFINITY;
}

mtp_status dense_launch(const PagedAttn& p, const Dense& d, uint8_t* ws, size_t ws_bytes, cudaStream_t st) {
  int32_t* ctx = reinterpret_cast<int32_t*>(ws + d.ctx);
  // not causal: every token sees all of the request's rows, and only those
  mtp_status s = kv_dense_launch(p.c, p.R, p.L, d.T, p.ctx_len, p.n_new, p.causal, ws + d.k, ws + d.v, ctx, st);
  if (s != MTP_OK) return s;
  PrefixAttn a;
  a.R = p.R, a.L = p.L, a.H = p.H, a.Hkv = p.c.n_kv_heads, a.hd = p.c.head_dim, a.T = static_cast<int>(d.T);
  a.causal = p.causal;
  a.scale = p.scale;
  a.q = p.q, a.q_r = p.q_r, a.q_l = p.q_l, a.q_h = p.q_h;
  a.kk = reinterpret_cast<const __nv_bfloat16*>(ws + d.k);
  a.kv = reinterpret_cast<const __nv_bfloat16*>(ws + d.v);
  a.k_h = a.hd, a.k_t = static_cast<long long>(a.Hkv) * a.hd, a.k_r = d.T * a.k_t;
  a.ctx_len = ctx;
  a.o = p.o, a.lse = p.lse;
  s = prefix_attn_launch(a, ws + d.ws, ws_bytes - d.ws, st);
  if (s != MTP_OK || !p.n_new) return s;
  const long long n = static_cast<long long>(p.R) * p.L * p.H * (p.c.head_dim / 8);
  paged_hide_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, st>>>(p.L, p.H, p.c.head_dim, n, p.n_new, p.o, p.lse);
  MTP_LAUNCH_CHECK();
  note_launch();
  return MTP_OK;
}

// An item of 16 rows is a CTA's where there are few rounds of them over the SMs and a table's rows, times the rounds, are few.
// In a graph, and as calls, against the kernels above: 64 items of 304 rows, hd 64, 8 bits 6.1 us instead of 11.9 (19 for 25);
// 128 items of 20 rows per key head, 1024 rows, hd 128 16.1 instead of 20.9 (19 for 26); 448 of 256 rows, bf16 17.9 instead of
// 17.1 (20 for 26); beyond: 256 of 1024 rows 34 instead of 30 (37 for 33), 1024 of 128 rows 32 instead of 19 (35 for 25).
constexpr int kItemRows = 1024, kItemRounds = 3;
bool item_ok(int R, int L, int H, const mtp_paged_cache& c) {
  const long long rows = static_cast<long long>(L) * (H / c.n_kv_heads), sms = std::max(1, sm_count_current());
  const long long rounds = ((rows + kTileRows - 1) / kTileRows * R * c.n_kv_heads + sms - 1) / sms;
  return rows < kDenseRows && rounds <= kItemRounds && rounds * c.table_len * c.page <= kItemRows;
}
template <int HD, bool kF8>
mtp_status item_launch(const PagedAttn& p, cudaStream_t st) {
  using C = Item<HD>;
  static PerDevice attr;
  if (!smem_limit(attr, paged_item_kernel<HD, kF8>, C::kSmemBytes)) return MTP_ERR_CUDA;
  Shape s = shape_of(p.R, p.L, p.H, p.c);
  s.tile_rows = kTileRows;
  s.tiles = (s.rows + kTileRows - 1) / kTileRows;
  s.keys = 16;
  s.causal = p.causal;
  s.ctx_len = p.ctx_len, s.n_new = p.n_new, s.table = p.c.page_table;
  s.ks = p.c.k_scale, s.vs = p.c.v_scale;
  s.q = p.q, s.q_r = p.q_r, s.q_l = p.q_l, s.q_h = p.q_h;
  paged_item_kernel<HD, kF8><<<s.R * s.Hkv * s.tiles, C::kThreads, C::kSmemBytes, st>>>(s, p.c, p.scale * kLog2e, p.o, p.lse);
  MTP_LAUNCH_CHECK();
  note_launch();
  return MTP_OK;
}

}  // namespace

bool paged_attn_sizes_ok(int R, int L, int H, const mtp_paged_cache& c) {
  if (R < 1 || L < 1 || H < 1 || R > 65535 || H % c.n_kv_heads || H / c.n_kv_heads > 128) return false;
  return static_cast<long long>(L) * H <= (1ll << 24) && static_cast<long long>(R) * L * H <= (1ll << 24);
}
size_t paged_attn_workspace_bytes(int R, int L, int H, const mtp_paged_cache& c) {
  const Dense d = dense_of(R, L, H, c);
  return d.use ? d.total : layout_of(shape_of(R, L, H, c), c.head_dim).total;
}
mtp_status paged_attn_launch(const PagedAttn& p, void* ws, size_t ws_bytes, cudaStream_t st) {
  if (const Dense d = dense_of(p.R, p.L, p.H, p.c); d.use && !p.rec) {
    if (ws_bytes < d.total) return MTP_ERR_WORKSPACE;
    return dense_launch(p, d, static_cast<uint8_t*>(ws), ws_bytes, st);
  }
  Shape s = shape_of(p.R, p.L, p.H, p.c);
  const Layout l = layout_of(s, p.c.head_dim);
  if (ws_bytes < l.total) return MTP_ERR_WORKSPACE;
  s.causal = p.causal;
  s.ctx_len = p.ctx_len, s.n_new = p.n_new, s.table = p.c.page_table;
  s.ks = p.c.k_scale, s.vs = p.c.v_scale;
  s.q = p.q, s.q_r = p.q_r, s.q_l = p.q_l, s.q_h = p.q_h;
  uint8_t* base = static_cast<uint8_t*>(ws);
  if (p.c.head_dim == 128)
    return p.c.dtype == MTP_E4M3 ? launch<128, true>(p, s, l, base, st) : launch<128, false>(p, s, l, base, st);
  return p.c.dtype == MTP_E4M3 ? launch<64, true>(p, s, l, base, st) : launch<64, false>(p, s, l, base, st);
}

}  // namespace mtp

using namespace mtp;

extern "C" size_t mtp_paged_attention_workspace_bytes(const mtp_paged_dims* dims, const mtp_paged_cache* cache) {
  if (!dims || paged_cache_check(cache, false) != MTP_OK) return 0;
  if (!paged_attn_sizes_ok(dims->R, dims->L, dims->n_heads, *cache)) return 0;
  if (item_ok(dims->R, dims->L, dims->n_heads, *cache)) return 0;
  return paged_attn_workspace_bytes(dims->R, dims->L, dims->n_heads, *cache);
}

extern "C" mtp_status mtp_paged_attention(const mtp_paged_dims* dims, const mtp_paged_cache* cache, const void* q,
                                          const int32_t* ctx_len, const int32_t* n_new, void* out, float* lse, void* ws,
                                          size_t ws_bytes, cudaStream_t st) {
  if (!dims) return MTP_ERR_INVALID_ARG;
  if (const mtp_status s = paged_cache_check(cache, true); s != MTP_OK) return s;
  if (!paged_attn_sizes_ok(dims->R, dims->L, dims->n_heads, *cache)) return MTP_ERR_SHAPE;
  const bool item = item_ok(dims->R, dims->L, dims->n_heads, *cache);
  if (!q || !ctx_len || !out || (!ws && !item)) return MTP_ERR_INVALID_ARG;
  if (!(dims->scale >= 0.f && dims->scale < 3.0e38f)) return MTP_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(ws)) return MTP_ERR_ALIGNMENT;
  if (((reinterpret_cast<uintptr_t>(ctx_len) | reinterpret_cast<uintptr_t>(n_new) | reinterpret_cast<uintptr_t>(lse)) & 3u))
    return MTP_ERR_ALIGNMENT;
  PagedAttn p;
  p.c = *cache;
  p.R = dims->R, p.L = dims->L, p.H = dims->n_heads;
  p.causal = dims->causal != 0;
  p.scale = dims->scale > 0.f ? dims->scale : 1.0f / sqrtf(static_cast<float>(cache->head_dim));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_h = dims->q_stride_h ? dims->q_stride_h : cache->head_dim;
  p.q_l = dims->q_stride_t ? dims->q_stride_t : static_cast<long long>(p.H) * cache->head_dim;
  p.q_r = dims->q_stride_r ? dims->q_stride_r : static_cast<long long>(p.L) * p.H * cache->head_dim;
  if (p.q_h % 8 || p.q_l % 8 || p.q_r % 8 || p.q_h < 0 || p.q_l < 0 || p.q_r < 0) return MTP_ERR_ALIGNMENT;
  if (!item && ws_bytes < paged_attn_workspace_bytes(p.R, p.L, p.H, p.c)) return MTP_ERR_WORKSPACE;
  // outputs are written while queries may still be looked at (rows of many tokens with values that are not finite)
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
  const unsigned long long q_span = 2ull * ((p.R - 1) * p.q_r + (p.L - 1) * p.q_l + (p.H - 1) * p.q_h + cache->head_dim);
  if (q0 < o0 + 2ull * p.R * p.L * p.H * cache->head_dim && o0 < q0 + q_span) return MTP_ERR_INVALID_ARG;
  p.ctx_len = ctx_len, p.n_new = n_new;
  p.o = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  if (item) {
    if (cache->head_dim == 128) return cache->dtype == MTP_E4M3 ? item_launch<128, true>(p, st) : item_launch<128, false>(p, st);
    return cache->dtype == MTP_E4M3 ? item_launch<64, true>(p, st) : item_launch<64, false>(p, st);
  }
  return paged_attn_launch(p, ws, ws_bytes, st);
}
