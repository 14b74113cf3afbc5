// Attention of a batch's new tokens over a prefix that all requests share and
// over each request's own cache.
//
// o = softmax(scale q [Kp; Kr]^T) [Vp; Vr] for every (request r, token i, head):
// Kp, Vp are the prefix, read once for the whole batch, Kr, Vr the request's own
// rows.  The softmax is taken in parts, (maximum m, sum l, output o) per part,
// and the parts joined at the end: o = Σ 2^(m_p - M) o_p / Σ 2^(m_p - M) l_p.
//
// Bound: HBM for few rows (the keys and values once: 4 hd bytes per key and
// head), the tensor cores once some 200 rows share a head's prefix (the weights' two
// parts make it three products instead of two).  Measured, call
// after call on inputs out of HBM: 32 requests, 56 heads of 128, 8192 shared and up
// to 256 own keys 77 us (4.5 TB/s); 6 requests, 64 heads over 8, 65000 shared keys
// 62 us (4.3 TB/s); 5 new tokens of 32 requests, 32 heads over 8, 8192 shared and up
// to 512 own keys 66 us (336 TFLOP/s).  Each further key of such a prefix costs its
// bytes at 6.9 TB/s in the first two cases, and 760 TFLOP/s (of the two products of the
// formula) in the third; the rest is three kernels' way to their first data, one after the other.
//
// All rows that see the same keys form one matrix: for the prefix the R L G rows
// (G = query heads per key head) of all requests, for a request's own cache its
// L G rows.  Work is cut into items -- (key head, rows) over the prefix, (request,
// key head, rows) over its cache -- and an item into blocks of keys.  The blocks of
// all items, weighted by their cost, are dealt to the CTAs in equal contiguous
// ranges, whatever the lengths; a CTA's range within an item (a segment) leaves
// records of partial results for each row, and a last kernel joins a row's records.
// Every kernel works the deal out from ctx_len.
//
// Many rows (prefix_attn_kernel): a row tile is as many whole requests as fit into
// 128 rows (or, with L G > 128, as many whole tokens of one request), so that one
// TMA box brings its q; an item has one or two row tiles, a block 128 keys.  TMA
// brings Q, K and V blocks, S = Q K^T and O += P V run on tcgen05 with S, P and O in
// TMEM, a softmax thread owns a row.  TMEM holds two tiles (S and P share columns),
// each with its own warpgroup.  With two row tiles both share every K/V block.  With
// one, the TMEM tiles take the blocks alternately, so that one's softmax runs under
// the other's products, each with a maximum, a sum and an output of its own (two
// records); the alternation runs on from segment to segment, so that short segments
// overlap as well.
//   softmax    warps 0-3 TMEM tile 0, warps 4-7 tile 1
//   K warp     walks the deal, publishes the segments in a ring and loads Q and K
//   V warp     loads V (as a second lane of the K warp it stood still whenever the
//              first was suspended in a wait: 4 us per short segment)
//   MMA warp   issues every product
// A last block is loaded as 64 rows where it has no more, and its products run over
// as many groups of 16 keys as it has.
//
// Few rows (small_attn_kernel): own caches with up to 32 rows per key head (8 beside a
// prefix on row tiles), and a prefix with up to 16 in all.  The kernel above spends
// 3.5 us on an item of one or two blocks, whatever its rows: the chain load, S, softmax,
// P V has two tiles to overlap with, and most of each is padding.  Here a warp takes 16
// rows and 16 keys with mma.sync.m16n8k16, and as many chains run as there are warps.
// Replayed from a graph, against the kernel above: own caches alone, 32 requests, 56
// heads, 256 keys 45 us instead of 69, 32 heads over 8 with 5 tokens (20 rows), 512 keys
// 26 instead of 32, 64 over 8 with 4 (32 rows) 31 instead of 34, 2048 keys 67 instead of
// 63.  Beside a prefix of 8192 keys on row tiles it is a launch more: up to 1024 keys, 56
// heads of one row 117 us instead of 145, 8 heads of 4 rows 38 and 39, 8 rows 45 and 43,
// 16 59 and 55, 20 71 and 65.  A prefix of 8192 keys, 56 heads and 16 rows 46 instead of
// 49, one row 42 instead of 47, 16 heads, 300 keys and 4 rows 5 instead of 9, but 8 heads
// of 16 rows on 65000 keys 55 instead of 52; with 32 rows 53 instead of 50.  It is launched
// beside the kernel above, whose CTAs fill an SM, and takes the SMs as they become free.
//
// Keys past a request's ctx_len may hold anything: their scores are replaced, and
// their V rows are cleared in shared memory (0 times NaN is NaN); rows of new tokens that
// an earlier token does not see may as well (see_again below).  P enters the second
// product as two bf16 parts, as in the draft step's own attention: its upper 16 bits
// (kept by the first part exactly) and the rest, rounded to bf16 (2^-15 of the weight
// together).  With one part the output was off by 1.4 of its own rounding; the second
// costs the tensor-bound case 66 us instead of 60, the others nothing.  Statistics, sums
// and records are fp32.  Every wait is bounded.
#include <cuda.h>

#include <algorithm>

#include "gemm_tc.cuh"
#include "mbarrier.cuh"
#include "prefix_attn.cuh"
#include "tcgen05.cuh"

MTP_DEFINE_ERROR_WORD(mtp_take_errors_prefix)

namespace mtp {
namespace {

constexpr int kRows = 128;   // rows per tile (MMA M, TMEM lanes)
constexpr int kKeys = 128;   // keys per block
constexpr float kStaleMaxLog2 = 8.0f;  // a running maximum is replaced only when exceeded by 2^8
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
// costs for the deal: a block with one row tile, with two, and what a segment
// of a request's own cache costs besides
constexpr int kCostOne = 6, kCostTwo = 11, kCostItem = 5;
// the small-row kernel: rows that it takes of a prefix, of an own cache alone and beside a
// prefix on row tiles; log2 of its blocks' keys, keys of a box
constexpr int kSmallPrefix = 16, kSmallOwn = 32, kSmallOwnBeside = 8, kSmallShift = 6, kSmallBox = 32, kSmallCost = 2, kSmallCostItem = 1;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tiled four-dimensional tensor copy global -> shared; x is the inner coordinate
__device__ __forceinline__ void tma_tile_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

__host__ __device__ constexpr int blocks_of(int keys, int shift) { return (keys + (1 << shift) - 1) >> shift; }

// Sizes of the two kinds of items (over the prefix, over a request's own cache),
// and where their records are.
struct Shape {
  int R, L, H, Hkv, G, P, T, causal;
  int tokens;        // new tokens of a request per row tile (L, or as many as fit)
  int groups;        // token groups per request: ceil(L / tokens)
  int requests;      // requests per row tile of the prefix
  int prefix_tiles, prefix_items, prefix_blocks;  // row tiles and items per key head; blocks
  int prefix_ctas;          // CTAs that share the prefix
  int own_items, own_cost, own_extra;  // row tiles of an own item: `groups` per key head; cost of a block, of an item besides
  int own_shift, own_ctas;  // log2 of a block's keys; CTAs that share the own caches
  int prefix_small, own_small;  // tiles of 16 rows where the prefix, the own caches are the small-row kernel's, else 0
  int prefix_per, own_per;  // parts that a segment leaves: 4 from the small-row kernel, else 2
  int prefix_rec, own_rec;  // record rows per row tile
  long long own_rec0;       // record row of the first own segment
  const int32_t* ctx_len;

  __device__ __forceinline__ int ctx(int r) const { return ctx_len ? min(max(ctx_len[r], 0), T) : T; }
  // cost of a block of prefix item k of a key head (with one row tile or two), where the item
  // starts in the head's, and what a head costs
  __host__ __device__ int prefix_cost(int k) const { return 2 * k + 1 < prefix_tiles ? kCostTwo : kCostOne; }
  __host__ __device__ long long prefix_at(int k) const { return static_cast<long long>(k) * prefix_blocks * kCostTwo; }
  __host__ __device__ long long prefix_head() const {
    return static_cast<long long>(prefix_blocks) * (prefix_tiles / 2 * kCostTwo + prefix_tiles % 2 * kCostOne);
  }
  // blocks of a request's own cache, cost of an item over them, and of all such items of the request
  __device__ __forceinline__ int own_blocks(int r) const { return blocks_of(ctx(r), own_shift); }
  __device__ __forceinline__ long long own_item(int blocks) const {
    return blocks > 0 ? static_cast<long long>(blocks) * own_cost + own_extra : 0;
  }
  __device__ __forceinline__ long long own_total(int blocks) const { return own_item(blocks) * Hkv * own_items; }
};

// A deal of the prefix's blocks, and one of the own caches': CTA k takes the
// blocks that start in [k total / n, (k + 1) total / n), n so small that every
// CTA gets a block.  The first block of an own item costs own_extra more.  Every
// CTA works on the prefix first and then on own caches: in one deal over both,
// the CTAs on the prefix kept the memory queues full, and those on short own
// items waited 6 us for each of their loads.
struct Deal {
  long long total;
  int n;
  __device__ __forceinline__ Deal(long long total_, int most_cost, int ctas) {
    total = total_;
    const long long most = total / most_cost;
    n = static_cast<int>(most < 1 ? 1 : most < ctas ? most : ctas);
  }
  __device__ __forceinline__ long long start(int k) const { return k * total / n; }
  // the CTA whose range the position is in
  __device__ __forceinline__ int owner(long long pos) const { return static_cast<int>(((pos + 1) * n + total - 1) / total - 1); }
  // blocks of an item (at `at`, its first block `extra` longer) that start before pos
  static __device__ __forceinline__ int before(long long pos, long long at, int extra, int cost, int blocks) {
    if (pos <= at) return 0;
    const long long later = pos - at - extra;  // block j >= 1 starts at extra + j cost
    const long long n = later > cost ? 1 + (later + cost - 1) / cost - 1 : 1;
    return static_cast<int>(n < blocks ? n : blocks);
  }
};

// a segment: blocks [b0, b0 + n) of an item
struct Segment {
  int kind;  // bit 0: own cache (else prefix), bit 1: two row tiles; -1 ends
  int head, item, r;
  int b0, n, keys;  // keys: of the item
  int rec;          // index of its records among the kind's
};
static_assert(sizeof(Segment) == 32, "two 16-byte words in the ring");

// take(segment), by a whole warp, for each segment of CTA `cta`'s part of the prefix's
// deal (if `prefix`), then of the own caches' (if `own`), until it returns false.
template <typename Take>
__device__ __forceinline__ bool each_segment(const Shape& sh, int cta, int lane, bool prefix, bool own, Take take) {
#pragma unroll 1
  for (int kind = prefix ? 0 : 1; kind < (own ? 2 : 1); ++kind) {
    long long total = 0;
    if (kind) {
      for (int r = lane; r < sh.R; r += 32) total += sh.own_total(sh.own_blocks(r));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    } else {
      total = sh.Hkv * sh.prefix_head();
    }
    const int extra = kind ? sh.own_extra : 0;
    const Deal deal(total, kind ? sh.own_cost + extra : sh.prefix_cost(0), kind ? sh.own_ctas : sh.prefix_ctas);
    if (total <= 0 || cta >= deal.n) continue;
    const long long from = deal.start(cta), to = deal.start(cta + 1);
    int r = 0;  // request that the range starts in, and where it starts
    long long start = 0;
    for (int base = 0; kind && base < sh.R; base += 32) {
      const long long c = base + lane < sh.R ? sh.own_total(sh.own_blocks(base + lane)) : 0;
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
    const int items = kind ? sh.own_items : sh.prefix_items, tiles = kind ? sh.groups : sh.prefix_tiles, per_r = sh.Hkv * items;
    for (; r < (kind ? sh.R : 1) && start < to; ++r) {
      const int keys = kind ? sh.ctx(r) : sh.P, nb = kind ? sh.own_blocks(r) : sh.prefix_blocks;
      if (nb == 0) continue;
      // items before item k of the request's (of the prefix's), by cost
      const long long own = kind ? sh.own_item(nb) : 0, head = kind ? own * items : sh.prefix_head();
      Segment s;
      s.r = r;
      s.keys = keys;
      const long long in = from > start ? from - start : 0;
      s.head = static_cast<int>(in / head);
      const long long left = in - s.head * head;
      s.item = static_cast<int>(min(kind ? left / own : left / sh.prefix_at(1), static_cast<long long>(items - 1)));
      long long at = start + s.head * head + (kind ? s.item * own : sh.prefix_at(s.item));
      for (int k = s.head * items + s.item; k < per_r && at < to; ++k) {
        const int block = kind ? sh.own_cost : sh.prefix_cost(s.item);
        const long long cost = static_cast<long long>(nb) * block + extra;
        // the item's blocks that start in [from, to)
        s.b0 = from <= at ? 0 : Deal::before(from, at, extra, block, nb);
        s.n = (to >= at + cost ? nb : Deal::before(to, at, extra, block, nb)) - s.b0;
        s.kind = kind | (2 * s.item + 1 < tiles ? 2 : 0);
        s.rec = r * per_r + k + cta;
        if (s.n > 0 && !take(s)) return false;
        at += cost;
        if (++s.item == items) {
          s.item = 0;
          ++s.head;
        }
      }
      start += head * sh.Hkv;
    }
  }
  return true;
}

template <int HD>
struct Cfg {
  static constexpr int kSoftmaxWarps = 8;
  static constexpr int kKWarp = 8, kMmaWarp = 9, kVWarp = 10;
  static constexpr int kThreads = 32 * 11;
  static constexpr int kChunks = HD / 64;
  static constexpr int kPiece = 128 * 128;       // one [128 rows x 128 B] swizzled piece
  static constexpr int kTileBytes = kRows * HD * 2;  // a Q, K or V tile
  static constexpr int kQTiles = HD == 64 ? 4 : 2;
  static constexpr int kKStages = HD == 64 ? 4 : 2;
  static constexpr int kVStages = HD == 64 ? 4 : 3;
  static constexpr int kOffK = kQTiles * kTileBytes;
  static constexpr int kOffV = kOffK + kKStages * kTileBytes;
  static constexpr int kOffBar = kOffV + kVStages * kTileBytes;
  static constexpr int kRing = 8;
  static constexpr int kReaders = 2 + kSoftmaxWarps;  // V warp, MMA warp, softmax warps
  // q, k, v full/empty; per tile s_full, p_full, pv_done, o_free; drain; segment ring full/empty
  static constexpr int kNumBars = 2 * (kQTiles + kKStages + kVStages) + 8 + 1 + 2 * kRing;
  static constexpr int kOffRing = (kOffBar + 8 * kNumBars + 15) / 16 * 16;
  static constexpr int kSmemBytes = kOffRing + 32 * kRing + 16;
  static constexpr uint32_t kColO = 256;
};

// tensor maps: q in boxes of a prefix tile's and of an own tile's rows, keys and
// values in boxes of 64 rows
struct Maps {
  CUtensorMap q_prefix, q_own, pk, pv, kk, kv;
};

template <int HD>
__global__ void __launch_bounds__(Cfg<HD>::kThreads, 1)
prefix_attn_kernel(const __grid_constant__ Maps maps, const Shape sh, float scale_log2, float2* __restrict__ rec_ml,
                   float* __restrict__ rec_o) {
  using C = Cfg<HD>;
  pdl_trigger();  // the joining kernel may start its setup
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t s0 = smem_u32(smem);
  if (s0 & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(&g_mtp_error_word, MTP_DEVERR_TIMEOUT);
    return;
  }
  const uint32_t sQ = s0, sK = s0 + C::kOffK, sV = s0 + C::kOffV, bar0 = s0 + C::kOffBar;
  auto q_full = [&](uint32_t i) { return bar0 + 8u * (i % C::kQTiles); };
  auto q_empty = [&](uint32_t i) { return bar0 + 8u * (C::kQTiles + i % C::kQTiles); };
  const uint32_t bark = bar0 + 16u * C::kQTiles;
  auto k_full = [&](uint32_t i) { return bark + 8u * (i % C::kKStages); };
  auto k_empty = [&](uint32_t i) { return bark + 8u * (C::kKStages + i % C::kKStages); };
  const uint32_t barv = bark + 16u * C::kKStages;
  auto v_full = [&](uint32_t i) { return barv + 8u * (i % C::kVStages); };
  auto v_empty = [&](uint32_t i) { return barv + 8u * (C::kVStages + i % C::kVStages); };
  const uint32_t barx = barv + 16u * C::kVStages;
  auto s_full = [&](int x) { return barx + 8u * x; };
  auto p_full = [&](int x) { return barx + 16u + 8u * x; };
  auto pv_done = [&](int x) { return barx + 32u + 8u * x; };
  auto o_free = [&](int x) { return barx + 48u + 8u * x; };
  const uint32_t drain_bar = barx + 64u;
  auto seg_full = [&](uint32_t i) { return barx + 72u + 8u * (i % C::kRing); };
  auto seg_empty = [&](uint32_t i) { return barx + 72u + 8u * (C::kRing + i % C::kRing); };
  int4* ring = reinterpret_cast<int4*>(smem + C::kOffRing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffRing + 32 * C::kRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  unsigned int* err = &g_mtp_error_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kQTiles; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 1);
    }
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(k_full(i), 1);
      mbar_init(k_empty(i), 1);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(v_full(i), 1);
      mbar_init(v_empty(i), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full(x), 1);
      mbar_init(p_full(x), kRows);
      mbar_init(pv_done(x), 1);
      mbar_init(o_free(x), kRows);
    }
    mbar_init(drain_bar, 1);
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(seg_full(i), 1);
      mbar_init(seg_empty(i), C::kReaders);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == C::kMmaWarp) tmem_alloc_cols(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_phase(bar, parity, abort_flag, err); };
  auto peek_segment = [&](uint32_t i, Segment& s) {
    if (!wait(seg_full(i), (i / C::kRing) & 1)) return false;
    const int4 a = ring[2 * (i % C::kRing)], b = ring[2 * (i % C::kRing) + 1];
    s = Segment{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    return s.kind >= 0;
  };
  // segment i, read by a warp: its slot is released once every lane has read it
  auto read_segment_warp = [&](uint32_t i, Segment& s) {
    if (!__all_sync(0xffffffffu, peek_segment(i, s))) return false;
    if (lane == 0) mbar_arrive1(seg_empty(i));
    return true;
  };

  if (warp == C::kKWarp || warp == C::kVWarp) {
    // ---------------- TMA producers: the deal, Q and K; V ----------------
    const bool kside = warp == C::kKWarp;
    const uint32_t stages = kside ? C::kKStages : C::kVStages;
    uint32_t g = 0, tile = 0;
    bool ok = true;
    auto wwait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
    // The whole warp walks along; lane 0 announces a copy's bytes and a lane per box issues it.
    auto load = [&](const Segment& s) {  // the segment's row tiles and blocks
      const bool own_kind = s.kind & 1;
      if (kside) {
        for (int x = 0; x < (s.kind & 2 ? 2 : 1); ++x, ++tile) {
          const uint32_t use = tile / C::kQTiles;
          if (use > 0 && !wwait(q_empty(tile), (use - 1) & 1)) { ok = false; return; }
          const int t = 2 * s.item + x;  // row tile
          const int first = sh.groups > 1 ? t / sh.groups : own_kind ? 0 : t;  // request (of a prefix tile)
          const int r = own_kind ? s.r : first * sh.requests, tok = (sh.groups > 1 ? t - first * sh.groups : 0) * sh.tokens;
          if (lane == 0) mbar_expect_tx(q_full(tile), (own_kind ? sh.own_rec : sh.prefix_rec) * HD * 2);
          __syncwarp();
          if (lane < C::kChunks)
            tma_tile_4d(sQ + (tile % C::kQTiles) * C::kTileBytes + lane * C::kPiece, own_kind ? &maps.q_own : &maps.q_prefix,
                        64 * lane, s.head * sh.G, tok, r, q_full(tile));
        }
      }
      for (int j = 0; j < s.n; ++j, ++g) {
        const uint32_t use = g / stages;
        if (use > 0 && !wwait(kside ? k_empty(g) : v_empty(g), (use - 1) & 1)) { ok = false; return; }
        const int key = (s.b0 + j) * kKeys;
        const uint32_t bar = kside ? k_full(g) : v_full(g);
        const bool half = s.keys - key <= kKeys / 2;  // the first 64 keys are all there are
        if (lane == 0) mbar_expect_tx(bar, half ? C::kTileBytes / 2 : C::kTileBytes);
        __syncwarp();
        if (lane < (half ? 1 : 2) * C::kChunks) {  // a box per 64 rows and 64 dimensions
          const int rows64 = lane / C::kChunks, c = lane % C::kChunks;
          const uint32_t dst = kside ? sK + (g % C::kKStages) * C::kTileBytes + c * C::kPiece + rows64 * 8192
                                     : sV + (g % C::kVStages) * C::kTileBytes + lane * 8192;
          const CUtensorMap* m = kside ? (own_kind ? &maps.kk : &maps.pk) : (own_kind ? &maps.kv : &maps.pv);
          tma_tile_4d(dst, m, 64 * c, s.head, key + 64 * rows64, s.r, bar);
        }
      }
    };
    if (kside) {
      uint32_t i = 0;
      auto publish = [&](const Segment& s) {
        if (i >= static_cast<uint32_t>(C::kRing) && !wwait(seg_empty(i), (i / C::kRing - 1) & 1)) { ok = false; return; }
        if (lane == 0) {
          ring[2 * (i % C::kRing)] = make_int4(s.kind, s.head, s.item, s.r);
          ring[2 * (i % C::kRing) + 1] = make_int4(s.b0, s.n, s.keys, s.rec);
          mbar_arrive1(seg_full(i));
        }
        ++i;
        if (s.kind >= 0) load(s);
      };
      const int cta = static_cast<int>(blockIdx.x);
      auto take = [&](const Segment& s) {
        publish(s);
        return ok;
      };
      each_segment(sh, cta, lane, !sh.prefix_small, !sh.own_small, take);
      Segment last{};
      last.kind = -1;
      if (ok) publish(last);
    } else {
      Segment s;
      for (uint32_t i = 0; ok && read_segment_warp(i, s); ++i) load(s);
    }
    // no copy may still be landing when the CTA leaves (matters only after an abort)
    for (uint32_t x = g > stages ? g - stages : 0; x < g; ++x)
      wait_drain(kside ? k_full(x) : v_full(x), (x / stages) & 1, kWaitLimitCycles);
    if (kside)
      for (uint32_t x = tile > C::kQTiles ? tile - C::kQTiles : 0; x < tile; ++x)
        wait_drain(q_full(x), (x / C::kQTiles) & 1, kWaitLimitCycles);
  } else if (warp == C::kMmaWarp) {
    // ---------------- MMA issuer ----------------
    // The whole warp walks along, so that what a product is given is uniform.  The row tiles'
    // blocks form one sequence, which takes the TMEM tiles alternately: S of a step, then P V
    // of the step before, whose softmax ran meanwhile.
    constexpr uint32_t idesc_o = idesc_bf16_f32(kRows, HD, 2);  // V read MN-major, P from TMEM
    auto wwait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
    uint32_t g = 0, tile = 0;     // key blocks and Q tiles consumed
    uint32_t turn = 0;            // blocks with one row tile so far: the TMEM tile is its parity
    // a bit per TMEM tile: parity of the S products issued; of the segments whose first P V has
    // been issued, and whether there are any
    uint32_t ns = 0, no = 0, had = 0;
    uint32_t i = 0;
    Segment s{};
    int tiles = 1, j = 0, t = 0;  // row tiles of the segment; block and row tile of the next step
    bool more = true, any = false;
    // the step whose P V is due: TMEM tile, ring block, groups of 16 keys, whether it is the segment's
    // first on that TMEM tile, and the block's last row tile
    bool due = false, due_first = false, due_last = false;
    int due_x = 0, due_keys = 0;
    uint32_t due_g = 0;
    while (more || due) {
      if (more && j == s.n) {
        more = read_segment_warp(i++, s);
        s.kind = __shfl_sync(0xffffffffu, s.kind, 0);
        s.b0 = __shfl_sync(0xffffffffu, s.b0, 0);
        s.n = __shfl_sync(0xffffffffu, s.n, 0);
        s.keys = __shfl_sync(0xffffffffu, s.keys, 0);
        tile += i > 1 ? tiles : 0;
        tiles = s.kind & 2 ? 2 : 1;
        j = 0;
      }
      const int x = tiles == 2 ? t : turn & 1;
      const int keys16 = (min(s.keys - (s.b0 + j) * kKeys, kKeys) + 15) / 16;
      const bool now = more && !(due && due_x == x);  // P of a due step may still be in S's columns
      if (now) {
        const uint32_t qt = tile + t;
        if (j == 0 && !wwait(q_full(qt), (qt / C::kQTiles) & 1)) break;
        if (t == 0 && !wwait(k_full(g), (g / C::kKStages) & 1)) break;
        tc_fence_after();
        const uint32_t idesc_s = idesc_bf16_f32(kRows, 16 * keys16, 0);
        const uint32_t q_at = sQ + (qt % C::kQTiles) * C::kTileBytes, k_at = sK + (g % C::kKStages) * C::kTileBytes;
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t off = (k >> 2) * C::kPiece + (k & 3) * 32;
          umma_bf16_ss_warp(tmem + 128u * x, sdesc_k_sw128(q_at + off), sdesc_k_sw128(k_at + off), idesc_s, k > 0);
        }
        umma_commit_warp(s_full(x));
        ns ^= 1u << x;
        any = true;
        if (t + 1 == tiles) umma_commit_warp(k_empty(g));
        if (j + 1 == s.n) umma_commit_warp(q_empty(qt));
      }
      if (due) {
        if (!wwait(v_full(due_g), (due_g / C::kVStages) & 1)) break;
        // P of this TMEM tile's last S but for the one just issued
        if (!wwait(p_full(due_x), ~ns >> due_x & 1)) break;
        if (due_first) {
          if ((had >> due_x & 1) && !wwait(o_free(due_x), ~no >> due_x & 1)) break;
          no ^= 1u << due_x;
          had |= 1u << due_x;
        }
        tc_fence_after();
        const uint32_t v_at = sV + (due_g % C::kVStages) * C::kTileBytes;
        auto product = [&](int k) {  // with both parts of P
          const uint32_t bv = v_at + (k >> 2) * (C::kChunks * 8192) + (k & 3) * 2048;
          const uint64_t v_desc = sdesc_mn_sw128(bv);
          const uint32_t p_at = tmem + 128u * due_x + 32u * (k >> 1) + 8u * (k & 1);
          umma_bf16_ts_warp(tmem + C::kColO + HD * due_x, p_at, v_desc, idesc_o, (!due_first || k > 0) ? 1u : 0u);
          umma_bf16_ts_warp(tmem + C::kColO + HD * due_x, p_at + 16, v_desc, idesc_o, 1u);
        };
        if (due_keys == kKeys / 16) {
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k) product(k);
        } else {
#pragma unroll 1
          for (int k = 0; k < due_keys; ++k) product(k);
        }
        umma_commit_warp(pv_done(due_x));
        if (due_last) umma_commit_warp(v_empty(due_g));
      }
      due = now;
      if (now) {
        due_x = x;
        due_keys = keys16;
        due_g = g;
        due_first = tiles == 2 ? j == 0 : j < 2;
        due_last = t + 1 == tiles;
        if (tiles == 1) ++turn;
        if (++t == tiles) {
          t = 0;
          ++j;
          ++g;
        }
      }
    }
    // every issued MMA has completed before TMEM is freed
    if (any) {
      umma_commit_warp(drain_bar);
      wait_drain(drain_bar, 0, kWaitLimitCycles);
    }
  } else {
    // ---------------- softmax: one row per thread of tile x ----------------
    const int x = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t colS = 128u * x, colO = C::kColO + HD * x;
    auto wwait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
    uint32_t n = 0;     // S products of this tile consumed
    uint32_t g = 0;     // key blocks of the CTA's earlier segments
    uint32_t turn = 0;  // ... of them with one row tile
    // this thread's row of a row tile: request and token from the tile's first
    const int in = row / (sh.tokens * sh.G), at_token = (row - in * sh.tokens * sh.G) / sh.G;
    Segment s;
    for (uint32_t i = 0; read_segment_warp(i, s); ++i) {
      const bool two = s.kind & 2, own = s.kind & 1;
      const int t = 2 * s.item + (two ? x : 0);
      const int first = sh.groups > 1 ? t / sh.groups : own ? 0 : t;
      const int token = (sh.groups > 1 ? t - first * sh.groups : 0) * sh.tokens + at_token;
      const int request = own ? s.r : first * sh.requests + in;
      const bool live = in < (own ? 1 : sh.requests) && request < sh.R && token < sh.L;
      const bool live_warp = __any_sync(0xffffffffu, live);
      // keys that the row sees
      int see = s.keys;
      if (own && sh.causal) see = max(0, s.keys - sh.L + 1 + token);
      // this tile's blocks of the segment: first, step, number
      const int j0 = two ? 0 : (turn ^ x) & 1, step = two ? 1 : 2;
      const int mine = two ? s.n : (s.n - j0 + 1) >> 1;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < mine; ++j, ++n) {
        if (!wwait(s_full(x), n & 1)) { ok = false; break; }
        tc_fence_after();
        const int jb = j0 + j * step;
        const int key0 = (s.b0 + jb) * kKeys;
        if (own && ((s.keys - key0) & 15) && s.keys - key0 < kKeys && (!two || x == 0)) {  // V rows past the end of the cache
          const uint32_t gu = g + jb;
          if (!wwait(v_full(gu), (gu / C::kVStages) & 1)) { ok = false; break; }
          if (row >= s.keys - key0 && row < (s.keys - key0 + 15) / 16 * 16) {
            uint8_t* v = smem + C::kOffV + (gu % C::kVStages) * C::kTileBytes + (row >> 6) * (C::kChunks * 8192) + (row & 63) * 128;
            for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
              for (int e = 0; e < 8; ++e) reinterpret_cast<uint4*>(v + c * 8192)[e] = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        if (live_warp) {
          // S is read twice, 32 keys at a time (held whole, its 128 registers and the loops' length
          // cost 3 us in 63): for the maximum, and for P, whose parts go over the columns that
          // have been read
          auto scores = [&](int c, float (&v)[32]) {
            tmem_ld32(lane_base + colS + 32 * c, v);
            const int left = see - key0 - 32 * c;
            if (left < 32) {  // keys the row sees only in part
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e >= left) v[e] = -INFINITY;
            }
          };
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float v[32];
            scores(c, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) mx4[e & 3] = fmaxf(mx4[e & 3], v[e]);
          }
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * scale_log2;
          // a new running maximum only when the block's exceeds the stale one by 2^8
          const float m_new = mx > m + kStaleMaxLog2 ? mx : m;
          const bool rescale = m_new != m && m != -INFINITY;
          const float neg = m_new == -INFINITY ? 0.f : -m_new;
          float rs4[4] = {};
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float v[32];
            scores(c, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              v[e] = ex2(fmaf(v[e], scale_log2, neg));
              rs4[e & 3] += v[e];
            }
            uint32_t high[16], low[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint32_t a = __float_as_uint(v[2 * e]), b = __float_as_uint(v[2 * e + 1]);
              high[e] = __byte_perm(a, b, 0x7632);
              low[e] = pack2_bf16(v[2 * e] - __uint_as_float(a & 0xFFFF0000u), v[2 * e + 1] - __uint_as_float(b & 0xFFFF0000u));
            }
            tmem_st16_nowait(lane_base + colS + 32 * c, high);
            tmem_st16_nowait(lane_base + colS + 32 * c + 16, low);
          }
          tmem_wait_st();
          if (__any_sync(0xffffffffu, rescale)) {  // O holds this segment's earlier P V: wait for the last one
            if (!wwait(pv_done(x), (n - 1) & 1)) { ok = false; break; }
            tc_fence_after();
            const float alpha = rescale ? ex2(m - m_new) : 1.f;
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
              float o[32];
              tmem_ld32(lane_base + colO + 32 * c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= alpha;
              tmem_st32(lane_base + colO + 32 * c, o);
            }
            l *= alpha;
          }
          m = m_new;
          l += (rs4[0] + rs4[1]) + (rs4[2] + rs4[3]);
        }
        tc_fence_before();
        mbar_arrive1(p_full(x));
      }
      if (!ok) break;
      g += s.n;
      if (!two) turn += s.n;
      // the segment's record of this row (of this tile's half of them with one row tile)
      const int rec_rows = own ? sh.own_rec : sh.prefix_rec;
      const long long at = (own ? sh.own_rec0 : 0) + (2ll * s.rec + x) * rec_rows + row;
      if (mine > 0) {
        if (!wwait(pv_done(x), (n - 1) & 1)) break;  // the segment's last P V
        tc_fence_after();
        if (live_warp) {
          // 4 x 4 transposes among four lanes, so that they write 64 bytes of one row at a time:
          // 8 lines per store instead of 32 half-written sectors (8000 cycles per segment)
#pragma unroll 1
          for (int c = 0; c < HD / 32; ++c) {
            float o[32];
            tmem_ld32(lane_base + colO + 32 * c, o);
#pragma unroll
            for (int q = 0; q < 32; q += 16) {
#pragma unroll
              for (int bit = 1; bit <= 2; bit <<= 1)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                  if (!(v & bit)) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      float &lo = o[q + 4 * v + e], &hi = o[q + 4 * (v | bit) + e];
                      const float other = __shfl_xor_sync(0xffffffffu, lane & bit ? lo : hi, bit);
                      if (lane & bit)
                        lo = other;
                      else
                        hi = other;
                    }
                  }
#pragma unroll
              for (int v = 0; v < 4; ++v)  // row v of the four, this lane's four columns
                if ((row & ~3) + v < rec_rows)
                  *reinterpret_cast<float4*>(rec_o + (at - (row & 3) + v) * HD + 32 * c + q + 4 * (lane & 3)) =
                      make_float4(o[q + 4 * v], o[q + 4 * v + 1], o[q + 4 * v + 2], o[q + 4 * v + 3]);
            }
          }
        }
        tc_fence_before();
        mbar_arrive1(o_free(x));
      }
      if (live) rec_ml[at] = make_float2(m, l);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMmaWarp) tmem_free_cols(tmem, 512);
}

// ---------------------------------------------------------------------------
// Own caches with few rows per key head
// ---------------------------------------------------------------------------
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the 16-byte piece with element (row, col) of rows of 64 elements that TMA wrote with the 128-byte swizzle
__device__ __forceinline__ uint32_t swz(uint32_t box, int row, int col) {
  return box + row * 128 + ((((col >> 3) ^ row) & 7) << 4);
}

// A CTA's ring holds blocks of keys and, with a segment's first block, its q.  Four
// warps have 16 rows, each 16 keys of a block, with a maximum, a sum and an output of
// its own: four parts per segment.  (Joined over shared memory first, they cost 2400
// cycles a segment, two waits for one another, against 300.)
template <int HD, int MT>
struct Small {
  static constexpr int kWarps = 4 * MT;
  static constexpr int kThreads = 32 * (kWarps + 1);  // and a warp that walks the deals and loads
  static constexpr int kCtas = 2 / MT;                // per SM
  static constexpr int kBlock = 1 << kSmallShift;
  static constexpr int kChunks = HD / 64, kChunkBytes = kBlock * 128;
  static constexpr int kTileBytes = kBlock * HD * 2;  // K or V of a block
  static constexpr int kOffQ = 2 * kTileBytes, kQChunk = 16 * MT * 128;
  static constexpr int kStageBytes = kOffQ + kChunks * kQChunk;
  static constexpr int kStages = 108 * 1024 * MT / kStageBytes;
  static constexpr int kOffBlocks = kStages * kStageBytes;       // what each stage holds
  static constexpr int kOffBar = kOffBlocks + 16 * kStages;      // full and empty per stage, abort flag
  static constexpr int kSmemBytes = kOffBar + 16 * kStages + 16;
};
// 16 rows of a warp
template <int HD>
struct SmallRows {
  uint32_t qa[HD / 16][4];
  float mx[2], sum[2], o[HD / 8][4];
  int hidden[2];  // keys at the item's end that rows g and g + 8 do not see
};
// ... and 16 keys of a block, `key` on, the item's last `left`
template <int HD>
__device__ __forceinline__ void small_block(SmallRows<HD>& w, uint32_t k_at, uint32_t v_at, int key, int left, float scale_log2, int lane) {
  constexpr int kChunk = Small<HD, 1>::kChunkBytes;
  const int t4 = lane & 3;
  float sc[2][4] = {};
#pragma unroll
  for (int k = 0; k < HD / 16; ++k) {  // keys 0-7 and 8-15, 16 dimensions
    uint32_t f[4];
    ldsm_x4(swz(k_at + (k >> 2) * kChunk, key + (lane & 7) + 8 * (lane >> 4), 16 * (k & 3) + (lane & 8)), f);
    mma_16816(sc[0], w.qa[k], f[0], f[1]);
    mma_16816(sc[1], w.qa[k], f[2], f[3]);
  }
  uint32_t pa[4], pl[4];  // P's two parts
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int see = left - w.hidden[e];  // of these keys
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = 8 * (i >> 1) + 2 * t4 + (i & 1) < see ? sc[i >> 1][2 * e + (i & 1)] : -INFINITY;
    float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)) * scale_log2;
    // a new running maximum only when the block's exceeds the stale one by 2^8
    const float now = top > w.mx[e] + kStaleMaxLog2 ? top : w.mx[e];
    const float neg = now == -INFINITY ? 0.f : -now;
    const float alpha = now == w.mx[e] ? 1.f : ex2(w.mx[e] + neg);
    w.mx[e] = now;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ex2(fmaf(v[i], scale_log2, neg));
    w.sum[e] = w.sum[e] * alpha + ((v[0] + v[1]) + (v[2] + v[3]));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      pa[e + 2 * i] = pack2_bf16(v[2 * i], v[2 * i + 1]);
      const float2 f = unpack2_bf16(pa[e + 2 * i]);
      pl[e + 2 * i] = pack2_bf16(v[2 * i] - f.x, v[2 * i + 1] - f.y);
    }
    if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
      for (int n = 0; n < HD / 8; ++n) {
        w.o[n][2 * e] *= alpha;
        w.o[n][2 * e + 1] *= alpha;
      }
    }
  }
#pragma unroll
  for (int n = 0; n < HD / 16; ++n) {
    uint32_t f[4];
    ldsm_x4_t(swz(v_at + (n >> 2) * kChunk, key + (lane & 15), 16 * (n & 3) + 8 * (lane >> 4)), f);
    mma_16816(w.o[2 * n], pa, f[0], f[1]);
    mma_16816(w.o[2 * n + 1], pa, f[2], f[3]);
    mma_16816(w.o[2 * n], pl, f[0], f[1]);
    mma_16816(w.o[2 * n + 1], pl, f[2], f[3]);
  }
}
enum : int { kFirst = 1, kLast = 2, kOwn = 4 };

template <int HD, int MT>
__global__ void __launch_bounds__(Small<HD, MT>::kThreads, Small<HD, MT>::kCtas)
small_attn_kernel(const __grid_constant__ Maps maps, const Shape sh, float scale_log2, float2* __restrict__ rec_ml,
                  float* __restrict__ rec_o, int after) {
  using C = Small<HD, MT>;
  pdl_trigger();
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t s0 = smem_u32(smem), bar0 = s0 + C::kOffBar;
  if (s0 & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(&g_mtp_error_word, MTP_DEVERR_TIMEOUT);
    return;
  }
  auto full = [&](uint32_t g) { return bar0 + 8u * (g % C::kStages); };
  auto empty = [&](uint32_t g) { return bar0 + 8u * (C::kStages + g % C::kStages); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffBar + 16 * C::kStages);
  int4* blocks = reinterpret_cast<int4*>(smem + C::kOffBlocks);  // keys of the item (< 0 ends), first key, flags, record
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), C::kWarps);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  auto wwait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_phase(bar, parity, abort_flag, &g_mtp_error_word));
  };
  if (warp == C::kWarps) {
    uint32_t g = 0;
    auto stage_free = [&]() { return g < C::kStages || wwait(empty(g), (g / C::kStages - 1) & 1); };
    auto take = [&](const Segment& s) {
      const bool own = s.kind & 1;
      for (int j = 0; j < s.n; ++j, ++g) {
        if (!stage_free()) return false;
        const int key0 = (s.b0 + j) * C::kBlock, boxes = min((s.keys - key0 + kSmallBox - 1) / kSmallBox, C::kBlock / kSmallBox);
        const uint32_t at = s0 + (g % C::kStages) * C::kStageBytes, bar = full(g);
        if (lane == 0) {
          blocks[g % C::kStages] =
              make_int4(s.keys, key0, (j == 0 ? kFirst : 0) | (j + 1 == s.n ? kLast : 0) | (own ? kOwn : 0), s.rec);
          mbar_expect_tx(bar, boxes * kSmallBox * HD * 4 + (j == 0 ? (own ? sh.own_rec : sh.prefix_rec) * HD * 2 : 0));
        }
        __syncwarp();
        constexpr int kPer = C::kBlock / kSmallBox * C::kChunks;  // boxes of K, of V
        const int i = lane % kPer, c = i % C::kChunks, b = i / C::kChunks;
        if (lane < 2 * kPer) {
          const bool k = lane < kPer;
          if (b < boxes)
            tma_tile_4d(at + (k ? 0 : C::kTileBytes) + c * C::kChunkBytes + b * (kSmallBox * 128),
                        own ? (k ? &maps.kk : &maps.kv) : (k ? &maps.pk : &maps.pv), 64 * c, s.head, key0 + b * kSmallBox, s.r, bar);
        } else if (j == 0 && lane < 2 * kPer + C::kChunks) {
          const int cq = lane - 2 * kPer;
          tma_tile_4d(at + C::kOffQ + cq * C::kQChunk, own ? &maps.q_own : &maps.q_prefix, 64 * cq, s.head * sh.G, 0, s.r, bar);
        }
      }
      return true;
    };
    const int cta = static_cast<int>(blockIdx.x);
    const bool ok = each_segment(sh, cta, lane, sh.prefix_small, sh.own_small, take);
    if (ok && stage_free()) {
      if (lane == 0) {
        blocks[g % C::kStages] = make_int4(-1, 0, 0, 0);
        mbar_arrive1(full(g));
      }
      ++g;
    }
    // no copy may still be landing when the CTA leaves (matters only after an abort)
    for (uint32_t x = g > C::kStages ? g - C::kStages : 0; x < g; ++x) wait_drain(full(x), (x / C::kStages) & 1, kWaitLimitCycles);
  } else {
    const int gr = lane >> 2, t4 = lane & 3;
    const int first = warp & 4, row0 = 4 * first;  // the first of the four warps, their first row
    const int key = 16 * (warp - first);           // a block's first key for this warp
    SmallRows<HD> w;
    for (uint32_t g = 0;; ++g) {
      if (!wwait(full(g), (g / C::kStages) & 1)) break;
      const int4 b = blocks[g % C::kStages];
      if (b.x < 0) break;
      const uint32_t k_at = s0 + (g % C::kStages) * C::kStageBytes, v_at = k_at + C::kTileBytes;
      const bool own = b.z & kOwn;
      const int rows = own ? sh.own_rec : sh.prefix_rec;
      if (b.z & kFirst) {
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)
          ldsm_x4(swz(k_at + C::kOffQ + (k >> 2) * C::kQChunk, row0 + (lane & 15), 16 * (k & 3) + 8 * (lane >> 4)), w.qa[k]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w.mx[e] = -INFINITY;
          w.sum[e] = 0.f;
          const int row = row0 + 8 * e + gr;
          w.hidden[e] = row >= rows ? 0x40000000 : own && sh.causal ? sh.L - 1 - row / sh.G : 0;
        }
#pragma unroll
        for (int n = 0; n < HD / 8; ++n) w.o[n][0] = w.o[n][1] = w.o[n][2] = w.o[n][3] = 0.f;
      }
      const int left = b.x - b.y - key;  // the item's keys from this warp's first on
      if (left > 0) {
        if (left < 16) {  // V rows past the end, by each warp that reads them (the same zeros)
          uint8_t* v = smem + (v_at - s0) + (key + left) * 128;
          for (int i = lane; i < (16 - left) * 8 * C::kChunks; i += 32)
            *reinterpret_cast<uint4*>(v + (i % C::kChunks) * C::kChunkBytes + i / C::kChunks * 16) = make_uint4(0, 0, 0, 0);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // a later copy overwrites them
          __syncwarp();
        }
        small_block<HD>(w, k_at, v_at, key, left, scale_log2, lane);
      }
      if (b.z & kLast) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w.sum[e] += __shfl_xor_sync(0xffffffffu, w.sum[e], 1);
          w.sum[e] += __shfl_xor_sync(0xffffffffu, w.sum[e], 2);
        }
        // a part of the segment's records per warp with the same rows
        const long long rec = (own ? sh.own_rec0 : 0) + (4ll * b.w + (warp & 3)) * rows + row0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * e + gr;
          if (row0 + row < rows) {
            if (t4 == 0) rec_ml[rec + row] = make_float2(w.mx[e], w.sum[e]);
            if (w.sum[e] != 0.f) {  // a part without a key is not read
              float* to = rec_o + (rec + row) * HD + 2 * t4;
#pragma unroll
              for (int n = 0; n < HD / 8; ++n) *reinterpret_cast<float2*>(to + 8 * n) = make_float2(w.o[n][2 * e], w.o[n][2 * e + 1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive1(empty(g));
    }
  }
  __syncthreads();
  if (after) pdl_wait();  // complete only once the kernel before is, which it may run beside
}

// Joins the records of one (request, token, head) per warp, or with kSplit = 4 per CTA,
// each warp every fourth of them: a lane per record for the maxima and the weights, then
// lanes over the head's dimensions.  The deals come from
// ctx_len alone, so all of that runs under the kernels before; what is left then is one
// chain of loads, in which the first records' outputs are asked for with their maxima.
constexpr int kJoinWarps = 4;
// Up to this many rows per SM have a CTA each: 128 rows (65000 keys) 56 us a call instead of 68,
// 512 60 instead of 61; 1792 (8192 keys) 93 instead of 90, 5120 83 instead of 72.
constexpr int kSplitRows = 8;
template <int kD>
__device__ __forceinline__ void store_row(__nv_bfloat16* to, const float (&acc)[kD], float inv) {
  if constexpr (kD == 4)
    *reinterpret_cast<uint2*>(to) = make_uint2(pack2_bf16(acc[0] * inv, acc[1] * inv), pack2_bf16(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(to) = pack2_bf16(acc[0] * inv, acc[1] * inv);
}
// what the join needs of the own caches where it takes them up itself (see_again)
struct OwnRows {
  const __nv_bfloat16 *q, *k, *v;
  long long q_r, q_l, q_h, k_r, k_t, k_h;
  float scale_log2;
};
// kD consecutive bf16
template <int kD>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* p, float (&f)[kD]) {
#pragma unroll
  for (int d = 0; d < kD; d += 2) {
    const float2 v = unpack2_bf16(*reinterpret_cast<const uint32_t*>(p + d));
    f[d] = v.x;
    f[d + 1] = v.y;
  }
}
// The output of a row (request r, token i, head h) over the prefix's n0 records and the first
// `see` rows of its own cache, one at a time, by a warp.  The products take 16 keys of all the
// rows together, with a weight of 0 where a row does not see a key, and 0 times the NaN or the
// infinity that a later token's value may hold (a padded draft's) is NaN.  The maxima and
// sums are free of it; where an output is not finite, it is worked out again from what it sees
// (5 tokens of 32 requests, 512 own keys, half of the requests padded: 191 us instead of 70).
// (A function of its own that writes the row, in a form of the join for such calls: within
// it, or in every form, it cost the others 1 to 1.5 us.)
template <int kD>
__device__ __noinline__ void see_again(const OwnRows& own, const float2* rec_ml, const float* rec_o, long long at0, int step0,
                                       int n0, int r, int i, int h, int head, int see, float M, float L, __nv_bfloat16* to) {
  const int lane = threadIdx.x & 31;
  float acc[kD];
#pragma unroll
  for (int d = 0; d < kD; ++d) acc[d] = 0.f;
#pragma unroll 1
  for (int p = 0; p < n0; ++p) {
    const long long at = at0 + static_cast<long long>(p) * step0;
    const float2 ml = rec_ml[at];
    if (!(ml.y > 0.f)) continue;
    const float w = ex2(ml.x - M);
#pragma unroll
    for (int d = 0; d < kD; ++d) acc[d] = fmaf(w, rec_o[at * (32 * kD) + lane * kD + d], acc[d]);
  }
  float q[kD];
  load_bf16<kD>(own.q + r * own.q_r + i * own.q_l + h * own.q_h + lane * kD, q);
  const long long at = r * own.k_r + head * own.k_h + lane * kD;
  constexpr int kU = 4;  // keys whose loads and sums are under way together
#pragma unroll 1
  for (int j0 = 0; j0 < see; j0 += kU) {
    float v[kU][kD], s[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float k[kD];
      const long long row = at + min(j0 + u, see - 1) * own.k_t;
      load_bf16<kD>(own.k + row, k);
      load_bf16<kD>(own.v + row, v[u]);
      s[u] = 0.f;
#pragma unroll
      for (int d = 0; d < kD; ++d) s[u] = fmaf(q[d], k[d], s[u]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const float w = ex2(fmaf(warp_sum(s[u]), own.scale_log2, -M));
      if (j0 + u < see) {
#pragma unroll
        for (int d = 0; d < kD; ++d) acc[d] = fmaf(w, v[u][d], acc[d]);
      }
    }
  }
  store_row<kD>(to, acc, 1.f / L);
}

template <int HD, int kSplit, bool kLater>
__global__ void __launch_bounds__(32 * kJoinWarps)
prefix_join_kernel(const Shape sh, const __grid_constant__ OwnRows own, const float2* __restrict__ rec_ml,
                   const float* __restrict__ rec_o, __nv_bfloat16* __restrict__ o, float* __restrict__ lse, float* __restrict__ rec, long long rec_stride) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  static_assert(kSplit == 1 || kSplit == kJoinWarps, "a row per warp, or per CTA");
  const int r = blockIdx.y, item = kSplit > 1 ? blockIdx.x : blockIdx.x * kJoinWarps + warp;
  if (item >= sh.L * sh.H) {
    pdl_wait();
    return;
  }
  const int i = item / sh.H, h = item - i * sh.H, head = h / sh.G, hg = h - head * sh.G;
  const int group = i / sh.tokens, in = (i - group * sh.tokens) * sh.G + hg;  // row of a tile that starts at the request
  // parts of a kind: `per` a segment from record row `at` on, `step` rows apart
  long long at0 = 0, at1 = 0;
  int n0 = 0, n1 = 0, step0 = 0, step1 = 0;
  if (sh.prefix_blocks > 0) {
    const Deal shared(sh.Hkv * sh.prefix_head(), sh.prefix_cost(0), sh.prefix_ctas);
    const int tile = r / sh.requests * sh.groups + group, row = r % sh.requests * sh.tokens * sh.G + in;
    const bool two = (tile | 1) < sh.prefix_tiles;
    const int k = head * sh.prefix_items + tile / 2;
    const long long at = head * sh.prefix_head() + sh.prefix_at(tile / 2);
    const int a = shared.owner(at), b = shared.owner(at + static_cast<long long>(sh.prefix_blocks - 1) * sh.prefix_cost(tile / 2));
    // two row tiles leave a part each and this row has every other one, else they are all this row's
    n0 = (b - a + 1) * (two ? 1 : sh.prefix_per);
    step0 = (two ? 2 : 1) * sh.prefix_rec;
    at0 = (static_cast<long long>(sh.prefix_per) * (k + a) + (two ? tile & 1 : 0)) * sh.prefix_rec + row;
  }
  const int nb = sh.own_blocks(r);
  if (nb > 0) {
    // cost of all requests' own caches, and of those before r
    long long all = 0, prev = 0;
    for (int q = lane; q < sh.R; q += 32) {
      const long long c = sh.own_total(sh.own_blocks(q));
      all += c;
      if (q < r) prev += c;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, d);
      prev += __shfl_xor_sync(0xffffffffu, prev, d);
    }
    const Deal each(all, sh.own_cost + sh.own_extra, sh.own_ctas);
    const bool two = (group | 1) < sh.groups;
    const int k = head * sh.own_items + group / 2;
    const long long cost = sh.own_item(nb), at = prev + k * cost;
    const int a = each.owner(at), b = each.owner(nb > 1 ? at + cost - sh.own_cost : at);
    n1 = (b - a + 1) * (two ? 1 : sh.own_per);
    step1 = (two ? 2 : 1) * sh.own_rec;
    at1 = sh.own_rec0 +
          (static_cast<long long>(sh.own_per) * (r * sh.Hkv * sh.own_items + k + a) + (two ? group & 1 : 0)) * sh.own_rec + in;
  }
  const int w0 = kSplit > 1 ? warp : 0, parts = (n0 + n1 - w0 + kSplit - 1) / kSplit;  // this warp's
  constexpr int kD = HD / 32;
  float acc[kD], L = 0.f, M = -INFINITY;  // L: this lane's records
#pragma unroll
  for (int d = 0; d < kD; ++d) acc[d] = 0.f;
  pdl_wait();  // the records are earlier kernels'
  for (int p0 = 0; p0 < parts; p0 += 32) {
    const int p = min(p0 + lane, parts - 1) * kSplit + w0, n = min(32, parts - p0);
    const long long at = p < n0 ? at0 + static_cast<long long>(p) * step0 : at1 + static_cast<long long>(p - n0) * step1;
    float v[8][kD];
    auto fetch = [&](int e0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float* src = rec_o + __shfl_sync(0xffffffffu, at, min(e0 + e, n - 1)) * HD + lane * kD;
        if constexpr (kD == 4) {
          const float4 f = *reinterpret_cast<const float4*>(src);
          v[e][0] = f.x; v[e][1] = f.y; v[e][2] = f.z; v[e][3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(src);
          v[e][0] = f.x; v[e][1] = f.y;
        }
      }
    };
    const float2 ml = rec_ml[at];
    fetch(0);
    const bool used = lane < n && (ml.y > 0.f || ml.y != ml.y);  // a part without a key has left no output
    const float now = fmaxf(M, warp_max(used ? ml.x : -INFINITY));
    const float z = now == -INFINITY ? 0.f : now, w = used ? ex2(ml.x - z) : 0.f;
    if (p0 > 0) {
      const float alpha = now == M ? 1.f : ex2(M - z);
      L *= alpha;
#pragma unroll
      for (int d = 0; d < kD; ++d) acc[d] *= alpha;
    }
    M = now;
    if (used) L += w * ml.y;
    for (int e0 = 0;;) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float we = __shfl_sync(0xffffffffu, w, min(e0 + e, 31));
        if (e0 + e < n && we != 0.f) {
#pragma unroll
          for (int d = 0; d < kD; ++d) acc[d] = fmaf(we, v[e][d], acc[d]);
        }
      }
      if ((e0 += 8) >= n) break;
      fetch(e0);
    }
  }
  L = warp_sum(L);
  if constexpr (kSplit > 1) {
    __shared__ float s_m[kSplit], s_l[kSplit], s_o[kSplit][HD];
    if (lane == 0) {
      s_m[warp] = M;
      s_l[warp] = L;
    }
#pragma unroll
    for (int d = 0; d < kD; ++d) s_o[warp][lane * kD + d] = acc[d];
    __syncthreads();
    if (warp != 0) return;
    L = 0.f;
#pragma unroll
    for (int d = 0; d < kD; ++d) acc[d] = 0.f;
#pragma unroll
    for (int w = 0; w < kSplit; ++w) M = fmaxf(M, s_m[w]);
    const float z = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < kSplit; ++w) {
      const float f = ex2(s_m[w] - z);
      L += f * s_l[w];
#pragma unroll
      for (int d = 0; d < kD; ++d) acc[d] += f * s_o[w][lane * kD + d];
    }
  }
  const long long out = (static_cast<long long>(r) * sh.L + i) * sh.H + h;
  if (rec) {
    float* to = rec + out * rec_stride;
    if (lane == 0) {
      to[0] = M * kLn2;
      to[1] = L;
    }
#pragma unroll
    for (int d = 0; d < kD; ++d) to[2 + lane * kD + d] = acc[d];
    return;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;  // a row that sees no key: zeros
  __nv_bfloat16* to = o + out * HD + lane * kD;
  store_row<kD>(to, acc, inv);
  if (lse && lane == 0) lse[out] = L == 0.f ? -INFINITY : M * kLn2 + logf(L);
  if constexpr (kLater) {
    if (nb > 0 && i + 1 < sh.L) {  // rows of later tokens stood beside this one's
      bool odd = false;
#pragma unroll
      for (int d = 0; d < kD; ++d) odd |= !(fabsf(acc[d]) < INFINITY);
      if (__any_sync(0xffffffffu, odd) && L == L)
        see_again<kD>(own, rec_ml, rec_o, at0, step0, n0, r, i, h, head, max(0, sh.ctx(r) - sh.L + 1 + i), M, L, to);
    }
  }
}

inline size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

Shape make_shape(int R, int L, int H, int Hkv, int P, int T) {
  Shape s{};
  s.R = R;
  s.L = L;
  s.H = H;
  s.Hkv = Hkv;
  s.G = H / Hkv;
  s.P = P;
  s.T = T;
  s.tokens = std::min(L, kRows / s.G);
  s.groups = (L + s.tokens - 1) / s.tokens;
  s.requests = s.groups > 1 ? 1 : std::min(R, kRows / (L * s.G));
  s.prefix_tiles = (R + s.requests - 1) / s.requests * s.groups;
  s.prefix_items = (s.prefix_tiles + 1) / 2;
  s.own_items = (s.groups + 1) / 2;
  s.own_rec = s.tokens * s.G;
  s.prefix_rec = s.requests * s.own_rec;
  s.prefix_small = P > 0 && static_cast<long long>(R) * L * s.G <= kSmallPrefix;
  const int most = P > 0 && !s.prefix_small ? kSmallOwnBeside : kSmallOwn;
  s.own_small = T > 0 && static_cast<long long>(L) * s.G <= most ? (L * s.G + 15) / 16 : 0;
  s.prefix_per = s.prefix_small ? 4 : 2;
  s.own_per = s.own_small ? 4 : 2;
  s.prefix_blocks = blocks_of(P, s.prefix_small ? kSmallShift : 7);
  s.own_shift = s.own_small ? kSmallShift : 7;
  s.own_cost = s.own_small ? kSmallCost : s.groups > 1 ? kCostTwo : kCostOne;
  s.own_extra = s.own_small ? kSmallCostItem : kCostItem;
  const int sms = sm_count_current();
  auto ctas = [&](int small, long long blocks) { return static_cast<int>(std::min<long long>(small == 1 ? 2 * sms : sms, blocks)); };
  s.prefix_ctas = ctas(s.prefix_small, static_cast<long long>(Hkv) * s.prefix_items * s.prefix_blocks);
  s.own_ctas = ctas(s.own_small, static_cast<long long>(R) * Hkv * s.own_items * blocks_of(T, s.own_shift));
  s.own_rec0 = s.prefix_per * (static_cast<long long>(Hkv) * s.prefix_items + s.prefix_ctas) * s.prefix_rec;
  return s;
}
long long record_rows(const Shape& s) {
  return s.own_rec0 + s.own_per * (static_cast<long long>(s.R) * s.Hkv * s.own_items + s.own_ctas) * s.own_rec;
}

// rows as (dimension, head, token, request); boxes of 64 dimensions of heads x tokens x requests
bool row_map(CUtensorMap* m, const void* p, int hd, int heads, int tokens, int requests, long long s_h, long long s_t,
             long long s_r, int box_h, int box_t, int box_r) {
  const uint64_t dims[4] = {static_cast<uint64_t>(hd), static_cast<uint64_t>(heads), static_cast<uint64_t>(tokens),
                            static_cast<uint64_t>(requests)};
  const uint64_t strides[3] = {static_cast<uint64_t>(s_h) * 2, static_cast<uint64_t>(s_t) * 2, static_cast<uint64_t>(s_r) * 2};
  const uint32_t boxes[4] = {64, static_cast<uint32_t>(box_h), static_cast<uint32_t>(box_t), static_cast<uint32_t>(box_r)};
  return tensor_map_bf16_4d(m, p, dims, strides, boxes);
}

template <int HD, int MT>
mtp_status launch_small(const Shape& s, const Maps& m, float scale_log2, float2* ml, float* ro, bool after, cudaStream_t st) {
  using C = Small<HD, MT>;
  static PerDevice attr;
  if (!smem_limit(attr, small_attn_kernel<HD, MT>, C::kSmemBytes)) return MTP_ERR_CUDA;
  const int ctas = std::max(s.prefix_small ? s.prefix_ctas : 0, s.own_small ? s.own_ctas : 0);
  if (after)
    MTP_CUDA_TRY(launch_pdl(small_attn_kernel<HD, MT>, dim3(ctas), dim3(C::kThreads), C::kSmemBytes, st, m, s, scale_log2, ml, ro, 1));
  else
    small_attn_kernel<HD, MT><<<ctas, C::kThreads, C::kSmemBytes, st>>>(m, s, scale_log2, ml, ro, 0);
  note_launch();
  MTP_LAUNCH_CHECK();
  return MTP_OK;
}

template <int HD>
mtp_status launch(const PrefixAttn& p, const Shape& s, float2* ml, float* ro, cudaStream_t st) {
  using C = Cfg<HD>;
  static PerDevice attr;
  if (!smem_limit(attr, prefix_attn_kernel<HD>, C::kSmemBytes)) return MTP_ERR_CUDA;
  Maps m{};
  const int pbox = s.prefix_small ? kSmallBox : 64, box = s.own_small ? kSmallBox : 64;
  if (p.P > 0 &&
      (!row_map(&m.q_prefix, p.q, HD, p.H, p.L, p.R, p.q_h, p.q_l, p.q_r, s.G, s.tokens, s.requests) ||
       !row_map(&m.pk, p.pk, HD, p.Hkv, p.P, 1, p.p_h, p.p_t, p.p_t, 1, pbox, 1) ||
       !row_map(&m.pv, p.pv, HD, p.Hkv, p.P, 1, p.p_h, p.p_t, p.p_t, 1, pbox, 1)))
    return MTP_ERR_CUDA;
  if (p.T > 0 &&
      (!row_map(&m.q_own, p.q, HD, p.H, p.L, p.R, p.q_h, p.q_l, p.q_r, s.G, s.tokens, 1) ||
       !row_map(&m.kk, p.kk, HD, p.Hkv, p.T, p.R, p.k_h, p.k_t, p.k_r, 1, box, 1) ||
       !row_map(&m.kv, p.kv, HD, p.Hkv, p.T, p.R, p.k_h, p.k_t, p.k_r, 1, box, 1)))
    return MTP_ERR_CUDA;
  const float scale = p.scale > 0.f ? p.scale : 1.0f / sqrtf(static_cast<float>(HD));
  const float scale_log2 = scale * kLog2e;
  const bool tiles = (p.P > 0 && !s.prefix_small) || (p.T > 0 && !s.own_small);
  if (tiles) {
    const int ctas = std::max(s.prefix_small ? 0 : s.prefix_ctas, s.own_small ? 0 : s.own_ctas);
    prefix_attn_kernel<HD><<<ctas, C::kThreads, C::kSmemBytes, st>>>(m, s, scale_log2, ml, ro);
    note_launch();
    MTP_LAUNCH_CHECK();
  }
  if (s.prefix_small || s.own_small) {
    const mtp_status e = std::max(s.prefix_small, s.own_small) == 1 ? launch_small<HD, 1>(s, m, scale_log2, ml, ro, tiles, st)
                                                                    : launch_small<HD, 2>(s, m, scale_log2, ml, ro, tiles, st);
    if (e != MTP_OK) return e;
  }
  // few rows: their records by four warps each
  const bool split = static_cast<long long>(s.R) * s.L * s.H <= kSplitRows * sm_count_current();
  const dim3 grid(split ? s.L * s.H : (s.L * s.H + kJoinWarps - 1) / kJoinWarps, s.R);
  const bool later = s.causal && s.L > 1 && p.T > 0;
  auto join = split ? (later ? prefix_join_kernel<HD, kJoinWarps, true> : prefix_join_kernel<HD, kJoinWarps, false>)
                    : (later ? prefix_join_kernel<HD, 1, true> : prefix_join_kernel<HD, 1, false>);
  const OwnRows own{p.q, p.kk, p.kv, p.q_r, p.q_l, p.q_h, p.k_r, p.k_t, p.k_h, scale_log2};
  if (p.P > 0 || p.T > 0)
    MTP_CUDA_TRY(launch_pdl(join, grid, dim3(32 * kJoinWarps), 0, st, s, own, ml, ro, p.o, p.lse, p.rec, p.rec_stride));
  else
    join<<<grid, 32 * kJoinWarps, 0, st>>>(s, own, ml, ro, p.o, p.lse, p.rec, p.rec_stride);
  note_launch();
  MTP_LAUNCH_CHECK();
  return MTP_OK;
}

}  // namespace

bool prefix_attn_sizes_ok(int R, int L, int H, int Hkv, int hd, int P, int T) {
  return R >= 1 && R <= 65535 && L >= 1 && H >= 1 && Hkv >= 1 && H % Hkv == 0 && H / Hkv <= kRows && (hd == 64 || hd == 128) && P >= 0 && T >= 0 &&
         static_cast<long long>(R) * L * H <= (1 << 24) && static_cast<long long>(P) + T <= 0x7FFFFF00ll;
}

size_t prefix_attn_workspace_bytes(int R, int L, int H, int Hkv, int hd, int P, int T) {
  if (!prefix_attn_sizes_ok(R, L, H, Hkv, hd, P, T)) return 0;
  const long long rows = record_rows(make_shape(R, L, H, Hkv, P, T));
  return up256(rows * sizeof(float2)) + up256(static_cast<size_t>(rows) * hd * 4) + 256;
}

mtp_status prefix_attn_launch(const PrefixAttn& p, void* ws, size_t ws_bytes, cudaStream_t st) {
  if (!prefix_attn_sizes_ok(p.R, p.L, p.H, p.Hkv, p.hd, p.P, p.T)) return MTP_ERR_SHAPE;
  if (ws_bytes < prefix_attn_workspace_bytes(p.R, p.L, p.H, p.Hkv, p.hd, p.P, p.T)) return MTP_ERR_WORKSPACE;
  Shape s = make_shape(p.R, p.L, p.H, p.Hkv, p.P, p.T);
  s.causal = p.causal;
  s.ctx_len = p.ctx_len;
  float2* ml = static_cast<float2*>(ws);
  float* ro = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + up256(record_rows(s) * sizeof(float2)));
  return p.hd == 64 ? launch<64>(p, s, ml, ro, st) : launch<128>(p, s, ml, ro, st);
}

}  // namespace mtp

extern "C" size_t mtp_prefix_attention_workspace_bytes(const mtp_prefix_dims* d) {
  return d ? mtp::prefix_attn_workspace_bytes(d->R, d->L, d->n_heads, d->n_kv_heads, d->head_dim, d->P, d->T) : 0;
}

extern "C" mtp_status mtp_prefix_attention(const mtp_prefix_dims* d, const void* q, const void* prefix_k, const void* prefix_v,
                                           const void* kv_k, const void* kv_v, const int32_t* ctx_len, void* out, float* lse,
                                           void* ws, size_t ws_bytes, cudaStream_t st) {
  if (!d) return MTP_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return MTP_ERR_UNSUPPORTED;
  if (!mtp::prefix_attn_sizes_ok(d->R, d->L, d->n_heads, d->n_kv_heads, d->head_dim, d->P, d->T)) return MTP_ERR_SHAPE;
  if (!(d->scale >= 0.f) || d->scale > 3.0e38f) return MTP_ERR_INVALID_ARG;
  if (!q || !out || !ws || (d->P > 0 && (!prefix_k || !prefix_v)) || (d->T > 0 && (!kv_k || !kv_v))) return MTP_ERR_INVALID_ARG;
  const long long hd = d->head_dim, row = hd * d->n_kv_heads, q_row = hd * d->n_heads;
  mtp::PrefixAttn p;
  p.R = d->R;
  p.L = d->L;
  p.H = d->n_heads;
  p.Hkv = d->n_kv_heads;
  p.hd = d->head_dim;
  p.P = d->P;
  p.T = d->T;
  p.causal = d->causal != 0;
  p.scale = d->scale;
  p.q_h = d->q_stride_h ? d->q_stride_h : hd;
  p.q_l = d->q_stride_t ? d->q_stride_t : q_row;
  p.q_r = d->q_stride_r ? d->q_stride_r : q_row * d->L;
  p.p_h = d->prefix_stride_h ? d->prefix_stride_h : hd;
  p.p_t = d->prefix_stride_t ? d->prefix_stride_t : row;
  p.k_h = d->kv_stride_h ? d->kv_stride_h : hd;
  p.k_t = d->kv_stride_t ? d->kv_stride_t : row;
  p.k_r = d->kv_stride_r ? d->kv_stride_r : row * std::max(d->T, 1);
  for (long long s : {p.q_h, p.q_l, p.q_r, p.p_h, p.p_t, p.k_h, p.k_t, p.k_r}) {
    if (s < 0 || s >= (1ll << 38)) return MTP_ERR_SHAPE;
    if (s % 8) return MTP_ERR_ALIGNMENT;  // 16-byte copies
  }
  for (const void* a : {q, prefix_k, prefix_v, kv_k, kv_v, static_cast<const void*>(out), static_cast<const void*>(ws)})
    if (!mtp::aligned16(a)) return MTP_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(ctx_len) & 3u)) return MTP_ERR_ALIGNMENT;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.pk = static_cast<const __nv_bfloat16*>(prefix_k);
  p.pv = static_cast<const __nv_bfloat16*>(prefix_v);
  p.kk = static_cast<const __nv_bfloat16*>(kv_k);
  p.kv = static_cast<const __nv_bfloat16*>(kv_v);
  p.ctx_len = ctx_len;
  p.o = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  return mtp::prefix_attn_launch(p, ws, ws_bytes, st);
}
