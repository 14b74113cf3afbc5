// 4-bit weight GEMM for 1..32 tokens: out[r, n] = Σ_k x[r, k] (q[n, k] - zero[n, k/G]) scale[n, k/G].
//
// Bound: HBM, half a byte per weight; what has to keep up with it is the
// unpacking.  18432 x 7168, groups of 128: one token 21 us (3.4 TB/s), 8 tokens 27,
// 16 29, 24 37, 32 42 (the tokens' share of the work, 7 us per 8: mma.sync alone
// takes 4 of them, the reads of their fragments 3.5); 73728 x 7168, one token 62 us
// (4.6 TB/s).  The products run on mma.sync.m16n8k16 with 16 weight rows as the
// A operand and 8 tokens as B: (q - zero) is an integer of at most 5 bits, so
// it is exact in bf16, the products with bf16 activations are exact in fp32
// and a group's sum is multiplied by its scale in fp32 -- nothing is rounded
// to fewer than 32 bits.  (On tcgen05, with the
// unpacked weights in shared memory as the N = 256 side, 32 tokens take 49 us
// instead of 42: each block is written and read there at four times its bytes.
// With e4m3 operands, for which a code is its own byte, mma.sync takes 93 us
// instead of 43 on 7168 x 18432 with 32 tokens.)
//
// The sum over k may be taken in any order, so a lane feeds the fragments
// straight from its own 16 bytes: the quad that shares a weight row reads 64
// consecutive bytes (128 weights) of it, and one 32-bit word of a lane, 8
// weights, is two MMA steps of that lane's share of k.  A word's nibbles i and
// i + 4 land in the two halves of a register with one shift and one
// and-or (0x4300 | q is bf16 128 + q), and one packed subtraction of
// 128 + zero leaves the integer.  The tokens' values are staged in shared
// memory in the same order: within 8 neighbours 0 4 1 5 2 6 3 7, and the four
// lanes' 16-byte units side by side, so the B fragments are conflict-free
// 16-byte reads.  All lanes of a quad have to be in one group of k while they
// accumulate: 128 weights are 128/G groups, and lane t takes
// 32 consecutive weights of one group (G = 128), 16 of each of two (64) or
// 8 of each of four (32), with 16-, 8- or 4-byte copies.
//
// A CTA's warps are WM along the rows (16 each) and the others along k; a
// cluster of up to 8 CTAs splits k further.  The partial sums meet in shared
// memory, then in the cluster's distributed shared memory, in a fixed order;
// there are no atomics and nothing is cleared first.
#include <cooperative_groups.h>

#include <algorithm>

#include "int4.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kPitchPad = 64;           // two token rows' units fall into different banks
constexpr int kMaxTokens = 32;
constexpr int kMaxSize = 1 << 30;       // rows and columns, so that rounded-up counts stay within 31 bits

// Variants by the number of 8-token tiles NT: with more than one, one CTA of 16
// warps per SM shares the staged activations (16 tokens, 18432 x 7168: 28 us;
// two CTAs of 8 warps 35; 32 tokens, 7168 x 18432: 43 and 47; 24 tokens on three
// tiles 37, on four 41; 32 rows per warp, which read the activations half as often,
// on 8 warps 47).  With one, the fixed part of a step weighs more: two CTAs of 8
// warps and 256 weights of a row per step (one token, 73728 x 7168: 62 us; three
// CTAs and 128 weights 72).
template <int NT> struct Cfg {
  static constexpr int kChunk = NT > 1 ? 128 : 256;       // weights of a row per step
  static constexpr int kUnitBytes = 2 * kChunk;           // a token's activations of one chunk
  static constexpr int kWords = kChunk / 32;              // words of a row per lane
  static constexpr int kWarps = NT > 1 ? 16 : 8;
  static constexpr int kCtas = NT > 1 ? 1 : 2;            // per SM
  static constexpr int kDepth = 4;                        // chunks of weights in flight per warp
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kSlotBytes = kChunk * 8;           // a warp's chunk: 16 bytes per lane, row and 128 weights
  static constexpr int kRingSlots = kDepth;               // a power of two: slots by mask
  static constexpr int kRingBytes = kWarps * kRingSlots * kSlotBytes;
  static constexpr int kSmem = 224 / kCtas * 1024;
};

struct Seg {
  const uint8_t* q;
  const __nv_bfloat16* scale;
  const uint8_t* zero;
  float* out;
  int n, tile0;  // rows; the segment's first tile
};

struct Args {
  Seg seg[3];
  int nseg, R, K, groups, ldo, accumulate;
  int wm;            // warps along the rows
  int chunks;        // chunks along K
  int cta_chunks;    // ... per CTA of the cluster
  int piece_chunks;  // ... of activations staged at a time
  int by4;           // groups are a multiple of 4 from 8-byte boundaries on: staged four at a time
  const __nv_bfloat16* x;
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// nibbles i and i + 4 of w as two bf16 integers, minus the zero point (z = two bf16 of 128 + zero)
__device__ __forceinline__ uint32_t unpack(uint32_t w, int i, uint32_t z) {
  uint32_t v;  // one instruction: (w & mask) | bf16 128 twice
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (4 * i)), "r"(0x000F000Fu), "r"(0x43004300u));
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                   *reinterpret_cast<const __nv_bfloat162*>(&z));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// first weight (within a chunk) of word w of lane t of the quad
template <int G>
__device__ __forceinline__ int word_k(int w, int t) {
  const int v = w & 3;
  return 128 * (w >> 2) + (G == 128 ? 32 * t + 8 * v : G == 64 ? 64 * (v >> 1) + 16 * t + 8 * (v & 1) : 32 * v + 8 * t);
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool in_range) {
  const int n = in_range ? BYTES : 0;  // the rest is filled with zeros
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}

// a lane's four words of 128 weights of a row (p: their bytes plus the lane's
// own offset) into its 16 bytes at dst; of the last ones only the `valid`
// weights that there are (p is not read where there are none)
template <int G, bool WHOLE>
__device__ __forceinline__ void fetch_words(uint32_t dst, const uint8_t* p, const uint8_t* q, int t, int valid) {
  constexpr int kBytes = G == 128 ? 16 : G == 64 ? 8 : 4;  // as word_k: pieces 4 kBytes apart
#pragma unroll
  for (int i = 0; i < 16 / kBytes; ++i) {
    const bool in = WHOLE || word_k<G>(i * kBytes / 4, t) < valid;
    copy_async<kBytes>(dst + i * kBytes, in ? p + 4 * kBytes * i : q, in);
  }
}

// i-th (row, column) pair of a rows x cols array, advanced by a fixed step
// without a division per step
struct Walk {
  int r, c, dr, dc, cols;
  __device__ __forceinline__ Walk(int i, int step, int cols_)
      : r(i / cols_), c(i - r * cols_), dr(step / cols_), dc(step - dr * cols_), cols(cols_) {}
  __device__ __forceinline__ void next() {
    r += dr;
    c += dc;
    if (c >= cols) {
      c -= cols;
      ++r;
    }
  }
};

// rows x cols elements, kU loads in flight per thread before the first is
// used.  `load` must neither branch nor use what it loads (indices past the end
// are clamped): with a branch around each load the latencies add up, 12 us for
// the scales of a tile whose weights take 5.
template <int kU, typename V, typename Load, typename Store>
__device__ __forceinline__ void stage(int step, int rows, int cols, Load load, Store store) {
  Walk at(threadIdx.x, step, cols);
  while (at.r < rows) {
    V v[kU];
    int r[kU], c[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      r[u] = at.r;
      c[u] = at.c;
      at.next();
      v[u] = load(min(r[u], rows - 1), c[u]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (r[u] < rows) store(r[u], c[u], v[u]);
  }
}

// scale in the upper half of a word, zero point in the lower
__device__ __forceinline__ uint32_t scale_word(uint32_t scale, uint32_t zero, bool has_zero) {
  return (scale << 16) | (has_zero ? zero & 15u : 8u);
}

template <int NT, int G>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, Cfg<NT>::kCtas) int4w_gemm_kernel(const __grid_constant__ Args a) {
  using F = Cfg<NT>;
  constexpr int kWarps = F::kWarps, kThreads = F::kThreads, kDepth = F::kDepth;
  constexpr int kChunk = F::kChunk, kUnitBytes = F::kUnitBytes, kWords = F::kWords;
  constexpr int kG = kChunk / G, kPer = kWords / kG;  // groups per chunk, words per group
  extern __shared__ __align__(16) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wk_n = kWarps / a.wm, wm = warp % a.wm, wk = warp / a.wm;
  const int bm = 16 * a.wm;
  const int tile = blockIdx.x / C;
  const Seg& s = a.seg[a.nseg > 2 && tile >= a.seg[2].tile0 ? 2 : a.nseg > 1 && tile >= a.seg[1].tile0 ? 1 : 0];
  const int row0 = (tile - s.tile0) * bm;
  const int c0 = rank * a.cta_chunks, c1 = min(c0 + a.cta_chunks, a.chunks);

  // This lane's weight rows, g and g + 8 of the warp's 16 (rows past the end
  // repeat the last one), stream through a ring of its own in shared memory: a
  // lane reads only what it copied, so nothing but its own copies is waited for.
  constexpr int kLaneBytes = G == 128 ? 16 : G == 64 ? 8 : 4;
  const uint8_t* rows[2];  // at the chunk to fetch next
  int next = c0 + wk;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    rows[h] = s.q + static_cast<size_t>(min(row0 + wm * 16 + 8 * h + g, s.n - 1)) * (a.K / 2) + next * (kChunk / 2) +
              kLaneBytes * t;
  const uint32_t smem_s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const uint32_t my_ring = smem_s + warp * F::kRingSlots * F::kSlotBytes + lane * 16;
  auto slot_addr = [&](uint32_t i) { return my_ring + (i % F::kRingSlots) * F::kSlotBytes; };
  const size_t row_step = static_cast<size_t>(wk_n) * (kChunk / 2);
  auto fetch = [&](uint32_t to) {
    if (next < c1) {
      const int valid = a.K - next * kChunk;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int b = 0; b < kChunk / 128; ++b) {
          const uint32_t dst = to + (h * (kChunk / 128) + b) * 512;
          if (valid >= kChunk) fetch_words<G, true>(dst, rows[h] + 64 * b, s.q, t, kChunk);
          else fetch_words<G, false>(dst, rows[h] + 64 * b, s.q, t, valid - 128 * b);
        }
        rows[h] += row_step;
      }
    }
    next += wk_n;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int d = 0; d < kDepth - 1; ++d) fetch(slot_addr(d));

  float tot[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) tot[n][0] = tot[n][1] = tot[n][2] = tot[n][3] = 0.f;

  // staged per piece of chunks: the tile's scales and zero points [row][group], and the activations
  const int pg = a.piece_chunks * kG;
  uint32_t* sz = reinterpret_cast<uint32_t*>(smem + F::kRingBytes);
  const int sz_pitch = pg + 1;  // a warp's rows in different banks
  uint8_t* xs = smem + F::kRingBytes + (bm * sz_pitch * 4 + 15) / 16 * 16;
  const int pitch = a.piece_chunks * kUnitBytes + kPitchPad;
  // this lane's B rows; columns past the last token repeat it and are not stored
  uint32_t xt[NT], szt[2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    xt[n] = static_cast<uint32_t>(__cvta_generic_to_shared(xs)) + min(8 * n + g, a.R - 1) * pitch + t * 16;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    szt[h] = static_cast<uint32_t>(__cvta_generic_to_shared(sz)) + (wm * 16 + 8 * h + g) * sz_pitch * 4;
  const bool has_zero = s.zero != nullptr;
  const uint8_t* zeros = has_zero ? s.zero : reinterpret_cast<const uint8_t*>(s.scale);  // any readable bytes
  uint32_t done = 0;  // this warp's chunks
  for (int p0 = c0; p0 < c1; p0 += a.piece_chunks) {
    const int p1 = min(p0 + a.piece_chunks, c1);
    if (p0 > c0) __syncthreads();
    const int g0 = p0 * kG;
    if (a.by4) {
      struct Raw { uint2 s; uint32_t z; };
      stage<4, Raw>(
          kThreads, bm, (p1 - p0) * kG / 4 + ((p1 - p0) * kG % 4 != 0),
          [&](int r, int c) {
            const size_t i = static_cast<size_t>(min(row0 + r, s.n - 1)) * a.groups + min(g0 + 4 * c, a.groups - 4);
            return Raw{__ldg(reinterpret_cast<const uint2*>(s.scale + i)), __ldg(reinterpret_cast<const uint32_t*>(zeros + i))};
          },
          [&](int r, int c, Raw v) {
            uint32_t* to = sz + r * sz_pitch + 4 * c;
            const int left = pg - 4 * c;  // the row's words end with the piece
            to[0] = scale_word(v.s.x & 0xFFFFu, v.z, has_zero);
            if (left > 1) to[1] = scale_word(v.s.x >> 16, v.z >> 8, has_zero);
            if (left > 2) to[2] = scale_word(v.s.y & 0xFFFFu, v.z >> 16, has_zero);
            if (left > 3) to[3] = scale_word(v.s.y >> 16, v.z >> 24, has_zero);
          });
    } else {
      struct Raw { uint16_t s; uint8_t z; };
      stage<8, Raw>(
          kThreads, bm, (p1 - p0) * kG,
          [&](int r, int c) {
            const size_t i = static_cast<size_t>(min(row0 + r, s.n - 1)) * a.groups + min(g0 + c, a.groups - 1);
            return Raw{__ldg(reinterpret_cast<const uint16_t*>(s.scale) + i), __ldg(zeros + i)};
          },
          [&](int r, int c, Raw v) { sz[r * sz_pitch + c] = scale_word(v.s, v.z, has_zero); });
    }
    // unit u of a token's chunk holds word u / 4 of lane u % 4; zeros past the end of K
    stage<4, uint4>(
        kThreads, a.R, (p1 - p0) * 4 * kWords,
        [&](int r, int u) {
          const int k = (p0 + u / (4 * kWords)) * kChunk + word_k<G>((u >> 2) % kWords, u & 3);
          return __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(r) * a.K + min(k, a.K - 8)));
        },
        [&](int r, int u, uint4 v) {
          if ((p0 + u / (4 * kWords)) * kChunk + word_k<G>((u >> 2) % kWords, u & 3) >= a.K) v = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(xs + r * pitch + u * 16) =
              make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                         __byte_perm(v.y, v.w, 0x7632));  // 0 4 1 5 2 6 3 7
        });
    __syncthreads();
    // pieces are whole rounds of the k-warps, so the chunks follow one another in the ring
    uint32_t x_at = wk * kUnitBytes, sz_at = wk * kG * 4;
    for (int c = p0 + wk; c < p1; c += wk_n, x_at += wk_n * kUnitBytes, sz_at += wk_n * kG * 4) {
      fetch(slot_addr(done + kDepth - 1));
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      const uint32_t from = slot_addr(done++);
      uint32_t f[2][kG];
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        f[0][i] = lds32(szt[0] + sz_at + i * 4);
        f[1][i] = lds32(szt[1] + sz_at + i * 4);
      }
      uint32_t q[2][kWords];
#pragma unroll
      for (int e = 0; e < 2 * kWords / 4; ++e) {
        const uint4 u = lds128(from + 512 * e);
        q[e / (kWords / 4)][4 * e % kWords] = u.x;
        q[e / (kWords / 4)][4 * e % kWords + 1] = u.y;
        q[e / (kWords / 4)][4 * e % kWords + 2] = u.z;
        q[e / (kWords / 4)][4 * e % kWords + 3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
        uint32_t z[2];  // 128 + zero twice
#pragma unroll
        for (int h = 0; h < 2; ++h) z[h] = 0x43004300u + 0x10001u * (f[h][i] & 0xFFFFu);
#pragma unroll
        for (int w = i * kPer; w < (i + 1) * kPer; ++w) {
          uint4 xb[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) xb[n] = lds128(xt[n] + x_at + w * 64);
          uint32_t lo[4], hi[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            lo[e] = unpack(q[0][w], e, z[0]);
            hi[e] = unpack(q[1][w], e, z[1]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_bf16(acc[n], lo[0], hi[0], lo[1], hi[1], xb[n].x, xb[n].y);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_bf16(acc[n], lo[2], hi[2], lo[3], hi[3], xb[n].z, xb[n].w);
        }
        const float fl = __uint_as_float(f[0][i] & 0xFFFF0000u), fh = __uint_as_float(f[1][i] & 0xFFFF0000u);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          tot[n][0] = fmaf(fl, acc[n][0], tot[n][0]);
          tot[n][1] = fmaf(fl, acc[n][1], tot[n][1]);
          tot[n][2] = fmaf(fh, acc[n][2], tot[n][2]);
          tot[n][3] = fmaf(fh, acc[n][3], tot[n][3]);
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

  // partial sums of the k-warps: part[wk][token][row of the tile]
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int tok = 8 * n + 2 * t + (e & 1), r = wm * 16 + g + 8 * (e >> 1);
      if (tok < a.R) part[(wk * a.R + tok) * bm + r] = tot[n][e];
    }
  __syncthreads();
  const int per = a.R * bm;
  if (wk_n > 1) {
    for (int i = threadIdx.x; i < per; i += kThreads) {
      float v = part[i];
      for (int w = 1; w < wk_n; ++w) v += part[w * per + i];
      part[i] = v;
    }
  }
  if (C > 1) cluster.sync();
  else __syncthreads();
  // every CTA of the cluster finishes its share of the tile
  for (int i = rank * kThreads + threadIdx.x; i < per; i += C * kThreads) {
    float v = 0.f;
    for (int c = 0; c < C; ++c) v += *cluster.map_shared_rank(part + i, c);
    const int tok = i / bm, r = row0 + i - tok * bm;
    if (r < s.n) {
      float* o = s.out + static_cast<size_t>(tok) * a.ldo + r;
      *o = a.accumulate ? *o + v : v;
    }
  }
  if (C > 1) cluster.sync();  // the others' reads of this CTA's sums
}

// shared memory of a piece: ring, scales, activations
template <int NT>
int piece_bytes(int R, int bm, int chunks, int group) {
  using F = Cfg<NT>;
  return F::kRingBytes + (bm * (chunks * (F::kChunk / group) + 1) * 4 + 15) / 16 * 16 + R * (chunks * F::kUnitBytes + kPitchPad);
}

template <int NT, int G>
mtp_status launch(const Args& a, int tiles, int C, int smem, cudaStream_t st) {
  static mtp::PerDevice attr;
  auto kernel = int4w_gemm_kernel<NT, G>;
  if (!mtp::smem_limit(attr, kernel, Cfg<NT>::kSmem)) return MTP_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * C));
  cfg.blockDim = dim3(Cfg<NT>::kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {static_cast<unsigned>(C), 1u, 1u};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  MTP_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, a));
  mtp::note_launch();
  return MTP_OK;
}

template <int NT>
mtp_status plan(Args& a, const mtp::Int4Seg* segs, int group, cudaStream_t st) {
  using F = Cfg<NT>;
  a.chunks = (a.K + F::kChunk - 1) / F::kChunk;
  long long n_all = 0;
  for (int i = 0; i < a.nseg; ++i) n_all += segs[i].n;
  // Rows per CTA and CTAs per cluster.  A large tile stages fewer activations
  // per weight, a split of k costs a join; what has to be met is a CTA for
  // every SM.  Up to 4 tokens: the largest tile that does so without a split
  // (18432 x 7168, one token: 64 rows 20.7 us, 128 rows on two CTAs 22.6, 16
  // rows 24.7); more tokens: the largest that does so with one (8 tokens: 128
  // rows on two CTAs 25 us, 64 rows 29).  Then k is split over as many CTAs as
  // the SMs hold at once (32 tokens, 7168 x 18432: 43 us on 5, 51 on 4, 56 on 8).
  const int sms = mtp::sm_count_current();
  auto tiles_of = [&](int w) { return (n_all + 16 * w - 1) / (16 * w); };
  int wm = F::kWarps;
  while (wm > 1 && tiles_of(wm) * (a.R > 4 ? 8 : 1) < sms) wm /= 2;
  int C = 8;
  while (C > 1 && (tiles_of(wm) * C > static_cast<long long>(sms) * F::kCtas || a.chunks / C < F::kWarps / wm)) --C;
  const int wk = F::kWarps / wm, bm = 16 * wm;
  a.wm = wm;
  a.cta_chunks = (a.chunks + C - 1) / C;
  // a piece is as many rounds of the k-warps as fit, at most the CTA's share
  // (no more than one token's activations alone would fill, so that the bytes stay within 31 bits)
  a.piece_chunks = std::min((a.cta_chunks + wk - 1) / wk * wk, F::kSmem / F::kUnitBytes / wk * wk);
  while (a.piece_chunks > wk && piece_bytes<NT>(a.R, bm, a.piece_chunks, group) > F::kSmem) a.piece_chunks -= wk;
  const int smem = std::max(piece_bytes<NT>(a.R, bm, a.piece_chunks, group), wk * a.R * bm * 4);
  if (smem > F::kSmem) return MTP_ERR_UNSUPPORTED;  // not reached: one round fits for every R
  long long tiles = 0;
  a.by4 = a.groups % 4 == 0 && a.cta_chunks * (F::kChunk / group) % 4 == 0 && a.piece_chunks * (F::kChunk / group) % 4 == 0;
  for (int i = 0; i < a.nseg; ++i) {
    if ((reinterpret_cast<uintptr_t>(segs[i].scale) & 7u) || (reinterpret_cast<uintptr_t>(segs[i].zero) & 3u)) a.by4 = 0;
    a.seg[i] = Seg{segs[i].q, segs[i].scale, segs[i].zero, segs[i].out, segs[i].n, static_cast<int>(tiles)};
    tiles += (segs[i].n + bm - 1) / bm;
  }
  if (tiles * C > 0x7FFFFFFFll) return MTP_ERR_UNSUPPORTED;
  const int tl = static_cast<int>(tiles);
  return group == 128 ? launch<NT, 128>(a, tl, C, smem, st)
         : group == 64 ? launch<NT, 64>(a, tl, C, smem, st)
                       : launch<NT, 32>(a, tl, C, smem, st);
}

}  // namespace

namespace mtp {

mtp_status int4w_gemm_launch(const Int4Seg* segs, int nseg, int K, int group, const __nv_bfloat16* x, int R, int ldo,
                             bool accumulate, cudaStream_t st) {
  if (nseg < 1 || nseg > 3 || R < 1 || R > kMaxTokens || K < 1 || K % 32) return MTP_ERR_SHAPE;
  if (group != 32 && group != 64 && group != 128) return MTP_ERR_UNSUPPORTED;
  Args a{};
  a.nseg = nseg;
  a.R = R;
  a.K = K;
  a.groups = (K + group - 1) / group;
  a.ldo = ldo;
  a.accumulate = accumulate;
  a.x = x;
  for (int i = 0; i < nseg; ++i)
    if (segs[i].n < 1) return MTP_ERR_SHAPE;
  for (int i = 0; i < nseg; ++i)
    if (segs[i].n > kMaxSize || K > kMaxSize) return MTP_ERR_UNSUPPORTED;
  return R <= 8 ? plan<1>(a, segs, group, st) : R <= 16 ? plan<2>(a, segs, group, st)
         : R <= 24 ? plan<3>(a, segs, group, st) : plan<4>(a, segs, group, st);
}

}  // namespace mtp

extern "C" mtp_status mtp_gemm_int4w(int R, int N, int K, int group, const void* x, const mtp_int4_matrix* w, float* out,
                                     int accumulate, cudaStream_t st) {
  if (!w || !x || !out || !w->q || !w->scale) return MTP_ERR_INVALID_ARG;
  if (R < 1 || R > kMaxTokens || N < 1 || K < 1) return MTP_ERR_SHAPE;
  if (K % 32) return MTP_ERR_ALIGNMENT;  // 16-byte rows of codes
  if (!mtp::aligned16(x) || !mtp::aligned16(w->q) || (reinterpret_cast<uintptr_t>(w->scale) & 1u) ||
      (reinterpret_cast<uintptr_t>(out) & 3u))
    return MTP_ERR_ALIGNMENT;
  mtp::Int4Seg s;
  s.q = static_cast<const uint8_t*>(w->q);
  s.scale = static_cast<const __nv_bfloat16*>(w->scale);
  s.zero = static_cast<const uint8_t*>(w->zero);
  s.n = N;
  s.out = out;
  return mtp::int4w_gemm_launch(&s, 1, K, group, static_cast<const __nv_bfloat16*>(x), R, N, accumulate != 0, st);
}
