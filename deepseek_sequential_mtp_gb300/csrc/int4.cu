// 4-bit weight GEMM for 1..32 tokens: out[r, n] = Σ_k x[r, k] (q[n, k] - zero[n, k/G]) scale[n, k/G].
//
// Bound: HBM, half a byte per weight; what has to be kept up with it is the
// unpacking.  The products run on mma.sync.m16n8k16 with 16 weight rows as the
// A operand and 8 tokens as B: (q - zero) is an integer of at most 5 bits, so
// it is exact in bf16, the products with bf16 activations are exact in fp32
// and a group's sum is multiplied by its scale in fp32 -- nothing is rounded
// to fewer than 32 bits.  (tcgen05 would want the unpacked weights in shared
// memory or TMEM first: 4 bytes moved per byte read, for an MMA of which at
// most 32 of 128 columns are tokens.)
//
// The sum over k may be taken in any order, so a lane feeds the fragments
// straight from its own 16-byte loads: the quad that shares a weight row reads
// 64 consecutive bytes (128 weights) of it, and one 32-bit word of a lane, 8
// weights, is two MMA steps of that lane's share of k.  A word's nibbles i and
// i + 4 land in the two halves of a register with one shift and one
// and-or (0x4300 | q is bf16 128 + q), and one packed subtraction of
// 128 + zero leaves the integer.  The tokens' values are staged in shared
// memory in the same order: within 8 neighbours 0 4 1 5 2 6 3 7, and the four
// lanes' 16-byte units side by side, so the B fragments are conflict-free
// 16-byte reads.  All lanes of a quad have to be in one group of k while they
// accumulate: a chunk of 128 weights is 128/G groups, and lane t takes
// 128/4 consecutive weights of one group (G = 128), 16 of each of two (64) or
// 8 of each of four (32), with 16-, 8- or 4-byte loads.
//
// A CTA is 8 warps: WM of them along the rows (16 MT rows each) and 8 / WM
// along k; a cluster of up to 8 CTAs splits k further.  The partial sums meet
// in shared memory, then in the cluster's distributed shared memory, in a
// fixed order; there are no atomics and nothing is cleared first.
#include <cooperative_groups.h>

#include <algorithm>

#include "int4.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kChunk = 128;                 // weights of a row per step
constexpr int kUnitBytes = 2 * kChunk;      // a token's activations of one chunk
constexpr int kPitchPad = 64;               // two token rows' units fall into different banks
constexpr int kMaxTokens = 32;

constexpr int ring_depth(int mt) { return mt == 1 ? 4 : 3; }
constexpr int x_bytes(int nt) { return nt == 4 ? 180 * 1024 : 96 * 1024; }  // staged activations: 1 or 2 CTAs per SM

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
  int chunks;        // chunks of 128 along K
  int cta_chunks;    // ... per CTA of the cluster
  int piece_chunks;  // ... of activations staged at a time
  const __nv_bfloat16* x;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// nibbles i and i + 4 of w as two bf16 integers, minus the zero point (z = two bf16 of 128 + zero)
__device__ __forceinline__ uint32_t unpack(uint32_t w, int i, uint32_t z) {
  const uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                   *reinterpret_cast<const __nv_bfloat162*>(&z));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// first weight (within a chunk) of word w of lane t of the quad
template <int G>
__device__ __forceinline__ int word_k(int w, int t) {
  return G == 128 ? 32 * t + 8 * w : G == 64 ? 64 * (w >> 1) + 16 * t + 8 * (w & 1) : 32 * w + 8 * t;
}

// the words of one weight row and chunk, and the row's scales and zero points there
template <int G>
struct RowChunk {
  static constexpr int kG = kChunk / G;
  uint32_t w[4];
  uint16_t scale[kG];
  uint8_t zero[kG];

  __device__ __forceinline__ void load(const Seg& s, int row, int c, int t, int K, int groups) {
    const uint8_t* p = s.q + static_cast<size_t>(row) * (K / 2) + c * (kChunk / 2);
    const int k0 = c * kChunk;
    if constexpr (G == 128) {
      const uint4 u = k0 + 32 * t < K ? __ldg(reinterpret_cast<const uint4*>(p + 16 * t)) : make_uint4(0, 0, 0, 0);
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else if constexpr (G == 64) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint2 u = k0 + 64 * i + 16 * t < K ? __ldg(reinterpret_cast<const uint2*>(p + 32 * i + 8 * t)) : make_uint2(0, 0);
        w[2 * i] = u.x; w[2 * i + 1] = u.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = k0 + 32 * i < K ? __ldg(reinterpret_cast<const uint32_t*>(p + 16 * i + 4 * t)) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kG; ++i) {
      const int g = c * kG + i;
      scale[i] = 0;
      zero[i] = 8;
      if (g < groups) {
        const size_t at = static_cast<size_t>(row) * groups + g;
        scale[i] = __ldg(reinterpret_cast<const uint16_t*>(s.scale) + at);
        if (s.zero) zero[i] = __ldg(s.zero + at);
      }
    }
  }
  __device__ __forceinline__ float factor(int i) const { return __uint_as_float(static_cast<uint32_t>(scale[i]) << 16); }
  // 128 + zero as two bf16: a step of 1 between 128 and 256
  __device__ __forceinline__ uint32_t offset(int i) const { return 0x43004300u + 0x10001u * (zero[i] & 15u); }
};

template <int NT, int MT, int G>
__global__ void __launch_bounds__(kThreads, NT == 4 ? 1 : 2) int4w_gemm_kernel(const __grid_constant__ Args a) {
  constexpr int kG = kChunk / G;
  constexpr int kDepth = ring_depth(MT);  // chunks of weights in flight per warp
  extern __shared__ __align__(16) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wk_n = kWarps / a.wm, wm = warp % a.wm, wk = warp / a.wm;
  const int bm = 16 * MT * a.wm;
  const int tile = blockIdx.x / C;
  const Seg& s = a.seg[a.nseg > 2 && tile >= a.seg[2].tile0 ? 2 : a.nseg > 1 && tile >= a.seg[1].tile0 ? 1 : 0];
  const int row0 = (tile - s.tile0) * bm;
  const int c0 = rank * a.cta_chunks, c1 = min(c0 + a.cta_chunks, a.chunks);

  // this lane's weight rows: g and g + 8 of each 16 (rows past the end repeat the last one)
  int rows[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) rows[m][h] = min(row0 + (wm * MT + m) * 16 + 8 * h + g, s.n - 1);
  RowChunk<G> ring[kDepth][MT][2];
  auto load = [&](int d, int c) {
    if (c < c1) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) ring[d][m][h].load(s, rows[m][h], c, t, a.K, a.groups);
    }
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d) load(d, c0 + wk + d * wk_n);

  float tot[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) tot[m][n][0] = tot[m][n][1] = tot[m][n][2] = tot[m][n][3] = 0.f;

  const int pitch = a.piece_chunks * kUnitBytes + kPitchPad;
  for (int p0 = c0; p0 < c1; p0 += a.piece_chunks) {
    const int p1 = min(p0 + a.piece_chunks, c1);
    if (p0 > c0) __syncthreads();
    // activations of chunks p0 .. p1 - 1: unit u of a token's chunk holds word u / 4 of lane u % 4
    const int units = (p1 - p0) * 16;
    for (int i = threadIdx.x; i < a.R * units; i += kThreads) {
      const int tok = i / units, u = i - tok * units, w = (u >> 2) & 3, tt = u & 3;
      const int k = (p0 + (u >> 4)) * kChunk + word_k<G>(w, tt);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (k < a.K) v = __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(tok) * a.K + k));
      // 0 4 1 5 2 6 3 7
      const uint4 o = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                 __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
      *reinterpret_cast<uint4*>(smem + tok * pitch + u * 16) = o;
    }
    __syncthreads();
    for (int cb = p0 + wk; cb < p1; cb += kDepth * wk_n) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int c = cb + d * wk_n;
        if (c < p1) {  // pieces are whole rounds of the ring, so slot d is chunk c's
          float acc[MT][NT][4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            constexpr int kPer = 4 / kG;  // words per group
            const int gi = w / kPer;
            uint4 xb[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const int tok = 8 * n + g;
              xb[n] = tok < a.R ? *reinterpret_cast<const uint4*>(smem + tok * pitch + (c - p0) * kUnitBytes + (4 * w + t) * 16)
                                : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              if (w % kPer == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
              }
              uint32_t lo[4], hi[4];
              const uint32_t zl = ring[d][m][0].offset(gi), zh = ring[d][m][1].offset(gi);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                lo[i] = unpack(ring[d][m][0].w[w], i, zl);
                hi[i] = unpack(ring[d][m][1].w[w], i, zh);
              }
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma_bf16(acc[m][n], lo[0], hi[0], lo[1], hi[1], xb[n].x, xb[n].y);
                mma_bf16(acc[m][n], lo[2], hi[2], lo[3], hi[3], xb[n].z, xb[n].w);
              }
              if (w % kPer == kPer - 1) {
                const float fl = ring[d][m][0].factor(gi), fh = ring[d][m][1].factor(gi);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  tot[m][n][0] = fmaf(fl, acc[m][n][0], tot[m][n][0]);
                  tot[m][n][1] = fmaf(fl, acc[m][n][1], tot[m][n][1]);
                  tot[m][n][2] = fmaf(fh, acc[m][n][2], tot[m][n][2]);
                  tot[m][n][3] = fmaf(fh, acc[m][n][3], tot[m][n][3]);
                }
              }
            }
          }
          load(d, c + kDepth * wk_n);
        }
      }
    }
  }

  // partial sums of the k-warps: part[wk][token][row of the tile]
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = 8 * n + 2 * t + (e & 1), r = (wm * MT + m) * 16 + g + 8 * (e >> 1);
        if (tok < a.R) part[(wk * a.R + tok) * bm + r] = tot[m][n][e];
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

template <int NT, int MT, int G>
mtp_status launch(const Args& a, int tiles, int C, int smem, cudaStream_t st) {
  static mtp::PerDevice attr;
  auto kernel = int4w_gemm_kernel<NT, MT, G>;
  if (!mtp::smem_limit(attr, kernel, x_bytes(NT))) return MTP_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * C));
  cfg.blockDim = dim3(kThreads);
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

template <int NT, int MT>
mtp_status launch_group(const Args& a, int group, int tiles, int C, int smem, cudaStream_t st) {
  return group == 128 ? launch<NT, MT, 128>(a, tiles, C, smem, st)
         : group == 64 ? launch<NT, MT, 64>(a, tiles, C, smem, st)
                       : launch<NT, MT, 32>(a, tiles, C, smem, st);
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
  a.chunks = (K + kChunk - 1) / kChunk;
  const int nt = R <= 8 ? 1 : R <= 16 ? 2 : 4, mt = nt == 4 ? 2 : 1, depth = ring_depth(mt);
  long long n_all = 0;
  for (int i = 0; i < nseg; ++i) n_all += segs[i].n;
  // Rows per CTA: the staged activations (2 R bytes per k) should not outweigh
  // the weights (half a byte per row and k) ...
  const int sms = sm_count_current();
  int wm = 1;
  while (wm < kWarps && 16 * mt * wm < 4 * R) wm *= 2;
  // ... and the cluster splits k until every SM has two CTAs or a CTA has one
  // round of chunks left
  auto split = [&](int w) {
    int c = 1;
    const long long tiles = (n_all + 16 * mt * w - 1) / (16 * mt * w);
    while (c < 8 && tiles * c < 2 * sms && a.chunks / (2 * c) >= kWarps / w) c *= 2;
    return c;
  };
  int C = split(wm);
  const int wk = kWarps / wm, bm = 16 * mt * wm;
  a.wm = wm;
  a.cta_chunks = (a.chunks + C - 1) / C;
  // pieces of activations are whole rounds of the warps' rings
  const int round = wk * depth;
  const int fit = (x_bytes(nt) / R - kPitchPad) / kUnitBytes / round * round;
  a.piece_chunks = std::min((a.cta_chunks + round - 1) / round * round, fit);
  if (a.piece_chunks < round) return MTP_ERR_UNSUPPORTED;  // not reached: 32 tokens fit one round of 16 chunks' worth
  const int smem = std::max(R * (a.piece_chunks * kUnitBytes + kPitchPad), wk * R * bm * 4);
  long long tiles = 0;
  for (int i = 0; i < nseg; ++i) {
    if (segs[i].n < 1) return MTP_ERR_SHAPE;
    a.seg[i] = Seg{segs[i].q, segs[i].scale, segs[i].zero, segs[i].out, segs[i].n, static_cast<int>(tiles)};
    tiles += (segs[i].n + bm - 1) / bm;
  }
  if (tiles * C > 0x7FFFFFFFll) return MTP_ERR_UNSUPPORTED;
  const int tl = static_cast<int>(tiles);
  return nt == 1 ? launch_group<1, 1>(a, group, tl, C, smem, st)
         : nt == 2 ? launch_group<2, 1>(a, group, tl, C, smem, st)
                   : launch_group<4, 2>(a, group, tl, C, smem, st);
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
