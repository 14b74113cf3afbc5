// Rotary positions, and the rows of a paged key/value cache: appending a step's, and
// reading them back as dense caches.
//
// All three move bytes: a few operations per element that is read and written once.
// Bound: HBM for large calls, the launch and one chain of loads for small ones.
#include <algorithm>
#include <cmath>

#include "paged.cuh"
#include "rotary.cuh"

MTP_DEFINE_ERROR_WORD(mtp_take_errors_paged)

namespace mtp {
namespace {

constexpr int kThreads = 256;

// 8 consecutive elements as floats
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2_bf16(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store_run(float* p, const float (&x)[4]) { *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void store_run(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]), pack2_bf16(x[4], x[5]), pack2_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store_run(__nv_bfloat16* p, const float (&x)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]));
}
// two runs of kP to kP pairs and back: neighbours (interleaved), or one of each run
template <int kP>
__device__ __forceinline__ void to_pairs(const float (&lo)[kP], const float (&hi)[kP], bool neighbours, float (&a)[kP], float (&b)[kP]) {
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    a[i] = !neighbours ? lo[i] : i < kP / 2 ? lo[2 * i % kP] : hi[2 * i % kP];
    b[i] = !neighbours ? hi[i] : i < kP / 2 ? lo[(2 * i + 1) % kP] : hi[(2 * i + 1) % kP];
  }
}
template <int kP>
__device__ __forceinline__ void to_runs(const float (&a)[kP], const float (&b)[kP], bool neighbours, float (&lo)[kP], float (&hi)[kP]) {
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    lo[i] = !neighbours ? a[i] : i & 1 ? b[i >> 1] : a[i >> 1];
    hi[i] = !neighbours ? b[i] : i & 1 ? b[kP / 2 + (i >> 1)] : a[kP / 2 + (i >> 1)];
  }
}
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
  const float x = fmaf(a, cs.x, -(b * cs.y));
  b = fmaf(b, cs.x, a * cs.y);
  a = x;
}

struct RopeArgs {
  long long N;
  int H, hd, rot, units;  // units per head
  int tokens, heads;      // of a block
  uint32_t per_magic, units_magic;  // 2^32 / (heads units), / units, rounded up (0: divided by 1)
  float mscale;
  int backward;
  const double* inv_freq;
  const int32_t* pos;
  long long xn, xh, on, oh;
};
// n / d for n, d < 2^16
__device__ __forceinline__ uint32_t divided(uint32_t n, uint32_t magic) { return magic ? __umulhi(n, magic) : n; }

// A run of elements as it lies in memory, and as floats
template <typename T, int kP> struct Run;
template <> struct Run<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const { unpack8(v, x); }
};
template <> struct Run<__nv_bfloat16, 4> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    const float2 a = unpack2_bf16(v.x), b = unpack2_bf16(v.y);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  }
};
template <> struct Run<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
};

// A block takes `tokens` positions and `heads` heads: their cosines and sines once into
// shared memory, then units, one per thread.  The loads of four units per thread are asked for
// before the angles are worked out, and further four after the ones before are stored; without that a block's
// loads wait for its angles, 4096 positions of 112 heads of 128 74 us instead of 44 (41 now).
// Bound: HBM.  That call moves 235 MB at 5.7 TB/s, the copy's own rate is 6.8; one of 32 positions takes
// 5 us, launch and one load after another.
template <typename T, int kP, bool kVec, bool kInter>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const RopeArgs g, const T* x, T* out) {
  extern __shared__ float2 cs[];  // [tokens][rot / 2]
  const long long n0 = static_cast<long long>(blockIdx.x) * g.tokens;
  const int h0 = blockIdx.y * g.heads;
  const int nt = static_cast<int>(min(static_cast<long long>(g.tokens), g.N - n0)), nh = min(g.heads, g.H - h0);
  const int half = g.rot / 2, per = g.heads * g.units, all = nt * per;
  constexpr int kAhead = 4;
  struct Unit {
    int t, h, u;
    bool is;
  };
  auto unit = [&](int i) {
    Unit q;
    q.t = divided(i, g.per_magic);
    const int k = i - q.t * per;
    q.h = divided(k, g.units_magic);
    q.u = k - q.h * g.units;
    q.is = i < all && q.h < nh;
    return q;
  };
  Run<T, kP> lo[kAhead], hi[kAhead];
  auto load = [&](int base) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const Unit q = unit(base + j * kThreads);
      if (q.is) {
        const T* from = x + (n0 + q.t) * g.xn + (h0 + q.h) * g.xh;
        const int2 run = unit_runs<kP>(q.u, g.rot, kInter);
        lo[j].load(from + run.x);
        hi[j].load(from + run.y);
      }
    }
  };
  if constexpr (kVec) load(threadIdx.x);
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, p = i - t * half;
    float2 v = turn_unit(g.pos[n0 + t], turn_fraction(g.inv_freq[p]));
    v.x *= g.mscale;
    v.y *= g.backward ? -g.mscale : g.mscale;
    // (two pairs are 16 bytes, those of neighbouring units neighbours: no conflicts where 8 lanes read 8 units)
    cs[kVec ? t * half + 2 * (p % kP / 2 * (half / kP) + p / kP) + (p & 1) : i] = v;
  }
  __syncthreads();
  for (int base = threadIdx.x; base < all; base += kThreads * kAhead) {
    if constexpr (kVec) {
      if (base != static_cast<int>(threadIdx.x)) load(base);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const Unit q = unit(base + j * kThreads);
        if (!q.is) continue;
        float rl[kP], rh[kP];
        lo[j].get(rl);
        hi[j].get(rh);
        if (2 * kP * q.u < g.rot) {
          const float4* c = reinterpret_cast<const float4*>(cs + q.t * half) + q.u;
          float a[kP], b[kP];
          to_pairs(rl, rh, kInter, a, b);
#pragma unroll
          for (int i = 0; i < kP; i += 2) {
            const float4 w = c[i / 2 * (half / kP)];
            turn(a[i], b[i], make_float2(w.x, w.y));
            turn(a[i + 1], b[i + 1], make_float2(w.z, w.w));
          }
          to_runs(a, b, kInter, rl, rh);
        }
        T* to = out + (n0 + q.t) * g.on + (h0 + q.h) * g.oh;
        const int2 run = unit_runs<kP>(q.u, g.rot, kInter);
        store_run(to + run.x, rl);
        store_run(to + run.y, rh);
      }
    } else {
#pragma unroll 1
      for (int j = 0; j < kAhead; ++j) {
        const Unit q = unit(base + j * kThreads);
        if (!q.is) continue;
        const T* from = x + (n0 + q.t) * g.xn + (h0 + q.h) * g.xh;
        T* to = out + (n0 + q.t) * g.on + (h0 + q.h) * g.oh;
#pragma unroll
        for (int e = 0; e < kP; ++e) {
          const int p = kP * q.u + e;
          if (2 * p >= g.hd) break;
          const int2 at = pair_elements(p, g.rot, kInter);
          float a = load_f32<T>(from + at.x), b = load_f32<T>(from + at.y);
          if (p < half) turn(a, b, cs[q.t * half + p]);
          to[at.x] = from_f32<T>(a);
          to[at.y] = from_f32<T>(b);
        }
      }
    }
  }
}

template <typename T, int kP>
mtp_status rope_launch(const RopeArgs& g, bool vec, bool inter, const void* x, void* out, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((g.N + g.tokens - 1) / g.tokens), static_cast<unsigned>((g.H + g.heads - 1) / g.heads));
  const size_t smem = static_cast<size_t>(g.tokens) * (g.rot / 2) * sizeof(float2);
  const T* xi = static_cast<const T*>(x);
  T* xo = static_cast<T*>(out);
  if (vec && inter) {
    rope_kernel<T, kP, true, true><<<grid, kThreads, smem, st>>>(g, xi, xo);
  } else if (vec) {
    rope_kernel<T, kP, true, false><<<grid, kThreads, smem, st>>>(g, xi, xo);
  } else if constexpr (kP == 4) {  // (8 are taken only where they fit)
    if (inter)
      rope_kernel<T, kP, false, true><<<grid, kThreads, smem, st>>>(g, xi, xo);
    else
      rope_kernel<T, kP, false, false><<<grid, kThreads, smem, st>>>(g, xi, xo);
  }
  note_launch();
  MTP_LAUNCH_CHECK();
  return MTP_OK;
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
constexpr int kWarps = kThreads / 32;

struct AppendArgs {
  mtp_paged_cache c;
  mtp_kv_rows w;
  int rot;
  float mscale;
  const double* inv_freq;
  int kv_blocks;  // blocks of 16 rows that a request's rows may touch
  int kv_groups, q_groups, q_chunks;  // groups of kWarps heads; runs of 16 tokens of q
  long long kv_ctas;
};

__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}
// values of four codes
__device__ __forceinline__ void unpack_e4m3(uint32_t w, float (&x)[4]) {
  uint32_t h[2];
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, u;\n}\n" : "=r"(h[0]), "=r"(h[1]) : "r"(w));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
// exponent of a scale byte, 1..254 or taken as the nearest of those
__device__ __forceinline__ int scale_exponent(uint8_t b) { return min(max(static_cast<int>(b), 1), 254) - 127; }

// 16 bf16 elements of unit u of a row, as 8 words: the runs' (kVec), or pairs
template <bool kVec, bool kInter>
__device__ __forceinline__ void load_unit(const __nv_bfloat16* row, int u, int rot, uint32_t (&w)[8]) {
  if constexpr (kVec) {
    const int2 run = unit_runs(u, rot, kInter);
    const uint4 a = *reinterpret_cast<const uint4*>(row + run.x), b = *reinterpret_cast<const uint4*>(row + run.y);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int2 at = pair_elements(8 * u + i, rot, kInter);
      w[i] = p[at.x] | static_cast<uint32_t>(p[at.y]) << 16;
    }
  }
}
// ... to turned pairs (cs: cosines and sines of the row, null: none)
template <bool kVec, bool kInter>
__device__ __forceinline__ void turn_unit_words(const uint32_t (&w)[8], int u, int rot, const float2* cs, float (&a)[8], float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (!kVec || kInter) {
      const float2 f = unpack2_bf16(w[i]);
      a[i] = f.x;
      b[i] = f.y;
    } else if (i < 4) {
      const float2 f = unpack2_bf16(w[i]), g = unpack2_bf16(w[4 + i]);
      a[2 * i] = f.x, a[2 * i + 1] = f.y, b[2 * i] = g.x, b[2 * i + 1] = g.y;
    }
  }
  if (cs) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (2 * (8 * u + i) < rot) turn(a[i], b[i], cs[8 * u + i]);
  }
}
template <bool kVec, bool kInter>
__device__ __forceinline__ void store_unit(__nv_bfloat16* row, int u, int rot, const float (&a)[8], const float (&b)[8]) {
  if constexpr (kVec) {
    const int2 run = unit_runs(u, rot, kInter);
    float lo[8], hi[8];
    to_runs(a, b, kInter, lo, hi);
    store_run(row + run.x, lo);
    store_run(row + run.y, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int2 at = pair_elements(8 * u + i, rot, kInter);
      row[at.x] = f32_to_bf16(a[i]);
      row[at.y] = f32_to_bf16(b[i]);
    }
  }
}
template <bool kVec, bool kInter>
__device__ __forceinline__ void store_unit_e4m3(uint8_t* row, int u, int rot, const float (&a)[8], const float (&b)[8]) {
  if constexpr (kVec) {
    const int2 run = unit_runs(u, rot, kInter);
    float lo[8], hi[8];
    to_runs(a, b, kInter, lo, hi);
    *reinterpret_cast<uint2*>(row + run.x) = make_uint2(pack_e4m3(lo[0], lo[1]) | pack_e4m3(lo[2], lo[3]) << 16,
                                                        pack_e4m3(lo[4], lo[5]) | pack_e4m3(lo[6], lo[7]) << 16);
    *reinterpret_cast<uint2*>(row + run.y) = make_uint2(pack_e4m3(hi[0], hi[1]) | pack_e4m3(hi[2], hi[3]) << 16,
                                                        pack_e4m3(hi[4], hi[5]) | pack_e4m3(hi[6], hi[7]) << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int2 at = pair_elements(8 * u + i, rot, kInter);
      const uint32_t v = pack_e4m3(a[i], b[i]);
      row[at.x] = static_cast<uint8_t>(v);
      row[at.y] = static_cast<uint8_t>(v >> 8);
    }
  }
}

// Rows of keys or of values: up to 16 of a block, tokens first .. first + n - 1 of the
// call, into slots slot .. of a page's head, by a warp: HD / 16 lanes per row.
template <int HD, bool kF8, bool kVec, bool kInter>
__device__ __forceinline__ void append_rows(const uint32_t (&raw)[HD / 32][8], int n, int slot, int rot, const float2* cs,
                                            int half, uint8_t* page, uint8_t* scale, bool begun) {
  constexpr int kUnits = HD / 16, kPer = 32 / kUnits, kIt = 16 / kPer;
  const int lane = threadIdx.x & 31, u = lane % kUnits, t = lane / kUnits;
  if constexpr (!kF8) {
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const int row = i * kPer + t;
      if (row < n) {
        float a[8], b[8];
        turn_unit_words<kVec, kInter>(raw[i], u, rot, cs ? cs + row * half : nullptr, a, b);
        store_unit<kVec, kInter>(reinterpret_cast<__nv_bfloat16*>(page) + static_cast<size_t>(slot + row) * HD, u, rot, a, b);
      }
    }
  } else {
    const int old = begun ? 0 : scale_exponent(*scale);
    float a[kIt][8], b[kIt][8], top = 0.f;
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const int row = i * kPer + t;
      if (row < n) {
        turn_unit_words<kVec, kInter>(raw[i], u, rot, cs ? cs + row * half : nullptr, a[i], b[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = fabsf(a[i][e]), y = fabsf(b[i][e]);
          if (x < INFINITY) top = fmaxf(top, x);
          if (y < INFINITY) top = fmaxf(top, y);
        }
      }
    }
    top = warp_max(top);
    // smallest 2^e >= top / 448, 448 = 1.75 * 2^8
    const uint32_t bits = __float_as_uint(top);
    int e = max(static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), -90);
    if (!begun) {
      if (e > old) {  // rows that are there to the new scale
        const float f = power_of_two(old - e);
        const int first = slot & ~15;
        for (int i = t; i < slot - first; i += kPer) {
          uint32_t* at = reinterpret_cast<uint32_t*>(page + static_cast<size_t>(first + i) * HD) + 4 * u;
          uint4 v = *reinterpret_cast<const uint4*>(at);
          uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x[4];
            unpack_e4m3(w[j], x);
            w[j] = pack_e4m3(x[0] * f, x[1] * f) | pack_e4m3(x[2] * f, x[3] * f) << 16;
          }
          *reinterpret_cast<uint4*>(at) = v;
        }
      } else {
        e = old;
      }
    }
    const float inv = power_of_two(-e);
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const int row = i * kPer + t;
      if (row < n) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // what is not finite to NaN, which x - x is then
          a[i][j] = fmaf(a[i][j], inv, a[i][j] - a[i][j]);
          b[i][j] = fmaf(b[i][j], inv, b[i][j] - b[i][j]);
        }
        store_unit_e4m3<kVec, kInter>(page + static_cast<size_t>(slot + row) * HD, u, rot, a[i], b[i]);
      }
    }
    if (lane == 0) *scale = static_cast<uint8_t>(e + 127);
  }
}

// Bound: HBM for many rows (32 requests x 8192 rows of 56 heads of 128: bf16 2.49 ms, 6.0 TB/s; e4m3 2.25 ms, 5.0 TB/s, with
// its quantising), for few of them the chain from lengths over the table to the rows, 7 us of a
// step's token of 32 requests, 9 us of 8 bits, whose block is read, scaled anew and written.
// A CTA takes a block of 16 rows of a request and 8 heads, a warp per head (keys and
// values), after the cosines and sines of the block's positions, once for the heads; or 16 tokens and 8
// heads of the queries.
template <int HD, bool kF8, bool kVec, bool kInter>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs g) {
  constexpr int kUnits = HD / 16, kPer = 32 / kUnits, kIt = 16 / kPer;
  __shared__ float2 cs[16 * (HD / 2)];
  // (the same in every lane, and known as such to the compiler: a shuffle where a warp may be apart takes 230 cycles instead of 36)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31, u = lane % kUnits, t = lane / kUnits;
  const int half = g.rot / 2, L = g.w.L;
  const bool kv = blockIdx.x < g.kv_ctas;
  long long id = kv ? blockIdx.x : blockIdx.x - g.kv_ctas;
  const int groups = kv ? g.kv_groups : g.q_groups, blocks = kv ? g.kv_blocks : g.q_chunks;
  const int h = static_cast<int>(id % groups) * kWarps + warp;
  id /= groups;
  const int r = static_cast<int>(id / blocks), j = static_cast<int>(id - static_cast<long long>(r) * blocks);
  const long long ctx = g.w.ctx_len[r];
  const int fresh = g.w.n_new ? min(max(g.w.n_new[r], 0), L) : L;
  const long long p0 = ctx - fresh;  // index of the call's first row
  int first, n;                      // tokens of this CTA
  long long b = 0;
  if (kv) {
    b = (p0 >> 4) + j;
    const long long lo = max(b << 4, p0), hi = min((b + 1) << 4, ctx);
    if (fresh == 0 || hi <= lo) return;
    if (b < 0 || (b << 4) >= static_cast<long long>(g.c.table_len) * g.c.page) {
      if (threadIdx.x == 0) atomicOr(&g_mtp_error_word, MTP_DEVERR_PAGE_RANGE);
      return;
    }
    first = static_cast<int>(lo - p0);
    n = static_cast<int>(hi - lo);
  } else {
    first = 16 * j;
    n = min(16, L - first);
  }
  const bool live = h < (kv ? g.c.n_kv_heads : g.w.n_heads);
  uint32_t raw[kIt][8];
  auto load = [&](const void* base, long long sr, long long st, long long sh) {
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const int row = i * kPer + t;
      if (live && row < n)
        load_unit<kVec, kInter>(static_cast<const __nv_bfloat16*>(base) + r * sr + (first + row) * st + h * sh, u, g.rot, raw[i]);
    }
  };
  if (kv)
    load(g.w.k, g.w.kv_stride_r, g.w.kv_stride_t, g.w.kv_stride_h);
  else
    load(g.w.q, g.w.q_stride_r, g.w.q_stride_t, g.w.q_stride_h);
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int row = i / half, p = i - row * half;
    const int at = g.w.pos ? g.w.pos[static_cast<long long>(r) * L + first + row] : static_cast<int>(p0 + first + row);
    float2 v = turn_unit(at, turn_fraction(g.inv_freq[p]));
    v.x *= g.mscale;
    v.y *= g.mscale;
    cs[i] = v;
  }
  __syncthreads();
  if (!live) return;
  const float2* turns = half ? cs : nullptr;
  if (!kv) {
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const int row = i * kPer + t;
      if (row < n) {
        float a[8], b8[8];
        turn_unit_words<kVec, kInter>(raw[i], u, g.rot, turns ? turns + row * half : nullptr, a, b8);
        store_unit<kVec, kInter>(static_cast<__nv_bfloat16*>(g.w.q_out) +
                                     ((static_cast<long long>(r) * L + first + row) * g.w.n_heads + h) * HD,
                                 u, g.rot, a, b8);
      }
    }
    return;
  }
  const int per_page = g.c.page >> 4;
  const int page = g.c.page_table[static_cast<long long>(r) * g.c.table_len + b / per_page];
  if (page < 0 || page >= g.c.n_pages) {
    if (lane == 0) atomicOr(&g_mtp_error_word, MTP_DEVERR_PAGE_RANGE);
    return;
  }
  const int block = static_cast<int>(b % per_page), slot = 16 * block + static_cast<int>((p0 + first) & 15);
  const long long head = static_cast<long long>(page) * g.c.n_kv_heads + h;
  const size_t at = static_cast<size_t>(head) * g.c.page * HD * (kF8 ? 1 : 2);
  const bool begun = (slot & 15) == 0;
  append_rows<HD, kF8, kVec, kInter>(raw, n, slot, g.rot, turns, half, static_cast<uint8_t*>(g.c.k) + at,
                                     kF8 ? g.c.k_scale + head * per_page + block : nullptr, begun);
  load(g.w.v, g.w.kv_stride_r, g.w.kv_stride_t, g.w.kv_stride_h);
  append_rows<HD, kF8, kVec, kInter>(raw, n, slot, g.rot, nullptr, half, static_cast<uint8_t*>(g.c.v) + at,
                                     kF8 ? g.c.v_scale + head * per_page + block : nullptr, begun);
}

template <int HD, bool kF8>
void append_launch(const AppendArgs& g, bool vec, bool inter, unsigned ctas, cudaStream_t st) {
  if (vec && inter)
    kv_append_kernel<HD, kF8, true, true><<<ctas, kThreads, 0, st>>>(g);
  else if (vec)
    kv_append_kernel<HD, kF8, true, false><<<ctas, kThreads, 0, st>>>(g);
  else if (inter)
    kv_append_kernel<HD, kF8, false, true><<<ctas, kThreads, 0, st>>>(g);
  else
    kv_append_kernel<HD, kF8, false, false><<<ctas, kThreads, 0, st>>>(g);
}

// ---------------------------------------------------------------------------
// Gather
// ---------------------------------------------------------------------------
// 16 elements of keys and of values per thread, neighbouring threads along a row and
// then over heads, as the dense rows lie.  Bound: HBM, 7.1 TB/s for large caches of bf16, 6.3 of 8 bits; 15000 rows of 8 heads
// 12 to 17 us, length, page and row one after another.
// kDense: rows behind a request's stay as they are, but for `more` of zeros (kv_dense_launch); a request without new tokens has none.
template <int HD, bool kF8, bool kDense>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const mtp_paged_cache c, int T, const int32_t* __restrict__ ctx_len,
                                                             __nv_bfloat16* __restrict__ k_out, __nv_bfloat16* __restrict__ v_out, int L,
                                                             const int32_t* __restrict__ n_new, int causal, int32_t* __restrict__ ctx_out) {
  constexpr int kUnits = HD / 16;
  const int r = blockIdx.y;
  int ctx = ctx_len[r], more = 0;
  if constexpr (kDense) {
    ctx = min(max(ctx, 0), c.table_len * c.page);
    const int fresh = n_new ? min(max(n_new[r], 0), L) : L;
    if (fresh == 0) ctx = 0;
    else if (causal) more = L - fresh;
    if (blockIdx.x == 0 && threadIdx.x == 0) ctx_out[r] = ctx + more;
  }
  const long long all = static_cast<long long>(kDense ? ctx + more : T) * c.n_kv_heads * kUnits, apart = static_cast<long long>(gridDim.x) * kThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < all; i += apart) {
    const int u = static_cast<int>(i % kUnits);
    const int row = static_cast<int>(i / (c.n_kv_heads * kUnits)), h = static_cast<int>(i / kUnits - static_cast<long long>(row) * c.n_kv_heads);
    const long long to = ((static_cast<long long>(r) * T + row) * c.n_kv_heads + h) * HD + 16 * u;
    uint4 k[2] = {}, v[2] = {};
    if (row < ctx) {
      const int page = c.page_table[static_cast<long long>(r) * c.table_len + row / c.page], slot = row % c.page;
      if (page < 0 || page >= c.n_pages) {
        atomicOr(&g_mtp_error_word, MTP_DEVERR_PAGE_RANGE);
      } else {
        const long long head = static_cast<long long>(page) * c.n_kv_heads + h;
        const size_t at = (static_cast<size_t>(head) * c.page + slot) * HD + 16 * u;
        if constexpr (kF8) {
          const long long s = head * (c.page >> 4) + (slot >> 4);
          const uint4 kc = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.k) + at);
          const uint4 vc = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.v) + at);
          const float ks = power_of_two(scale_exponent(c.k_scale[s])), vs = power_of_two(scale_exponent(c.v_scale[s]));
          const uint32_t kw[4] = {kc.x, kc.y, kc.z, kc.w}, vw[4] = {vc.x, vc.y, vc.z, vc.w};
          uint32_t* ko = reinterpret_cast<uint32_t*>(k);
          uint32_t* vo = reinterpret_cast<uint32_t*>(v);
  #pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x[4];
            unpack_e4m3(kw[j], x);
            ko[2 * j] = pack2_bf16(x[0] * ks, x[1] * ks);
            ko[2 * j + 1] = pack2_bf16(x[2] * ks, x[3] * ks);
            unpack_e4m3(vw[j], x);
            vo[2 * j] = pack2_bf16(x[0] * vs, x[1] * vs);
            vo[2 * j + 1] = pack2_bf16(x[2] * vs, x[3] * vs);
          }
        } else {
          const uint4* kp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c.k) + at);
          const uint4* vp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c.v) + at);
          k[0] = kp[0], k[1] = kp[1], v[0] = vp[0], v[1] = vp[1];
        }
      }
    }
    uint4* ko = reinterpret_cast<uint4*>(k_out + to);
    uint4* vo = reinterpret_cast<uint4*>(v_out + to);
    ko[0] = k[0], ko[1] = k[1], vo[0] = v[0], vo[1] = v[1];
  }
}

template <int HD, bool kDense>
void gather_launch(const mtp_paged_cache& c, const dim3& grid, int T, const int32_t* ctx_len, void* k_out, void* v_out, int L,
                   const int32_t* n_new, int causal, int32_t* ctx_out, cudaStream_t st) {
  __nv_bfloat16 *k = static_cast<__nv_bfloat16*>(k_out), *v = static_cast<__nv_bfloat16*>(v_out);
  if (c.dtype == MTP_E4M3)
    kv_gather_kernel<HD, true, kDense><<<grid, kThreads, 0, st>>>(c, T, ctx_len, k, v, L, n_new, causal, ctx_out);
  else
    kv_gather_kernel<HD, false, kDense><<<grid, kThreads, 0, st>>>(c, T, ctx_len, k, v, L, n_new, causal, ctx_out);
}

mtp_status rotation_check(const mtp_rotation* rot, int head_dim) {
  if (!rot || !rot->inv_freq) return MTP_OK;
  if (rot->rot < 2 || rot->rot % 2 || rot->rot > head_dim) return MTP_ERR_SHAPE;
  if (!(std::fabs(rot->mscale) <= 3.4e38f)) return MTP_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(rot->inv_freq) & 7u) return MTP_ERR_ALIGNMENT;
  return MTP_OK;
}
// whether two rows of hd elements at n on + h oh, n < N and h < H, share one
bool rows_meet(long long N, long long H, int hd, long long on, long long oh) {
  if ((N > 1 && on < hd) || (H > 1 && oh < hd)) return true;
  if (N == 1 || H == 1) return false;
  if (on > oh ? on - hd >= (H - 1) * oh : oh - hd >= (N - 1) * on) return false;  // one within a step of the other
  for (long long h = 1; h < H; ++h) {  // the two rows n below and above h oh
    const long long n = h * oh / on, over = h * oh - n * on;
    if ((n < N && over < hd) || (n + 1 < N && on - over < hd)) return true;
  }
  return false;
}
// whether [a, a + a_bytes) and [b, b + b_bytes) share a byte
bool ranges_meet(const void* a, unsigned long long a_bytes, const void* b, unsigned long long b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

mtp_status kv_dense_launch(const mtp_paged_cache& c, int R, int L, long long T, const int32_t* ctx_len, const int32_t* n_new,
                           bool causal, void* k_out, void* v_out, int32_t* ctx_out, cudaStream_t st) {
  const long long blocks = (T * c.n_kv_heads * (c.head_dim / 16) + kThreads - 1) / kThreads;
  if (T > 0x7FFFFFFFll || R > 65535) return MTP_ERR_UNSUPPORTED;
  // the lengths are the device's: some 16 CTAs per SM go over what there is
  const long long most = std::max(1ll, 16ll * sm_count_current() / R);
  const dim3 grid(static_cast<unsigned>(std::min(blocks, most)), static_cast<unsigned>(R));
  if (c.head_dim == 128)
    gather_launch<128, true>(c, grid, static_cast<int>(T), ctx_len, k_out, v_out, L, n_new, causal, ctx_out, st);
  else
    gather_launch<64, true>(c, grid, static_cast<int>(T), ctx_len, k_out, v_out, L, n_new, causal, ctx_out, st);
  note_launch();
  MTP_LAUNCH_CHECK();
  return MTP_OK;
}

mtp_status paged_cache_check(const mtp_paged_cache* c, bool pointers) {
  if (!c) return MTP_ERR_INVALID_ARG;
  if (c->dtype != MTP_BF16 && c->dtype != MTP_E4M3) return MTP_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return MTP_ERR_UNSUPPORTED;
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->table_len < 1 || c->page < 1) return MTP_ERR_SHAPE;
  if (c->page % 16 || c->page > 1024) return MTP_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->n_pages) * c->n_kv_heads > 0x7FFFFFFFll) return MTP_ERR_SHAPE;
  if (static_cast<long long>(c->table_len) * c->page > 0x7FFFFFFFll - 255) return MTP_ERR_SHAPE;
  if (!pointers) return MTP_OK;
  if (!c->k || !c->v || !c->page_table) return MTP_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->page_table)) return MTP_ERR_ALIGNMENT;
  if (c->dtype == MTP_E4M3) {
    if (!c->k_scale || !c->v_scale) return MTP_ERR_INVALID_ARG;
    if (!aligned4(c->k_scale) || !aligned4(c->v_scale)) return MTP_ERR_ALIGNMENT;
  }
  return MTP_OK;
}

}  // namespace mtp

using namespace mtp;

extern "C" mtp_status mtp_rope_frequencies(int rot, double base, int scaling, double factor, double original, double beta_slow,
                                           double beta_fast, double* out, float* mscale) {
  if (!out || rot < 2 || rot % 2) return MTP_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base)) return MTP_ERR_INVALID_ARG;
  if (scaling < MTP_ROPE_NONE || scaling > MTP_ROPE_BANDS) return MTP_ERR_INVALID_ARG;
  if (scaling != MTP_ROPE_NONE && !(factor >= 1.0 && std::isfinite(factor))) return MTP_ERR_INVALID_ARG;
  if (scaling >= MTP_ROPE_YARN && !(original > 0.0 && beta_slow > 0.0 && beta_fast > beta_slow && std::isfinite(original) &&
                                    std::isfinite(beta_fast)))
    return MTP_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  const int n = rot / 2;
  double low = 0.0, high = 1.0;
  if (scaling == MTP_ROPE_YARN) {  // index of the pair that turns so many times within `original` positions
    const auto at = [&](double turns) { return rot * std::log(original / (turns * two_pi)) / (2.0 * std::log(base)); };
    low = std::fmax(std::floor(at(beta_fast)), 0.0);
    high = std::fmin(std::ceil(at(beta_slow)), rot - 1.0);  // (behind the last pair too: the ramp's slope is the method's)
    high = std::fmax(high, low + 1e-3);
  }
  for (int p = 0; p < n; ++p) {
    const double f = std::pow(base, -2.0 * p / rot);
    double keep = 1.0;  // share of the unscaled frequency
    if (scaling == MTP_ROPE_LINEAR) keep = 0.0;
    if (scaling == MTP_ROPE_YARN) keep = 1.0 - std::fmin(std::fmax((p - low) / (high - low), 0.0), 1.0);
    if (scaling == MTP_ROPE_BANDS)
      keep = std::fmin(std::fmax((original * f / two_pi - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0);
    out[p] = scaling == MTP_ROPE_NONE ? f : f * keep + f / factor * (1.0 - keep);
  }
  if (mscale) *mscale = scaling == MTP_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return MTP_OK;
}

extern "C" mtp_status mtp_rope(long long N, int H, int head_dim, int dtype, const mtp_rotation* rotation, const int32_t* pos,
                               int backward, const void* x, long long xn, long long xh, void* out, long long on, long long oh,
                               cudaStream_t st) {
  if (!rotation || !rotation->inv_freq) return MTP_ERR_INVALID_ARG;
  if (N < 0 || H < 1 || head_dim < 2) return MTP_ERR_INVALID_ARG;
  if (dtype != MTP_F32 && dtype != MTP_BF16) return MTP_ERR_UNSUPPORTED;
  if (head_dim % 2 || head_dim > 1024 || H > 65535 || N > 0x7FFFFFFFll) return MTP_ERR_UNSUPPORTED;
  if (const mtp_status s = rotation_check(rotation, head_dim); s != MTP_OK) return s;
  if (N == 0) return MTP_OK;
  if (!x || !out || !pos) return MTP_ERR_INVALID_ARG;
  const long long dense = static_cast<long long>(H) * head_dim;
  if (xh == 0) xh = head_dim;
  if (xn == 0) xn = dense;
  if (oh == 0) oh = head_dim;
  if (on == 0) on = dense;
  if (xn < 0 || xh < 0 || on < 0 || oh < 0) return MTP_ERR_SHAPE;
  if (rows_meet(N, H, head_dim, on, oh)) return MTP_ERR_SHAPE;
  const int bytes = dtype == MTP_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & (bytes - 1)) return MTP_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(pos) & 3u) return MTP_ERR_ALIGNMENT;
  if (x == out) {
    if ((N > 1 && xn != on) || (H > 1 && xh != oh)) return MTP_ERR_INVALID_ARG;
  } else {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(out);
    const uintptr_t ea = a + ((N - 1) * xn + (H - 1) * xh + head_dim) * bytes, eb = b + ((N - 1) * on + (H - 1) * oh + head_dim) * bytes;
    if (a < eb && b < ea) {
      // parts of one buffer that lie side by side within a row (both with its stride) do not meet
      const uintptr_t gap = a < b ? b - a : a - b;
      const long long span_x = (H - 1) * xh + head_dim, span_o = (H - 1) * oh + head_dim;
      const long long off = static_cast<long long>(gap / bytes) % (xn > 0 ? xn : 1);
      const bool apart = gap % bytes == 0 && xn == on && N > 1 &&
                         (a < b ? off >= span_x && off + span_o <= xn : off >= span_o && off + span_x <= xn);
      if (!apart) return MTP_ERR_INVALID_ARG;
    }
  }
  RopeArgs g{};
  // runs of 16 bytes per thread, bf16 also of 8 (921 x 118 heads of 128, 24 elements turned: 24 us, 21 of neighbours; all of them in
  // runs of 16 bytes 14, element by element 29)
  const auto fits = [&](int run) {  // elements
    const uintptr_t at = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out);
    return rotation->rot % (2 * run) == 0 && head_dim % (2 * run) == 0 && at % (run * bytes) == 0 && (xn | xh | on | oh) % run == 0;
  };
  const bool narrow = dtype == MTP_BF16 && !fits(8), vec = fits(narrow || dtype == MTP_F32 ? 4 : 8);
  const int pairs = narrow || dtype == MTP_F32 ? 4 : 8;
  g.N = N, g.H = H, g.hd = head_dim, g.rot = rotation->rot, g.units = (head_dim + 2 * pairs - 1) / (2 * pairs);
  g.mscale = rotation->mscale, g.backward = backward, g.inv_freq = rotation->inv_freq, g.pos = pos;
  g.xn = xn, g.xh = xh, g.on = on, g.oh = oh;
  // A block's work: four units per thread, the loads that are asked for at once (4096 positions of 112 heads of 128 41 us; eight 44,
  // sixteen 50, for fewer blocks at a time leave SMs waiting at the end; two 51, as a position's angles are worked out
  // twice).  Where that leaves SMs without any, one.
  const int most = kThreads * 4;
  g.heads = H * g.units <= most ? H : most / g.units;
  g.tokens = most / (g.heads * g.units) < 1 ? 1 : most / (g.heads * g.units);
  if (g.tokens > 8) g.tokens = 8;
  if ((N + g.tokens - 1) / g.tokens * ((H + g.heads - 1) / g.heads) < 2 * sm_count_current()) {
    g.tokens = 1;
    g.heads = H * g.units <= kThreads ? H : kThreads / g.units < 1 ? 1 : kThreads / g.units;
  }
  const auto magic = [](int d) { return d == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + d - 1) / d); };
  g.per_magic = magic(g.heads * g.units), g.units_magic = magic(g.units);
  const bool inter = rotation->interleaved != 0;
  if (dtype == MTP_F32) return rope_launch<float, 4>(g, vec, inter, x, out, st);
  return narrow ? rope_launch<__nv_bfloat16, 4>(g, vec, inter, x, out, st) : rope_launch<__nv_bfloat16, 8>(g, vec, inter, x, out, st);
}

extern "C" mtp_status mtp_kv_append(const mtp_paged_cache* cache, const mtp_kv_rows* rows, const mtp_rotation* rotation,
                                    cudaStream_t st) {
  if (const mtp_status s = paged_cache_check(cache, false); s != MTP_OK) return s;
  if (!rows) return MTP_ERR_INVALID_ARG;
  AppendArgs g{};
  g.c = *cache;
  g.w = *rows;
  mtp_kv_rows& w = g.w;
  const int hd = cache->head_dim, Hkv = cache->n_kv_heads;
  if (w.R < 0 || w.L < 0 || w.n_heads < 0) return MTP_ERR_INVALID_ARG;
  if (const mtp_status s = rotation_check(rotation, hd); s != MTP_OK) return s;
  if ((w.q == nullptr) != (w.q_out == nullptr) || (w.q && w.n_heads < 1)) return MTP_ERR_INVALID_ARG;
  if (w.R == 0 || w.L == 0) return MTP_OK;  // (a table without requests has no address)
  if (const mtp_status s = paged_cache_check(cache, true); s != MTP_OK) return s;
  if (!w.k || !w.v || !w.ctx_len) return MTP_ERR_INVALID_ARG;
  if (!aligned16(w.k) || !aligned16(w.v) || !aligned16(w.q) || !aligned16(w.q_out)) return MTP_ERR_ALIGNMENT;
  if (!aligned4(w.ctx_len) || !aligned4(w.n_new) || !aligned4(w.pos)) return MTP_ERR_ALIGNMENT;
  auto fill = [](long long& v, long long dense) {
    if (v == 0) v = dense;
    return v > 0 && v % 8 == 0;
  };
  if (!fill(w.kv_stride_h, hd) || !fill(w.kv_stride_t, static_cast<long long>(Hkv) * hd) ||
      !fill(w.kv_stride_r, static_cast<long long>(w.L) * Hkv * hd))
    return MTP_ERR_ALIGNMENT;
  if (w.q && (!fill(w.q_stride_h, hd) || !fill(w.q_stride_t, static_cast<long long>(w.n_heads) * hd) ||
              !fill(w.q_stride_r, static_cast<long long>(w.L) * w.n_heads * hd)))
    return MTP_ERR_ALIGNMENT;
  if (w.q == w.q_out && w.q && (w.q_stride_h != hd || w.q_stride_t != static_cast<long long>(w.n_heads) * hd ||
                                w.q_stride_r != static_cast<long long>(w.L) * w.n_heads * hd))
    return MTP_ERR_INVALID_ARG;
  if (w.q) {  // q_out is written while other blocks read
    const auto span = [&](long long heads, long long sr, long long st, long long sh) {
      return 2ull * ((w.R - 1) * sr + (w.L - 1) * st + (heads - 1) * sh + hd);
    };
    const unsigned long long out = 2ull * w.R * w.L * w.n_heads * hd, kv = span(Hkv, w.kv_stride_r, w.kv_stride_t, w.kv_stride_h);
    if (ranges_meet(w.q_out, out, w.k, kv) || ranges_meet(w.q_out, out, w.v, kv) ||
        (w.q != w.q_out && ranges_meet(w.q_out, out, w.q, span(w.n_heads, w.q_stride_r, w.q_stride_t, w.q_stride_h))))
      return MTP_ERR_INVALID_ARG;
  }
  const bool turned = rotation && rotation->inv_freq;
  g.rot = turned ? rotation->rot : 0;
  g.mscale = turned ? rotation->mscale : 1.f;
  g.inv_freq = turned ? rotation->inv_freq : nullptr;
  g.kv_blocks = static_cast<int>((w.L + 14ll) / 16 + 1);
  g.kv_groups = (Hkv + kWarps - 1) / kWarps;
  g.kv_ctas = static_cast<long long>(w.R) * g.kv_blocks * g.kv_groups;
  g.q_groups = w.q ? (w.n_heads + kWarps - 1) / kWarps : 0;
  g.q_chunks = static_cast<int>((w.L + 15ll) / 16);
  const long long ctas = g.kv_ctas + static_cast<long long>(w.R) * g.q_chunks * g.q_groups;
  if (ctas > 0x7FFFFFFFll) return MTP_ERR_UNSUPPORTED;
  const bool inter = turned && rotation->interleaved, vec = g.rot % 16 == 0;
  const bool f8 = cache->dtype == MTP_E4M3;
  if (hd == 128)
    f8 ? append_launch<128, true>(g, vec, inter, static_cast<unsigned>(ctas), st) : append_launch<128, false>(g, vec, inter, static_cast<unsigned>(ctas), st);
  else
    f8 ? append_launch<64, true>(g, vec, inter, static_cast<unsigned>(ctas), st) : append_launch<64, false>(g, vec, inter, static_cast<unsigned>(ctas), st);
  note_launch();
  MTP_LAUNCH_CHECK();
  return MTP_OK;
}

extern "C" mtp_status mtp_kv_gather(const mtp_paged_cache* cache, int R, int T, const int32_t* ctx_len, void* k_out, void* v_out,
                                    cudaStream_t st) {
  if (const mtp_status s = paged_cache_check(cache, false); s != MTP_OK) return s;
  if (R < 0 || T < 0) return MTP_ERR_INVALID_ARG;
  if (R > 65535) return MTP_ERR_UNSUPPORTED;
  if (T > static_cast<long long>(cache->table_len) * cache->page) return MTP_ERR_SHAPE;
  if (R == 0 || T == 0) return MTP_OK;
  if (const mtp_status s = paged_cache_check(cache, true); s != MTP_OK) return s;
  if (!ctx_len || !k_out || !v_out) return MTP_ERR_INVALID_ARG;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned4(ctx_len)) return MTP_ERR_ALIGNMENT;
  const long long units = static_cast<long long>(T) * cache->n_kv_heads * (cache->head_dim / 16);
  const long long blocks = (units + kThreads - 1) / kThreads;
  if (blocks > 0x7FFFFFFFll) return MTP_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(R));
  if (cache->head_dim == 128)
    gather_launch<128, false>(*cache, grid, T, ctx_len, k_out, v_out, 0, nullptr, 0, nullptr, st);
  else
    gather_launch<64, false>(*cache, grid, T, ctx_len, k_out, v_out, 0, nullptr, 0, nullptr, st);
  note_launch();
  MTP_LAUNCH_CHECK();
  return MTP_OK;
}
