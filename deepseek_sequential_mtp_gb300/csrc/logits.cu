// mtp_logits_probs: logits of the target's (or the draft's) head to the
// probability rows that spec_verify reads.
//
// Row (r, j) is position j of request r: its text is the request's tokens so
// far followed by the drafts y_0 .. y_{j-1}.  With n(v) the number of times v
// was generated (prompt tokens do not count) and seen(v) whether it occurs at
// all, the row's logits become
//   z(v) = seen(v) ? (x(v) > 0 ? x(v) / rep : x(v) rep) : x(v)
//   z(v) -= freq n(v) + pres [n(v) > 0];  z(v) += bias(v);  z(v) = -inf where the mask bit is 0
//   p = softmax(z / temperature), or the one-hot of the lowest index of the maximum at temperature 0.
//
// Bound: HBM.  A row is read once and written once (4 or 2 bytes in, 4 out, one
// mask bit).  A cluster of C CTAs holds the row in registers (kThreads x 4 NV
// values per CTA), so the maximum and the sum need one exchange: every CTA
// forms e = exp((z - m_c) / T) against its own maximum m_c, sums it, and sends
// (m_c, s_c) to the cluster's CTAs, after which each scales its values by
// exp((m_c - M) / T) / S.  Sums are fp32 over at most 64 values per thread
// and a tree above that.
//
// Penalties and biases are sparse, the row is dense: one 32-bit word of shared
// memory per vocabulary entry of the CTA's slice collects them -- bits 0-18
// count the generated occurrences, bit 19 marks any occurrence, bits 20-31
// hold 1 + the index of the request's bias entry (the last entry of an id
// wins) -- by integer atomics, whose order cannot change the result.  The
// history is scanned while the row's loads are in flight.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "mbarrier.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxNV = 16;                                         // 4-value vectors per thread
constexpr int kMaxVocab = kMaxCluster * kMaxNV * 4 * kThreads;     // 524288
constexpr uint32_t kSeenBit = 1u << 19, kCountMask = kSeenBit - 1;
constexpr int kBiasShift = 20, kMaxBias = (1 << 12) - 1;
constexpr int kMaxHist = 1 << 18;  // hist_cap + drafts stay below the 19-bit count
constexpr int kMaxDrafts = 1 << 16;

struct Args {
  const void* logits;
  long long ld;
  float* p;
  int32_t* status;
  mtp_logits_params prm;
  int L, V, slice, use_words, has_pen;
};

// what a CTA tells its cluster about its slice
struct Part {
  float m, s;
  int best;  // lowest index of the maximum (greedy rows)
  int bad;   // a NaN or +inf among the allowed logits
};

__device__ __forceinline__ float exp_scaled(float x) {  // e^x
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = mtp::unpack2_bf16(u.x), b = mtp::unpack2_bf16(u.y);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  }
}

// Value e of vector i of a thread is entry off(i, e) of the CTA's slice: with
// VEC four neighbours per thread (16-byte accesses), else one entry per
// thread and access (rows that are not 16-byte aligned).
template <int NV, bool VEC, typename T>
__global__ void __launch_bounds__(kThreads)
logits_probs_kernel(const Args a) {
  extern __shared__ __align__(16) uint32_t words[];
  __shared__ float s_red[kWarps];
  __shared__ int s_redi[kWarps];
  __shared__ Part parts[kMaxCluster];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  // the other CTAs' shared memory may be written once they have started
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const long long row = blockIdx.x / C;
  const int r = static_cast<int>(row / a.L), j = static_cast<int>(row % a.L);
  const int lo = rank * a.slice;
  const int n = min(max(a.V - lo, 0), a.slice);
  const mtp_logits_params& q = a.prm;

  auto off = [&](int i, int e) { return VEC ? (i * kThreads + t) * 4 + e : (i * 4 + e) * kThreads + t; };
  const T* src = static_cast<const T*>(a.logits) + row * a.ld + lo;
  float z[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (VEC) {  // n is a multiple of 4
      if (off(i, 0) < n) load4(src + off(i, 0), z[i]);
      else z[i][0] = z[i][1] = z[i][2] = z[i][3] = -INFINITY;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) z[i][e] = off(i, e) < n ? mtp::load_f32<T>(src + off(i, e)) : -INFINITY;
    }
  }
  const float temp = q.temperature ? q.temperature[r] : 1.f;
  const float rep = q.repetition ? q.repetition[r] : 1.f;
  const float freq = q.frequency ? q.frequency[r] : 0.f;
  const float pres = q.presence ? q.presence[r] : 0.f;
  const bool params_ok = temp >= 0.f && temp < INFINITY && rep > 0.f && rep < INFINITY && fabsf(freq) < INFINITY &&
                         fabsf(pres) < INFINITY;

  if (a.use_words) {
    for (int i = t * 4; i < n; i += kThreads * 4) *reinterpret_cast<uint4*>(words + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (q.n_bias > 0) {
      const int32_t* ids = q.bias_ids + static_cast<size_t>(r) * q.n_bias;
      for (int i = t; i < q.n_bias; i += kThreads) {
        const unsigned v = static_cast<unsigned>(ids[i]) - static_cast<unsigned>(lo);
        if (ids[i] >= 0 && v < static_cast<unsigned>(n)) atomicMax(&words[v], static_cast<uint32_t>(i + 1) << kBiasShift);
      }
      __syncthreads();
    }
    if (a.has_pen) {
      const int len = q.hist ? min(max(q.hist_len ? q.hist_len[r] : q.hist_cap, 0), q.hist_cap) : 0;
      const int made = q.prompt_len ? q.prompt_len[r] : 0;  // tokens from here on were generated
      const int32_t* h = q.hist + static_cast<size_t>(r) * q.hist_cap;
      for (int i = t; i < len; i += kThreads) {
        const int id = h[i];
        const unsigned v = static_cast<unsigned>(id) - static_cast<unsigned>(lo);
        if (id >= 0 && v < static_cast<unsigned>(n)) {
          if (i < made) atomicOr(&words[v], kSeenBit);
          else atomicAdd(&words[v], 1u);
        }
      }
      if (q.draft) {
        const int32_t* y = q.draft + static_cast<size_t>(r) * (a.L - 1);
        for (int i = t; i < j; i += kThreads) {
          const int id = y[i];
          const unsigned v = static_cast<unsigned>(id) - static_cast<unsigned>(lo);
          if (id >= 0 && v < static_cast<unsigned>(n)) atomicAdd(&words[v], 1u);
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t w4[4];
      if constexpr (VEC) {
        const uint4 u = off(i, 0) < n ? *reinterpret_cast<const uint4*>(words + off(i, 0)) : make_uint4(0, 0, 0, 0);
        w4[0] = u.x; w4[1] = u.y; w4[2] = u.z; w4[3] = u.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w4[e] = off(i, e) < n ? words[off(i, e)] : 0u;
      }
      if ((w4[0] | w4[1] | w4[2] | w4[3]) == 0u) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = w4[e];
        if (w == 0u) continue;
        float v = z[i][e];
        const uint32_t cnt = w & kCountMask;
        if (w & (kSeenBit | kCountMask)) v = v > 0.f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
        if (cnt) v = __fsub_rn(v, __fadd_rn(__fmul_rn(freq, static_cast<float>(cnt)), pres));
        if (w >> kBiasShift) v = __fadd_rn(v, q.bias[static_cast<size_t>(r) * q.n_bias + (w >> kBiasShift) - 1]);
        z[i][e] = v;
      }
    }
  }
  if (q.mask) {  // a CTA's slice starts at a multiple of 32
    const uint32_t* mw = q.mask + row * ((a.V + 31) / 32) + lo / 32;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (VEC) {
        const uint32_t bits = off(i, 0) < n ? mw[off(i, 0) >> 5] >> (off(i, 0) & 31) : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((bits >> e) & 1u)) z[i][e] = -INFINITY;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (off(i, e) >= n || !((mw[off(i, e) >> 5] >> (off(i, e) & 31)) & 1u)) z[i][e] = -INFINITY;
      }
    }
  }
  // the slice's maximum; fmaxf drops a NaN, so the flag looks for it beside +inf
  float m = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bad |= !(z[i][e] < INFINITY);
      m = fmaxf(m, z[i][e]);
    }
  m = mtp::warp_max(m);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    s_red[warp] = m;
    s_redi[warp] = bad;
  }
  __syncthreads();
  m = -INFINITY;
  int any_bad = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    m = fmaxf(m, s_red[w]);
    any_bad |= s_redi[w];
  }
  __syncthreads();
  const bool greedy = temp == 0.f;
  const float inv_t = greedy ? 0.f : fminf(1.f / temp, 3.4028234e38f);
  float sum = 0.f;
  int best = 0x7fffffff;
  if (!greedy) {
    // a slice without a finite maximum has e = 0 everywhere (its z are -inf)
    const float mz = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) z[i][e] = exp_scaled((z[i][e] - mz) * inv_t);
      sum += (z[i][0] + z[i][1]) + (z[i][2] + z[i][3]);
    }
    sum = mtp::warp_sum(sum);
    if (lane == 0) s_red[warp] = sum;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (z[i][e] == m && off(i, e) < n) best = min(best, lo + off(i, e));
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0) s_redi[warp] = best;
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (warp == 0) {
    if (!greedy) {
      sum = mtp::warp_sum(lane < kWarps ? s_red[lane] : 0.f);
    } else {
      best = __reduce_min_sync(0xffffffffu, lane < kWarps ? s_redi[lane] : 0x7fffffff);
    }
    if (lane < C) {
      Part* dst = cluster.map_shared_rank(parts, lane) + rank;
      *dst = Part{m, sum, best, any_bad};
    }
  }
  cluster.sync();  // nobody touches another CTA's shared memory after this
  float M = -INFINITY;
  any_bad = 0;
  for (int c = 0; c < C; ++c) {
    M = fmaxf(M, parts[c].m);
    any_bad |= parts[c].bad;
  }
  float factor = 0.f;
  best = 0x7fffffff;
  const bool row_ok = params_ok && !any_bad && M != -INFINITY;
  if (row_ok) {
    if (!greedy) {
      float S = 0.f;
      for (int c = 0; c < C; ++c)
        if (parts[c].m != -INFINITY) S += parts[c].s * exp_scaled((parts[c].m - M) * inv_t);
      if (m != -INFINITY) factor = exp_scaled((m - M) * inv_t) / S;
    } else {
      for (int c = 0; c < C; ++c)
        if (parts[c].m == M) best = min(best, parts[c].best);
    }
  }
  float* dst = a.p + row * a.V + lo;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = !row_ok ? 0.f : greedy ? (lo + off(i, e) == best ? 1.f : 0.f) : z[i][e] * factor;
    if constexpr (VEC) {
      if (off(i, 0) < n) *reinterpret_cast<float4*>(dst + off(i, 0)) = make_float4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (off(i, e) < n) dst[off(i, e)] = o[e];
    }
  }
  if (rank == 0 && t == 0 && a.status)
    a.status[row] = !params_ok ? MTP_LOGITS_INVALID_PARAM
                    : any_bad  ? MTP_LOGITS_INVALID
                    : M == -INFINITY ? MTP_LOGITS_EMPTY
                                     : MTP_LOGITS_OK;
}

template <int NV, bool VEC, typename T>
mtp_status launch(const Args& a, long long rows, int C, cudaStream_t st) {
  static mtp::PerDevice attr_smem, attr_cluster;
  const int smem = a.use_words ? a.slice * 4 : 0;
  auto kernel = logits_probs_kernel<NV, VEC, T>;
  if (!mtp::smem_limit(attr_smem, kernel, NV * 4 * kThreads * 4)) return MTP_ERR_CUDA;
  const int dev = mtp::current_device();
  if (C > 8 && dev >= 0 && (dev >= mtp::kMaxDevices || !attr_cluster.v[dev].load(std::memory_order_acquire))) {
    MTP_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    if (dev < mtp::kMaxDevices) attr_cluster.v[dev].store(1, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(C), 1u, 1u};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MTP_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, a));
  mtp::note_launch();
  return MTP_OK;
}

template <int NV, typename T>
mtp_status launch_vec(const Args& a, long long rows, int C, bool vec, cudaStream_t st) {
  return vec ? launch<NV, true, T>(a, rows, C, st) : launch<NV, false, T>(a, rows, C, st);
}

template <typename T>
mtp_status launch_nv(const Args& a, long long rows, int C, int nv, bool vec, cudaStream_t st) {
  switch (nv) {
    case 1: return launch_vec<1, T>(a, rows, C, vec, st);
    case 2: return launch_vec<2, T>(a, rows, C, vec, st);
    case 4: return launch_vec<4, T>(a, rows, C, vec, st);
    case 8: return launch_vec<8, T>(a, rows, C, vec, st);
    default: return launch_vec<16, T>(a, rows, C, vec, st);
  }
}

}  // namespace

extern "C" mtp_status mtp_logits_probs(int R, int L, int V, int dtype, const void* logits, long long ld,
                                       const mtp_logits_params* prm, float* p, int32_t* status, cudaStream_t st) {
  if (R < 0 || L < 1 || V < 1) return MTP_ERR_INVALID_ARG;
  if (dtype != MTP_F32 && dtype != MTP_BF16) return MTP_ERR_INVALID_ARG;
  if (R == 0) return MTP_OK;
  if (!logits || !p) return MTP_ERR_INVALID_ARG;
  if (V > kMaxVocab || L > kMaxDrafts) return MTP_ERR_UNSUPPORTED;
  if (ld < V) return MTP_ERR_SHAPE;
  const int esize = dtype == MTP_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(logits) % esize) || (reinterpret_cast<uintptr_t>(p) & 3u) ||
      (reinterpret_cast<uintptr_t>(status) & 3u))
    return MTP_ERR_ALIGNMENT;
  // the rows may be rewritten in place, but not through another row's logits
  if (static_cast<const void*>(p) == logits && (dtype != MTP_F32 || ld != V)) return MTP_ERR_INVALID_ARG;
  Args a{};
  if (prm) a.prm = *prm;
  const mtp_logits_params& q = a.prm;
  if (q.hist_cap < 0 || q.n_bias < 0) return MTP_ERR_INVALID_ARG;
  if (q.hist_cap > kMaxHist || q.n_bias > kMaxBias) return MTP_ERR_UNSUPPORTED;
  if (q.hist_cap > 0 && !q.hist) return MTP_ERR_INVALID_ARG;
  if (q.n_bias > 0 && (!q.bias_ids || !q.bias)) return MTP_ERR_INVALID_ARG;
  for (const void* ptr : {static_cast<const void*>(q.temperature), static_cast<const void*>(q.repetition),
                          static_cast<const void*>(q.frequency), static_cast<const void*>(q.presence),
                          static_cast<const void*>(q.hist), static_cast<const void*>(q.hist_len),
                          static_cast<const void*>(q.prompt_len), static_cast<const void*>(q.draft),
                          static_cast<const void*>(q.bias_ids), static_cast<const void*>(q.bias),
                          static_cast<const void*>(q.mask)})
    if (reinterpret_cast<uintptr_t>(ptr) & 3u) return MTP_ERR_ALIGNMENT;
  const long long rows = static_cast<long long>(R) * L;
  if (rows > 0x7FFFFFFFll / kMaxCluster) return MTP_ERR_UNSUPPORTED;

  a.logits = logits;
  a.ld = ld;
  a.p = p;
  a.status = status;
  a.L = L;
  a.V = V;
  a.has_pen = (q.repetition || q.frequency || q.presence) && (q.hist_cap > 0 || (q.draft && L > 1));
  if (L == 1) a.prm.draft = nullptr;
  a.use_words = a.has_pen || q.n_bias > 0;
  // Cluster size: the fewest CTAs that hold the row with 8 vectors per thread
  // (16 only where 16 CTAs need it); twice as many for as long as that still
  // leaves SMs idle and threads with more than one vector.
  auto vectors = [&](int c) {
    const int need = ((V + c - 1) / c + 4 * kThreads - 1) / (4 * kThreads);
    int nv = 1;
    while (nv < need) nv *= 2;
    return nv;
  };
  int C = 1;
  while (C < kMaxCluster && vectors(C) > 8) C *= 2;
  const int sms = mtp::sm_count_current();
  while (C < kMaxCluster && vectors(C) > 1 && rows * C * 2 <= sms) C *= 2;
  const int nv = vectors(C);
  a.slice = ((V + C - 1) / C + 31) / 32 * 32;
  if (a.slice > nv * 4 * kThreads) return MTP_ERR_UNSUPPORTED;  // not reached: both sides are multiples of 32
  const bool vec = V % 4 == 0 && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) % (4 * esize)) == 0 &&
                   mtp::aligned16(p);
  return dtype == MTP_F32 ? launch_nv<float>(a, rows, C, nv, vec, st)
                          : launch_nv<__nv_bfloat16>(a, rows, C, nv, vec, st);
}
