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
// Bound: HBM.  A row has to be read once (4 or 2 bytes a value and one mask bit)
// and written once (4 bytes).  A cluster of C CTAs takes a row, each CTA a slice:
// pass 1 streams the slice and keeps a running maximum and sum per thread,
// the cluster exchanges (maximum, sum), and pass 2 streams the slice again,
// out of L2 (or out of registers, where one batch of loads covers it), and
// writes p.  Holding the slices in registers instead reads nothing twice but
// leaves two CTAs per SM that wait for one phase after the other (120 us on
// 320 rows of 129280 bf16 logits with a 2048-token history, mask and biases;
// this form 74 us, 3.4 TB/s; of that the mask alone 59 us, a plain softmax 54, a
// streaming copy of the same bytes 41).  What is left is the marking's phases, in
// which every CTA of a cluster goes through the whole history.
//
// Penalties and biases are sparse, the row is dense.  A bit per vocabulary
// entry of the slice marks the ids that occur; the ranks of the set bits
// number them, and one 32-bit word per marked id collects what happens to it
// -- bits 0-18 count the generated occurrences, bit 19 marks any occurrence,
// bits 20-31 hold 1 + the index of the request's bias entry (the last entry of
// an id wins) -- by integer atomics, whose order cannot change the result.
// One thread per marked id forms its z; both passes leave these ids out, by
// the same bits as the grammar's, and their p are written last.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace {

// 256 threads with four vectors in flight, five CTAs per SM: over (threads,
// vectors, CTAs per SM) = (512, 8, 2), (512, 4, 3), (1024, 2, 2) this one was
// fastest on 320 rows of 129280 (by 2, 4 and 8 us).  Where the SMs hold the call's
// CTAs three at a time, the form with room for the registers that five leave in
// memory: one row of 32000 11.5 us instead of 16.5 in a graph, 28 rows 17.5 instead of
// 19.6, 32 rows of 129280 21.6 instead of 23.6; 320 rows 81 instead of 73.
constexpr int kThreads = 256;
constexpr int kManyCtas = 5, kFewCtas = 3;  // per SM
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;                 // 4-value vectors a thread has in flight
constexpr int kBatchValues = kBatch * 4 * kThreads;
constexpr int kMaxCluster = 16;
constexpr int kMaxVocab = 524288;                // as spec_verify
constexpr int kTargetSlice = 32768;              // entries of a CTA's slice where there are rows enough
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
  int L, V, slice, slots, has_pen, sparse, live;
};

// what a thread, a warp, a CTA knows about its values: their maximum, the sum
// of their exponentials against it (NaN where one of them is NaN or +inf) and,
// in greedy rows, the lowest index of the maximum
struct Part {
  float m, s;
  int best;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// four values as they are stored: 16 bytes of fp32 or 8 of bf16
template <typename T> struct Raw4;
template <> struct Raw4<float> {
  float4 v;
  __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
};
template <> struct Raw4<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xFFFF0000u);
    f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
};

// Vector i of batch b of a thread holds the slice's entries off(b, i, 0..3):
// with VEC four neighbours (16-byte accesses), else entries kThreads apart
// (rows that are not 16-byte aligned).
template <bool VEC, typename T, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas)
logits_probs_kernel(const Args a) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ Part warp_part[kWarps];
  __shared__ Part parts[kMaxCluster];
  __shared__ int warp_count[kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  // the other CTAs' shared memory may be written once they have started
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const long long row = blockIdx.x / static_cast<unsigned>(C);
  const unsigned r = static_cast<unsigned>(row) / static_cast<unsigned>(a.L);
  const int j = static_cast<int>(static_cast<unsigned>(row) - r * static_cast<unsigned>(a.L));
  const int lo = rank * a.slice;
  const int n = min(max(a.V - lo, 0), a.slice);
  const int nw = a.slice / 32;
  const mtp_logits_params& q = a.prm;
  uint32_t* live = smem;          // [nw] entries that the passes take: allowed and not marked
  uint32_t* marks = live + nw;    // [nw] ids that occur, or have a bias
  uint32_t* before = marks + nw;  // [nw] marked ids in the words before
  uint32_t* word = before + nw;   // [slots] what happens to a marked id, later its z
  uint16_t* token = reinterpret_cast<uint16_t*>(word + a.slots);  // [slots] its entry of the slice

  auto off = [&](int b, int i, int e) {
    return b * kBatchValues + (VEC ? (i * kThreads + t) * 4 + e : (i * 4 + e) * kThreads + t);
  };
  const T* src = static_cast<const T*>(a.logits) + row * a.ld + lo;
  const uint32_t* mask = q.mask ? q.mask + row * ((a.V + 31) / 32) + lo / 32 : nullptr;
  using Raw = typename std::conditional<VEC, Raw4<T>, float4>::type;
  Raw raw[kBatch];
  // `whole`: no entry of the batch is past the end
  auto fetch = [&](int b, auto whole) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if constexpr (VEC) {  // n is a multiple of 4
        if (whole.value || off(b, i, 0) < n) raw[i] = *reinterpret_cast<const Raw*>(src + off(b, i, 0));
      } else {
        raw[i].x = off(b, i, 0) < n ? mtp::load_f32<T>(src + off(b, i, 0)) : -INFINITY;
        raw[i].y = off(b, i, 1) < n ? mtp::load_f32<T>(src + off(b, i, 1)) : -INFINITY;
        raw[i].z = off(b, i, 2) < n ? mtp::load_f32<T>(src + off(b, i, 2)) : -INFINITY;
        raw[i].w = off(b, i, 3) < n ? mtp::load_f32<T>(src + off(b, i, 3)) : -INFINITY;
      }
    }
  };
  // the live values of vector i, -inf for the others
  auto values = [&](int b, int i, float (&z)[4], auto whole) {
    if constexpr (VEC) {
      const int o = off(b, i, 0);
      raw[i].get(z);
      if (whole.value) {
        if (a.live) {
          const uint32_t on = live[o >> 5] >> (4 * t & 31);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(on & (1u << e))) z[e] = -INFINITY;
        }
      } else {
        uint32_t on = o < n ? 0xFu : 0u;
        if (a.live && o < n) on = live[o >> 5] >> (o & 31);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!(on & (1u << e))) z[e] = -INFINITY;
      }
    } else {
      z[0] = raw[i].x; z[1] = raw[i].y; z[2] = raw[i].z; z[3] = raw[i].w;
      if (a.live) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int o = off(b, i, e);
          if (o < n && !((live[o >> 5] >> (o & 31)) & 1u)) z[e] = -INFINITY;
        }
      }
    }
  };
  const int batches = (n + kBatchValues - 1) / kBatchValues;
  // runs f(b, whole) on batch b, with a form of its own for the whole ones
  auto batch = [&](int b, auto f) {
    if (VEC && (b + 1) * kBatchValues <= n)
      f(std::true_type());
    else
      f(std::false_type());
  };
  fetch(0, std::false_type());

  const float temp = q.temperature ? q.temperature[r] : 1.f;
  const float rep = q.repetition ? q.repetition[r] : 1.f;
  const float freq = q.frequency ? q.frequency[r] : 0.f;
  const float pres = q.presence ? q.presence[r] : 0.f;
  const bool params_ok = temp >= 0.f && temp < INFINITY && rep > 0.f && rep < INFINITY && fabsf(freq) < INFINITY &&
                         fabsf(pres) < INFINITY;
  const bool greedy = temp == 0.f;
  const float k = fminf(1.4426950408889634f / temp, 3.4028234e38f);  // e^(x / T) = 2^(x k)

  Part mine{-INFINITY, 0.f, 0x7fffffff};
  // one value more (greedy rows keep s = NaN for a NaN or +inf)
  auto add = [&](float z, int index) {
    if (greedy) {
      if (!(z < INFINITY)) mine.s = NAN;
      if (z > mine.m || (z == mine.m && index < mine.best)) {
        mine.m = z;
        mine.best = index;
      }
    } else {
      const float mn = fmaxf(mine.m, z), mz = mn == -INFINITY ? 0.f : mn;
      mine.s = mine.s * ex2((mine.m - mz) * k) + ex2((z - mz) * k);
      mine.m = mn;
    }
  };

  int n_marked = 0;
  if (a.sparse) {
    const int len = a.has_pen && q.hist ? min(max(q.hist_len ? q.hist_len[r] : q.hist_cap, 0), q.hist_cap) : 0;
    const int made = q.prompt_len ? q.prompt_len[r] : 0;  // tokens from here on were generated
    const int32_t* h = q.hist + static_cast<size_t>(r) * q.hist_cap;
    const int32_t* y = q.draft + static_cast<size_t>(r) * (a.L - 1);
    const int n_draft = a.has_pen && q.draft ? j : 0;
    const int32_t* ids = q.bias_ids + static_cast<size_t>(r) * q.n_bias;
    auto entry = [&](int id) {  // index within the slice, or -1
      const unsigned v = static_cast<unsigned>(id) - static_cast<unsigned>(lo);
      return id >= 0 && v < static_cast<unsigned>(n) ? static_cast<int>(v) : -1;
    };
    auto mark = [&](int id) {
      const int v = entry(id);
      if (v >= 0) atomicOr(&marks[v >> 5], 1u << (v & 31));
    };
    for (int i = t; i < nw; i += kThreads) marks[i] = 0u;
    for (int i = t; i < a.slots; i += kThreads) word[i] = 0u;
    __syncthreads();
    // f(id, place) for a list's ids, four loads in flight per thread (one after the other they
    // took a third of the marking's time)
    auto each = [&](const int32_t* list, int count, auto f) {
      for (int i = t; i < count; i += 4 * kThreads) {
        int id[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) id[u] = i + u * kThreads < count ? list[i + u * kThreads] : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u) f(id[u], i + u * kThreads);
      }
    };
    each(h, len, [&](int id, int) { mark(id); });
    each(y, n_draft, [&](int id, int) { mark(id); });
    each(ids, q.n_bias, [&](int id, int) { mark(id); });
    __syncthreads();
    {  // ranks: every thread counts a run of words, scanned over the CTA
      const int per = (nw + kThreads - 1) / kThreads, w0 = t * per;
      int count = 0;
      for (int i = w0; i < min(w0 + per, nw); ++i) {
        const uint32_t mk = marks[i];
        live[i] = (mask ? (i * 32 < n ? mask[i] : 0u) : 0xFFFFFFFFu) & ~mk;
        count += __popc(mk);
      }
      int incl = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      if (lane == 31) warp_count[warp] = incl;
      __syncthreads();
      int base = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) base += warp_count[w];
        n_marked += warp_count[w];
      }
      base += incl - count;
      for (int i = w0; i < min(w0 + per, nw); ++i) {
        before[i] = static_cast<uint32_t>(base);
        base += __popc(marks[i]);
      }
    }
    __syncthreads();
    auto slot = [&](int v) { return before[v >> 5] + __popc(marks[v >> 5] & ((1u << (v & 31)) - 1u)); };
    if (q.n_bias > 0) {  // before the counts: a maximum over whole words
      each(ids, q.n_bias, [&](int id, int i) {
        const int v = entry(id);
        if (v >= 0) {
          const uint32_t s = slot(v);
          token[s] = static_cast<uint16_t>(v);
          atomicMax(&word[s], static_cast<uint32_t>(i + 1) << kBiasShift);
        }
      });
      __syncthreads();
    }
    auto count = [&](int id, uint32_t made_here) {
      const int v = entry(id);
      if (v >= 0) {
        const uint32_t s = slot(v);
        token[s] = static_cast<uint16_t>(v);
        if (made_here) atomicAdd(&word[s], 1u);
        else atomicOr(&word[s], kSeenBit);
      }
    };
    each(h, len, [&](int id, int i) { count(id, i >= made); });
    each(y, n_draft, [&](int id, int) { count(id, 1u); });
  } else if (a.live) {
    for (int i = t; i * 32 < n; i += kThreads) live[i] = mask[i];
    __syncthreads();
  }

  // pass 1: maximum and sum
  for (int b = 0; b < batches; ++b) {
    batch(b, [&](auto whole) {
      if (b > 0) fetch(b, whole);
      if (!greedy) {
        float z[kBatch][4], mb = -INFINITY;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          values(b, i, z[i], whole);
          mb = fmaxf(mb, fmaxf(fmaxf(z[i][0], z[i][1]), fmaxf(z[i][2], z[i][3])));  // passes over a NaN
        }
        // A NaN makes the sum NaN, and so does +inf (inf - inf).  (z k - m k
        // would save an instruction, but overflows for logits at the type's
        // lowest value and for small T.)
        const float mn = fmaxf(mine.m, mb), mz = mn == -INFINITY ? 0.f : mn;
        float s4[4] = {mine.s * ex2((mine.m - mz) * k), 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s4[e] += ex2((z[i][e] - mz) * k);
        mine.s = (s4[0] + s4[1]) + (s4[2] + s4[3]);
        mine.m = mn;
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          float z[4];
          values(b, i, z, whole);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (off(b, i, e) < n) add(z[e], lo + off(b, i, e));
        }
      }
    });
  }
  if (a.sparse) {  // the marked ids, each step rounded once
    __syncthreads();
    for (int i = t; i < n_marked; i += kThreads) {
      const uint32_t w = word[i], cnt = w & kCountMask;
      const int v = token[i];
      float z = mtp::load_f32<T>(src + v);
      if (w & (kSeenBit | kCountMask)) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
      if (cnt) z = __fsub_rn(z, __fadd_rn(__fmul_rn(freq, static_cast<float>(cnt)), pres));
      if (w >> kBiasShift) z = __fadd_rn(z, q.bias[static_cast<size_t>(r) * q.n_bias + (w >> kBiasShift) - 1]);
      if (mask && !((mask[v >> 5] >> (v & 31)) & 1u)) z = -INFINITY;
      word[i] = __float_as_uint(z);
      add(z, lo + v);
    }
  }
  // merge: thread -> warp -> CTA -> cluster
  auto weight = [&](float pm, float M) {  // a part without a maximum has s = 0 or NaN
    return greedy || pm == -INFINITY ? 1.f : ex2((pm - M) * k);
  };
  {
    const float m = mtp::warp_max(mine.m);
    mine.s = mtp::warp_sum(mine.s * weight(mine.m, m));
    mine.best = __reduce_min_sync(0xffffffffu, mine.m == m ? mine.best : 0x7fffffff);
    mine.m = m;
  }
  auto merge = [&](const Part* p, int count) {
    Part o{-INFINITY, 0.f, 0x7fffffff};
    for (int i = 0; i < count; ++i) o.m = fmaxf(o.m, p[i].m);
    for (int i = 0; i < count; ++i) {
      o.s += p[i].s * weight(p[i].m, o.m);
      if (p[i].m == o.m) o.best = min(o.best, p[i].best);
    }
    return o;
  };
  if (lane == 0) warp_part[warp] = mine;
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (t < C) *(cluster.map_shared_rank(parts, t) + rank) = merge(warp_part, kWarps);
  cluster.sync();  // nobody touches another CTA's shared memory after this
  const Part all = merge(parts, C);
  const bool bad = !(all.s == all.s);
  const bool row_ok = params_ok && !bad && all.m != -INFINITY;

  // pass 2
  const float M = all.m, scale = greedy ? 1.f : 1.f / all.s;
  float* dst = a.p + row * a.V + lo;
  for (int b = 0; b < batches; ++b) {
    batch(b, [&](auto whole) {
      if (batches > 1) fetch(b, whole);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        float z[4];
        if (row_ok && !greedy) {
          values(b, i, z, whole);
#pragma unroll
          for (int e = 0; e < 4; ++e) z[e] = ex2((z[e] - M) * k) * scale;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) z[e] = row_ok && lo + off(b, i, e) == all.best ? 1.f : 0.f;
        }
        if constexpr (VEC) {
          if (whole.value || off(b, i, 0) < n)
            *reinterpret_cast<float4*>(dst + off(b, i, 0)) = make_float4(z[0], z[1], z[2], z[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (off(b, i, e) < n) dst[off(b, i, e)] = z[e];
        }
      }
    });
  }
  if (a.sparse && row_ok && !greedy) {  // over the zeros that the pass wrote for the marked ids
    __syncthreads();
    for (int i = t; i < n_marked; i += kThreads) dst[token[i]] = ex2((__uint_as_float(word[i]) - M) * k) * scale;
  }
  if (rank == 0 && t == 0 && a.status)
    a.status[row] = !params_ok ? MTP_LOGITS_INVALID_PARAM
                    : bad      ? MTP_LOGITS_INVALID
                    : all.m == -INFINITY ? MTP_LOGITS_EMPTY
                                         : MTP_LOGITS_OK;
}

// What the largest slice needs with all of its entries marked: no call is beyond it, whatever
// the sizes allowed below.
constexpr int kMaxSlice = kMaxVocab / kMaxCluster;
static_assert(kMaxSlice == kTargetSlice && kMaxSlice <= 65536, "a slice's entries are 16-bit numbers");
constexpr int smem_for(int slice, int slots, bool sparse) { return 4 * (slice / 32) * (sparse ? 3 : 1) + 6 * slots; }
constexpr int kMaxSmem = smem_for(kMaxSlice, kMaxSlice, true);
static_assert(kMaxSmem <= 226 * 1024, "beside the static arrays");

int smem_bytes(const Args& a) { return a.live ? smem_for(a.slice, a.slots, a.sparse) : 0; }

template <bool VEC, typename T, int kCtas>
mtp_status launch_as(const Args& a, long long rows, int C, cudaStream_t st) {
  static mtp::PerDevice attr_smem, attr_cluster;
  auto kernel = logits_probs_kernel<VEC, T, kCtas>;
  if (!mtp::smem_limit(attr_smem, kernel, kMaxSmem)) return MTP_ERR_CUDA;
  const int dev = mtp::current_device();
  if (C > 8 && dev >= 0 && (dev >= mtp::kMaxDevices || !attr_cluster.v[dev].load(std::memory_order_acquire))) {
    MTP_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    if (dev < mtp::kMaxDevices) attr_cluster.v[dev].store(1, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes(a));
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

template <bool VEC, typename T>
mtp_status launch(const Args& a, long long rows, int C, cudaStream_t st) {
  return rows * C <= kFewCtas * mtp::sm_count_current() ? launch_as<VEC, T, kFewCtas>(a, rows, C, st)
                                                        : launch_as<VEC, T, kManyCtas>(a, rows, C, st);
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
  // the rows may be rewritten in place, but not through another row's logits
  const uintptr_t l0 = reinterpret_cast<uintptr_t>(logits), p0 = reinterpret_cast<uintptr_t>(p);
  if (ld > 1ll << 33) return MTP_ERR_UNSUPPORTED;
  const uintptr_t l1 = l0 + (static_cast<uintptr_t>(rows - 1) * ld + V) * esize, p1 = p0 + static_cast<uintptr_t>(rows) * V * 4;
  if (l0 < p1 && p0 < l1 && (l0 != p0 || dtype != MTP_F32 || ld != V)) return MTP_ERR_INVALID_ARG;

  a.logits = logits;
  a.ld = ld;
  a.p = p;
  a.status = status;
  a.L = L;
  a.V = V;
  if (L == 1) a.prm.draft = nullptr;
  a.has_pen = (q.repetition || q.frequency || q.presence) && (q.hist_cap > 0 || q.draft);
  a.sparse = a.has_pen || q.n_bias > 0;
  a.live = a.sparse || q.mask;
  const int listed = (a.has_pen ? q.hist_cap + L - 1 : 0) + q.n_bias;  // marked ids at most
  auto cut = [&](int c) {
    a.slice = ((V + c - 1) / c + 31) / 32 * 32;
    a.slots = a.sparse ? std::min(a.slice, listed) : 0;
  };
  // Cluster size: slices of at most kTargetSlice entries whose marked ids fit
  // into shared memory (65536 entries are within 5%, 16384 take 40% longer on
  // 320 rows of 129280); then twice as many CTAs for as long as no SM gets
  // more than two of them and every thread has more than one vector.
  int C = 1;
  for (cut(C); C < kMaxCluster && (a.slice > kTargetSlice || smem_bytes(a) > kMaxSmem); cut(C)) C *= 2;
  const int sms = mtp::sm_count_current();
  while (C < kMaxCluster && a.slice > 4 * kThreads && rows * C <= sms) cut(C *= 2);
  const bool vec = V % 4 == 0 && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) % (4 * esize)) == 0 &&
                   mtp::aligned16(p);
  if (dtype == MTP_F32) return vec ? launch<true, float>(a, rows, C, st) : launch<false, float>(a, rows, C, st);
  return vec ? launch<true, __nv_bfloat16>(a, rows, C, st) : launch<false, __nv_bfloat16>(a, rows, C, st);
}
