// Log probabilities of given tokens, entropy and top alternatives.
#include <algorithm>
#include <cmath>

#include "msk_ops.cuh"

namespace msk {
namespace {

constexpr int kMaxTop = 32;

struct LogProbs {
  const void* logits;
  const int32_t* tokens;
  float* logprob;
  int32_t* rank;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  long long rows, ld, V;
  int top;
  float inv_t;
};

template <int DT>
__device__ __forceinline__ float load1(const void* p, long long i) {
  if (DT == MSK_FP32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t u = __ldg(static_cast<const uint16_t*>(p) + i);
  return DT == MSK_FP16 ? __half2float(__ushort_as_half(u)) : __uint_as_float((uint32_t)u << 16);
}

// 16 aligned bytes, read once.
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int DT>
struct Vec {  // a 16-byte vector of logits
  static constexpr int N = DT == MSK_FP32 ? 4 : 8;
  uint4 u;
  __device__ __forceinline__ void none() {
    const uint32_t w = DT == MSK_FP32 ? 0xFF800000u : DT == MSK_FP16 ? 0xFC00FC00u : 0xFF80FF80u;  // -inf
    u = make_uint4(w, w, w, w);
  }
  __device__ __forceinline__ void get(float (&x)[N]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == MSK_FP32) {
        x[i] = __uint_as_float(w[i]);
      } else {
        const float2 f = unpack16(w[i], DT == MSK_FP16);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
      }
    }
  }
};

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Greatest value of N vectors.
template <int DT, int K>
__device__ __forceinline__ float vec_max(const Vec<DT> (&v)[K]) {
  if (DT == MSK_FP32) {
    float m = __uint_as_float(v[0].u.x);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      m = max_nan(max_nan(m, __uint_as_float(v[k].u.x)), __uint_as_float(v[k].u.y));
      m = max_nan(max_nan(m, __uint_as_float(v[k].u.z)), __uint_as_float(v[k].u.w));
    }
    return m;
  }
  uint32_t m = v[0].u.x;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const uint32_t w[4] = {v[k].u.x, v[k].u.y, v[k].u.z, v[k].u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == MSK_FP16) asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
      else asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    }
  }
  const float2 f = unpack16(m, DT == MSK_FP16);
  return max_nan(f.x, f.y);
}

// Ordered key of (value descending, index ascending): greater keys come
// first.  -0 and 0 are one value; every NaN is above every number.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = x != x ? 0x7FFFFFFFu : __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// Softmax statistics relative to a maximum m: s = sum 2^t and u = sum 2^t t,
// t = (x - m) log2(e) / temperature <= 0.  m starts at the lowest number, so
// that every difference is defined; +inf and NaN end in an s that is not a
// positive number, and so does a row without any number above -inf.
struct Stat {
  float m, s, u;
};
constexpr float kLowest = -3.402823466e38f;
__device__ __forceinline__ Stat stat_join(const Stat& a, const Stat& b, float c) {
  const float m = max_nan(a.m, b.m);
  const float da = fmaxf((a.m - m) * c, -200.f), db = fmaxf((b.m - m) * c, -200.f);
  const float fa = ex2((a.m - m) * c), fb = ex2((b.m - m) * c);
  return {m, a.s * fa + b.s * fb, fa * (a.u + da * a.s) + fb * (b.u + db * b.s)};
}

// `key` into the warp's list of its 32 greatest keys (lane i holds the i-th).
__device__ __forceinline__ void list_insert(unsigned long long& list, unsigned long long key, int lane) {
  const int at = __popc(__ballot_sync(0xFFFFFFFFu, list > key));
  const unsigned long long up = __shfl_up_sync(0xFFFFFFFFu, list, 1);
  if (lane >= at) list = lane == at ? key : up;
}

// One row, or one of `gridDim.x` segments of a row that a cluster of blocks
// works on.  One pass over the logits: every thread keeps a running maximum
// and the sums relative to it over vectors of 16 bytes, four at a time, so
// that the sums are rescaled once for 16 or 32 logits.  DRAM bounds it.
//
// Alternatives cost no second pass: the top k logits lie in the threads whose
// own maxima are at least the k-th greatest thread maximum, so a bisection on
// those maxima names the few threads (k of them unless maxima tie) whose
// logits are looked at again, a warp for each, against a sorted list in the
// warp's lanes.
template <int DT, int NT>
__global__ void __launch_bounds__(NT) logprobs_kernel(const __grid_constant__ LogProbs a) {
  constexpr int VN = Vec<DT>::N, NW = NT / 32, U = 4;
  __shared__ Stat st[NW];
  __shared__ int cnt[NW];
  __shared__ int owners[NT];
  __shared__ int n_owners, n_cand;
  __shared__ unsigned long long cand[NW * 32];
  __shared__ unsigned long long best[kMaxTop];  // this segment's greatest keys; read by the cluster
  __shared__ Stat seg;                          // ... and its statistics
  __shared__ int seg_above;
  const long long row = blockIdx.y + (long long)blockIdx.z * gridDim.y;
  if (row >= a.rows) return;  // (the whole cluster)
  const int S = gridDim.x, part = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const char* x = static_cast<const char*>(a.logits) + row * a.ld * (DT == MSK_FP32 ? 4 : 2);
  const int tok = a.tokens ? a.tokens[row] : -1;
  const bool given = tok >= 0 && tok < a.V;
  const float xg = given ? load1<DT>(x, tok) : INFINITY;

  // the aligned vectors of this segment; single logits before (first
  // segment) and behind them (last segment)
  const int es = DT == MSK_FP32 ? 4 : 2;
  const int head = (int)min(a.V, (long long)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / es);
  const long long nv = (a.V - head) / VN;
  const int tail = (int)(a.V - head - nv * VN);
  const long long v0 = nv * part / S, v1 = nv * (part + 1) / S;
  const char* xv = x + head * es;
  // the single logit of this thread, if it has one
  const long long mine = part == 0 && tid < head                       ? tid
                         : part == S - 1 && tid >= 32 && tid < 32 + tail ? a.V - tail + (tid - 32)
                                                                         : -1;

  const float c = a.inv_t * 1.4426950408889634f;
  Stat q = {kLowest, 0.f, 0.f};
  int above = 0;
  if (mine >= 0) {
    const float v = load1<DT>(x, mine);
    above += v > xg;
    q.m = max_nan(q.m, v);
    const float t = fmaxf((v - q.m) * c, -200.f);
    q.s = v == v ? ex2(t) : NAN;
  }
  for (long long v = v0 + tid; v < v1; v += U * NT) {
    Vec<DT> w[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (v + k * NT < v1) w[k].u = load_stream(xv + (v + k * NT) * 16);
      else w[k].none();
    }
    const float bm = vec_max<DT, U>(w);
    const float mn = max_nan(q.m, bm);
    const float d = (q.m - mn) * c, f = ex2(d);
    q.u = f * (q.u + fmaxf(d, -200.f) * q.s);
    q.s *= f;
    q.m = mn;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      float y[VN];
      w[k].get(y);
#pragma unroll
      for (int i = 0; i < VN; ++i) {
        const float t = fmaxf((y[i] - mn) * c, -200.f), e = ex2(t);  // (-200: 2^t is 0 and 2^t t a number)
        q.s += e;
        q.u = fmaf(e, t, q.u);
      }
      if (bm > xg) {
#pragma unroll
        for (int i = 0; i < VN; ++i) above += y[i] > xg;
      }
    }
  }
  const float my_max = q.m;
  for (int o = 16; o; o >>= 1) {
    const Stat b = {__shfl_xor_sync(0xFFFFFFFFu, q.m, o), __shfl_xor_sync(0xFFFFFFFFu, q.s, o),
                    __shfl_xor_sync(0xFFFFFFFFu, q.u, o)};
    q = stat_join(q, b, c);
  }
  above = __reduce_add_sync(0xFFFFFFFFu, above);
  if (lane == 0) st[warp] = q, cnt[warp] = above;
  if (tid == 0) n_owners = 0, n_cand = 0;
  if (tid < kMaxTop) best[tid] = 0ull;
  __syncthreads();
  if (warp == 0) {
    q = lane < NW ? st[lane] : Stat{kLowest, 0.f, 0.f};
    above = lane < NW ? cnt[lane] : 0;
    for (int o = NW / 2; o; o >>= 1) {
      const Stat b = {__shfl_xor_sync(0xFFFFFFFFu, q.m, o), __shfl_xor_sync(0xFFFFFFFFu, q.s, o),
                      __shfl_xor_sync(0xFFFFFFFFu, q.u, o)};
      q = stat_join(q, b, c);
      above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
    }
    if (lane == 0) seg = q, seg_above = above;
  }

  if (a.top > 0) {
    // a bound that at least `top` thread maxima reach: the greatest one, or
    // one that few reach (0, which every thread reaches, if there are no
    // `top` maxima above the lowest number)
    const uint32_t key = my_max == kLowest ? 0u : ordered(my_max);
    uint32_t lo = 0, hi = 0xFFFFFFFFu;  // (reached by >= top threads; by fewer)
    while (hi - lo > 1) {
      const uint32_t mid = lo + (hi - lo) / 2;
      const int n = __syncthreads_count(key >= mid);
      if (n >= a.top) {
        lo = mid;
        if (n <= 2 * kMaxTop) break;
      } else {
        hi = mid;
      }
    }
    if (key >= lo) owners[atomicAdd(&n_owners, 1)] = tid;
    __syncthreads();
    const int no = n_owners;
    unsigned long long list = 0ull;
    for (int i = warp; i < no; i += NW) {
      const int o = owners[i];
      // the owner's single logit
      const long long single = part == 0 && o < head                       ? o
                               : part == S - 1 && o >= 32 && o < 32 + tail ? a.V - tail + (o - 32)
                                                                           : -1;
      if (single >= 0) {
        const uint32_t k = ordered(load1<DT>(x, single));
        if (k >= lo) list_insert(list, ((unsigned long long)k << 32) | (0xFFFFFFFFu - (uint32_t)single), lane);
      }
      for (long long vb = v0 + o; vb < v1; vb += 32 * NT) {
        const long long v = vb + (long long)lane * NT;
        Vec<DT> w;
        w.none();
        const bool in = v < v1;
        if (in) w.u = load_stream(xv + v * 16);
        float y[VN];
        w.get(y);
#pragma unroll
        for (int j = 0; j < VN; ++j) {
          const uint32_t k = ordered(y[j]);
          const unsigned long long full =
              ((unsigned long long)k << 32) | (0xFFFFFFFFu - (uint32_t)(head + v * VN + j));
          // (the list's last key bounds what can still enter)
          const unsigned long long last = __shfl_sync(0xFFFFFFFFu, list, 31);
          uint32_t hit = __ballot_sync(0xFFFFFFFFu, in && k >= lo && full > last);
          while (hit) {
            const int src = __ffs(hit) - 1;
            hit &= hit - 1;
            list_insert(list, __shfl_sync(0xFFFFFFFFu, full, src), lane);
          }
        }
      }
    }
    // the warps' lists, joined by counting how many keys are greater
    const uint32_t have = __ballot_sync(0xFFFFFFFFu, list != 0ull);
    int base = 0;
    if (lane == 0 && have) base = atomicAdd(&n_cand, __popc(have));
    base = __shfl_sync(0xFFFFFFFFu, base, 0);
    if (list != 0ull) cand[base + lane] = list;
    __syncthreads();
    const int n = n_cand;
    for (int i = tid; i < n; i += NT) {
      const unsigned long long k = cand[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += cand[j] > k;
      if (r < a.top) best[r] = k;
    }
  }
  if (S > 1) {
    // segments meet in the first block, through the cluster's shared memory
    cluster_sync();
    if (part == 0) {
      auto remote = [](const void* p, int rank) { return mapa(smem_u32(p), rank); };
      auto ld32 = [](uint32_t at) { return __float_as_uint(ld_cluster(at)); };
      const int n = S * a.top;  // <= 256
      for (int i = tid; i < n; i += NT) {
        const uint32_t at = remote(&best[i % a.top], i / a.top);
        cand[i] = ((unsigned long long)ld32(at + 4) << 32) | ld32(at);
      }
      __syncthreads();
      if (tid == 0) {
        for (int r = 1; r < S; ++r) {
          const uint32_t at = remote(&seg, r);
          seg = stat_join(seg, {__uint_as_float(ld32(at)), __uint_as_float(ld32(at + 4)), __uint_as_float(ld32(at + 8))}, c);
          seg_above += (int)ld32(remote(&seg_above, r));
        }
      }
      for (int i = tid; i < n; i += NT) {
        const unsigned long long k = cand[i];
        int r = 0;
        for (int j = 0; j < n; ++j) r += cand[j] > k;
        if (k != 0ull && r < a.top) best[r] = k;
      }
    }
    cluster_sync();
    if (part != 0) return;
  }
  __syncthreads();
  const bool bad = !(seg.s > 0.f && seg.s < INFINITY);
  const float log_s = bad ? NAN : logf(seg.s);
  if (tid == 0) {
    if (a.logprob) a.logprob[row] = given ? (xg - seg.m) * a.inv_t - log_s : 0.f;
    if (a.rank) a.rank[row] = given ? seg_above : -1;
    if (a.entropy) a.entropy[row] = bad ? NAN : log_s - 0.6931471805599453f * (seg.u / seg.s);
  }
  if (tid < a.top) {
    const unsigned long long k = best[tid];
    if (a.top_ids) a.top_ids[row * a.top + tid] = (int32_t)(0xFFFFFFFFu - (uint32_t)k);
    if (a.top_logprobs) a.top_logprobs[row * a.top + tid] = bad ? NAN : (key_value(k) - seg.m) * a.inv_t - log_s;
  }
}

template <int DT>
cudaError_t launch_logprobs(const LogProbs& a, int nsm, cudaStream_t st) {
  // Few rows: up to 8 segments a row (a cluster, portable size), as long as
  // they all fit the GPU at once and are worth a block; small vocabularies:
  // blocks of 128 threads.
  int S = 1;
  while (S < 8 && a.rows * S * 2 <= 4ll * nsm && a.V / (S * 2) >= 4096) S *= 2;
  cudaLaunchConfig_t cfg = {};
  const unsigned gy = (unsigned)std::min<long long>(a.rows, 65535);
  cfg.gridDim = dim3((unsigned)S, gy, (unsigned)((a.rows + gy - 1) / gy));
  const bool small = S == 1 && a.V <= 4096;
  cfg.blockDim = dim3(small ? 128 : 512);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)S, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return small ? cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, 128>, a) : cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, 512>, a);
}

}  // namespace
}  // namespace msk

using namespace msk;

extern "C" msk_status msk_token_logprobs(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t ld,
                                         const int32_t* tokens, float temperature, int32_t top, float* logprob,
                                         int32_t* rank, float* entropy, int32_t* top_ids, float* top_logprobs,
                                         void* stream) {
  if (!dtype_ok(dtype) || rows < 0 || !(temperature >= 1e-30f && temperature <= 1e30f)) return MSK_ERR_INVALID_ARG;
  if (vocab <= 0 || vocab > 0x7FFFFFFFll || rows > 0x7FFFFFFFll || top < 0 || top > kMaxTop) return MSK_ERR_SHAPE;
  if (top > vocab) return MSK_ERR_INVALID_ARG;
  if (rows == 0) return MSK_OK;
  if (logits == nullptr || (rows > 1 && ld < vocab)) return MSK_ERR_INVALID_ARG;
  if (tokens == nullptr && (logprob != nullptr || rank != nullptr)) return MSK_ERR_INVALID_ARG;
  const uintptr_t words = reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(logprob) |
                          reinterpret_cast<uintptr_t>(rank) | reinterpret_cast<uintptr_t>(entropy) |
                          reinterpret_cast<uintptr_t>(top_ids) | reinterpret_cast<uintptr_t>(top_logprobs);
  if (reinterpret_cast<uintptr_t>(logits) % dtype_bytes(dtype) || words % 4) return MSK_ERR_ALIGNMENT;
  int nsm = 0;
  const msk_status s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  LogProbs a{};
  a.logits = logits, a.tokens = tokens, a.logprob = logprob, a.rank = rank, a.entropy = entropy;
  a.top_ids = top_ids, a.top_logprobs = top_logprobs, a.rows = rows, a.ld = ld, a.V = vocab, a.top = top, a.inv_t = 1.f / temperature;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MSK_FP32   ? launch_logprobs<MSK_FP32>(a, nsm, st)
                        : dtype == MSK_FP16 ? launch_logprobs<MSK_FP16>(a, nsm, st)
                                            : launch_logprobs<MSK_BF16>(a, nsm, st);
  return e == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}
