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
  // below this a clamp of 16-bit logits would meet the type's lowest number
  static constexpr float LOW = DT == MSK_FP16 ? -65000.f : -1e37f;
  uint4 u;
  __device__ __forceinline__ void none() {
    const uint32_t w = DT == MSK_FP32 ? 0xFF800000u : DT == MSK_FP16 ? 0xFC00FC00u : 0xFF80FF80u;  // -inf
    u = make_uint4(w, w, w, w);
  }
  __device__ __forceinline__ void at_least(uint32_t lb) {  // (16-bit types)
    uint32_t* w = &u.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == MSK_FP16) asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(lb));
      else asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(lb));
    }
  }
  // How many are greater than x (a 16-bit type's number twice, or fp32).
  __device__ __forceinline__ void count_above(uint32_t x, uint32_t& n2) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == MSK_FP32) {
        n2 += __uint_as_float(w[i]) > __uint_as_float(x);
      } else {  // 1 or 0 for each half, added up as 16-bit floats (at most 16 a half)
        uint32_t g;
        if (DT == MSK_FP16) {
          asm("set.gt.f16x2.f16x2 %0, %1, %2;" : "=r"(g) : "r"(w[i]), "r"(x));
          asm("add.f16x2 %0, %0, %1;" : "+r"(n2) : "r"(g));
        } else {
          asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(g) : "r"(w[i]), "r"(x));
          asm("add.bf16x2 %0, %0, %1;" : "+r"(n2) : "r"(g));
        }
      }
    }
  }
  static __device__ __forceinline__ int counted(uint32_t n2) {
    if (DT == MSK_FP32) return (int)n2;
    const float2 f = unpack16(n2, DT == MSK_FP16);
    return (int)(f.x + f.y);
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

// Softmax statistics of logits with maximum m: s = sum 2^t and u = sum 2^t t,
// t = (x - m) c <= 0, c = log2(e) / temperature.  The difference is taken before
// the product, so that the maximum's t is 0 and steep temperatures stay exact.
// +inf and NaN end in an s that is not a positive number, and so does a row of
// nothing but -inf (m = -inf, s = 0).
struct Stat {
  float m, s, u;
};
__device__ __forceinline__ float anchor(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ Stat stat_join(const Stat& a, const Stat& b, float c) {
  const float m = max_nan(a.m, b.m), r = anchor(m);
  const float da = (a.m - r) * c, db = (b.m - r) * c, fa = ex2(da), fb = ex2(db);
  return {m, a.s * fa + b.s * fb, fa * (a.u + fmaxf(da, -200.f) * a.s) + fb * (b.u + fmaxf(db, -200.f) * b.s)};
}
__device__ __forceinline__ Stat stat_shfl(const Stat& a, int o) {
  return {__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o), __shfl_xor_sync(0xFFFFFFFFu, a.u, o)};
}

// K vectors' sums relative to the maximum m.  A logit far below it counts as one
// some 300 powers of two below, so that 2^t t is a number (0) for -inf too:
// 16-bit logits are clamped in pairs at `lb`, or (SLOW: fp32, a type without a
// number that low) every t is.
template <int DT, int K, bool SLOW>
__device__ __forceinline__ void vec_sums(const Vec<DT> (&v)[K], float c, float m, float lb, unsigned long long& s,
                                         unsigned long long& u) {
  constexpr int N = Vec<DT>::N;
  const unsigned long long cc = pair(c, c), nm = pair(-m, -m);
  const uint32_t lb2 = pack16(lb, lb, DT == MSK_FP16);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    Vec<DT> w = v[k];
    if (!SLOW) w.at_least(lb2);
    float y[N];
    w.get(y);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float t0, t1;
      unpair(mul2(add2(pair(y[i], y[i + 1]), nm), cc), t0, t1);
      if (SLOW) t0 = max_nan(t0, -300.f), t1 = max_nan(t1, -300.f);
      const unsigned long long e = pair(ex2(t0), ex2(t1));
      s = add2(s, e);
      u = fma2(e, pair(t0, t1), u);
    }
  }
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
// Alternatives cost no second pass: of 32 groups of threads, k have maxima that
// reach the k-th greatest group maximum, so the top k logits lie in the (few)
// threads whose own maxima reach it.  Those threads' logits are looked at again,
// a warp for each thread, against a sorted list in the warp's lanes.
template <int DT, int NT>
__global__ void __launch_bounds__(NT) logprobs_kernel(const __grid_constant__ LogProbs a) {
  constexpr int VN = Vec<DT>::N, NW = NT / 32, U = 4;
  __shared__ Stat st[NW];
  __shared__ int cnt[NW];
  __shared__ int owners[NT];
  __shared__ int n_owners, n_cand;
  __shared__ uint32_t group_max[32], bound;  // (a thread without a logit: 0)
  __shared__ unsigned long long cand[NW * 32];
  __shared__ unsigned long long best[kMaxTop];  // this segment's greatest keys; read by the cluster
  __shared__ Stat seg;                          // ... and its statistics
  __shared__ int seg_above;
  __shared__ Stat joined;  // all segments'
  __shared__ int joined_above;
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
  // the clamp's distance below the maximum: at least 300 powers of two, and
  // enough steps of the type (|m| / 64; fp16's smallest) that rounding it keeps
  // more than 260 of them
  const float reach = fmaxf(300.f / c, 0x1p-20f);
  Stat q = {-INFINITY, 0.f, 0.f};
  int above = 0;
  if (mine >= 0) {
    const float v = load1<DT>(x, mine);
    above += v > xg;
    q.m = max_nan(q.m, v);
    q.s = v == -INFINITY ? 0.f : ex2((v - v) * c);  // (NaN for what is no number)
  }
  unsigned long long s2 = pair(q.s, 0.f), u2 = pair(q.u, 0.f);
  const uint32_t xg2 = DT == MSK_FP32 ? __float_as_uint(xg) : pack16(xg, xg, DT == MSK_FP16);
  for (long long v = v0 + tid; v < v1; v += U * NT) {
    Vec<DT> w[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (v + k * NT < v1) w[k].u = load_stream(xv + (v + k * NT) * 16);
      else w[k].none();
    }
    const float bm = vec_max<DT, U>(w);
    const float mn = max_nan(q.m, bm);
    const float r = anchor(mn);
    if (mn != q.m) {
      const float d = (q.m - r) * c, f = ex2(d), dd = fmaxf(d, -300.f);
      u2 = mul2(fma2(s2, pair(dd, dd), u2), pair(f, f));
      s2 = mul2(s2, pair(f, f));
      q.m = mn;
    }
    const float lb = r - fmaxf(reach, fabsf(r) * 0.015625f);
    if (DT != MSK_FP32 && lb > Vec<DT>::LOW) vec_sums<DT, U, false>(w, c, r, lb, s2, u2);
    else vec_sums<DT, U, true>(w, c, r, lb, s2, u2);
    if (!(bm <= xg)) {
      uint32_t n2 = 0;
#pragma unroll
      for (int k = 0; k < U; ++k) w[k].count_above(xg2, n2);
      above += Vec<DT>::counted(n2);
    }
  }
  {
    float s0, s1, u0, u1;
    unpair(s2, s0, s1);
    unpair(u2, u0, u1);
    q.s = s0 + s1, q.u = u0 + u1;
  }
  const uint32_t key = v0 + tid < v1 || mine >= 0 ? ordered(q.m) : 0u;  // of this thread's greatest logit
#pragma unroll
  for (int o = 16; o; o >>= 1) q = stat_join(q, stat_shfl(q, o), c);
  above = __reduce_add_sync(0xFFFFFFFFu, above);
  if (lane == 0) st[warp] = q, cnt[warp] = above;
  if (tid == 0) n_owners = 0, n_cand = 0;
  if (tid < kMaxTop) best[tid] = 0ull;
  if (a.top > 0) {
    uint32_t gm = key;
#pragma unroll
    for (int o = 1; o < NT / 32; o <<= 1) gm = max(gm, __shfl_xor_sync(0xFFFFFFFFu, gm, o));
    if (lane % (NT / 32) == 0) group_max[tid / (NT / 32)] = gm;
  }
  __syncthreads();
  if (warp == 0) {
    q = lane < NW ? st[lane] : Stat{-INFINITY, 0.f, 0.f};
    above = __reduce_add_sync(0xFFFFFFFFu, lane < NW ? cnt[lane] : 0);
#pragma unroll
    for (int o = NW / 2; o; o >>= 1) q = stat_join(q, stat_shfl(q, o), c);
    if (lane == 0) seg = q, seg_above = above;
  } else if (warp == 1 && a.top > 0) {
    // the bound: the `top`-th greatest group maximum
    const uint32_t g = group_max[lane];
    int r = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const uint32_t o = __shfl_sync(0xFFFFFFFFu, g, j);
      r += o > g || (o == g && j < lane);
    }
    if (r == a.top - 1) bound = g;
  }

  if (a.top > 0) {
    __syncthreads();
    const uint32_t lo = bound;
    if (key >= lo) owners[atomicAdd(&n_owners, 1)] = tid;
    __syncthreads();
    const int no = n_owners;
    const float lo_value = lo == 0u ? -INFINITY : key_value((unsigned long long)lo << 32);
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
        if (v < v1) w.u = load_stream(xv + v * 16);
        float y[VN];
        w.get(y);
        uint32_t in = 0;  // which of them reach the bound (few)
#pragma unroll
        for (int j = 0; j < VN; ++j) in |= (uint32_t)!(y[j] < lo_value) << j;
        if (v >= v1) in = 0;
        while (uint32_t hit = __ballot_sync(0xFFFFFFFFu, in != 0)) {
          const int j = __ffs(in) - 1;
          float best_y = 0.f;
#pragma unroll
          for (int k = 0; k < VN; ++k) best_y = k == j ? y[k] : best_y;
          const unsigned long long full =
              ((unsigned long long)ordered(best_y) << 32) | (0xFFFFFFFFu - (uint32_t)(head + v * VN + j));
          in &= in - 1;
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
      if (warp == 1) {  // the segments' statistics, a lane for each
        Stat z = {-INFINITY, 0.f, 0.f};
        int n_above = 0;
        if (lane < S) {
          const uint32_t at = remote(&seg, lane);
          z = {__uint_as_float(ld32(at)), __uint_as_float(ld32(at + 4)), __uint_as_float(ld32(at + 8))};
          n_above = (int)ld32(remote(&seg_above, lane));
        }
        n_above = __reduce_add_sync(0xFFFFFFFFu, n_above);
#pragma unroll
        for (int o = 4; o; o >>= 1) z = stat_join(z, stat_shfl(z, o), c);
        if (lane == 0) joined = z, joined_above = n_above;
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
  const Stat z = S > 1 ? joined : seg;
  const bool bad = !(z.s > 0.f && z.s < INFINITY);
  // in log2 units, then nats
  constexpr float kLn2 = 0.6931471805599453f;
  const float log_s = bad ? NAN : log2f(z.s);
  if (tid == 0) {
    if (a.logprob) a.logprob[row] = given ? ((xg - z.m) * c - log_s) * kLn2 : 0.f;
    if (a.rank) a.rank[row] = given ? (S > 1 ? joined_above : seg_above) : -1;
    if (a.entropy) a.entropy[row] = bad ? NAN : (log_s - z.u / z.s) * kLn2;
  }
  if (tid < a.top) {
    const unsigned long long k = best[tid];
    if (a.top_ids) a.top_ids[row * a.top + tid] = (int32_t)(0xFFFFFFFFu - (uint32_t)k);
    if (a.top_logprobs) a.top_logprobs[row * a.top + tid] = bad ? NAN : ((key_value(k) - z.m) * c - log_s) * kLn2;
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
