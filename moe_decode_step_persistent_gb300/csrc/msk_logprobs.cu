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
  long long ld, V;
  int top;
  float inv_t;
};

template <int DT>
__device__ __forceinline__ float load1(const void* p, long long i) {
  if (DT == MSK_FP32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t u = __ldg(static_cast<const uint16_t*>(p) + i);
  return DT == MSK_FP16 ? __half2float(__ushort_as_half(u)) : __uint_as_float((uint32_t)u << 16);
}

// Ordered key of (value descending, index ascending): greater keys come
// first.  -0 and 0 are one value; every NaN is above every number.
__device__ __forceinline__ unsigned long long logit_key(float x, uint32_t i) {
  const uint32_t u = x != x ? 0x7FFFFFFFu : __float_as_uint(x + 0.f);
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return ((unsigned long long)o << 32) | (0xFFFFFFFFu - i);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// Softmax statistics relative to a maximum m: s = sum e^(x - m), u = sum
// e^(x - m) (m - x), both over scaled logits.
struct Stat {
  float m, s, u;
};
__device__ __forceinline__ Stat stat_join(const Stat& a, const Stat& b) {
  const float m = fmaxf(a.m, b.m), r = m == -INFINITY ? 0.f : m;
  const float da = a.m - r, db = b.m - r, fa = expf(da), fb = expf(db);
  // (a part that holds nothing has s = u = 0; its distance is infinite)
  return {m, a.s * fa + b.s * fb,
          (a.s > 0.f ? fa * (a.u - da * a.s) : 0.f) + (b.s > 0.f ? fb * (b.u - db * b.s) : 0.f)};
}

template <int DT>
__global__ void __launch_bounds__(512) logprobs_kernel(const __grid_constant__ LogProbs a) {
  __shared__ Stat st[16];
  __shared__ int cnt[16];
  __shared__ bool nan[16];
  __shared__ unsigned long long best[16];
  const long long row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const void* x = static_cast<const char*>(a.logits) + row * a.ld * (DT == MSK_FP32 ? 4 : 2);
  const int tok = a.tokens ? a.tokens[row] : -1;
  const bool given = tok >= 0 && tok < a.V;
  const float xg = given ? load1<DT>(x, tok) : 0.f;
  Stat q = {-INFINITY, 0.f, 0.f};
  int above = 0;
  bool bad = false;
  for (long long i = threadIdx.x; i < a.V; i += 512) {
    const float raw = load1<DT>(x, i), v = raw * a.inv_t;
    above += raw > xg;
    bad |= !(raw < INFINITY);
    if (v == -INFINITY) continue;
    if (v > q.m) {
      const float f = expf(q.m - v);
      q.u = q.s > 0.f ? f * (q.u + (v - q.m) * q.s) : 0.f;
      q.s = q.s * f + 1.f;
      q.m = v;
    } else {
      const float e = expf(v - q.m);
      q.s += e;
      q.u += e * (q.m - v);
    }
  }
  for (int o = 16; o; o >>= 1) {
    const Stat b = {__shfl_xor_sync(0xFFFFFFFFu, q.m, o), __shfl_xor_sync(0xFFFFFFFFu, q.s, o),
                    __shfl_xor_sync(0xFFFFFFFFu, q.u, o)};
    q = stat_join(q, b);
    above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
  }
  bad = __any_sync(0xFFFFFFFFu, bad);
  if (lane == 0) st[warp] = q, cnt[warp] = above, nan[warp] = bad;
  __syncthreads();
  q = st[0], above = cnt[0], bad = nan[0];
  for (int w = 1; w < 16; ++w) q = stat_join(q, st[w]), above += cnt[w], bad |= nan[w];
  bad |= q.m == -INFINITY;
  const float log_s = bad ? NAN : logf(q.s);
  if (threadIdx.x == 0) {
    if (a.logprob) a.logprob[row] = given ? (xg * a.inv_t - q.m) - log_s : 0.f;
    if (a.rank) a.rank[row] = given ? above : -1;
    if (a.entropy) a.entropy[row] = bad ? NAN : log_s + q.u / q.s;
  }
  // alternatives, one after the other
  unsigned long long last = ~0ull;
  for (int k = 0; k < a.top; ++k) {
    unsigned long long b = 0;
    for (long long i = threadIdx.x; i < a.V; i += 512) {
      const unsigned long long key = logit_key(load1<DT>(x, i), (uint32_t)i);
      if (key < last && key > b) b = key;
    }
    for (int o = 16; o; o >>= 1) b = max(b, __shfl_xor_sync(0xFFFFFFFFu, b, o));
    if (lane == 0) best[warp] = b;
    __syncthreads();
    b = best[0];
    for (int w = 1; w < 16; ++w) b = max(b, best[w]);
    __syncthreads();
    last = b;
    if (threadIdx.x == 0) {
      if (a.top_ids) a.top_ids[row * a.top + k] = (int32_t)(0xFFFFFFFFu - (uint32_t)b);
      if (a.top_logprobs) a.top_logprobs[row * a.top + k] = bad ? NAN : (key_value(b) * a.inv_t - q.m) - log_s;
    }
  }
}

}  // namespace
}  // namespace msk

using namespace msk;

extern "C" size_t msk_token_logprobs_workspace(int64_t rows, int64_t vocab, int32_t top) {
  (void)rows, (void)vocab, (void)top;
  return 0;
}

extern "C" msk_status msk_token_logprobs(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t ld,
                                         const int32_t* tokens, float temperature, int32_t top, float* logprob,
                                         int32_t* rank, float* entropy, int32_t* top_ids, float* top_logprobs,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || rows < 0 || !(temperature > 0.f && temperature < INFINITY)) return MSK_ERR_INVALID_ARG;
  if (vocab <= 0 || vocab > 0x7FFFFFFFll || rows > 0x7FFFFFFFll || top < 0 || top > kMaxTop) return MSK_ERR_SHAPE;
  if (top > vocab) return MSK_ERR_INVALID_ARG;
  if (rows == 0) return MSK_OK;
  if (logits == nullptr || (rows > 1 && ld < vocab)) return MSK_ERR_INVALID_ARG;
  if (tokens == nullptr && (logprob != nullptr || rank != nullptr)) return MSK_ERR_INVALID_ARG;
  const uintptr_t words = reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(logprob) |
                          reinterpret_cast<uintptr_t>(rank) | reinterpret_cast<uintptr_t>(entropy) |
                          reinterpret_cast<uintptr_t>(top_ids) | reinterpret_cast<uintptr_t>(top_logprobs);
  if (reinterpret_cast<uintptr_t>(logits) % dtype_bytes(dtype) || words % 4 || !ops_aligned16(workspace))
    return MSK_ERR_ALIGNMENT;
  const size_t need = msk_token_logprobs_workspace(rows, vocab, top);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MSK_ERR_INVALID_ARG;
  int nsm = 0;
  const msk_status s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  LogProbs a{};
  a.logits = logits, a.tokens = tokens, a.logprob = logprob, a.rank = rank, a.entropy = entropy;
  a.top_ids = top_ids, a.top_logprobs = top_logprobs, a.ld = ld, a.V = vocab, a.top = top, a.inv_t = 1.f / temperature;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == MSK_FP32) logprobs_kernel<MSK_FP32><<<(unsigned)rows, 512, 0, st>>>(a);
  else if (dtype == MSK_FP16) logprobs_kernel<MSK_FP16><<<(unsigned)rows, 512, 0, st>>>(a);
  else logprobs_kernel<MSK_BF16><<<(unsigned)rows, 512, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}
