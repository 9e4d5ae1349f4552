// Products of up to 16 rows of 16-bit activations with NVFP4 weights.
#include <algorithm>

#include "msk_internal.h"
#include "msk_ops.cuh"

namespace msk {
namespace {

struct Lin4 {
  const uint16_t* x;
  const uint8_t* codes;
  const uint8_t* scales;
  void* y;
  long long x_stride, y_stride, N;
  int K, T, y_dtype;
  bool fp16;
  float ts;
};

__device__ __forceinline__ void store_y(const Lin4& a, int t, long long n, float v) {
  const long long i = t * a.y_stride + n;
  if (a.y_dtype == MSK_FP32) static_cast<float*>(a.y)[i] = v;
  else if (a.y_dtype == MSK_FP16) static_cast<__half*>(a.y)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(a.y)[i] = __float2bfloat16_rn(v);
}

// A block takes 16 weight rows, its 8 warps the 128-column chunks in turn.
// W is the MMA's A operand (16 rows), the tokens are its columns.  A lane
// takes 32 consecutive columns of a chunk (16 bytes of codes a row, two
// scales), four for each step of the contraction, and of x the same ones.
__global__ void __launch_bounds__(256) linear4_kernel(const __grid_constant__ Lin4 a) {
  __shared__ float red[8][16][17];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const long long n0 = blockIdx.x * 16ll;
  const int chunks = a.K / 128;
  // the scaling of this warp's share of x, token by token
  int shift[2];
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    const int t = nt * 8 + g;
    float amax = 0.f;
    if (t < a.T)
      for (int ch = warp; ch < chunks; ch += 8) {
        const uint4* p = reinterpret_cast<const uint4*>(a.x + t * a.x_stride + ch * 128 + c * 32);
        for (int i = 0; i < 4; ++i) {
          const uint4 u = __ldg(p + i);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack16(w[j], a.fp16);
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
      }
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    shift[nt] = row_shift(amax);
  }
  float acc[2][4] = {};
  const long long r0 = min(n0 + g, a.N - 1), r1 = min(n0 + g + 8, a.N - 1);
  for (int ch = warp; ch < chunks; ch += 8) {
    const uint4 u0 = __ldg(reinterpret_cast<const uint4*>(a.codes + r0 * (a.K / 2) + ch * 64 + c * 16));
    const uint4 u1 = __ldg(reinterpret_cast<const uint4*>(a.codes + r1 * (a.K / 2) + ch * 64 + c * 16));
    const uint32_t e0 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(a.scales + r0 * (a.K / 16) + ch * 8 + c * 2));
    const uint32_t e1 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(a.scales + r1 * (a.K / 16) + ch * 8 + c * 2));
    const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
    uint32_t xf[2][16];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int t = nt * 8 + g;
      const float mul = exp2i(shift[nt]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (t < a.T) u = __ldg(reinterpret_cast<const uint4*>(a.x + t * a.x_stride + ch * 128 + c * 32) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = unpack16(w[j], a.fp16);
          xf[nt][4 * i + j] = pack_f16x2(f.x * mul, f.y * mul);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t f0 = f16x2_bcast(e0, k >= 4), f1 = f16x2_bcast(e1, k >= 4);
      const uint32_t af[4] = {hmul2(e2m1_byte_to_f16x2(w0[k >> 1], 2 * (k & 1)), f0),
                              hmul2(e2m1_byte_to_f16x2(w1[k >> 1], 2 * (k & 1)), f1),
                              hmul2(e2m1_byte_to_f16x2(w0[k >> 1], 2 * (k & 1) + 1), f0),
                              hmul2(e2m1_byte_to_f16x2(w1[k >> 1], 2 * (k & 1) + 1), f1)};
      mma_f16(acc[0], af, xf[0][2 * k], xf[0][2 * k + 1]);
      mma_f16(acc[1], af, xf[1][2 * k], xf[1][2 * k + 1]);
    }
  }
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float f = exp2i(-__shfl_sync(0xFFFFFFFFu, shift[nt], (2 * c + i) * 4));
      red[warp][g][nt * 8 + 2 * c + i] = acc[nt][i] * f;
      red[warp][g + 8][nt * 8 + 2 * c + i] = acc[nt][2 + i] * f;
    }
  __syncthreads();
  const int t = threadIdx.x >> 4, r = threadIdx.x & 15;
  float s = 0.f;
  for (int w = 0; w < 8; ++w) s += red[w][r][t];
  if (t < a.T && n0 + r < a.N) store_y(a, t, n0 + r, s * a.ts);
}

}  // namespace
}  // namespace msk

using namespace msk;

extern "C" size_t msk_linear_fp4_workspace(int32_t tokens, int64_t rows, int64_t cols) {
  (void)tokens, (void)rows, (void)cols;
  return 0;
}

extern "C" msk_status msk_linear_fp4(const void* x, int32_t x_dtype, int64_t x_stride, const msk_nvfp4_desc* w,
                                     int32_t tokens, void* y, int32_t y_dtype, int64_t y_stride, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  if (w == nullptr || (x_dtype != MSK_BF16 && x_dtype != MSK_FP16) || !dtype_ok(y_dtype)) return MSK_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > kMaxT || w->rows < 0 || w->rows > (1ll << 31) || w->cols <= 0 || w->cols % 128 ||
      w->cols > 32768)
    return MSK_ERR_SHAPE;
  if (tokens == 0 || w->rows == 0) return MSK_OK;
  if (x == nullptr || y == nullptr || w->packed == nullptr || w->scales == nullptr) return MSK_ERR_INVALID_ARG;
  if (tokens > 1 && (x_stride < w->cols || y_stride < w->rows)) return MSK_ERR_INVALID_ARG;
  if (!ops_aligned16(x) || x_stride % 8 || !ops_aligned16(w->packed) || !ops_aligned16(w->scales) ||
      reinterpret_cast<uintptr_t>(y) % dtype_bytes(y_dtype))
    return MSK_ERR_ALIGNMENT;
  if (!ops_aligned16(workspace)) return MSK_ERR_ALIGNMENT;
  const size_t need = msk_linear_fp4_workspace(tokens, w->rows, w->cols);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MSK_ERR_INVALID_ARG;
  int nsm = 0;
  const msk_status s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  Lin4 a{};
  a.x = static_cast<const uint16_t*>(x), a.codes = w->packed, a.scales = w->scales, a.y = y;
  a.x_stride = x_stride, a.y_stride = y_stride, a.N = w->rows, a.K = (int)w->cols, a.T = tokens;
  a.y_dtype = y_dtype, a.fp16 = x_dtype == MSK_FP16, a.ts = w->tensor_scale;
  linear4_kernel<<<(unsigned)((w->rows + 15) / 16), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}
