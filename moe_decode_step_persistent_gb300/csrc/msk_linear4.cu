// Products of up to 16 rows of 16-bit activations with NVFP4 weights.
#include <algorithm>

#include "msk_internal.h"
#include "msk_ops.cuh"

namespace msk {
namespace {

constexpr int kGroup = 256;      // columns a warp takes: 64 consecutive ones a lane
constexpr int kMaxGroups = 16;   // groups (warps along the columns) of a pass
constexpr int kTokStride = 20;   // words between tokens of a warp's partial sums (no bank is hit twice)

struct Lin4 {
  const uint16_t* x;
  const uint8_t* codes;
  const uint8_t* scales;
  void* y;
  float* ws;  // [T][N] partial sums between passes
  long long x_stride, y_stride, N;
  int K, T, y_dtype;
  int groups, per_pass, passes;  // column groups, those of one pass, passes over the columns
  int wr;                        // 16-row tiles side by side in a block
  bool fp16, wide;               // codes aligned to 32 bytes
  float ts;
};

// A lane's share of 16 weight rows: 64 columns of rows g and g + 8.
struct WTile {
  uint32_t c[2][8];
  uint32_t e[2];
};

__device__ __forceinline__ void ld_codes(uint32_t (&w)[8], const uint8_t* p, bool wide) {
  if (wide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p + 16));
  }
}

// (col: the lane's first column, or -1 past the matrix)
__device__ __forceinline__ void ld_tile(WTile& t, const Lin4& a, long long row, int col) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const long long r = row + 8 * i;
    if (col >= 0 && r < a.N) {
      ld_codes(t.c[i], a.codes + r * (a.K / 2) + col / 2, a.wide);
      asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(t.e[i]) : "l"(a.scales + r * (a.K / 16) + col / 16));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) t.c[i][j] = 0;
      t.e[i] = 0;
    }
  }
}

__device__ __forceinline__ void store_y(const Lin4& a, int t, long long n, float v) {
  const long long i = t * a.y_stride + n;
  if (a.y_dtype == MSK_FP32) static_cast<float*>(a.y)[i] = v;
  else if (a.y_dtype == MSK_FP16) static_cast<__half*>(a.y)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(a.y)[i] = __float2bfloat16_rn(v);
}

// Persistent blocks of up to 16 warps.  A warp keeps its 256 columns of x in
// registers for the whole pass, as the MMA's B fragments (NT tiles of 8
// tokens), and streams weight rows through its A fragments, 16 rows at a
// time: decoded to fp16 in registers, exact, with one multiply by the block
// scale for two weights.  Of x and W a lane takes the same 64 columns, so a
// row's codes are one 32-byte load and its scales one 4-byte load, and
// neither passes through shared memory.  The warps of a row tile add their
// partial sums up in shared memory.
//
// The next tile's loads are issued before the current one is computed: two
// tiles of up to 36 KB in flight per SM are what DRAM's latency asks for.
template <int NT>
__global__ void __launch_bounds__(512, 1) linear4_kernel(const __grid_constant__ Lin4 a) {
  constexpr int TOK = 8 * NT;
  __shared__ float red[2][kMaxGroups][TOK * kTokStride];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int wk = warp % a.per_pass, tile = warp / a.per_pass;
  const long long step = 16ll * a.wr * gridDim.x, first = 16ll * a.wr * blockIdx.x;
  int buf = 0;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int grp = pass * a.per_pass + wk;
    int col = grp * kGroup + c * 64;
    if (grp >= a.groups || col >= a.K) col = -1;
    WTile cur;
    ld_tile(cur, a, first + tile * 16 + g, col);
    // x: scaled by a power of two for each (token, warp), then fp16
    uint32_t xf[NT][32];
    float back[NT][2];  // the scalings of this lane's accumulator columns, undone
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int t = nt * 8 + g;
      const uint4* p = reinterpret_cast<const uint4*>(a.x + t * a.x_stride + (col < 0 ? 0 : col));
      const bool in = t < a.T && col >= 0;
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (in) u = __ldg(p + i);
        xf[nt][4 * i] = u.x, xf[nt][4 * i + 1] = u.y, xf[nt][4 * i + 2] = u.z, xf[nt][4 * i + 3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float2 f = unpack16(xf[nt][i], a.fp16);
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      const int sh = row_shift(amax);
      const float mul = exp2i(sh);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float2 f = unpack16(xf[nt][i], a.fp16);
        xf[nt][i] = pack_f16x2(f.x * mul, f.y * mul);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) back[nt][i] = exp2i(-__shfl_sync(0xFFFFFFFFu, sh, (2 * c + i) * 4));
    }

    for (long long r0 = first; r0 < a.N; r0 += step) {
      WTile nxt;
      ld_tile(nxt, a, r0 + step + tile * 16 + g, col);
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
      uint32_t sc[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sc[i][0] = e4m3_pair_to_f16x2(cur.e[i], 0);
        sc[i][1] = e4m3_pair_to_f16x2(cur.e[i], 1);
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint32_t f0 = f16x2_bcast(sc[0][k >> 3], (k >> 2) & 1), f1 = f16x2_bcast(sc[1][k >> 3], (k >> 2) & 1);
        const uint32_t af[4] = {hmul2(e2m1_byte_to_f16x2(cur.c[0][k >> 1], 2 * (k & 1)), f0),
                                hmul2(e2m1_byte_to_f16x2(cur.c[1][k >> 1], 2 * (k & 1)), f1),
                                hmul2(e2m1_byte_to_f16x2(cur.c[0][k >> 1], 2 * (k & 1) + 1), f0),
                                hmul2(e2m1_byte_to_f16x2(cur.c[1][k >> 1], 2 * (k & 1) + 1), f1)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], af, xf[nt][2 * k], xf[nt][2 * k + 1]);
      }
      float* part = red[buf][warp];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          part[(nt * 8 + 2 * c + i) * kTokStride + g] = acc[nt][i] * back[nt][i];
          part[(nt * 8 + 2 * c + i) * kTokStride + g + 8] = acc[nt][2 + i] * back[nt][i];
        }
      __syncthreads();  // (the other buffer's readers are past it too)
      for (int o = threadIdx.x; o < 16 * TOK * a.wr; o += blockDim.x) {
        const int r = o & 15, t = (o >> 4) % TOK, rt = (o >> 4) / TOK;
        const long long n = r0 + rt * 16 + r;
        if (t >= a.T || n >= a.N) continue;
        float s = 0.f;
        for (int w = 0; w < a.per_pass; ++w) s += red[buf][rt * a.per_pass + w][t * kTokStride + r];
        // (a later pass of the same thread takes the partial sum up again)
        if (pass > 0) s += a.ws[t * a.N + n];
        if (pass + 1 < a.passes) a.ws[t * a.N + n] = s;
        else store_y(a, t, n, s * a.ts);
      }
      buf ^= 1;
      cur = nxt;
    }
  }
}

}  // namespace
}  // namespace msk

using namespace msk;

extern "C" size_t msk_linear_fp4_workspace(int32_t tokens, int64_t rows, int64_t cols) {
  if (tokens <= 0 || rows <= 0 || cols <= kGroup * kMaxGroups) return 0;
  return (size_t)tokens * (size_t)rows * 4;
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
  a.ws = static_cast<float*>(workspace);
  a.wide = reinterpret_cast<uintptr_t>(w->packed) % 32 == 0;
  a.groups = (a.K + kGroup - 1) / kGroup;
  a.passes = (a.groups + kMaxGroups - 1) / kMaxGroups;
  a.per_pass = (a.groups + a.passes - 1) / a.passes;
  // row tiles side by side: as many as warps allow, fewer where that would
  // leave SMs without rows
  const long long tiles = (a.N + 15) / 16;
  a.wr = (int)std::max<long long>(1, std::min<long long>(kMaxGroups / a.per_pass, tiles / nsm));
  const unsigned grid = (unsigned)std::min<long long>(nsm, (tiles + a.wr - 1) / a.wr);
  const unsigned threads = 32u * a.per_pass * a.wr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (tokens <= 8) linear4_kernel<1><<<grid, threads, 0, st>>>(a);
  else linear4_kernel<2><<<grid, threads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}
