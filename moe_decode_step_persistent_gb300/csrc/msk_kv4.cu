// The 4-bit KV cache: writing rows (quantise), reading them back, and GQA
// attention over them.
#include <algorithm>
#include <cmath>

#include "msk_internal.h"
#include "msk_ops.cuh"

namespace msk {
namespace {

// ---------------------------------------------------------------------------
// rows in and out
// ---------------------------------------------------------------------------

struct Kv4Rows {
  uint8_t* codes;
  uint8_t* scales;
  const void* k;
  const void* v;
  const int32_t* pos0_dev;
  long long token_stride, head_stride;
  int Hkv, max_seq, tokens, pos0;
  float k_scale, v_scale;
};

// 16 consecutive elements of type T as floats.
template <int DT>
__device__ __forceinline__ void load16(const void* base, long long off, float (&x)[16]) {
  if (DT == MSK_FP32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldg(p + i);
      x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = f.z, x[4 * i + 3] = f.w;
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = __ldg(p + i);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack16(w[j], DT == MSK_FP16);
        x[8 * i + 2 * j] = f.x, x[8 * i + 2 * j + 1] = f.y;
      }
    }
  }
}

// One thread per block of 16 elements: two 16-byte loads (of 16-bit rows),
// one 8-byte and one 1-byte store.  Bound by DRAM for long conversions and by
// the launch for a step's 16 rows.
template <int HD, int DT>
__global__ void __launch_bounds__(256) kv4_write_kernel(const Kv4Rows a) {
  constexpr int NB = HD / 16;
  const long long idx = blockIdx.x * 256ll + threadIdx.x;
  const int b = (int)(idx % NB);
  const long long r = idx / NB;  // ((kv * Hkv) + h) * tokens + t
  if (r >= 2ll * a.Hkv * a.tokens) return;
  const int t = (int)(r % a.tokens);
  const int kvh = (int)(r / a.tokens);
  const int h = kvh % a.Hkv;
  const bool is_v = kvh >= a.Hkv;
  float x[16];
  load16<DT>(is_v ? a.v : a.k, t * a.token_stride + h * a.head_stride + b * 16, x);
  const float ts = is_v ? a.v_scale : a.k_scale;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    x[i] = __fdiv_rn(x[i], ts);
    amax = fmaxf(amax, fabsf(x[i]));
  }
  const uint32_t sc = f32_to_e4m3(__fdiv_rn(amax, 6.0f));
  const float dec = e4m3_to_f32(sc);
  uint32_t w[2] = {0u, 0u};
  if (dec > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i >> 2] |= f32x2_to_e2m1x2(__fdiv_rn(x[2 * i], dec), __fdiv_rn(x[2 * i + 1], dec)) << (8 * (i & 3));
  }
  int pos0 = a.pos0;
  if (a.pos0_dev) pos0 = max(0, min(*a.pos0_dev, a.max_seq - a.tokens));
  const long long row = (long long)kvh * a.max_seq + pos0 + t;
  *reinterpret_cast<uint2*>(a.codes + row * (HD / 2) + b * 8) = make_uint2(w[0], w[1]);
  a.scales[row * NB + b] = (uint8_t)sc;
}

template <int HD, int DT>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4Rows a) {
  constexpr int NB = HD / 16;
  const long long idx = blockIdx.x * 256ll + threadIdx.x;
  const int b = (int)(idx % NB);
  const long long r = idx / NB;
  if (r >= 2ll * a.Hkv * a.tokens) return;
  const int t = (int)(r % a.tokens);
  const int kvh = (int)(r / a.tokens);
  const int h = kvh % a.Hkv;
  const bool is_v = kvh >= a.Hkv;
  const long long row = (long long)kvh * a.max_seq + a.pos0 + t;
  const uint2 c = *reinterpret_cast<const uint2*>(a.codes + row * (HD / 2) + b * 8);
  const float dec = e4m3_to_f32(a.scales[row * NB + b]);
  const float ts = is_v ? a.v_scale : a.k_scale;
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpack_f16x2(e2m1_byte_to_f16x2(i < 4 ? c.x : c.y, i & 3));
    x[2 * i] = f.x * dec * ts, x[2 * i + 1] = f.y * dec * ts;
  }
  void* base = const_cast<void*>(is_v ? a.v : a.k);
  const long long off = t * a.token_stride + h * a.head_stride + b * 16;
  if (DT == MSK_FP32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack16(x[2 * i], x[2 * i + 1], DT == MSK_FP16);
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off);
    p[0] = make_uint4(w[0], w[1], w[2], w[3]);
    p[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int HD>
void launch_rows(bool write, int32_t dt, const Kv4Rows& a, cudaStream_t st) {
  const long long n = 2ll * a.Hkv * a.tokens * (HD / 16);
  const unsigned grid = (unsigned)((n + 255) / 256);
#define MSK_ROWS(D)                                                    \
  do {                                                                 \
    if (write) kv4_write_kernel<HD, D><<<grid, 256, 0, st>>>(a);       \
    else kv4_read_kernel<HD, D><<<grid, 256, 0, st>>>(a);              \
  } while (0)
  if (dt == MSK_BF16) MSK_ROWS(MSK_BF16);
  else if (dt == MSK_FP16) MSK_ROWS(MSK_FP16);
  else MSK_ROWS(MSK_FP32);
#undef MSK_ROWS
}

msk_status check_cache(const msk_kv4_desc* c) {
  if (c == nullptr || c->codes == nullptr || c->scales == nullptr) return MSK_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return MSK_ERR_SHAPE;
  if (c->n_kv_heads <= 0 || c->max_seq <= 0) return MSK_ERR_SHAPE;
  // (also false for NaN)
  if (!(c->k_scale > 0.f && c->k_scale <= 3e38f) || !(c->v_scale > 0.f && c->v_scale <= 3e38f)) return MSK_ERR_INVALID_ARG;
  if (!ops_aligned16(c->codes) || !ops_aligned16(c->scales)) return MSK_ERR_ALIGNMENT;
  return MSK_OK;
}

msk_status rows_call(bool write, const msk_kv4_desc* c, const void* k, const void* v, int32_t dtype, int32_t tokens,
                     int64_t ts, int64_t hs, int32_t pos0, const int32_t* pos0_dev, void* stream) {
  msk_status s = check_cache(c);
  if (s != MSK_OK) return s;
  if (!dtype_ok(dtype) || tokens < 0) return MSK_ERR_INVALID_ARG;
  if (tokens == 0) return MSK_OK;
  if (k == nullptr || v == nullptr || ts < 0 || hs < 0) return MSK_ERR_INVALID_ARG;
  if (tokens > c->max_seq || (pos0_dev == nullptr && (pos0 < 0 || pos0 > c->max_seq - tokens))) return MSK_ERR_INVALID_ARG;
  const int per16 = 16 / dtype_bytes(dtype);
  if (!ops_aligned16(k) || !ops_aligned16(v) || ts % per16 || hs % per16) return MSK_ERR_ALIGNMENT;
  // the kernels' grid is one-dimensional
  if (2ll * c->n_kv_heads * tokens * (c->head_dim / 16) / 256 >= 0x7FFFFFFFll) return MSK_ERR_SHAPE;
  int nsm = 0;
  s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  Kv4Rows a{};
  a.codes = c->codes, a.scales = c->scales, a.k = k, a.v = v, a.pos0_dev = pos0_dev;
  a.token_stride = ts, a.head_stride = hs;
  a.Hkv = c->n_kv_heads, a.max_seq = c->max_seq, a.tokens = tokens, a.pos0 = pos0;
  a.k_scale = c->k_scale, a.v_scale = c->v_scale;
  if (c->head_dim == 128) launch_rows<128>(write, dtype, a, static_cast<cudaStream_t>(stream));
  else launch_rows<64>(write, dtype, a, static_cast<cudaStream_t>(stream));
  return cudaGetLastError() == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------

constexpr int kMaxSplits = 64;  // key ranges per kv head

struct Kv4Attn {
  const uint16_t* q;
  uint16_t* out;
  const uint8_t* codes;
  const uint8_t* scales;
  const int32_t* len_dev;
  float* o_part;    // [tiles][Hkv][splits][16][HD]
  float2* ml_part;  // [tiles][Hkv][splits][16] (maximum in log2 units, sum)
  long long q_stride;
  int T, Hq, Hkv, G, max_seq, len, window, splits;
  bool fp16;
  float qk_scale;  // softmax scale * k_scale * log2(e)
  float v_scale;
  int depth[kMaxT];
  uint32_t vis[kMaxT];
};

__device__ __forceinline__ int cached_len(const Kv4Attn& a) {
  return a.len_dev ? max(0, min(*a.len_dev, a.max_seq - a.T)) : a.len;
}

// Does query slot t (position len + depth) see cache row j?
__device__ __forceinline__ bool sees(const Kv4Attn& a, int t, int j, int len) {
  if (j >= len) return j - len < a.T && ((a.vis[t] >> (j - len)) & 1u);
  return a.window == 0 || j > len + a.depth[t] - a.window;
}

// A warp takes 16 keys at a time for a tile of 16 query rows (row = token *
// group + head of the group).  S = Q K^T and O = P V on mma.sync with K and V
// decoded straight into its B fragments: no shared memory on the way.
//  K: lane (g, c) of a fragment holds key g and, of each 16 dimensions, any
//     four, as long as Q's fragments hold the same: it takes the HD / 4
//     dimensions from c HD / 4 (16 bytes of codes at HD = 128), four a step.
//  V: the fragment pairs two keys for one dimension; lane (g, c) holds four
//     keys and takes the HD / 8 dimensions from g HD / 8.  Nibbles of two
//     keys are put into one byte before the decoding, so a byte decodes to
//     the pair.
// Values are exact in fp16 (at most 6 significant bits, at most 2688).
template <int HD>
__global__ void __launch_bounds__(256) kv4_attention_kernel(const __grid_constant__ Kv4Attn a) {
  constexpr int KS = HD / 16;   // steps of S's contraction
  constexpr int NT = HD / 8;    // n tiles of O
  constexpr int KW = HD / 32;   // code words of a lane's K piece
  constexpr int VW = HD / 64;   // code words of a lane's V piece of one key
  extern __shared__ float smem[];  // [8 warps][16][HD + 1], then [8][16] (m, l)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int split = blockIdx.x, h = blockIdx.y, tile = blockIdx.z;
  const int len = cached_len(a);
  const int rows = a.T * a.G;

  // this lane's query rows g and g + 8
  uint32_t qf[KS][4];
  float fac[2];
  int tok[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = tile * 16 + g + 8 * i;
    tok[i] = row < rows ? row / a.G : -1;
    uint32_t w[HD / 8];
#pragma unroll
    for (int j = 0; j < HD / 8; ++j) w[j] = 0;
    if (tok[i] >= 0) {
      const uint16_t* p = a.q + tok[i] * a.q_stride + (long long)(h * a.G + row % a.G) * HD + c * (HD / 4);
#pragma unroll
      for (int j = 0; j < HD / 32; ++j) {
        const uint4 u = *reinterpret_cast<const uint4*>(p + 8 * j);
        w[4 * j] = u.x, w[4 * j + 1] = u.y, w[4 * j + 2] = u.z, w[4 * j + 3] = u.w;
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < HD / 8; ++j) {
      const float2 f = unpack16(w[j], a.fp16);
      amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    const int sh = row_shift(amax);
    const float mul = exp2i(sh);
    fac[i] = a.qk_scale * exp2i(-sh);
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      const float2 lo = unpack16(w[2 * j], a.fp16), hi = unpack16(w[2 * j + 1], a.fp16);
      qf[j][i] = pack_f16x2(lo.x * mul, lo.y * mul);
      qf[j][i + 2] = pack_f16x2(hi.x * mul, hi.y * mul);
    }
  }

  // this block's keys: [lo, hi), in steps of 16 handed round the warps
  const int n = len + a.T;
  const int lo = a.window > 0 ? max(0, len - a.window + 1) : 0, first = lo & ~15;  // (no query sees a key before lo)
  const int steps = (n - first + 15) / 16;
  const int per = (steps + a.splits - 1) / a.splits;
  const int s0 = split * per, s1 = min(steps, s0 + per);
  const uint8_t* kc = a.codes + (long long)h * a.max_seq * (HD / 2);
  const uint8_t* ks = a.scales + (long long)h * a.max_seq * (HD / 16);
  const uint8_t* vc = kc + (long long)a.Hkv * a.max_seq * (HD / 2);
  const uint8_t* vs = ks + (long long)a.Hkv * a.max_seq * (HD / 16);

  float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

  for (int s = s0 + warp; s < s1; s += 8) {
    const int j0 = first + s * 16;
    float sc[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const long long j = min(j0 + nt * 8 + g, n - 1);
      uint32_t w[KW], e;
      if (KW == 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(kc + j * (HD / 2) + c * 16);
        w[0] = u.x, w[1] = u.y, w[KW - 2] = u.z, w[KW - 1] = u.w;
        e = *reinterpret_cast<const uint16_t*>(ks + j * (HD / 16) + c * 2);
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(kc + j * (HD / 2) + c * 8);
        w[0] = u.x, w[1] = u.y;
        e = ks[j * (HD / 16) + c];
      }
      const uint32_t ef = e4m3x2_to_f16x2(e);
      sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint32_t f = f16x2_bcast(ef, k >= 4);
        mma_f16(sc[nt], qf[k], hmul2(e2m1_byte_to_f16x2(w[k >> 1], 2 * (k & 1)), f),
                hmul2(e2m1_byte_to_f16x2(w[k >> 1], 2 * (k & 1) + 1), f));
      }
    }
    // scores in log2 units, masked
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + nt * 8 + 2 * c + (i & 1), t = tok[i >> 1];
        sc[nt][i] = t >= 0 && sees(a, t, j, len) ? sc[nt][i] * fac[i >> 1] : -INFINITY;
      }
    uint32_t pa[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = fmaxf(fmaxf(sc[0][2 * i], sc[0][2 * i + 1]), fmaxf(sc[1][2 * i], sc[1][2 * i + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      const float mn = fmaxf(m[i], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float al = exp2f(m[i] - ref);
      m[i] = mn;
      float p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = exp2f(sc[k >> 1][2 * i + (k & 1)] - ref);
      l[i] = l[i] * al + (p[0] + p[1]) + (p[2] + p[3]);
      pa[i] = pack_f16x2(p[0], p[1]);
      pa[i + 2] = pack_f16x2(p[2], p[3]);
#pragma unroll
      for (int k = 0; k < NT; ++k) o[k][2 * i] *= al, o[k][2 * i + 1] *= al;
    }
    // O += P V
    uint32_t vw[4][VW], ve[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int jj = j0 + (k >> 1) * 8 + 2 * c + (k & 1);
      const long long j = min(jj, n - 1);
      if (VW == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(vc + j * (HD / 2) + g * 8);
        vw[k][0] = u.x, vw[k][VW - 1] = u.y;
      } else {
        vw[k][0] = *reinterpret_cast<const uint32_t*>(vc + j * (HD / 2) + g * 4);
      }
      ve[k] = jj >= lo && jj < n ? vs[j * (HD / 16) + (g * NT) / 16] : 0u;  // (rows outside may hold anything)
    }
    const uint32_t e0 = e4m3x2_to_f16x2(ve[0] | ve[1] << 8), e1 = e4m3x2_to_f16x2(ve[2] | ve[3] << 8);
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      const uint32_t M = 0x0F0F0F0Fu;
      const uint32_t a0 = (vw[0][w] & M) | ((vw[1][w] & M) << 4), a1 = ((vw[0][w] >> 4) & M) | (vw[1][w] & ~M);
      const uint32_t b0 = (vw[2][w] & M) | ((vw[3][w] & M) << 4), b1 = ((vw[2][w] >> 4) & M) | (vw[3][w] & ~M);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        mma_f16(o[w * 8 + 2 * k], pa, hmul2(e2m1_byte_to_f16x2(a0, k), e0), hmul2(e2m1_byte_to_f16x2(b0, k), e1));
        mma_f16(o[w * 8 + 2 * k + 1], pa, hmul2(e2m1_byte_to_f16x2(a1, k), e0), hmul2(e2m1_byte_to_f16x2(b1, k), e1));
      }
    }
  }

  // merge the warps
  float* so = smem;                                              // [8][16][HD + 1]
  float2* sml = reinterpret_cast<float2*>(smem + 8 * 16 * (HD + 1));  // [8][16]
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
    l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
    const int r = g + 8 * i;
    if (c == 0) sml[warp * 16 + r] = make_float2(m[i], l[i]);
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      so[(warp * 16 + r) * (HD + 1) + 2 * c * NT + k] = o[k][2 * i];
      so[(warp * 16 + r) * (HD + 1) + (2 * c + 1) * NT + k] = o[k][2 * i + 1];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * HD; i += 256) {
    const int r = i / HD, d = i % HD, row = tile * 16 + r;
    if (row >= rows) break;
    float mm = -INFINITY;
    for (int w = 0; w < 8; ++w) mm = fmaxf(mm, sml[w * 16 + r].x);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float sum = 0.f, ll = 0.f;
    for (int w = 0; w < 8; ++w) {
      const float f = exp2f(sml[w * 16 + r].x - ref);
      sum += f * so[(w * 16 + r) * (HD + 1) + d];
      ll += f * sml[w * 16 + r].y;
    }
    const long long part = (((long long)tile * a.Hkv + h) * a.splits + split) * 16 + r;
    a.o_part[part * HD + d] = sum;
    if (d == 0) a.ml_part[part] = make_float2(mm, ll);
  }
}

// One block per (token, query head), HD threads.
template <int HD>
__global__ void __launch_bounds__(HD) kv4_combine_kernel(const __grid_constant__ Kv4Attn a) {
  const int t = blockIdx.x, hq = blockIdx.y, d = threadIdx.x;
  const int h = hq / a.G, row = t * a.G + hq % a.G;
  const long long base = ((long long)(row >> 4) * a.Hkv + h) * a.splits * 16 + (row & 15);
  float mm = -INFINITY;
  for (int s = 0; s < a.splits; ++s) mm = fmaxf(mm, a.ml_part[base + s * 16].x);
  float sum = 0.f, ll = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const float2 ml = a.ml_part[base + s * 16];
    const float f = exp2f(ml.x - mm);
    sum += f * a.o_part[(base + s * 16) * HD + d];
    ll += f * ml.y;
  }
  const float y = sum / ll * a.v_scale;
  uint16_t* p = a.out + (long long)t * a.Hq * HD + (long long)hq * HD + d;
  *p = a.fp16 ? __half_as_ushort(__float2half_rn(y)) : __bfloat16_as_ushort(__float2bfloat16_rn(y));
}

int attention_splits(int tiles, int Hkv) { return std::max(1, std::min(kMaxSplits, 2 * kOpsSms / (tiles * Hkv))); }

template <int HD>
cudaError_t launch_attention(const Kv4Attn& a, int tiles, cudaStream_t st) {
  const int smem = 8 * 16 * (HD + 1) * 4 + 8 * 16 * 8;
  cudaError_t e = cudaFuncSetAttribute(kv4_attention_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kv4_attention_kernel<HD><<<dim3(a.splits, a.Hkv, tiles), 256, smem, st>>>(a);
  kv4_combine_kernel<HD><<<dim3(a.T, a.Hq), HD, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace msk

using namespace msk;

extern "C" msk_status msk_kv4_write(const msk_kv4_desc* cache, const void* k, const void* v, int32_t dtype,
                                    int32_t tokens, int64_t token_stride, int64_t head_stride, int32_t pos0,
                                    const int32_t* pos0_dev, void* stream) {
  return rows_call(true, cache, k, v, dtype, tokens, token_stride, head_stride, pos0, pos0_dev, stream);
}

extern "C" msk_status msk_kv4_read(const msk_kv4_desc* cache, int32_t pos0, int32_t tokens, void* k, void* v,
                                   int32_t dtype, int64_t token_stride, int64_t head_stride, void* stream) {
  return rows_call(false, cache, k, v, dtype, tokens, token_stride, head_stride, pos0, nullptr, stream);
}

extern "C" size_t msk_attention_kv4_workspace(int32_t tokens, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (tokens <= 0 || tokens > kMaxT || n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads || head_dim <= 0) return 0;
  const int tiles = (tokens * (n_q_heads / n_kv_heads) + 15) / 16;
  return (size_t)tiles * n_kv_heads * attention_splits(tiles, n_kv_heads) * 16 * (head_dim + 2) * 4;
}

extern "C" msk_status msk_attention_kv4(const void* q, int32_t dtype, int64_t q_stride, const msk_kv4_desc* cache,
                                        int32_t tokens, int32_t n_q_heads, int32_t cache_len,
                                        const int32_t* cache_len_dev, const int32_t* parents, int32_t window,
                                        float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  msk_status s = check_cache(cache);
  if (s != MSK_OK) return s;
  if (q == nullptr || out == nullptr) return MSK_ERR_INVALID_ARG;
  if (dtype != MSK_BF16 && dtype != MSK_FP16) return MSK_ERR_INVALID_ARG;
  if (tokens <= 0 || tokens > kMaxT || n_q_heads <= 0 || n_q_heads % cache->n_kv_heads) return MSK_ERR_SHAPE;
  const int G = n_q_heads / cache->n_kv_heads, tiles = (tokens * G + 15) / 16;
  if (cache->n_kv_heads > 65535 || tiles > 65535 || n_q_heads > 65535) return MSK_ERR_SHAPE;  // (grid limits)
  if (window < 0 || tokens > cache->max_seq) return MSK_ERR_INVALID_ARG;
  if (cache_len_dev == nullptr && (cache_len < 0 || cache_len > cache->max_seq - tokens)) return MSK_ERR_INVALID_ARG;
  if (!(softmax_scale >= 0.f && softmax_scale <= 3e38f)) return MSK_ERR_INVALID_ARG;
  if (q_stride < (int64_t)n_q_heads * cache->head_dim && tokens > 1) return MSK_ERR_INVALID_ARG;
  if (!ops_aligned16(q) || !ops_aligned16(out) || !ops_aligned16(workspace) || q_stride % 8) return MSK_ERR_ALIGNMENT;
  Kv4Attn a{};
  if (!tree_masks(parents, tokens, window, a.depth, a.vis)) return MSK_ERR_INVALID_ARG;
  if (workspace == nullptr ||
      workspace_bytes < msk_attention_kv4_workspace(tokens, n_q_heads, cache->n_kv_heads, cache->head_dim))
    return MSK_ERR_INVALID_ARG;
  int nsm = 0;
  s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.codes = cache->codes;
  a.scales = cache->scales;
  a.len_dev = cache_len_dev;
  a.q_stride = q_stride;
  a.T = tokens, a.Hq = n_q_heads, a.Hkv = cache->n_kv_heads, a.G = G;
  a.max_seq = cache->max_seq, a.len = cache_len, a.window = window;
  a.splits = attention_splits(tiles, a.Hkv);
  a.fp16 = dtype == MSK_FP16;
  const float scale = softmax_scale > 0.f ? softmax_scale : (float)(1.0 / std::sqrt((double)cache->head_dim));
  a.qk_scale = scale * cache->k_scale * 1.4426950408889634f;
  a.v_scale = cache->v_scale;
  const size_t parts = (size_t)tiles * a.Hkv * a.splits * 16;
  a.o_part = static_cast<float*>(workspace);
  a.ml_part = reinterpret_cast<float2*>(a.o_part + parts * cache->head_dim);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->head_dim == 128 ? launch_attention<128>(a, tiles, st) : launch_attention<64>(a, tiles, st);
  return e == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}
