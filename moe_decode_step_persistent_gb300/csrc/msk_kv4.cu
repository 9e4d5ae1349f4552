// The 4-bit KV cache: writing rows (quantise), reading them back, and GQA
// attention over them.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "msk_internal.h"
#include "msk_ops.cuh"
#include "msk_tc.cuh"

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

// 16 consecutive elements of type DT as floats.
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

// Two -x / d rounded to nearest (my: two rounded reciprocals of d, negative;
// quotients and remainders within the normal range): Markstein's correction of
// x my by its remainder (IBM J. Res. Dev. 34, 1990).  The codes depend on the
// quotient's last bit where it lies half way between two of them.  The negative
// quotient, because a remainder of 0 is +0: times my it is -0, which leaves the
// sign of a zero alone, and +0, times y, would not.
__device__ __forceinline__ void minus_quotients(float& x0, float& x1, unsigned long long d, unsigned long long my) {
  const unsigned long long x = pair(x0, x1), q = mul2(x, my);
  unpair(fma2(fma2(q, d, x), my, q), x0, x1);
}

// Both kernels: blockIdx.y is K's and then V's heads, a block takes `per`
// consecutive pieces of its head's rows.
struct RowsAt {
  int h;
  bool is_v;
  long long at;     // first piece of the rows in the cache, in pieces
  long long piece;  // this thread's first
  long long n;      // pieces of the head's rows
};
template <int NP>
__device__ __forceinline__ RowsAt rows_at(const Kv4Rows& a, int pos0, int per) {
  const int kvh = blockIdx.y;
  const bool is_v = kvh >= a.Hkv;
  return {is_v ? kvh - a.Hkv : kvh, is_v, ((long long)kvh * a.max_seq + pos0) * NP, (long long)blockIdx.x * per + threadIdx.x,
          (long long)a.tokens * NP};
}

// A piece is a block of 16 elements, one a thread.  16384 rows of 8 heads of 128
// in bf16: 17.0 us with scales of 1, 19.1 with others (without the signs of zeros
// 16.4 and 18.9; two pieces a thread 4 us more, half a piece, so that two threads do
// each block's scale, 8): the quantiser's instructions bound it beside DRAM (12.7 us
// for the bytes).
template <int HD, int DT>
__global__ void __launch_bounds__(256) kv4_write_kernel(const Kv4Rows a) {
  constexpr int NP = HD / 16;
  grid_dep_wait();
  grid_dep_launch();
  int pos0 = a.pos0;
  if (a.pos0_dev) pos0 = max(0, min(*a.pos0_dev, a.max_seq - a.tokens));
  const RowsAt w = rows_at<NP>(a, pos0, 256);
  if (w.piece >= w.n) return;
  const float ts = w.is_v ? a.v_scale : a.k_scale, yts = __frcp_rn(ts);
  const unsigned long long ts2 = pair(ts, ts), myts2 = pair(-yts, -yts);
  const bool plain = ts > 1e-18f && ts < 1e18f;
  const void* src = w.is_v ? a.v : a.k;
  const long long from = w.piece / NP * a.token_stride + w.h * a.head_stride + w.piece % NP * 16;
  float x[16];
  load16<DT>(src, from, x);
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(x[j]));
  const bool whole = ts == 1.f;
  if (!whole) {  // x becomes -x / ts
    if (plain && amax < 1e18f) {  // (smaller quotients than normal ones leave codes of 0)
#pragma unroll
      for (int j = 0; j < 16; j += 2) minus_quotients(x[j], x[j + 1], ts2, myts2);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = __fdiv_rn(x[j], -ts);
    }
    amax = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(x[j]));
  }
  // amax / 6 (what is beyond 448 saturates)
  const float y6 = 1.f / 6.f, am = fminf(amax, 1e6f), q6 = am * y6;
  const uint32_t sc = f32_to_e4m3(fmaf(fmaf(-q6, 6.f, am), y6, q6));
  const float dec = e4m3_to_f32(sc);
  uint32_t c[2] = {0u, 0u};
  if (amax > 2688.f) {  // saturates, with infinities perhaps
    const float d = whole ? dec : -dec;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      c[j >> 2] |= f32x2_to_e2m1x2(__fdiv_rn(x[2 * j], d), __fdiv_rn(x[2 * j + 1], d)) << (8 * (j & 3));
  } else if (dec > 0.f) {
    const float y = __frcp_rn(dec);
    auto codes = [&](auto negate) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float u = x[2 * j], v = x[2 * j + 1];
        minus_quotients(u, v, pair(dec, dec), pair(-y, -y));
        c[j >> 2] |= (negate() ? f32x2_to_e2m1x2(-u, -v) : f32x2_to_e2m1x2(u, v)) << (8 * (j & 3));
      }
    };
    if (whole) codes(std::true_type());
    else codes(std::false_type());  // (two negative quotients)
  }
  const long long at = w.at + w.piece;  // (rows of a head are consecutive)
  *reinterpret_cast<uint2*>(a.codes + at * 8) = make_uint2(c[0], c[1]);
  a.scales[at] = (uint8_t)sc;
}

// A piece is what fills 16 bytes of the rows, so that a warp's stores are one
// run; four a thread, all loaded first.  16384 rows of 8 heads of 128 in bf16:
// 11.8 us, as fast as DRAM takes the bytes (two a thread 13.0, one 17.4).
constexpr int kReadUnroll = 4;
template <int HD, int DT>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4Rows a) {
  constexpr int E = DT == MSK_FP32 ? 4 : 8, NP = HD / E, U = kReadUnroll;
  using Codes = std::conditional_t<E == 4, uint16_t, uint32_t>;
  grid_dep_wait();
  grid_dep_launch();
  const RowsAt w = rows_at<NP>(a, a.pos0, 256 * U);
  const float ts = w.is_v ? a.v_scale : a.k_scale;
  uint32_t c[U], e[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const long long at = w.at + w.piece + k * 256;
    if (w.piece + k * 256 < w.n) {
      c[k] = __ldg(reinterpret_cast<const Codes*>(a.codes) + at);
      e[k] = __ldg(a.scales + at / (16 / E));
    }
  }
  void* dst = const_cast<void*>(w.is_v ? a.v : a.k);
  const long long to = w.piece / NP * a.token_stride + w.h * a.head_stride + w.piece % NP * E;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (w.piece + k * 256 >= w.n) break;
    const float dec = e4m3_to_f32(e[k]);
    float x[E];
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const float2 f = unpack_f16x2(e2m1_byte_to_f16x2(c[k], j));
      x[2 * j] = f.x * dec * ts, x[2 * j + 1] = f.y * dec * ts;
    }
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = DT == MSK_FP32 ? __float_as_uint(x[j]) : pack16(x[2 * j % E], x[(2 * j + 1) % E], DT == MSK_FP16);
    const long long off = to + k * (256 / NP) * a.token_stride;
    *reinterpret_cast<uint4*>(static_cast<char*>(dst) + off * (16 / E)) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int HD>
cudaError_t launch_rows(bool write, int32_t dt, const Kv4Rows& a, cudaStream_t st) {
  const int piece = write ? 16 : dt == MSK_FP32 ? 4 : 8, per = write ? 256 : 256 * kReadUnroll;
  const long long n = (long long)a.tokens * HD / piece;
  const dim3 grid((unsigned)((n + per - 1) / per), 2u * a.Hkv);
  const OpsLaunch l(grid, 256, 0, st);
  auto launch = [&](void (*write_kernel)(Kv4Rows), void (*read_kernel)(Kv4Rows)) {
    return cudaLaunchKernelEx(&l.cfg, write ? write_kernel : read_kernel, a);
  };
  return dt == MSK_BF16   ? launch(kv4_write_kernel<HD, MSK_BF16>, kv4_read_kernel<HD, MSK_BF16>)
         : dt == MSK_FP16 ? launch(kv4_write_kernel<HD, MSK_FP16>, kv4_read_kernel<HD, MSK_FP16>)
                          : launch(kv4_write_kernel<HD, MSK_FP32>, kv4_read_kernel<HD, MSK_FP32>);
}

constexpr int kMaxRows = 1 << 30;  // of a cache: positions and steps stay within 32 bits

msk_status check_cache(const msk_kv4_desc* c) {
  if (c == nullptr || c->codes == nullptr || c->scales == nullptr) return MSK_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return MSK_ERR_SHAPE;
  if (c->n_kv_heads <= 0 || c->max_seq <= 0 || c->max_seq > kMaxRows) return MSK_ERR_SHAPE;
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
  // (rows that are read may be one and the same, those that are written may not)
  if (!write && ((tokens > 1 && ts == 0) || (c->n_kv_heads > 1 && hs == 0))) return MSK_ERR_INVALID_ARG;
  if (tokens > c->max_seq || (pos0_dev == nullptr && (pos0 < 0 || pos0 > c->max_seq - tokens))) return MSK_ERR_INVALID_ARG;
  const int per16 = 16 / dtype_bytes(dtype);
  if (!ops_aligned16(k) || !ops_aligned16(v) || ts % per16 || hs % per16) return MSK_ERR_ALIGNMENT;
  if (c->n_kv_heads > 32767) return MSK_ERR_SHAPE;  // (the grid's second axis)
  int nsm = 0;
  s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  Kv4Rows a{};
  a.codes = c->codes, a.scales = c->scales, a.k = k, a.v = v, a.pos0_dev = pos0_dev;
  a.token_stride = ts, a.head_stride = hs;
  a.Hkv = c->n_kv_heads, a.max_seq = c->max_seq, a.tokens = tokens, a.pos0 = pos0;
  a.k_scale = c->k_scale, a.v_scale = c->v_scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = c->head_dim == 128 ? launch_rows<128>(write, dtype, a, st) : launch_rows<64>(write, dtype, a, st);
  return e == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------

constexpr int kMaxSplits = 128;   // key ranges of a kv head, each a block's, joined by a second kernel
constexpr int kMaxCluster = 9;    // or, of few keys, the blocks of a cluster (as many clusters of 9 run at once as of 8)
// Up to so many keys (of a tile of 8 rows, of more) a cluster and its one launch
// beat ranges and a second kernel.  4 rows (1 token of a group of 4) x 6000 keys 7.4 us
// and 8.8, 12000 10.3 and 9.9; 12 rows x 2000 8.4 and 9.0, 4000 9.8 either way, 6000
// 10.9 and 9.8; 64 rows x 2000 11.3 and 12.1, 4000 13.4 and 12.5, 8000 17.5 and 14.9.
constexpr int cluster_keys(int rows) { return rows <= 8 ? 8192 : 256 * kMaxCluster; }
constexpr int kRing = 5;          // steps of 16 keys in a warp's ring

struct Kv4Attn {
  const uint16_t* q;
  uint16_t* out;
  const uint8_t* codes;
  const uint8_t* scales;
  const int32_t* len_dev;
  float* o_part;    // [tiles][Hkv][splits][rows of a tile][HD]
  float2* ml_part;  // [tiles][Hkv][splits][rows of a tile] (reference in log2 units, sum)
  long long q_stride;
  int T, Hq, Hkv, G, max_seq, len, window, splits, cluster;
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

__device__ __forceinline__ void store_out(const Kv4Attn& a, int hd, int h, int row, int d, float y) {
  uint16_t* p = a.out + ((long long)(row / a.G) * a.Hq + h * a.G + row % a.G) * hd + d;
  *p = a.fp16 ? __half_as_ushort(__float2half_rn(y)) : __bfloat16_as_ushort(__float2bfloat16_rn(y));
}

// 8 x 8 fp16 matrix across a warp (lane (g, c): row g, columns 2c and 2c + 1),
// transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// 16 keys and their values in shared memory, as in the cache (rows one behind
// the other), and the fragments that a lane takes from there.
template <int HD>
struct Kv16 {
  static constexpr int KW = HD / 32, VW = HD / 64;                 // code words of a lane's key, value
  static constexpr int CODES = 16 * HD / 2, SCALES = HD;           // bytes of 16 rows
  static constexpr int BYTES = 2 * (CODES + SCALES);               // K codes, V codes, K scales, V scales
};

template <int W>
__device__ __forceinline__ void lds_words(uint32_t (&w)[W], uint32_t at) {
  if (W == 4) {
    const uint4 u = lds128(at);
    w[0] = u.x, w[1] = u.y, w[W - 2] = u.z, w[W - 1] = u.w;
  } else if (W == 2) {
    const uint2 u = lds64(at);
    w[0] = u.x, w[W - 1] = u.y;
  } else {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
  }
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// A softmax's reference lies kBelow powers of two under the greatest score that it
// was set from, and is raised when a weight would pass 2^kMost: weights reach 2^15 of
// fp16's 65504, and the sums are rescaled a few times in all.
constexpr float kBelow = 7.f, kMost = 15.f;

// Two weights for an fp16 operand, and what their rounding left out for a second
// one: together 22 bits, and off by at most 2^-25 where that is more, 2^-32 of the
// greatest weight.  (In one operand of 11 bits the weights differ from those in the
// fp32 sum of weights by up to 2^-12, and all below 2^-25 are lost.)
struct Split {
  uint32_t hi, lo;
};
__device__ __forceinline__ Split split_f16x2(float x, float y) {
  const uint32_t hi = pack_f16x2(x, y);
  const float2 f = unpack_f16x2(hi);
  return {hi, pack_f16x2(x - f.x, y - f.y)};
}

// Four elements of an output row.
__device__ __forceinline__ void store_out4(const Kv4Attn& a, int hd, int h, int row, int d, float4 y) {
  uint16_t* p = a.out + ((long long)(row / a.G) * a.Hq + h * a.G + row % a.G) * hd + d;
  *reinterpret_cast<uint2*>(p) = make_uint2(pack16(y.x, y.y, a.fp16), pack16(y.z, y.w, a.fp16));
}

// The end of an attention block: its sums, smem[row][PITCH] with the reference
// and the sum of weights behind each row's elements, go to the workspace or
// straight to the output; or to the block of the cluster that joins the row, rank
// r mod cluster: all blocks push into `recv` there, so that one barrier lies
// between the sums and the output and nothing remote is read.  (The cluster's
// first barrier, which the block has entered before, says that all blocks are there
// and that their `recv` is free.)
constexpr int recv_bytes(int rows, int hd) { return (rows + kMaxCluster - 1) * (hd + 4) * 4; }
template <int HD, int ROWS, int THREADS>
__device__ __forceinline__ void finish_block(const Kv4Attn& a, float* smem, float* recv, int split, int h, int tile) {
  constexpr int PITCH = HD + 4, Q4 = HD / 4;
  const int rows = min(ROWS, a.T * a.G - tile * ROWS), tid = threadIdx.x;
  if (a.splits > 1) {
    const long long part = (((long long)tile * a.Hkv + h) * a.splits + split) * ROWS;
    for (int e = tid; e < rows * Q4; e += THREADS) {
      const int r = e / Q4, q = e % Q4;
      *reinterpret_cast<float4*>(a.o_part + (part + r) * HD + q * 4) = *reinterpret_cast<const float4*>(smem + r * PITCH + q * 4);
    }
    for (int r = tid; r < rows; r += THREADS) a.ml_part[part + r] = make_float2(smem[r * PITCH + HD], smem[r * PITCH + HD + 1]);
    return;
  }
  const int n = a.cluster, rank = n > 1 ? split : 0;
  const float* from = smem;
  if (n > 1) {
    cluster_wait();
    for (int e = tid; e < rows * Q4; e += THREADS) {
      const int r = e / Q4, q = e % Q4, to = r % n;
      const float* x = smem + r * PITCH + q * 4;
      const uint32_t at = smem_u32(recv + (r / n * n + rank) * PITCH + q * 4);
      st_cluster4(mapa(at, to), *reinterpret_cast<const float4*>(x));
      if (q == Q4 - 1) st_cluster4(mapa(at + 16, to), *reinterpret_cast<const float4*>(x + 4));
    }
    cluster_arrive();
    cluster_wait();
    from = recv;
  }
  for (int e = tid; e < (rows - rank + n - 1) / n * Q4; e += THREADS) {
    const int i = e / Q4, q = e % Q4;
    const float* x = from + i * n * PITCH;
    float mm = -INFINITY, ll = 0.f;
    for (int b = 0; b < n; ++b) mm = fmaxf(mm, x[b * PITCH + HD]);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = 0; b < n; ++b) {
      const float f = ex2(x[b * PITCH + HD] - mm);  // (a block without a visible key: 0)
      const float4 v = *reinterpret_cast<const float4*>(x + b * PITCH + q * 4);
      ll += f * x[b * PITCH + HD + 1];
      y.x += f * v.x, y.y += f * v.y, y.z += f * v.z, y.w += f * v.w;
    }
    const float f = a.v_scale / ll;
    store_out4(a, HD, h, tile * ROWS + i * n + rank, q * 4, make_float4(y.x * f, y.y * f, y.z * f, y.w * f));
  }
}

// Few query rows (8 NT of them in a tile; row = token * group + head of the
// group): a warp takes 16 keys at a time, as the M of S^T = K Q^T and O^T =
// V^T P^T, so that NT n-tiles hold all rows and a key is decoded once, into the
// A fragments:
//  K: lane (g, c) holds the keys of A rows g and g + 8 and, of each 16
//     dimensions, any four, as long as Q's fragments hold the same: it takes
//     the HD / 4 dimensions from c HD / 4 (16 bytes of codes at HD = 128).
//  V: the fragment pairs two keys for one dimension; the lane holds four keys
//     and takes the HD / 8 dimensions from g HD / 8, two for each m-tile (one
//     byte).  Nibbles of two keys are put into one byte before the decoding,
//     so a byte decodes to the pair.
//  P: S^T's accumulators, as fp16, are P^T's B fragments after one 8 x 8
//     transposition each.
// A row 2i stands for the step's key i, row 2i + 1 for key 4 + i (+ 8 in the
// second half), so that the lanes' values lie next to each other.  Elements
// are exact in fp16 (at most 6 significant bits, at most 2688).
//
// A warp's keys come through a ring of kRing steps of its own, by asynchronous
// copies; warps meet only at the end.  One token, 131071 keys of 8 kv heads: 36.0
// us (4.2 TB/s, 62% of what a copy reaches; with weights of one part 34.3).  Bound by
// the decoding (a conversion and a multiply for two elements; the ALU 55%, issue
// slots 60% in use) beside DRAM.  Q in shared memory for three blocks an SM instead
// of two lost 8 us.
template <int HD, int NT>
constexpr int rows_smem() {  // the rings, then the warps' sums
  return std::max(8 * kRing * Kv16<HD>::BYTES, 8 * 8 * NT * (HD + 4) * 4 + 8 * 8 * NT * 8);
}
template <int HD, int NT>
__global__ void __launch_bounds__(256, NT == 1 ? 2 : 1) kv4_rows_kernel(const __grid_constant__ Kv4Attn a) {
  constexpr int KS = HD / 16, MT = HD / 16, ROWS = 8 * NT, PITCH = HD + 4;
  using K16 = Kv16<HD>;
  // the warps' rings; after the last step [8 warps][ROWS][PITCH] sums, [8][ROWS] (reference, sum)
  extern __shared__ __align__(16) float smem[];
  float2* sml = reinterpret_cast<float2*>(smem + 8 * ROWS * PITCH);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int split = blockIdx.x, h = blockIdx.y, tile = blockIdx.z;
  if (a.cluster > 1) cluster_arrive();
  grid_dep_wait();
  const int len = cached_len(a), rows = a.T * a.G;

  // this block's keys: in steps of 16 handed round the warps
  const int n = len + a.T;
  const int lo = a.window > 0 ? max(0, len - a.window + 1) : 0, first = lo & ~15;  // (no query sees a key before lo)
  const int steps = (n - first + 15) / 16;
  const int per = (steps + (int)gridDim.x - 1) / (int)gridDim.x;
  const int s0 = split * per, s1 = min(steps, s0 + per);
  const uint8_t* kc = a.codes + (long long)h * a.max_seq * (HD / 2);
  const uint8_t* ks = a.scales + (long long)h * a.max_seq * (HD / 16);
  const long long vc = (long long)a.Hkv * a.max_seq * (HD / 2), vs = (long long)a.Hkv * a.max_seq * (HD / 16);
  const uint32_t ring = smem_u32(smem) + warp * kRing * K16::BYTES;
  // the next step to fetch, this lane's parts of it: 16 bytes of codes in each
  // half kilobyte of keys and of values, one row's scales (lanes 0-15 the
  // keys', 16-31 the values')
  int fs = s0 + warp;
  uint32_t fslot = ring;
  const uint8_t* fk = kc + (long long)(first + fs * 16) * (HD / 2) + lane * 16;
  const uint8_t* fe = ks + (lane < 16 ? 0 : vs) + (long long)(first + fs * 16 + (lane & 15)) * (HD / 16);
  const uint32_t fet = 2 * K16::CODES + (lane < 16 ? 0 : K16::SCALES) + (lane & 15) * (HD / 16);
  auto fetch = [&]() {
    if (fs < s1) {
      const int have = n - (first + fs * 16);  // (rows past the last one are not read)
      if (have >= 16) {
#pragma unroll
        for (int i = 0; i < K16::CODES / 512; ++i) {
          cp_async16(fslot + i * 512 + lane * 16, fk + i * 512);
          cp_async16(fslot + K16::CODES + i * 512 + lane * 16, fk + vc + i * 512);
        }
        if (HD == 128) cp_async8(fslot + fet, fe);
        else cp_async4(fslot + fet, fe);
      } else {
#pragma unroll
        for (int i = 0; i < K16::CODES / 512; ++i)
          if (i * 512 + lane * 16 < have * (HD / 2)) {
            cp_async16(fslot + i * 512 + lane * 16, fk + i * 512);
            cp_async16(fslot + K16::CODES + i * 512 + lane * 16, fk + vc + i * 512);
          }
        if ((lane & 15) < have) {
          if (HD == 128) cp_async8(fslot + fet, fe);
          else cp_async4(fslot + fet, fe);
        }
      }
    }
    cp_async_commit();
    fs += 8, fk += 8 * K16::CODES, fe += 8 * K16::SCALES;
    fslot = fslot == ring + (kRing - 1) * K16::BYTES ? ring : fslot + K16::BYTES;
  };
  // Q: lane (g, c) of n-tile nt holds row 8 nt + g
  // (its loads go out before the ring's, which would keep them waiting)
  uint32_t qf[NT][KS][2], w[NT][HD / 8];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = tile * ROWS + nt * 8 + g;
#pragma unroll
    for (int j = 0; j < HD / 8; ++j) w[nt][j] = 0;
    if (row < rows) {
      const uint16_t* p = a.q + (row / a.G) * a.q_stride + (long long)(h * a.G + row % a.G) * HD + c * (HD / 4);
#pragma unroll
      for (int j = 0; j < HD / 32; ++j) {
        const uint4 u = *reinterpret_cast<const uint4*>(p + 8 * j);
        w[nt][4 * j] = u.x, w[nt][4 * j + 1] = u.y, w[nt][4 * j + 2] = u.z, w[nt][4 * j + 3] = u.w;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch();
  float fac[NT][2];
  int tok[NT][2];  // the tokens of this lane's accumulator columns, -1 past the last row
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < HD / 8; ++j) {
      const float2 f = unpack16(w[nt][j], a.fp16);
      amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    const int sh = row_shift(amax);
    const float mul = exp2i(sh);
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 f = unpack16(w[nt][2 * j + i], a.fp16);
        qf[nt][j][i] = pack_f16x2(f.x * mul, f.y * mul);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fac[nt][i] = a.qk_scale * exp2i(-__shfl_sync(0xFFFFFFFFu, sh, (2 * c + i) * 4));
      const int r = tile * ROWS + nt * 8 + 2 * c + i;
      tok[nt][i] = r < rows ? r / a.G : -1;
    }
  }
  // keys that every query sees: [seen, len)
  const int deepest = a.T - 1;
  const int seen = a.window > 0 ? max(0, len + deepest - a.window + 1) : 0;

  float o[MT][NT][4], nm[NT][2], l[NT][2];  // (nm: the reference's negative)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    nm[nt][0] = nm[nt][1] = INFINITY, l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
  }

  const int kg = (g >> 1) + (g & 1) * 4;  // the key of A row g
  const uint32_t ka = kg * (HD / 2) + c * (HD / 8), kea = 2 * K16::CODES + kg * (HD / 16) + c * (HD / 64);
  const uint32_t va = K16::CODES + c * (HD / 2) + g * (HD / 16);
  const uint32_t vea = 2 * K16::CODES + K16::SCALES + c * (HD / 16) + g * (HD / 8) / 16;
  uint32_t slot = ring;
  for (int s = s0 + warp; s < s1; s += 8) {
    const int j0 = first + s * 16;
    cp_async_wait_group<kRing - 2>();
    __syncwarp();
    float sc[NT][4];
    bool hidden[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[nt][i] = 0.f, hidden[nt][i] = false;
    uint32_t k0[K16::KW], k1[K16::KW], vw[4][K16::VW], ve[4];
    lds_words(k0, slot + ka);
    lds_words(k1, slot + ka + 8 * (HD / 2));
    const uint32_t e0 = e4m3x2_to_f16x2(HD == 128 ? lds_u16(slot + kea) : lds_u8(slot + kea));
    const uint32_t e1 = e4m3x2_to_f16x2(HD == 128 ? lds_u16(slot + kea + 8 * (HD / 16)) : lds_u8(slot + kea + 8 * (HD / 16)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // A rows 2c, 2c + 1, 8 + 2c, 9 + 2c: keys c, 4 + c, 8 + c, 12 + c
      lds_words(vw[i], slot + va + i * 4 * (HD / 2));
      ve[i] = lds_u8(slot + vea + i * 4 * (HD / 16));
      if (j0 < lo || j0 + 16 > n) {  // (rows that no query sees may hold anything, NaN scales too)
        const int j = j0 + i * 4 + c;
        if (j < lo || j >= n) ve[i] = 0;
      }
    }
    fetch();  // (into the slot of the step before: every lane is past it)
    slot = slot == ring + (kRing - 1) * K16::BYTES ? ring : slot + K16::BYTES;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const uint32_t f0 = f16x2_bcast(e0, k >= 4), f1 = f16x2_bcast(e1, k >= 4);
      const uint32_t af[4] = {hmul2(e2m1_byte_to_f16x2(k0[k >> 1], 2 * (k & 1)), f0),
                              hmul2(e2m1_byte_to_f16x2(k1[k >> 1], 2 * (k & 1)), f1),
                              hmul2(e2m1_byte_to_f16x2(k0[k >> 1], 2 * (k & 1) + 1), f0),
                              hmul2(e2m1_byte_to_f16x2(k1[k >> 1], 2 * (k & 1) + 1), f1)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_f16(sc[nt], af, qf[nt][k][0], qf[nt][k][1]);
    }
    // scores in log2 units: A row g, query rows 2c and 2c + 1; A row g + 8, the same
    if (j0 < seen || j0 + 16 > len) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tk = tok[nt][i & 1];
          hidden[nt][i] = !(tk >= 0 && sees(a, tk, j0 + kg + 8 * (i >> 1), len));
        }
    }
    float y[NT][4];  // relative to the reference; a row without one: +inf
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[nt][i] = fmaf(sc[nt][i], fac[nt][i & 1], nm[nt][i & 1]);
        if (hidden[nt][i]) y[nt][i] = -INFINITY;
        raise |= y[nt][i] > kMost;
      }
    if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x0 = hidden[nt][i] ? -INFINITY : sc[nt][i] * fac[nt][i];
          const float x1 = hidden[nt][i + 2] ? -INFINITY : sc[nt][i + 2] * fac[nt][i];
          float mx = fmaxf(x0, x1);
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, k));
          const float ref = fmaxf(-nm[nt][i], mx - kBelow), al = ref == -INFINITY ? 1.f : ex2(-nm[nt][i] - ref);
          nm[nt][i] = -ref;
          l[nt][i] *= al;
#pragma unroll
          for (int k = 0; k < MT; ++k) o[k][nt][i] *= al, o[k][nt][i + 2] *= al;
          y[nt][i] = hidden[nt][i] ? -INFINITY : x0 - ref;
          y[nt][i + 2] = hidden[nt][i + 2] ? -INFINITY : x1 - ref;
        }
    }
    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = ex2(y[nt][i]);
      l[nt][0] += p[0] + p[2], l[nt][1] += p[1] + p[3];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Split w = split_f16x2(p[2 * i], p[2 * i + 1]);
        ph[nt][i] = movmatrix_trans(w.hi), pl[nt][i] = movmatrix_trans(w.lo);
      }
    }
    const uint32_t v0 = e4m3x2_to_f16x2(__byte_perm(ve[0], ve[1], 0x0040)), v1 = e4m3x2_to_f16x2(__byte_perm(ve[2], ve[3], 0x0040));
#pragma unroll
    for (int w = 0; w < K16::VW; ++w) {
      constexpr uint32_t M = 0x0F0F0F0Fu;
      const uint32_t a0 = (vw[0][w] & M) | ((vw[1][w] & M) << 4), a1 = ((vw[0][w] >> 4) & M) | (vw[1][w] & ~M);
      const uint32_t b0 = (vw[2][w] & M) | ((vw[3][w] & M) << 4), b1 = ((vw[2][w] >> 4) & M) | (vw[3][w] & ~M);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t af[4] = {hmul2(e2m1_byte_to_f16x2(a0, k), v0), hmul2(e2m1_byte_to_f16x2(a1, k), v0),
                                hmul2(e2m1_byte_to_f16x2(b0, k), v1), hmul2(e2m1_byte_to_f16x2(b1, k), v1)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(o[w * 4 + k][nt], af, ph[nt][0], ph[nt][1]);
          mma_f16(o[w * 4 + k][nt], af, pl[nt][0], pl[nt][1]);
        }
      }
    }
  }
  grid_dep_launch();
  cp_async_wait_all();
  __syncthreads();  // (the sums take the rings' place)

  // the warps' sums to shared memory
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float s = l[nt][i];
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
      const int r = nt * 8 + 2 * c + i;
      if (g == 0) sml[warp * ROWS + r] = make_float2(-nm[nt][i], s);
#pragma unroll
      for (int k = 0; k < MT; ++k)
        *reinterpret_cast<float2*>(smem + (warp * ROWS + r) * PITCH + g * (HD / 8) + 2 * k) =
            make_float2(o[k][nt][i], o[k][nt][i + 2]);
    }
  __syncthreads();
  // joined, an element a thread; the first warp's place takes the sum
  for (int e = tid; e < ROWS * HD; e += 256) {
    const int r = e / HD, d = e % HD;
    float mm = -INFINITY, sum = 0.f, ll = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) mm = fmaxf(mm, sml[w * ROWS + r].x);
    const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float2 ml = sml[w * ROWS + r];
      const float f = exp2f(ml.x - ref);
      sum += f * smem[(w * ROWS + r) * PITCH + d];
      ll += f * ml.y;
    }
    smem[r * PITCH + d] = sum;  // (this thread's own element)
    if (d == 0) smem[r * PITCH + HD] = mm, smem[r * PITCH + HD + 1] = ll;
  }
  __syncthreads();
  finish_block<HD, ROWS, 256>(a, smem, smem + rows_smem<HD, NT>() / 4, split, h, tile);
}

// ---------------------------------------------------------------------------
// many query rows: the fifth-generation tensor cores
// ---------------------------------------------------------------------------

constexpr int kTcRows = 64;    // query rows of a tile (the MMAs' N)
constexpr int kTcKeys = 128;   // keys of a step (the MMAs' M, and K)
constexpr int kTcTeams = 2;    // teams of eight warps that take the steps in turn
constexpr int kTcWorkers = 8 * kTcTeams;
constexpr int kTcThreads = 32 * (kTcWorkers + kTcTeams);
constexpr int kTcSlots = 2;    // steps that a team has in shared memory
static __device__ uint32_t g_error;  // nonzero once a wait has run out

template <int HD>
struct Tc {
  static constexpr int CODES = kTcKeys * HD / 2;                // bytes of a step's keys (or values)
  static constexpr int Q = kTcRows * HD * 2, V = kTcKeys * HD * 2, P = kTcKeys * kTcRows * 2;
  static constexpr int TEAM = V + 2 * P + kTcSlots * 2 * CODES;  // a team's shared memory (P: the weights' two parts)
  static constexpr int SMEM = 1024 + Q + kTcTeams * TEAM;
  // tensor memory columns: decoded keys, scores, output sums of the weights' two parts
  static constexpr int A0 = 0, S0 = kTcTeams * HD / 2, O0 = S0 + kTcTeams * kTcRows, COLS = 512;
  static_assert(O0 + kTcTeams * 2 * kTcRows <= COLS);
  // at the end the first team's place takes the block's sums, the second one's those
  // that the cluster's blocks push
  static_assert(kTcRows * (HD + 4) * 4 <= TEAM && recv_bytes(kTcRows, HD) <= TEAM && kTcTeams == 2);
};

struct TcBars {
  uint64_t full[kTcTeams][kTcSlots], empty[kTcTeams][kTcSlots];
  uint64_t kready[kTcTeams], sdone[kTcTeams], pready[kTcTeams], pvdone[kTcTeams];
};

struct TcQuery {  // what the block holds of its query rows
  float fac[kTcRows];            // scores in log2 units: times this
  int unseen[kTcRows];           // the last cached key that the row does not see
  uint32_t own[kTcRows];         // which of the tokens' own keys it sees (all, past the last row)
  float nm[kTcTeams][kTcRows];   // the references' negatives (+inf: none yet)
  float al[kTcTeams][kTcRows];   // factors of a rescaling
};

struct Kv4AttnTc {
  CUtensorMap map;  // [2 Hkv][max_seq][HD / 2] bytes, boxes of 1 x 128 x HD / 2
  Kv4Attn a;
};

// OR of a truth value over four warps (a barrier of their 128 threads).
__device__ __forceinline__ bool half_any(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void sts128(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Row of 16-byte pieces with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t piece) { return row * 128 + (((piece ^ row) & 7) << 4); }

// N values a lane (32 or 16), combined over the lanes: lane i gets value i mod
// N's result.
template <int N, typename F>
__device__ __forceinline__ float spread(float (&z)[N], int lane, F f) {
  if (N == 16) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = f(z[i], __shfl_xor_sync(0xFFFFFFFFu, z[i], 16));
  }
#pragma unroll
  for (int w = N / 2; w > 0; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float give = up ? z[i] : z[i + w], keep = up ? z[i + w] : z[i];
      z[i] = f(keep, __shfl_xor_sync(0xFFFFFFFFu, give, w));
    }
  }
  return z[0];
}

// 32 N elements decoded to fp16: N 16-byte pieces of codes, two block scales
// each.
template <int N>
__device__ __forceinline__ void decode_codes(uint32_t (&v)[32], const uint4 (&c)[2], uint32_t e) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t f = f16x2_bcast(e4m3_pair_to_f16x2(e, i), b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i * 16 + b * 8 + j] = hmul2(e2m1_byte_to_f16x2(w[2 * b + (j >> 2)], j & 3), f);
    }
  }
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t at, float (&v)[N]) {
  if constexpr (N == 32) tmem_ld32(at, v);
  else tmem_ld16(at, v);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&v)[N]) {
  if constexpr (N == 32) tmem_st32(at, v);
  else tmem_st16(at, v);
}

// Up to 64 query rows of a kv head at once: S^T = K Q^T (M = 128 keys, N = 64
// rows, K = HD) and O^T = V^T P^T (M = HD, N = 64, K = 128 keys), fp16 operands,
// fp32 accumulators in tensor memory.
//
// Two teams of eight warps take steps of 128 keys in turn, two threads for a
// key: each decodes half of the key's dimensions into the A operand in tensor
// memory (exactly) and half of the value's into shared memory while the scores
// are computed, then takes its half of the query rows: the key's scores, turned
// into weights and written as the B operand.  Each team has a softmax of its own
// (references, sums, output sums); the two are joined at the end.  A warp for
// each team issues its MMAs and copies.  The reference of a row is raised when a
// score passes it by 2^8, and the sums rescaled: a few times in all.  On mma.sync
// 64 rows cost four times the decoding or do not fit the registers: 53 us for
// 16 tokens over 32768 keys of 8 kv heads, here 28.0 (131072 keys: 77.3).  Bound
// by the chain of a step (decoding, scores, softmax, weights, each through
// tensor memory; 2.4 us) with two teams: issue slots 50%, tensor pipe 30% in
// use.  A third team has no room in tensor memory and registers.
//
// The weights' two parts (see Split) lie side by side as the N of one MMA, columns r
// and NR + r of the sums, which are added at the end (one MMA after the other, V read
// twice: 30.0 us for 28.0).  The second part costs 2.8 us of the 28.0.
//
// NR: rows of the 64 that are in use, 32 or 64 (the softmax skips the rest: 32
// rows, 32768 keys 22.0 us, as 64 26.8).
template <int HD, int NR>
__global__ void __launch_bounds__(kTcThreads, 1) kv4_tc_kernel(const __grid_constant__ Kv4AttnTc args) {
  using L = Tc<HD>;
  constexpr int PITCH = HD + 4, PIECES = HD / 32;  // 16-byte pieces of a row's codes
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ TcBars bars;
  __shared__ __align__(16) TcQuery query;
  __shared__ float wmax[kTcTeams][4][kTcRows];            // a warp's maxima; its sums at the end
  __shared__ float jf[kTcTeams][kTcRows];                 // a team's share when the two are joined
  __shared__ uint32_t tmem_base;
  __shared__ int abort, never;
  const Kv4Attn& a = args.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x, h = blockIdx.y, tile = blockIdx.z;
  grid_dep_wait();
  const int len = cached_len(a), rows = a.T * a.G;
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  auto bar = [](uint64_t& b) { return smem_u32(&b); };

  // this block's keys: steps of 128
  const int n = len + a.T;
  const int lo = a.window > 0 ? max(0, len - a.window + 1) : 0;  // (no query sees a key before lo)
  const int steps = (n - lo + kTcKeys - 1) / kTcKeys;
  const int per = (steps + (int)gridDim.x - 1) / (int)gridDim.x;
  const int s0 = min(steps, split * per), s1 = min(steps, s0 + per);
  const int seen = a.window > 0 ? max(0, len + a.T - a.window) : 0;  // keys that every query sees: [seen, len)
  const uint64_t deadline = gtimer() + kOpsWaitNs + (uint64_t)(s1 - s0) * kOpsStepNs;

  if (tid < kTcRows) {
    const int row = tile * kTcRows + tid;
    const int t = row < rows ? row / a.G : -1;
    query.unseen[tid] = t >= 0 && a.window > 0 ? len + a.depth[t] - a.window : -1;
    query.own[tid] = t >= 0 ? a.vis[t] : ~0u;
    for (int i = 0; i < kTcTeams; ++i) query.nm[i][tid] = t >= 0 ? INFINITY : 0.f;
  }
  const int team = warp < kTcWorkers ? warp >> 3 : warp - kTcWorkers;
  const int mine = max(0, (s1 - s0 - team + kTcTeams - 1) / kTcTeams);  // this team's steps
  uint8_t* tsm = smem + L::Q + team * L::TEAM;
  const uint32_t vbuf = smem_u32(tsm), pbuf = vbuf + L::V, raw = pbuf + 2 * L::P;
  auto load = [&](int it) {  // a step's keys and values
    const int slot = it % kTcSlots, j0 = lo + (s0 + team + it * kTcTeams) * kTcKeys;
    const uint32_t b = bar(bars.full[team][slot]), dst = raw + slot * 2 * L::CODES;
    mbar_arrive_expect_tx(b, 2 * L::CODES);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile(
          "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
              dst + i * L::CODES),
          "l"(&args.map), "r"(0), "r"(j0), "r"(i * a.Hkv + h), "r"(b)
          : "memory");
  };
  const bool issuer = warp >= kTcWorkers && lane == 0;

  // everything from memory that the first step needs is under way before the
  // block's set-up: the keys and values, their scales, the queries
  if (issuer) {
    prefetch_tensormap(&args.map);
    for (int i = 0; i < kTcSlots; ++i) mbar_init(bar(bars.full[team][i]), 1), mbar_init(bar(bars.empty[team][i]), 8);
    mbar_init(bar(bars.kready[team]), 8), mbar_init(bar(bars.sdone[team]), 1);
    mbar_init(bar(bars.pready[team]), 8), mbar_init(bar(bars.pvdone[team]), 1);
    mbar_fence_init();
    fence_proxy_async_shared();
    for (int it = 0; it < min(mine, kTcSlots); ++it) load(it);
  }
  const int quad = warp & 3, half = (warp >> 2) & 1, r = quad * 32 + lane;  // (workers) r: the thread's key of a step
  // block scales of this thread's key and value, a step ahead
  const uint8_t* es = a.scales + (long long)h * a.max_seq * (HD / 16) + half * (HD / 32);
  const long long vs = (long long)a.Hkv * a.max_seq * (HD / 16);
  uint32_t ek = 0, ev = 0;
  auto scales = [&](int it) {
    const int j = lo + (s0 + team + it * kTcTeams) * kTcKeys + r;
    ek = ev = 0;  // (rows past the last one may hold anything, NaN scales too)
    if (it < mine && j < n) {
      const uint8_t* p = es + (long long)j * (HD / 16);
      if (HD == 128) {
        ek = __ldg(reinterpret_cast<const uint32_t*>(p));
        ev = __ldg(reinterpret_cast<const uint32_t*>(p + vs));
      } else {
        ek = __ldg(reinterpret_cast<const uint16_t*>(p));
        ev = __ldg(reinterpret_cast<const uint16_t*>(p + vs));
      }
    }
  };
  constexpr int RP = HD / 8, QN = kTcRows * RP / (32 * kTcWorkers);  // 16-byte pieces of a query row, a lane for each
  uint4 qv[QN];
  if (warp < kTcWorkers) {
    scales(0);
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int e = tid + i * 32 * kTcWorkers, row = tile * kTcRows + e / RP;
      qv[i] = make_uint4(0, 0, 0, 0);
      if (row < rows)
        qv[i] = *reinterpret_cast<const uint4*>(a.q + (row / a.G) * a.q_stride + (long long)(h * a.G + row % a.G) * HD + e % RP * 8);
    }
  }
  if (tid == 0) abort = 0, never = 0;
  if (warp == 0) tmem_alloc(smem_u32(&tmem_base), L::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const volatile int* ab = &abort;
  auto wait = [&](uint64_t& b, uint32_t parity) {
    if (mbar_wait(bar(b), parity, deadline, ab)) return true;
    abort = 1;
    return false;
  };
  auto wait_warp = [&](uint64_t& b, uint32_t parity) { return (bool)__all_sync(0xFFFFFFFFu, wait(b, parity)); };

  if (warp < kTcWorkers) {
    // Q as the B operand: fp16 after a scaling of each row by a power of two
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int e = tid + i * 32 * kTcWorkers, r = e / RP, piece = e % RP;
      uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
      float most = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack16(w[j], a.fp16);
        most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
#pragma unroll
      for (int k = 1; k < RP; k <<= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, k));
      const int sh = row_shift(most);
      const float mul = exp2i(sh);
      if (piece == 0) query.fac[r] = a.qk_scale * exp2i(-sh);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack16(w[j], a.fp16);
        w[j] = pack_f16x2(f.x * mul, f.y * mul);
      }
      *reinterpret_cast<uint4*>(smem + (piece >> 3) * (kTcRows * 128) + swz(r, piece & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_shared();
  }
  __syncthreads();

  if (warp < kTcWorkers) {
    constexpr int RW = NR / 2, CP = PIECES / 2;  // query rows, pieces of codes of a thread
    const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t tk = tl + L::A0 + team * HD / 2 + half * HD / 4, ts = tl + L::S0 + team * kTcRows + half * RW;
    const uint32_t to = tl + L::O0 + team * 2 * kTcRows + half * RW;
    const int id = 1 + 2 * team + half;  // the barrier of the four warps with the same rows
    // this thread's rows; its team's references lie 3 arrays on, their factors 2 more
    float* hq = query.fac + half * RW;
    const float* hfac = hq;
    float *hnm = hq + (3 + team) * kTcRows, *hal = hnm + 2 * kTcRows;
    static_assert(offsetof(TcQuery, nm) == 3 * kTcRows * 4 && kTcTeams == 2);
    float l[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) l[i] = 0.f;
    // (a wait that runs out sets `abort`, after which no wait waits: the warps
    // still come to each of the team's barriers)
    for (int it = 0; it < mine; ++it) {
      const int slot = it % kTcSlots, j0 = lo + (s0 + team + it * kTcTeams) * kTcKeys;
      wait_warp(bars.full[team][slot], (it / kTcSlots) & 1);
      const uint32_t kc = raw + slot * 2 * L::CODES + r * (HD / 2), vc = kc + L::CODES;
      // (the copies' swizzle: piece p of row r lies at p ^ (r / 2 mod 4), of 32-byte rows at p ^ (r / 4 mod 2))
      const uint32_t x = HD == 128 ? (r >> 1) & 3 : (r >> 2) & 1;
      uint4 c[2];
      uint32_t v[32];
#pragma unroll
      for (int i = 0; i < CP; ++i) c[i] = lds128(kc + (((half * CP + i) ^ x) << 4));
      decode_codes<CP>(v, c, ek);
      if (HD == 128) tmem_st32(tk, v);
      else tmem_st16(tk, reinterpret_cast<const uint32_t(&)[16]>(v));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.kready[team]));
      // the value, while the scores are computed
#pragma unroll
      for (int i = 0; i < CP; ++i) c[i] = lds128(vc + (((half * CP + i) ^ x) << 4));
      decode_codes<CP>(v, c, ev);
      if (it > 0) wait_warp(bars.pvdone[team], (it - 1) & 1);
#pragma unroll
      for (int q = 0; q < 4 * CP; ++q) {  // 8 dimensions
        const int piece = half * 4 * CP + q;
        sts128(vbuf + (piece >> 3) * (kTcKeys * 128) + swz(r, piece & 7),
               make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.empty[team][slot]));
      scales(it + 1);
      wait_warp(bars.sdone[team], it & 1);
      tc_fence_after();
      const bool edge = j0 < seen || j0 + kTcKeys > len;
      float y[RW];  // the scores of this key
      auto mask = [&]() {
        const int j = j0 + r, bit = min(j - len, 31);  // (a real row sees none of the keys past its own)
#pragma unroll
        for (int i = 0; i < RW; i += 4) {
          if (j < len) {
            const int4 u = *reinterpret_cast<const int4*>(hq + kTcRows + i);
            y[i] = j > u.x ? y[i] : -INFINITY, y[i + 1] = j > u.y ? y[i + 1] : -INFINITY;
            y[i + 2] = j > u.z ? y[i + 2] : -INFINITY, y[i + 3] = j > u.w ? y[i + 3] : -INFINITY;
          } else {
            const uint4 u = *reinterpret_cast<const uint4*>(hq + 2 * kTcRows + i);
            y[i] = u.x >> bit & 1 ? y[i] : -INFINITY, y[i + 1] = u.y >> bit & 1 ? y[i + 1] : -INFINITY;
            y[i + 2] = u.z >> bit & 1 ? y[i + 2] : -INFINITY, y[i + 3] = u.w >> bit & 1 ? y[i + 3] : -INFINITY;
          }
        }
      };
      auto scores = [&]() {  // in log2 units, relative to the references
        tmem_ld<RW>(ts, y);
#pragma unroll
        for (int i = 0; i < RW; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(hfac + i), m = *reinterpret_cast<const float4*>(hnm + i);
          y[i] = fmaf(y[i], f.x, m.x), y[i + 1] = fmaf(y[i + 1], f.y, m.y);
          y[i + 2] = fmaf(y[i + 2], f.z, m.z), y[i + 3] = fmaf(y[i + 3], f.w, m.w);
        }
        if (edge) mask();
      };
      bool raise = it == 0;
      if (!raise) {
        scores();
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < RW; ++i) most = fmaxf(most, y[i]);
        raise = half_any(id, most > kMost);
      }
      if (raise) {
        // raise the references: the rows' maxima over the step's keys, lane i
        // ending with row i's
        tmem_ld<RW>(ts, y);
#pragma unroll
        for (int i = 0; i < RW; ++i) y[i] *= hfac[i];
        if (edge) mask();
        const float zm = spread(y, lane, [](float u, float w) { return fmaxf(u, w); });
        if (lane < RW) wmax[team][quad][half * RW + lane] = zm;
        named_bar(id, 128);
        if (r < RW) {
          const int row = half * RW + r;
          const float old = -hnm[r];
          const float mx =
              fmaxf(fmaxf(wmax[team][0][row], wmax[team][1][row]), fmaxf(wmax[team][2][row], wmax[team][3][row]));
          const float ref = tile * kTcRows + row < rows ? fmaxf(old, mx - kBelow) : old;
          hal[r] = ref == -INFINITY ? 1.f : ex2(old - ref);
          hnm[r] = -ref;
        }
        named_bar(id, 128);
        if (it > 0) {  // (the last step's output sums are complete: pvdone was waited for)
#pragma unroll
          for (int i = 0; i < RW; ++i) l[i] *= hal[i];
#pragma unroll 1
          for (int p = 0; p < RW / 8; ++p) {  // 16 rows of each part at a time
            const int row = p % (RW / 16) * 16;
            const uint32_t at = to + p / (RW / 16) * NR + row;
            float z[16];
            uint32_t w[16];
            tmem_ld16(at, z);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(z[i] * hal[row + i]);
            tmem_st16(at, w);
          }
        }
        // (a row still without a reference sees none of these keys; the maxima
        // and factors are written again after another barrier of these warps)
        scores();
      }
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        y[i] = ex2(y[i]);
        l[i] += y[i];
      }
#pragma unroll
      for (int i = 0; i < RW / 8; ++i) {
        Split w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = split_f16x2(y[8 * i + 2 * j], y[8 * i + 2 * j + 1]);
        const uint32_t piece = half * (RW / 8) + i;
        sts128(pbuf + swz(r, piece), make_uint4(w[0].hi, w[1].hi, w[2].hi, w[3].hi));
        sts128(NR == kTcRows ? pbuf + L::P + swz(r, piece) : pbuf + swz(r, 4 + piece), make_uint4(w[0].lo, w[1].lo, w[2].lo, w[3].lo));
      }
      fence_proxy_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.pready[team]));
    }
    if (mine > 0) wait_warp(bars.pvdone[team], (mine - 1) & 1);
    tc_fence_after();
    // weights summed over the team's keys: lane i ends with its warp's sum for row i
    const float ls = spread(l, lane, [](float u, float w) { return u + w; });
    if (lane < RW) wmax[team][quad][half * RW + lane] = ls;
  } else if (issuer) {
    // --- a team's MMAs and copies -------------------------------------------
    constexpr uint32_t idesc_s = (1u << 4) | ((kTcRows / 8u) << 17) | ((128u / 16) << 24);
    // A and B with M and N contiguous, N = the weights' two parts
    constexpr uint32_t idesc_o = (1u << 4) | (2 * NR / 8u << 17) | ((128u / 16) << 24) | (1u << 15) | (1u << 16);
    const uint32_t tk = tmem + L::A0 + team * HD / 2, ts = tmem + L::S0 + team * kTcRows, to = tmem + L::O0 + team * 2 * kTcRows;
    const uint64_t qd = umma_desc(smem_u32(smem), 16, 1024) | kSwizzle128;
    // V: blocks of 64 dimensions 16 KB apart (64 dimensions in all: the second one is the first again)
    const uint64_t vd = umma_desc(vbuf, HD == 128 ? kTcKeys * 128 : 0, 1024) | kSwizzle128;
    const uint64_t pd = umma_desc(pbuf, L::P, 1024) | kSwizzle128;  // (64 columns, then the next 64)
    bool ok = true;
    for (int it = 0; it < mine; ++it) {
      ok = wait(bars.kready[team], it & 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < HD / 16; ++k)
        mma_f16_ts(ts, tk + k * 8, qd + (k >> 2) * (kTcRows * 128 >> 4) + (k & 3) * 2, idesc_s, k > 0);
      tc_commit(bar(bars.sdone[team]));
      if (it + kTcSlots < mine) {
        ok = wait(bars.empty[team][it % kTcSlots], (it / kTcSlots) & 1);
        if (!ok) break;
        load(it + kTcSlots);
      }
      ok = wait(bars.pready[team], it & 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < kTcKeys / 16; ++k)
        mma_f16_ss(to, vd + k * (2048 >> 4), pd + k * (2048 >> 4), idesc_o, it > 0 || k > 0);
      tc_commit(bar(bars.pvdone[team]));
    }
    if (!ok) {  // what is in flight ends before the block does
      for (int i = 0; i < kTcSlots; ++i)
        for (uint32_t q = 0; q < 2; ++q) mbar_wait(bar(bars.full[team][i]), q, gtimer() + kOpsWaitNs / 100, &never);
      for (uint32_t q = 0; q < 2; ++q) {
        mbar_wait(bar(bars.sdone[team]), q, gtimer() + kOpsWaitNs / 100, &never);
        mbar_wait(bar(bars.pvdone[team]), q, gtimer() + kOpsWaitNs / 100, &never);
      }
    }
  }
  grid_dep_launch();
  __syncwarp();
  __syncthreads();
  if (a.cluster > 1) cluster_arrive();  // (the operands' places are free)
  tc_fence_after();

  // the teams joined: smem[row][PITCH] (over the first team's operands)
  float* out = reinterpret_cast<float*>(smem + L::Q);
  const bool one = s0 < s1, two = s0 + 1 < s1;  // teams that had steps
  if (tid < NR) {
    const float m0 = one ? -query.nm[0][tid] : -INFINITY, m1 = two ? -query.nm[1][tid] : -INFINITY, mm = fmaxf(m0, m1);
    const float ref = mm == -INFINITY ? 0.f : mm, f0 = ex2(m0 - ref), f1 = ex2(m1 - ref);
    jf[0][tid] = f0, jf[1][tid] = f1;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) s += (one ? f0 * wmax[0][w][tid] : 0.f) + (two ? f1 * wmax[1][w][tid] : 0.f);
    out[tid * PITCH + HD] = mm, out[tid * PITCH + HD + 1] = s;
  }
  __syncthreads();
  if (warp < 4 * (NR / 16)) {  // 16 rows a warp
    const int quad = warp & 3, d = quad * 32 + lane, q = (warp >> 2) * 16;
    const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
    float z[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
#pragma unroll
    for (int t = 0; t < kTcTeams; ++t)
      if (t == 0 ? one : two) {
        const uint32_t at = tl + L::O0 + t * 2 * kTcRows + q;
        float y[16];
        tmem_ld16(at, y);
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] += jf[t][q + i] * y[i];
        tmem_ld16(at + NR, y);
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] += jf[t][q + i] * y[i];
      }
    if (HD == 128 || d < HD) {
#pragma unroll
      for (int i = 0; i < 16; ++i) out[(q + i) * PITCH + d] = z[i];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_relinquish();
    tmem_dealloc(tmem, L::COLS);
  }
  if (tid == 0 && abort) atomicExch(&g_error, 1u);
  finish_block<HD, kTcRows, kTcThreads>(a, out, reinterpret_cast<float*>(smem + L::Q + L::TEAM), split, h, tile);
}

// The key ranges of a (token, query head): a block of four groups of HD
// threads.  A group takes every fourth range, all that it needs of N of them at
// once (their references too: nothing waits for a maximum over all), and the
// groups meet in shared memory.
template <int HD, int N>
__global__ void __launch_bounds__(4 * HD, N > 8 ? 1 : 4) kv4_combine_kernel(const __grid_constant__ Kv4Attn a, int tile_rows) {
  __shared__ float part[4][HD], pm[4], pl[4];
  const int row = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, d = tid % HD, q = tid / HD;
  const long long base = ((long long)(row / tile_rows) * a.Hkv + h) * a.splits * tile_rows + row % tile_rows;
  float mm = -INFINITY, l = 0.f, sum = 0.f;
  grid_dep_wait();
  grid_dep_launch();
  for (int s0 = q; s0 < a.splits; s0 += 4 * N) {
    float o[N];
    float2 ml[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int s = s0 + 4 * i;
      o[i] = 0.f, ml[i] = make_float2(-INFINITY, 0.f);
      if (s < a.splits) {
        ml[i] = a.ml_part[base + (long long)s * tile_rows];
        o[i] = a.o_part[(base + (long long)s * tile_rows) * HD + d];
      }
    }
    float m = mm;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, ml[i].x);
    const float ref = m == -INFINITY ? 0.f : m, f = ex2(mm - ref);
    mm = m, l *= f, sum *= f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float g = ex2(ml[i].x - ref);  // (a range without a visible key: 0)
      l += g * ml[i].y, sum += g * o[i];
    }
  }
  part[q][d] = sum;
  if (d == 0) pm[q] = mm, pl[q] = l;
  __syncthreads();
  if (q == 0) {
    const float m = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
    float total = 0.f, y = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = ex2(pm[i] - m);
      total += f * pl[i], y += f * part[i][d];
    }
    store_out(a, HD, h, row, d, y / total * a.v_scale);
  }
}

// How a call is laid out.  `keys`: the most keys that a head may have to read.
struct Kv4Plan {
  int tile_rows, tiles, cluster, splits;
};
Kv4Plan plan_attention(int tokens, int group, int Hkv, int keys) {
  Kv4Plan p{};
  const int rows = tokens * group;
  // (16 rows, 16384 keys of 8 kv heads: 13.8 us in a tile of 16, 14.7 in one of 64)
  p.tile_rows = rows <= 8 ? 8 : rows <= 16 ? 16 : kTcRows;
  p.tiles = (rows + p.tile_rows - 1) / p.tile_rows;
  p.cluster = p.splits = 1;
  if (keys <= cluster_keys(rows)) {
    // a block for every 128 keys (16 a warp), or 256 (a step for each team)
    const int block = p.tile_rows == kTcRows ? kTcTeams * kTcKeys : 128;
    // (a window of 2048 and the tokens' own keys: 9 blocks, not 8 of which some
    // have a step more)
    p.cluster = std::max(1, std::min(kMaxCluster, (keys + block - 1) / block));
  } else {
    const int per_sm = p.tile_rows == 8 ? 2 : 1;  // blocks that an SM holds
    // up to 64 ranges; more only of 1024 keys each (1 row, 131071 keys, one kv
    // head: 128 ranges 12.2 us, 64 15.4; 65536 keys, two: 13.2 and 11.3)
    const int most = std::min(kMaxSplits, std::max(64, keys / 1024));
    p.splits = std::max(2, std::min(most, per_sm * kOpsSms / (p.tiles * Hkv)));
  }
  return p;
}
size_t plan_bytes(const Kv4Plan& p, int Hkv, int hd) {
  return p.splits == 1 ? 0 : (size_t)p.tiles * Hkv * p.splits * p.tile_rows * (hd + 2) * 4;
}
int most_keys(int tokens, int window, int len) {
  const long long keys = std::min<long long>(len, window > 0 ? (long long)window + tokens : len) + tokens;
  return (int)std::min<long long>(keys, kMaxRows);
}

// A kernel over (key ranges, kv heads, row tiles), its shared-memory limit set
// once a device (`ready`; by two threads at once does no harm).
template <typename Args>
cudaError_t launch_blocks(void (*kernel)(Args), const Args& args, std::atomic<bool> (&ready)[64], int threads, int smem,
                          const Kv4Plan& p, int Hkv, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  const OpsLaunch l(dim3((unsigned)(p.cluster * p.splits), (unsigned)Hkv, (unsigned)p.tiles), threads, smem, st, p.cluster);
  return cudaLaunchKernelEx(&l.cfg, kernel, args);
}

template <int HD, int NT>
cudaError_t launch_rows_kernel(const Kv4Attn& a, const Kv4Plan& p, cudaStream_t st) {
  static std::atomic<bool> ready[64] = {};
  constexpr int smem = rows_smem<HD, NT>() + recv_bytes(8 * NT, HD);
  return launch_blocks(kv4_rows_kernel<HD, NT>, a, ready, 256, smem, p, a.Hkv, st);
}

template <int HD, int NR>
cudaError_t launch_tc_kernel(const Kv4Attn& a, const Kv4Plan& p, cudaStream_t st) {
  static std::atomic<bool> ready[64] = {};
  Kv4AttnTc t{};
  t.a = a;
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  const cuuint64_t dims[3] = {HD / 2, (cuuint64_t)a.max_seq, 2ull * a.Hkv}, pitch[2] = {HD / 2, (cuuint64_t)a.max_seq * (HD / 2)};
  const cuuint32_t box[3] = {HD / 2, kTcKeys, 1}, es[3] = {1, 1, 1};
  if (enc == nullptr ||
      enc(&t.map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(a.codes), dims, pitch, box, es,
          CU_TENSOR_MAP_INTERLEAVE_NONE, HD == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return launch_blocks(kv4_tc_kernel<HD, NR>, t, ready, kTcThreads, Tc<HD>::SMEM, p, a.Hkv, st);
}

template <int HD>
cudaError_t launch_attention(const Kv4Attn& a, const Kv4Plan& p, cudaStream_t st) {
  cudaError_t e = p.tile_rows == 8            ? launch_rows_kernel<HD, 1>(a, p, st)
                  : p.tile_rows == 16         ? launch_rows_kernel<HD, 2>(a, p, st)
                  : a.T * a.G <= kTcRows / 2  ? launch_tc_kernel<HD, 32>(a, p, st)
                                              : launch_tc_kernel<HD, 64>(a, p, st);
  if (e != cudaSuccess || p.splits == 1) return e;
  const OpsLaunch l(dim3((unsigned)(a.T * a.G), (unsigned)a.Hkv), 4 * HD, 0, st);
  // many blocks: few registers, so that all run at once (16 tokens x 32 heads, 19
  // ranges: 25.7 us in all, with 16 at once a group 30.7; one token, 38 ranges: 35.4
  // and 35.1)
  return a.T * a.Hq > kOpsSms ? cudaLaunchKernelEx(&l.cfg, kv4_combine_kernel<HD, 5>, a, p.tile_rows)
                              : cudaLaunchKernelEx(&l.cfg, kv4_combine_kernel<HD, 16>, a, p.tile_rows);
}

}  // namespace

cudaError_t kv4_error(uint32_t* e) {
  cudaError_t r = cudaMemcpyFromSymbol(e, g_error, sizeof(*e));
  const uint32_t zero = 0;
  if (r == cudaSuccess && *e != 0) r = cudaMemcpyToSymbol(g_error, &zero, sizeof(zero));
  return r;
}

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

extern "C" size_t msk_attention_kv4_workspace(int32_t tokens, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                              int32_t window, int32_t cache_len) {
  if (tokens <= 0 || tokens > kMaxT || n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads || head_dim <= 0 ||
      window < 0 || cache_len < 0)
    return 0;
  return plan_bytes(plan_attention(tokens, n_q_heads / n_kv_heads, n_kv_heads, most_keys(tokens, window, cache_len)),
                    n_kv_heads, head_dim);
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
  const int G = n_q_heads / cache->n_kv_heads;
  if (cache->n_kv_heads > 65535 || G > 32768) return MSK_ERR_SHAPE;  // (grid limits)
  if (window < 0 || tokens > cache->max_seq) return MSK_ERR_INVALID_ARG;
  if (cache_len_dev == nullptr && (cache_len < 0 || cache_len > cache->max_seq - tokens)) return MSK_ERR_INVALID_ARG;
  if (!(softmax_scale >= 0.f && softmax_scale <= 3e38f)) return MSK_ERR_INVALID_ARG;
  const float scale = softmax_scale > 0.f ? softmax_scale : (float)(1.0 / std::sqrt((double)cache->head_dim));
  const float qk_scale = scale * cache->k_scale * 1.4426950408889634f;
  if (!std::isfinite(qk_scale)) return MSK_ERR_INVALID_ARG;  // (every score would be a NaN)
  if (q_stride < (int64_t)n_q_heads * cache->head_dim && tokens > 1) return MSK_ERR_INVALID_ARG;
  if (!ops_aligned16(q) || !ops_aligned16(out) || !ops_aligned16(workspace) || q_stride % 8) return MSK_ERR_ALIGNMENT;
  Kv4Attn a{};
  if (!tree_masks(parents, tokens, window, a.depth, a.vis)) return MSK_ERR_INVALID_ARG;
  // (a cache of few rows is laid out by its size, whatever its length now, and so is
  // any where the length is read on the device: 4 rows x 128 keys in a cache of 20000 7.5
  // us, of a length known here 4.6, 4000 8.5 and 6.6; 64 rows 11.7 and 10.4, 12.6 and 12.5)
  int keys = most_keys(tokens, window, cache->max_seq - tokens);
  if (cache_len_dev == nullptr && keys > cluster_keys(tokens * G)) keys = most_keys(tokens, window, cache_len);
  const Kv4Plan plan = plan_attention(tokens, G, cache->n_kv_heads, keys);
  const size_t need = plan_bytes(plan, cache->n_kv_heads, cache->head_dim);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MSK_ERR_INVALID_ARG;
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
  a.splits = plan.splits, a.cluster = plan.cluster;
  a.fp16 = dtype == MSK_FP16;
  a.qk_scale = qk_scale;
  a.v_scale = cache->v_scale;
  const size_t parts = (size_t)plan.tiles * a.Hkv * a.splits * plan.tile_rows;
  a.o_part = static_cast<float*>(workspace);
  a.ml_part = reinterpret_cast<float2*>(a.o_part + parts * cache->head_dim);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->head_dim == 128 ? launch_attention<128>(a, plan, st) : launch_attention<64>(a, plan, st);
  return e == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}
