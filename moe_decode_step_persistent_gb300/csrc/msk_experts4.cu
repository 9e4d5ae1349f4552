// 4-bit matrices: rows quantised and read back, and products of quantised rows,
// sorted by expert, with each expert's 4-bit weights.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "msk_internal.h"
#include "msk_ops.cuh"
#include "msk_quant.cuh"
#include "msk_tc.cuh"

namespace msk {
namespace {

// ---------------------------------------------------------------------------
// rows in and out
// ---------------------------------------------------------------------------

struct Rows4 {
  const void* x;
  uint8_t* codes;
  uint8_t* scales;
  long long n, x_stride;  // pieces in all
  int pieces;             // of a row; 0 where rows lie one behind the other
  float ts;
};

// Where piece i of E elements begins in x, in elements.
template <int E>
__device__ __forceinline__ long long piece_at(const Rows4& a, long long i) {
  if (a.pieces == 0) return i * E;
  // (a division of 64 bits is some 40 instructions)
  const long long r = a.n <= 0xFFFFFFFFll ? (long long)((uint32_t)i / (uint32_t)a.pieces) : i / a.pieces;
  return r * a.x_stride + (i - r * a.pieces) * E;
}

// A block of 16 elements a thread, as in the 4-bit cache's writer.  WIDE: rows of
// 16-bit elements are aligned to 32 bytes, one load's.
template <int DT, bool WIDE>
__global__ void __launch_bounds__(256) quantize_kernel(const Rows4 a) {
  grid_dep_wait();
  grid_dep_launch();
  const long long step = (long long)gridDim.x * 256;
  long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (WIDE) {
    // (the next block's elements are on their way while one is quantised)
    uint32_t w[8];
    if (i < a.n) ldg256(static_cast<const uint16_t*>(a.x) + piece_at<16>(a, i), w);
    for (; i < a.n; i += step) {
      float x[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = unpack16(w[j], DT == MSK_FP16);
        x[2 * j] = f.x, x[2 * j + 1] = f.y;
      }
      if (i + step < a.n) ldg256(static_cast<const uint16_t*>(a.x) + piece_at<16>(a, i + step), w);
      uint32_t sc;
      const uint2 c = quantise16(x, a.ts, sc);
      *reinterpret_cast<uint2*>(a.codes + i * 8) = c;
      a.scales[i] = (uint8_t)sc;
    }
    return;
  }
  if (i >= a.n) return;
  float x[16];
  load16<DT>(a.x, piece_at<16>(a, i), x);
  uint32_t sc;
  const uint2 c = quantise16(x, a.ts, sc);
  *reinterpret_cast<uint2*>(a.codes + i * 8) = c;
  a.scales[i] = (uint8_t)sc;
}

// 16 bytes of the row a thread and step, four steps, all loaded first.
constexpr int kReadUnroll = 4;
template <int DT>
__global__ void __launch_bounds__(256) dequantize_kernel(const Rows4 a) {
  constexpr int E = DT == MSK_FP32 ? 4 : 8, U = kReadUnroll;
  using Codes = std::conditional_t<E == 4, uint16_t, uint32_t>;
  grid_dep_wait();
  grid_dep_launch();
  const long long i0 = (long long)blockIdx.x * (256 * U) + threadIdx.x, n = a.n;
  uint32_t c[U], e[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const long long i = i0 + k * 256;
    if (i < n) {
      c[k] = __ldg(reinterpret_cast<const Codes*>(a.codes) + i);
      e[k] = __ldg(a.scales + i / (16 / E));
    }
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const long long i = i0 + k * 256;
    if (i >= n) break;
    const float dec = e4m3_to_f32(e[k]);
    float x[E];
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const float2 f = unpack_f16x2(e2m1_byte_to_f16x2(c[k], j));
      x[2 * j] = f.x * dec * a.ts, x[2 * j + 1] = f.y * dec * a.ts;
    }
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = DT == MSK_FP32 ? __float_as_uint(x[j]) : pack16(x[2 * j % E], x[(2 * j + 1) % E], DT == MSK_FP16);
    const long long off = piece_at<E>(a, i);
    *reinterpret_cast<uint4*>(static_cast<char*>(const_cast<void*>(a.x)) + off * (16 / E)) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

msk_status rows_call(bool write, const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride, float ts,
                     const uint8_t* codes, const uint8_t* scales, void* stream) {
  if (!dtype_ok(dtype) || rows < 0) return MSK_ERR_INVALID_ARG;
  if (cols <= 0 || cols % 16 || cols > (1ll << 24) || rows > (1ll << 31) - 1 || rows * cols > (1ll << 38)) return MSK_ERR_SHAPE;
  if (!(ts > 0.f && ts <= 3e38f)) return MSK_ERR_INVALID_ARG;  // (also false for NaN)
  if (rows == 0) return MSK_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr) return MSK_ERR_INVALID_ARG;
  // (rows that are read may be one and the same, those that are written may not overlap)
  if (rows > 1 && (stride < 0 || (!write && stride < cols))) return MSK_ERR_INVALID_ARG;
  if (!ops_aligned16(x) || (rows > 1 && stride % (16 / dtype_bytes(dtype))) || !ops_aligned16(codes) || !ops_aligned16(scales))
    return MSK_ERR_ALIGNMENT;
  int nsm = 0;
  const msk_status s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  Rows4 a{};
  a.x = x, a.codes = const_cast<uint8_t*>(codes), a.scales = const_cast<uint8_t*>(scales);
  const int piece = write ? 16 : dtype == MSK_FP32 ? 4 : 8, per = write ? 256 : 256 * kReadUnroll;
  a.n = rows * (cols / piece), a.x_stride = rows > 1 ? stride : 0, a.ts = ts;
  a.pieces = rows == 1 || stride == cols ? 0 : (int)(cols / piece);
  const bool wide = write && dtype != MSK_FP32 && ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)(a.x_stride * 2)) & 31) == 0;
  // (wide: as many blocks as run at once, each going on)
  const long long blocks = (a.n + per - 1) / per;
  const OpsLaunch l(dim3((unsigned)(wide ? std::min<long long>(blocks, 8ll * nsm) : blocks)), 256, 0, static_cast<cudaStream_t>(stream));
  auto launch = [&](void (*q)(Rows4), void (*qw)(Rows4), void (*d)(Rows4)) {
    return cudaLaunchKernelEx(&l.cfg, !write ? d : wide ? qw : q, a);
  };
  const cudaError_t e =
      dtype == MSK_BF16   ? launch(quantize_kernel<MSK_BF16, false>, quantize_kernel<MSK_BF16, true>, dequantize_kernel<MSK_BF16>)
      : dtype == MSK_FP16 ? launch(quantize_kernel<MSK_FP16, false>, quantize_kernel<MSK_FP16, true>, dequantize_kernel<MSK_FP16>)
                          : launch(quantize_kernel<MSK_FP32, false>, quantize_kernel<MSK_FP32, false>, dequantize_kernel<MSK_FP32>);
  return e == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

constexpr int kM = 128;            // weight rows of a block (a pair's MMA has M = 256)
constexpr int kStageK = 256;       // columns of a stage
constexpr int kSteps = kStageK / 64;  // MMAs of a stage
constexpr int kMaxN = 256;         // tokens of a tile at most (the MMA's N); half of it where a tile has gate and up
constexpr int kStepN = 32;         // ... and what they are filled up to: each block has half of them
constexpr int kMaxStages = 10;
constexpr int kMaxE = 1024;
constexpr int kScaleWarps = 4, kEpiWarps = 8;
constexpr int kScaleWarp0 = 4, kEpiWarp0 = kScaleWarp0 + kScaleWarps;
constexpr int kProductThreads = 32 * (kEpiWarp0 + kEpiWarps);
// Tiles whose places are known ahead: four are at the warps that write scales where
// a tile is one stage, and two at their ends.
constexpr int kTiles = 8;
constexpr int kACodes = kM * kStageK / 2, kSfABytes = kM * kStageK / 16;
// Weights' scales as they come: 32 bytes of a row, which hold the stage's 16, where rows lie
// no multiple of 16 bytes apart.
__host__ __device__ constexpr int weight_scales_bytes(int group) { return group > 1 ? 2 * kSfABytes : kSfABytes; }
constexpr int kRing = 204 * 1024;  // (dynamic shared memory: beside it the tables below and what aligns the ring)
// Gathered tokens' scales: of four stages and 128 tokens, twice.
constexpr int kQuadBytes = 128 * kStageK / 16 * 4, kQuads = 2 * kQuadBytes;
constexpr int kTables = 3 * kMaxE * 4;
constexpr int kSmem = 1024 + kRing + kTables;
// Tensor memory columns: two accumulators, which overlap where a tile has more
// than kAcc1 columns (a token's, or a token's gate and up), then the scales of a
// stage: of weights and up to 256 tokens, or of gate, up and up to 128 tokens.
constexpr int kAcc1 = 208, kSf = kAcc1 + 256;
static_assert(kSf + 12 * kSteps == 512, "tensor memory");

static __device__ uint32_t g_error;  // nonzero once a wait has run out

struct Experts4 {
  CUtensorMap w_map, up_map;     // [E rows][cols / 2] bytes, boxes of 128 x 128
  CUtensorMap x_map, x16_map, x8_map;  // [x_rows][cols / 2] bytes, boxes of 64 x 128, of 16 x 128, of 8 x 128
  CUtensorMap ws_map, us_map;    // scales: [E rows / w_group][w_group cols / 16] bytes, boxes of 128 rows
  CUtensorMap xs_map, xs32_map, xs8_map;  // [x_rows][cols / 16], boxes of nt x 16, of 32 x 16, of 8 x 16
  const uint8_t *x_codes, *x_scales, *w_scales, *up_scales;
  const float *w_ts, *up_ts;
  const int32_t *offsets, *slots;
  void* y;
  long long y_stride, x_rows;
  int n, E, rows, K, top_k, y_dtype, nt, stages, mblocks;
  float x_ts;
  int w_group;  // weights' scales come by copies of so many rows as one (0: threads load them)
  int withheld;       // tests: of this one of a pair's tiles nobody says that it is complete (-1: of none)
  uint64_t wait_ns;   // bound of every wait, beside the time for each step
};

// A tile: the pair's 256 weight rows of an expert and up to nt of its tokens.
struct Tile {
  int e, m;       // expert, block of weight rows
  int p0, count;  // first place and number of places
  int n;          // count, up to the MMA's next N
};

struct Bars {
  // a stage is full (weights, tokens, and both blocks' scales in order); its scales have come; it may be filled
  uint64_t full[kMaxStages], rfull[kMaxStages], empty[kMaxStages];
  uint64_t accf[2], acce[2], over[2];
  uint64_t tfull[kTiles], tempty[kTiles];
  uint64_t qfull[2], qempty[2];  // gathered tokens' scales
  uint64_t done;
};

// --- what a pair of blocks does together (the first block's thread issues) ------

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred q; elect.sync _|q, 0xFFFFFFFF; selp.u32 %0, 1, 0, q; }" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_tmem_free(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         bool accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p; }" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// 32 rows x 16 bytes of each block's shared memory into its tensor memory.
__device__ __forceinline__ void pair_cp_sf(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
// Arrives on the barrier of both blocks (or of `mask`'s) when the MMAs before are complete.
__device__ __forceinline__ void pair_commit(uint32_t mbar, uint16_t mask) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(mbar),
               "h"(mask)
               : "memory");
}
// A box into this block's shared memory, counted by a barrier of the first block's.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Arrives on a barrier of the pair's first block.  At the block's scope: a release
// at the cluster's waits for everything that the thread has under way, some 1200
// clocks.  What is said is that tensor memory has been read (tcgen05's own fences
// order that), or that this block's shared memory is ready for its own SM's tensor
// core (the fence between the proxies orders that).
__device__ __forceinline__ void pair_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// v = m 2^e, m's magnitude in [1, 2) (v finite and not 0; a subnormal number is made a
// normal one first).
__device__ __forceinline__ float significand(float v, int& e) {
  e = -127;
  if (fabsf(v) < 0x1p-126f) v *= 0x1p24f, e -= 24;
  e += (__float_as_uint(v) >> 23) & 255;
  return __uint_as_float((__float_as_uint(v) & 0x807FFFFFu) | 0x3F800000u);
}

// Two tensors' scales as a factor and 1 or, where the product leaves the range of
// fp32's normal numbers, as a significand with a half of the power of two and the other
// half, so that no product with them leaves it unless the result does (and the other way
// round: a subnormal factor would have lost digits that the result has).
__device__ __forceinline__ float2 scale_factors(float w, float x) {
  const float p = w * x;
  if (fabsf(p) >= 0x1p-126f && fabsf(p) <= 3e38f) return make_float2(p, 1.f);
  if (w == 0.f || x == 0.f || !(fabsf(w) < INFINITY) || !(fabsf(x) < INFINITY)) return make_float2(p, 1.f);
  int ew, ex;
  const float m = significand(w, ew) * significand(x, ex);
  const int e2 = max(-250, min(250, ew + ex)), e1 = e2 / 2;
  return make_float2(m * exp2i(e1), exp2i(e2 - e1));
}

// `bytes` (0 or 16) of 16, zeros for the rest.
__device__ __forceinline__ void cp_async16_some(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// silu(g) = g / (1 + e^-g) of two numbers, off by some 2^-21: 2^t for t = -g
// log2(e), times a factor for what t's rounding and the constant's leave; 0 for
// g below some -87.3 (the reciprocal leaves fp32's normal numbers).
__device__ __forceinline__ unsigned long long silu2(unsigned long long g) {
  const unsigned long long one = pair(1.f, 1.f), l = pair(-1.4426950409f, -1.4426950409f);
  float g0, g1, t0, t1, r0, r1;
  unpair(g, g0, g1);
  const unsigned long long m = pair(fminf(g0, 1e30f), fminf(g1, 1e30f));  // (an infinity stays one)
  const unsigned long long t = mul2(m, l);
  const unsigned long long rest = fma2(m, pair(-1.9259629911e-8f, -1.9259629911e-8f), fma2(m, l, mul2(t, pair(-1.f, -1.f))));
  unpair(t, t0, t1);
  const unsigned long long p = mul2(pair(ex2(t0), ex2(t1)), fma2(rest, pair(0.6931471806f, 0.6931471806f), one));
  unpair(add2(p, one), t0, t1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(t0));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(t1));
  return mul2(g, pair(r0, r1));
}

// y^T = W x^T by block-scaled NVFP4 on the fifth-generation tensor cores.  A pair
// of blocks (a cluster) has a tile of M = 256 weight rows, 128 each, and N = up to
// 256 tokens of one expert, of which each block loads half: alone, a block would
// load 384 rows where it loads 256 now, and loads bound the kernel as much as MMAs.
// GLU: a tile has 256 rows of gate and the same of up, and up to 128 tokens, so that
// a lane's accumulators hold both of its row.
// Weights and tokens come by tiled copies with the 128-byte swizzle, tokens named
// by slots by asynchronous copies of 16 bytes (gathering tiled copies take 66
// clocks for four rows of 128 bytes).  Scales, row-major in memory, come by tiled
// copies too and are put into the tensor cores' order by threads; where columns are
// no multiple of 256 (!TILED) tokens' are loaded by threads (128 rows hold the load unit
// for 256 clocks) and weights' come as scale_group has it.  Tiles run over experts, then blocks of weight rows, then tokens, so
// that neighbouring pairs share weights in L2; a pair takes every one that is a
// multiple of the pairs on.
//
// 65536 rows of 256 experts, gate and up of 1024 x 2048: 150 us, 3.7 PFLOP/s, 5.0 TB/s
// (168 to 170 in a row of seconds, where the power limit holds the clock at 1.55 GHz);
// 8192 x 8192 x 8192: 180 us, 6.1 PFLOP/s; 1 to 128 tokens with 4096 x 4096: 7.6 to 8.9 us,
// 16 pairs of 76 and a chain of latencies.  What bounds full tiles is what a stage takes
// of shared memory's 128 bytes a clock (copies in, the MMAs' reads, scales in, read,
// put in order and read again: 94 KB, with gate and up 110 to 130), and, with weights
// from DRAM, its latency behind four or five stages.
//
// Roles: a warp that finds the tiles and their tokens, one that copies weights, one
// that copies tokens, one that issues (of the pair's first block), four that write
// scales and gather, eight that end the tiles from one of two accumulators while
// the other fills.  Everything that one thread issues is issued by the elected lane
// of a warp that stays together: from a branch of one lane an MMA or a copy takes
// three times as long.
template <bool GLU, bool GATHER, bool TILED>
__global__ void __launch_bounds__(kProductThreads, 1) experts4_kernel(const __grid_constant__ Experts4 a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ Tile tile_ring[kTiles];
  __shared__ int source_ring[kTiles][kMaxN];  // rows of x of a tile's tokens
  __shared__ uint32_t tmem_base;
  __shared__ int abort, never, tiles_all, warp_tiles[kProductThreads / 32];
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const int rank = blockIdx.x & 1, team = blockIdx.x >> 1, teams = gridDim.x >> 1;
  // (dynamic shared memory starts at a multiple of 1024 in the shared window)
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t ring = smem_u32(smem);
  int* starts = reinterpret_cast<int*>(smem + kRing);  // [E]: first place of each expert
  int* counts = starts + kMaxE;                         // [E]
  int* ends = counts + kMaxE;                           // [E]: tiles up to and with each expert
  const int chunks = a.nt > 128 ? 2 : 1;                // of tokens' scales, 128 rows each
  const int slot_b = a.nt / 2 * (kStageK / 2);
  // in a slot: weights (gate, up), tokens, the weights' scales, the tokens'.  Scales are put in
  // order where they have come to: a warp's threads write what they have read.
  constexpr int kMats = GLU ? 2 : 1, off_b = kMats * kACodes;
  const int w_group = TILED ? 1 : a.w_group, sfa = weight_scales_bytes(w_group);
  const int off_sfa = off_b + slot_b, off_sfb = off_sfa + kMats * sfa, slot_bytes = off_sfb + chunks * 512 * kSteps;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  auto first = [&](uint64_t& b) { return mapa(smem_u32(&b), 0); };  // the pair's first block's

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&a.w_map);
    if (GLU) prefetch_tensormap(&a.up_map);
    if (!GATHER) prefetch_tensormap(&a.x8_map);
    if (w_group > 0) {
      prefetch_tensormap(&a.ws_map);
      if (GLU) prefetch_tensormap(&a.us_map);
    }
    if (!GATHER && TILED) prefetch_tensormap(&a.xs8_map);
  }
  if (tid == 32) {
    abort = 0, never = 0;
    for (int i = 0; i < a.stages; ++i)
      mbar_init(bar(bars.full[i]), (GATHER ? 1 : 2) + 2), mbar_init(bar(bars.rfull[i]), 1 + (!GATHER && TILED)), mbar_init(bar(bars.empty[i]), 1);
    for (int i = 0; i < 2; ++i)
      mbar_init(bar(bars.accf[i]), 1), mbar_init(bar(bars.acce[i]), 2 * kEpiWarps), mbar_init(bar(bars.over[i]), 2 * kEpiWarps);
    for (int i = 0; i < kTiles; ++i)
      mbar_init(bar(bars.tfull[i]), 1), mbar_init(bar(bars.tempty[i]), 1 + (!GATHER || TILED) + !rank + kScaleWarps + kEpiWarps);
    for (int i = 0; i < 2; ++i) mbar_init(bar(bars.qfull[i]), 1), mbar_init(bar(bars.qempty[i]), kScaleWarps);
    mbar_init(bar(bars.done), 1);
    mbar_fence_init();
    fence_proxy_async_shared();
  }
  if (warp == 3) pair_tmem_alloc(smem_u32(&tmem_base), 512);
  grid_dep_wait();
  grid_dep_launch();

  // The experts' places and tiles.  Whatever the offsets hold, ranges lie in [0, n]
  // and do not overlap: an expert begins where the ones before have ended.
  constexpr int kPer = kMaxE / kProductThreads;
  {
    int from[kPer], last[kPer];
    bool rising = true;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = kPer * tid + j;
      from[j] = e < a.E ? max(0, min(a.n, __ldg(a.offsets + e))) : 0;
      last[j] = e < a.E ? max(0, min(a.n, __ldg(a.offsets + e + 1))) : 0;
      rising = rising && from[j] <= last[j];
    }
    if (!__syncthreads_and(rising)) {  // (not what a sort gives)
      for (int j = 0; j < kPer; ++j) counts[kPer * tid + j] = last[j];
      __syncthreads();
      if (tid == 0) {
        int at = 0;
        for (int e = 0; e < a.E; ++e) {
          starts[e] = max(at, e > 0 ? counts[e - 1] : max(0, min(a.n, __ldg(a.offsets))));
          at = max(starts[e], counts[e]);
          if (e > 0) counts[e - 1] = ends[e - 1];
          ends[e] = max(0, counts[e] - starts[e]);
        }
        counts[a.E - 1] = ends[a.E - 1];
      }
      __syncthreads();
      for (int j = 0; j < kPer; ++j)
        if (kPer * tid + j < a.E) from[j] = starts[kPer * tid + j], last[j] = from[j] + counts[kPer * tid + j];
      __syncthreads();
    }
    int sum = 0, upto[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) sum += (last[j] - from[j] + a.nt - 1) / a.nt * a.mblocks, upto[j] = sum;
    int scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) warp_tiles[warp] = scan;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kProductThreads / 32; ++w) {
      const int v = warp_tiles[w];
      before += w < warp ? v : 0, all += v;
    }
    if (tid == 0) tiles_all = all;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = kPer * tid + j;
      if (e < a.E) starts[e] = from[j], counts[e] = last[j] - from[j], ends[e] = before + scan - sum + upto[j];
    }
  }
  tc_fence_before();
  cluster_sync();  // (of the block too)
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const int mine = team < tiles_all ? (tiles_all - team + teams - 1) / teams : 0;
  const int kst = (a.K + kStageK - 1) / kStageK;  // stages of a tile
  const uint64_t deadline = gtimer() + a.wait_ns + (uint64_t)mine * kst * kOpsStepNs;
  const volatile int* ab = &abort;
  // Waits by whole warps.
  auto wait = [&](uint64_t& b, uint32_t parity) {
    const bool ok = mbar_wait(bar(b), parity, deadline, ab);
    if (!ok) abort = 1;
    return (bool)__all_sync(0xFFFFFFFFu, ok);
  };
  auto wait_tile = [&](int i) { return wait(bars.tfull[i % kTiles], (i / kTiles) & 1); };
  auto leave_tile = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(bars.tempty[i % kTiles]));
  };

  if (warp == 3) {
    // --- tiles ----------------------------------------------------------------
    for (int i = 0; i < mine; ++i) {
      if (!wait(bars.tempty[i % kTiles], ((i / kTiles) & 1) ^ 1)) break;
      const int t = team + i * teams;
      int lo = 0, hi = a.E - 1;  // the first expert whose tiles go beyond t
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > t) hi = mid;
        else lo = mid + 1;
      }
      const int all = counts[lo], nb = (all + a.nt - 1) / a.nt;
      const int local = t - (lo > 0 ? ends[lo - 1] : 0);
      const int m = local / nb, j = local - m * nb;
      const int step = ((all + nb - 1) / nb + kStepN - 1) / kStepN * kStepN;  // tokens of a tile, the same for all but the last
      const int p0 = starts[lo] + j * step, count = min(step, all - j * step);
      Tile& r = tile_ring[i % kTiles];
      int p[kMaxN / 32];
#pragma unroll
      for (int k = 0; k < kMaxN / 32; ++k) {
        p[k] = lane + 32 * k < count ? p0 + lane + 32 * k : -1;
        if (GATHER && p[k] >= 0) p[k] = __ldg(a.slots + p[k]);
      }
#pragma unroll
      for (int k = 0; k < kMaxN / 32; ++k) {
        if (GATHER && lane + 32 * k < count) p[k] = min((int)a.x_rows - 1, (int)((unsigned)max(p[k], 0) / (unsigned)a.top_k));
        source_ring[i % kTiles][lane + 32 * k] = p[k];
      }
      if (lane == 0) r.e = lo, r.m = m, r.p0 = p0, r.count = count, r.n = (count + kStepN - 1) / kStepN * kStepN;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.tfull[i % kTiles]));
    }
  } else if (warp == 0 || (!GATHER && warp == 1)) {
    // --- copies of weights (warp 0) and tokens (warp 1) --------------------------
    const bool el = elect_one();
    const int groups = max(1, w_group), part = sfa / groups;
    int st = 0;
    uint32_t ph = 1;  // (a fresh barrier passes a wait for phase 1)
    bool ok = true;
    for (int i = 0; i < mine && ok; ++i) {
      ok = wait_tile(i);
      if (!ok) break;
      const Tile& t = tile_ring[i % kTiles];
      const int n = t.n, count = t.count;
      // Tokens that each block copies.  Rows behind a tile's are others' tokens, which no
      // one needs here, and where experts have few all pairs would read the same few lines: 512
      // rows of 256 experts, 2048 x 1024, 62 us, in copies of no more than these 43.
      const int few = (count + 7) & ~7, in_first = min(few, n / 2), copied = rank == 0 ? in_first : few - in_first;
      const int with_scales = few <= 8 ? 8 : few <= 64 ? (few + 31) & ~31 : a.nt;  // (a copy more takes 40 clocks a stage)
      const int row = warp == 0 ? t.e * a.rows + t.m * 256 + rank * 128 : t.p0 + rank * (n / 2), p0 = t.p0, row_group = row / groups;
      for (int s = 0; s < kst; ++s) {
        ok = wait(bars.empty[st], ph);
        if (!ok) break;
        if (el) {
          const uint32_t dst = ring + st * slot_bytes, b = first(bars.full[st]);
          const int x = s * (kStageK / 2);
          // (scales first: they are put in order while the codes are on their way)
          const uint32_t r = bar(bars.rfull[st]);
          const int xs = s * (kStageK / 16);
          if (warp == 1) {
            if (TILED) {
              mbar_arrive_expect_tx(r, with_scales * (kStageK / 16));
              tma_load_2d(dst + off_sfb, few <= 8 ? &a.xs8_map : few <= 64 ? &a.xs32_map : &a.xs_map, xs, p0, r);
              if (with_scales == 64) tma_load_2d(dst + off_sfb + 32 * (kStageK / 16), &a.xs32_map, xs, p0 + 32, r);
            }
          } else if (w_group > 0) {
            mbar_arrive_expect_tx(r, kMats * sfa);
            for (int u = 0; u < w_group; ++u) {  // the rows that are u of their group
              const uint32_t to = dst + off_sfa + u * part;
              const int xu = (u * (a.K / 16) + xs) & ~15;
              tma_load_2d(to, &a.ws_map, xu, row_group, r);
              if (GLU) tma_load_2d(to + sfa, &a.us_map, xu, row_group, r);
            }
          }
          if (rank == 0) mbar_arrive_expect_tx(bar(bars.full[st]), warp == 0 ? 2 * kMats * kACodes : few * (kStageK / 2));
          if (warp == 1) {
            int j = 0;
            for (; j + 64 <= copied; j += 64) pair_load_2d(dst + off_b + j * 128, &a.x_map, x, row + j, b);
            for (; j + 16 <= copied; j += 16) pair_load_2d(dst + off_b + j * 128, &a.x16_map, x, row + j, b);
            if (j < copied) pair_load_2d(dst + off_b + j * 128, &a.x8_map, x, row + j, b);
          } else {
            pair_load_2d(dst, &a.w_map, x, row, b);
            if (GLU) pair_load_2d(dst + kACodes, &a.up_map, x, row, b);
          }
        }
        __syncwarp();
        if (++st == a.stages) st = 0, ph ^= 1;
      }
      leave_tile(i);
    }
  } else if (warp == 1) {
    // --- gathered tokens' scales, four stages at a time -----------------------------
    // (four lanes have 64 bytes of a row: a load of 16 bytes each of 32 rows would
    // hold the load unit four times as long)
    if (TILED) {
      const int pitch = a.K / 16, piece = lane & 3;
      int quad = 0;
      bool ok = true;
      for (int i = 0; i < mine && ok; ++i) {
        ok = wait_tile(i);
        const int count = ok ? tile_ring[i % kTiles].count : 0;
        for (int s = 0; s < kst && ok; s += 4, ++quad) {
          ok = wait(bars.qempty[quad & 1], ((quad >> 1) & 1) ^ 1);
          if (!ok) break;
          const uint32_t dst = ring + kRing - kQuads + (quad & 1) * kQuadBytes;
          if (s + piece < kst) {
#pragma unroll 4
            for (int k = lane >> 2; k < count; k += 8)  // (columns behind them may have any scales)
              cp_async16(dst + k * 64 + ((piece ^ ((k >> 1) & 3)) << 4),
                         a.x_scales + (long long)source_ring[i % kTiles][k] * pitch + (s + piece) * 16);
          }
          cp_async_wait_all();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bars.qfull[quad & 1]));
        }
        leave_tile(i);
      }
    }
  } else if (warp == 2) {
    // --- MMAs -----------------------------------------------------------------
    if (rank == 0) {
      const bool el = elect_one();
      int st = 0, before = 0;  // (the tokens of the tile before)
      uint32_t ph = 0;
      bool ok = true;
      for (int i = 0; i < mine && ok; ++i) {
        ok = wait_tile(i);
        if (!ok) break;
        const int n = __shfl_sync(0xFFFFFFFFu, tile_ring[i % kTiles].n, 0), d = i & 1;
        leave_tile(i);
        ok = wait(bars.acce[d], ((i >> 1) & 1) ^ 1);
        // (accumulators that overlap: the tile before has been read there)
        if (ok && i > 0 && kMats * (d ? before : n) > kAcc1) ok = wait(bars.over[d ^ 1], ((i - 1) >> 1) & 1);
        if (!ok) break;
        before = n;
        tc_fence_after();
        const uint32_t acc = tmem + d * kAcc1, idesc = idesc_mxf4nvf4(n) + (1u << 27);  // (M = 256)
        for (int s = 0; s < kst; ++s) {
          ok = wait(bars.full[st], ph);
          if (!ok) break;
          tc_fence_after();
          if (el) {
            const uint32_t at = ring + st * slot_bytes;
            const uint64_t ad = umma_desc(at, 16, 1024) | kSwizzle128, bd = umma_desc(at + off_b, 16, 1024) | kSwizzle128;
            const uint64_t fa = umma_desc(at + off_sfa, 128, 128), fb = umma_desc(at + off_sfb, 128, 128);
            const uint32_t ta = tmem + kSf, tb = ta + 4 * kMats * kSteps;
            auto step = [&](int k, bool two) {
              pair_cp_sf(ta + 4 * k, fa + 32 * k);
              if (GLU) pair_cp_sf(ta + 4 * kSteps + 4 * k, fa + (sfa >> 4) + 32 * k);
              pair_cp_sf(tb + (GLU ? 4 : 8) * k, fb + (two ? 64 : 32) * k);
              if (two && n > 128) pair_cp_sf(tb + 8 * k + 4, fb + 64 * k + 32);
              pair_mma(acc, ad + 2 * k, bd + 2 * k, idesc, ta + 4 * k, tb + (GLU ? 4 : 8) * k, s > 0 || k > 0);
              if (GLU)
                pair_mma(acc + n, ad + (kACodes >> 4) + 2 * k, bd + 2 * k, idesc, ta + 4 * kSteps + 4 * k, tb + 4 * k, s > 0 || k > 0);
            };
            auto steps = [&](bool two) {
              if (a.K - s * kStageK >= kStageK) {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) step(k, two);
              } else {
                for (int k = 0; k < (a.K - s * kStageK) / 64; ++k) step(k, two);
              }
            };
            if (!GLU && chunks == 2) steps(true);
            else steps(false);
            pair_commit(bar(bars.empty[st]), 3);
          }
          __syncwarp();
          if (++st == a.stages) st = 0, ph ^= 1;
        }
        if (ok && el && i != a.withheld) pair_commit(bar(bars.accf[d]), 3);
        __syncwarp();
      }
      // what is still in flight ends before the block does
      if (el) {
        pair_commit(bar(bars.done), 1);
        if (!mbar_wait(bar(bars.done), 0, gtimer() + kOpsWaitNs, &never)) abort = 1;
      }
      __syncwarp();
    }
  } else if (warp >= kScaleWarp0 && warp < kEpiWarp0) {
    // --- scales, and gathered tokens ----------------------------------------------
    // Of four stages each of these warps takes one, so that four are under way: a stage
    // takes some 700 clocks from its first wait to its hand-over, 1300 where tokens are
    // gathered.  A lane has every 8th row and token of a block's 128, of which four make 16
    // bytes that follow each other in order: all steps of four or, where scales have come
    // by threads' loads or 32 bytes of a row, one step of 16.
    constexpr int kOf = 3;  // rows' scales of a stage, 128 each: weights (gate), tokens or up, tokens
    constexpr int kTok = GLU ? 2 : 1, kChunks = GLU || GATHER ? 1 : 2;
    const int sw = warp - kScaleWarp0, r8 = lane & 7, r4 = lane >> 3;
    const int pitch = a.K / 16;
    // at [q][j]: of row 32 r4 + 8 q + r8 step j's where TILED, else of row 32 j + 8 q + r8 step r4's
    uint32_t w[kOf][4][4];
    auto put = [&](uint32_t (&v)[4], uint4 u) { v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w; };
    // Scales that do not come by copies: eight rows' 16 bytes at a time (what holds the load
    // unit is rows, two clocks each, whatever it takes of them).
    auto fetch = [&](int i, int s) {
      const int at = 16 * s + 4 * r4;
      const bool in = at < pitch;
      auto word = [](const uint8_t* p) { return __ldg(reinterpret_cast<const uint32_t*>(p)); };
      if (w_group == 0) {
        const Tile& t = tile_ring[i % kTiles];
        const int row0 = t.m * 256 + rank * 128 + r8;
        const long long from = ((long long)t.e * a.rows + row0) * pitch + at;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = 32 * j + 8 * q;
            const bool have = in && row0 + row < a.rows;
            w[0][q][j] = have ? word(a.w_scales + from + row * pitch) : 0;
            if (GLU) w[1][q][j] = have ? word(a.up_scales + from + row * pitch) : 0;
          }
      }
      if (!TILED) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              const int src = source_ring[i % kTiles][128 * c + 32 * j + 8 * q + r8];
              w[kTok + c][q][j] = in && src >= 0 ? word(a.x_scales + (long long)src * pitch + at) : 0;
            }
      }
    };
    // Where the copies put this lane's of weights' rows, and how far on the next eight rows are.
    const int group = max(w_group, 1), u = r8 & (group - 1);
    const int w_at = off_sfa + u * (sfa / group) + r8 / group * 32 + ((u * pitch) & 15) + 4 * r4;
    const int w_next = group == 4 ? 64 : 128;
    // Of stages s0 .. s0 + 3 of tile i this warp's is s (there may be none), every
    // fourth of all tiles' (no more apart than there are slots: a slot's barrier would
    // be mistaken for its next but one use); st: the slot it goes to.
    int i = 0, s0 = 0, s = sw, st = sw, quad = 0;
    uint32_t ph = 1;
    bool ok = mine > 0 && wait_tile(0);
    if (ok && s < kst) fetch(i, s);
    for (; ok && i < mine; ++quad) {
      const uint32_t slot = ring + st * slot_bytes;
      if (s < kst) {
        ok = wait(bars.empty[st], ph);
        if (!ok) break;
        if (GATHER) {
          // eight lanes have a row's 128 bytes (columns behind the tokens get none of it)
          const int n = tile_ring[i % kTiles].n, col = s * (kStageK / 2) + r8 * 16;
          const int* rows = source_ring[i % kTiles] + rank * (n / 2) + r4;
          const bool inside = col < a.K / 2;
          int r[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (8 * j < n) r[j] = rows[4 * j];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (8 * j >= n) break;
            const int k = r4 + 4 * j;
            cp_async16_some(slot + off_b + k * 128 + (((r8 ^ k) & 7) << 4), a.x_codes + (long long)max(r[j], 0) * (a.K / 2) + (inside ? col : 0),
                            r[j] >= 0 && inside ? 16 : 0);
          }
        }
      }
      if (GATHER && TILED) {
        ok = wait(bars.qfull[quad & 1], (quad >> 1) & 1);
        if (!ok) break;
        if (s < kst) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int row = 32 * r4 + 8 * q + r8;
            put(w[kTok][q], lds128(ring + kRing - kQuads + (quad & 1) * kQuadBytes + row * 64 + (((s - s0) ^ ((row >> 1) & 3)) << 4)));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bars.qempty[quad & 1]));
      }
      if (s < kst) {
        if (w_group > 0) {
          ok = wait(bars.rfull[st], ph ^ 1);
          if (!ok) break;
          if (TILED) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t at = slot + 16 * (32 * r4 + 8 * q + r8);
              put(w[0][q], lds128(at + off_sfa));
              if (GLU) put(w[1][q], lds128(at + off_sfa + sfa));
              if (!GATHER) {
                put(w[kTok][q], lds128(at + off_sfb));
                if (!GLU && chunks == 2) put(w[2][q], lds128(at + off_sfb + 2048));
              }
            }
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t at = slot + w_at + (4 * j + q) * w_next;
                w[0][q][j] = lds32(at);
                if (GLU) w[1][q][j] = lds32(at + sfa);
              }
          }
          __syncwarp();  // (they are put in order where they have come to)
        }
        // (chunk c of step k at 512 (chunks k + c))
        if (TILED) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t to = slot + 16 * (8 * q + r8) + 4 * r4;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              sts32(to + off_sfa + 512 * k, w[0][q][k]);
              if (GLU) sts32(to + off_sfa + sfa + 512 * k, w[1][q][k]);
              sts32(to + off_sfb + 512 * (GLU ? 1 : chunks) * k, w[kTok][q][k]);
              if (!GLU && chunks == 2) sts32(to + off_sfb + 512 + 1024 * k, w[2][q][k]);
            }
          }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t to = slot + 16 * (8 * q + r8), to_b = to + off_sfb + 512 * (GLU ? 1 : chunks) * r4;
            sts128(to + off_sfa + 512 * r4, w[0][q]);
            if (GLU) sts128(to + off_sfa + sfa + 512 * r4, w[1][q]);
            sts128(to_b, w[kTok][q]);
            if (!GLU && chunks == 2) sts128(to_b + 512, w[2][q]);
          }
        }
        // what this warp's threads have written is seen by the tensor cores
        if (GATHER) cp_async_wait_all();
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) pair_arrive(first(bars.full[st]));
      }
      // on to the next four
      if (s < kst && (st += kScaleWarps) >= a.stages) st -= a.stages, ph ^= 1;
      if (s0 + 4 < kst) {
        s0 += 4, s += 4;
      } else {
        leave_tile(i);
        ++i, s0 = 0, s = (int)((unsigned)sw - (unsigned)i * (unsigned)kst) & 3;
        ok = i >= mine || wait_tile(i);
      }
      if (ok && i < mine && s < kst) fetch(i, s);
    }
    if (GATHER) cp_async_wait_all();  // (behind a wait that ran out)
  } else if (warp >= kEpiWarp0) {
    // --- epilogue -------------------------------------------------------------
    const int quad = warp & 3, half = (warp - kEpiWarp0) >> 2;
    auto run = [&](auto type) {
      using T = decltype(type);
      bool ok = true;
      for (int i = 0; i < mine && ok; ++i) {
        const int d = i & 1;
        ok = wait_tile(i);
        if (!ok) break;
        const Tile& t = tile_ring[i % kTiles];
        const int n = t.n, count = t.count;
        const float2 f = scale_factors(a.w_ts != nullptr ? __ldg(a.w_ts + t.e) : 1.f, a.x_ts);
        const float2 g = GLU ? scale_factors(a.up_ts != nullptr ? __ldg(a.up_ts + t.e) : 1.f, a.x_ts) : f;
        const float f0 = f.x, f1 = f.y, u0 = g.x, u1 = g.y;
        ok = wait(bars.accf[d], (i >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16) + d * kAcc1;
        const int row = t.m * 256 + rank * 128 + quad * 32 + lane;
        T* y = static_cast<T*>(a.y) + (long long)t.p0 * a.y_stride + row;
        const bool in = row < a.rows;
        const bool one = f1 == 1.f && (!GLU || u1 == 1.f);
        // Chunks of 32 tokens, in turn with the other warps of these lanes, those first
        // that overlap the other accumulator: the first chunk of each.
        const int nc = (n / 32 + 1 - half) / 2;
        for (int c = 0; c < nc; ++c) {
          const int c0 = 32 * (half + 2 * (d ? c : nc - 1 - c));
          float v[32], u[32];
          __syncwarp();  // (lanes behind the last row store nothing and are here first)
          tmem_ld32(at + c0, v);
          if (GLU) tmem_ld32(at + n + c0, u);
          if (c == 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) pair_arrive(first(bars.over[d]));
          }
          if (c == nc - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) pair_arrive(first(bars.acce[d]));
          }
          if (!in) continue;
          T* p = y + (long long)c0 * a.y_stride;
          auto values = [&](auto single, int j, float& x, float& z) {  // tokens j and j + 1
            unsigned long long g = mul2(pair(v[j], v[j + 1]), pair(f0, f0));
            if (!single()) g = mul2(g, pair(f1, f1));
            if (GLU) {
              unsigned long long h = mul2(pair(u[j], u[j + 1]), pair(u0, u0));
              if (!single()) h = mul2(h, pair(u1, u1));
              g = mul2(silu2(g), h);
            }
            unpair(g, x, z);
          };
          if (one && c0 + 32 <= count) {
#pragma unroll
            for (int j = 0; j < 32; j += 2, p += 2 * a.y_stride) {
              float x, z;
              values(std::true_type(), j, x, z);
              p[0] = static_cast<T>(x), p[a.y_stride] = static_cast<T>(z);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 2, p += 2 * a.y_stride) {
              if (c0 + j >= count) break;
              float x, z;
              values(std::false_type(), j, x, z);
              p[0] = static_cast<T>(x);
              if (c0 + j + 1 < count) p[a.y_stride] = static_cast<T>(z);
            }
          }
        }
        if (nc == 0) {
          __syncwarp();
          if (lane == 0) pair_arrive(first(bars.over[d])), pair_arrive(first(bars.acce[d]));
        }
        leave_tile(i);
      }
    };
    if (a.y_dtype == MSK_FP32) run(float());
    else if (a.y_dtype == MSK_FP16) run(__half());
    else run(__nv_bfloat16());
  }
  tc_fence_before();
  cluster_sync();  // (no block leaves while the pair's MMAs, copies or arrivals may come to it)
  tc_fence_after();
  if (warp == 3) {
    // Read here, where none of the block's waits can run out any more (a barrier of its threads in
    // front of the pair's, for this alone, took 0.4 us of a product of one token, 7.5 us).
    if (*ab) {
      if (lane == 0) {
        atomicExch(&g_error, 1u);
        // copies end before the block does: a slot's newest may be a use ahead of what was waited for
        // (those of the second block are counted by the first one, so that the second waits for as
        // long as the limit is; where only the other block gave up, this one's have all been used)
        for (uint32_t q = 0; q < 2; ++q)
          for (int k = 0; k < a.stages; ++k) {
            mbar_wait(bar(bars.full[k]), q, gtimer() + kOpsWaitNs / 100, &never);
            mbar_wait(bar(bars.rfull[k]), q, gtimer() + kOpsWaitNs / 100, &never);
          }
      }
      __syncwarp();
    }
    pair_tmem_free(tmem, 512);
  }
}

// Clusters of two that run at a time, looked up once a device.
template <bool GLU, bool GATHER, bool TILED>
int pairs_at_once() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev].load(std::memory_order_acquire);
  if (n == 0) {
    if (cudaFuncSetAttribute(experts4_kernel<GLU, GATHER, TILED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return 0;
    const OpsLaunch l(dim3(2), kProductThreads, kSmem, nullptr, 2);
    cudaLaunchConfig_t cfg = l.cfg;
    cudaLaunchAttribute at = l.at[1];
    cfg.attrs = &at, cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, experts4_kernel<GLU, GATHER, TILED>, &cfg) != cudaSuccess || n < 1) return 0;
    known[dev].store(n, std::memory_order_release);
  }
  return n;
}

template <bool GLU, bool GATHER, bool TILED>
cudaError_t launch_products(const Experts4& a, long long tiles, cudaStream_t st) {
  const int pairs = pairs_at_once<GLU, GATHER, TILED>();
  if (pairs == 0) return cudaErrorInvalidConfiguration;
  const OpsLaunch l(dim3(2 * (unsigned)std::min<long long>(pairs, tiles)), kProductThreads, kSmem, st, 2);
  return cudaLaunchKernelEx(&l.cfg, experts4_kernel<GLU, GATHER, TILED>, a);
}

msk_status check_experts(const msk_fp4_experts* w) {
  if (w->n_experts < 1 || w->n_experts > kMaxE || w->rows < 0 || w->rows > (1 << 24) || w->cols < 64 || w->cols > (1 << 17) ||
      w->cols % 64 || (int64_t)w->n_experts * w->rows > (1ll << 31) - 256)
    return MSK_ERR_SHAPE;
  return MSK_OK;
}

// What msk_fp4_experts_maps writes.
struct WeightMaps {
  CUtensorMap codes, scales;
  const uint8_t *packed, *scale_codes;
  int64_t experts, rows, cols, group;
};
static_assert(sizeof(WeightMaps) <= MSK_FP4_MAPS_BYTES && alignof(WeightMaps) <= 128, "msk.h");

// A tiled copy's rows lie a multiple of 16 bytes apart, so scales' one, two or four rows
// (of one expert) are one of a map, and a copy takes 32 bytes of each one's first, its
// second ..: a stage's 16 from a multiple of 4 on.  Loaded by threads, which is left for
// rows that are no such multiple, they hold the load unit for 256 clocks a stage and
// matrix: 32768 rows of 8 experts, gate and up of 1024 x 3968, 161 us, by copies 136 (of 4096
// columns 108); 16384 of 256, 2048 x 1088, 75 and 65.
int scale_group(const msk_fp4_experts* w) {
  const int group = w->cols % 256 == 0 ? 1 : w->cols % 128 == 0 ? 2 : 4;
  return w->rows % group == 0 ? group : 0;
}

// Rows of codes in boxes of `box` x 128 bytes, of scales in boxes of `box` x 16.
bool codes_map(CUtensorMap* m, const uint8_t* p, long long rows, long long cols, int box) {
  return matrix_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, rows, cols / 2, cols / 2, box, kStageK / 2, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool scales_map(CUtensorMap* m, const uint8_t* p, long long rows, long long cols, int box, int group) {
  const long long bytes = cols / 16 * group;
  return matrix_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, rows / group, bytes, bytes, box / group, group > 1 ? 32 : kStageK / 16,
                    CU_TENSOR_MAP_SWIZZLE_NONE);
}

bool make_maps(const msk_fp4_experts* w, WeightMaps* m) {
  const long long rows = (long long)w->n_experts * w->rows;
  m->packed = w->packed, m->scale_codes = w->scales, m->experts = w->n_experts, m->rows = w->rows, m->cols = w->cols;
  m->group = scale_group(w);
  return codes_map(&m->codes, w->packed, rows, w->cols, kM) &&
         (m->group == 0 || scales_map(&m->scales, w->scales, rows, w->cols, kM, (int)m->group));
}

// The weights' maps, the caller's or new ones.
msk_status weight_maps(const msk_fp4_experts* w, CUtensorMap* codes, CUtensorMap* scales) {
  WeightMaps own;
  const WeightMaps* m = static_cast<const WeightMaps*>(w->maps);
  if (m == nullptr) {
    if (!make_maps(w, &own)) return MSK_ERR_CUDA;
    m = &own;
  } else if (m->packed != w->packed || m->scale_codes != w->scales || m->experts != w->n_experts || m->rows != w->rows || m->cols != w->cols) {
    return MSK_ERR_INVALID_ARG;
  }
  *codes = m->codes;
  if (m->group > 0) *scales = m->scales;
  return MSK_OK;
}

std::atomic<int32_t> g_withheld{-1};
std::atomic<uint64_t> g_wait_ns{kOpsWaitNs};

}  // namespace

cudaError_t experts4_error(uint32_t* e) {
  cudaError_t r = cudaMemcpyFromSymbol(e, g_error, sizeof(*e));
  const uint32_t zero = 0;
  if (r == cudaSuccess && *e != 0) r = cudaMemcpyToSymbol(g_error, &zero, sizeof(zero));
  return r;
}

}  // namespace msk

using namespace msk;

extern "C" msk_status msk_quantize_fp4(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t x_stride,
                                       float tensor_scale, uint8_t* codes, uint8_t* scales, void* stream) {
  return rows_call(true, x, dtype, rows, cols, x_stride, tensor_scale, codes, scales, stream);
}

extern "C" msk_status msk_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, float tensor_scale, int64_t rows,
                                         int64_t cols, void* x, int32_t dtype, int64_t x_stride, void* stream) {
  return rows_call(false, x, dtype, rows, cols, x_stride, tensor_scale, codes, scales, stream);
}

extern "C" msk_status msk_fp4_experts_maps(const msk_fp4_experts* w, void* maps) {
  if (w == nullptr || maps == nullptr) return MSK_ERR_INVALID_ARG;
  const msk_status s = check_experts(w);
  if (s != MSK_OK) return s;
  if (w->rows == 0) return MSK_ERR_SHAPE;
  if (w->packed == nullptr || w->scales == nullptr) return MSK_ERR_INVALID_ARG;
  if (!ops_aligned16(w->packed) || !ops_aligned16(w->scales) || (reinterpret_cast<uintptr_t>(maps) & 127)) return MSK_ERR_ALIGNMENT;
  return make_maps(w, static_cast<WeightMaps*>(maps)) ? MSK_OK : MSK_ERR_CUDA;
}

extern "C" msk_status msk_debug_experts_fault(int32_t tile, uint64_t wait_ns) {
  if (tile < -1 || wait_ns > kOpsWaitNs) return MSK_ERR_INVALID_ARG;
  g_withheld.store(tile, std::memory_order_relaxed);
  g_wait_ns.store(wait_ns > 0 ? wait_ns : kOpsWaitNs, std::memory_order_relaxed);
  return MSK_OK;
}

extern "C" msk_status msk_experts_fp4(const msk_nvfp4_desc* x, const int32_t* slots, int32_t top_k, int64_t n,
                                      const int32_t* offsets, const msk_fp4_experts* w, const msk_fp4_experts* up, void* y,
                                      int32_t y_dtype, int64_t y_stride, void* stream) {
  if (x == nullptr || w == nullptr || !dtype_ok(y_dtype) || n < 0) return MSK_ERR_INVALID_ARG;
  msk_status s = check_experts(w);
  if (s == MSK_OK && up != nullptr) s = check_experts(up);
  if (s != MSK_OK) return s;
  if (up != nullptr && (up->n_experts != w->n_experts || up->rows != w->rows || up->cols != w->cols)) return MSK_ERR_INVALID_ARG;
  if (x->cols != w->cols) return MSK_ERR_INVALID_ARG;
  if (n > (1ll << 30) || x->rows < 0 || x->rows > (1ll << 30)) return MSK_ERR_SHAPE;
  if (slots != nullptr && top_k < 1) return MSK_ERR_INVALID_ARG;
  if (slots == nullptr && n > x->rows) return MSK_ERR_INVALID_ARG;
  if (n == 0 || w->rows == 0) return MSK_OK;
  if (x->rows == 0 || x->packed == nullptr || x->scales == nullptr || offsets == nullptr || w->packed == nullptr ||
      w->scales == nullptr || y == nullptr || (up != nullptr && (up->packed == nullptr || up->scales == nullptr)))
    return MSK_ERR_INVALID_ARG;
  if (n > 1 && y_stride < w->rows) return MSK_ERR_INVALID_ARG;
  if (!ops_aligned16(x->packed) || !ops_aligned16(x->scales) || !ops_aligned16(w->packed) || !ops_aligned16(w->scales) ||
      (up != nullptr && (!ops_aligned16(up->packed) || !ops_aligned16(up->scales))) ||
      ((reinterpret_cast<uintptr_t>(w->maps) | (up != nullptr ? reinterpret_cast<uintptr_t>(up->maps) : 0)) & 127) ||
      reinterpret_cast<uintptr_t>(y) % dtype_bytes(y_dtype) ||
      ((reinterpret_cast<uintptr_t>(slots) | reinterpret_cast<uintptr_t>(offsets) | reinterpret_cast<uintptr_t>(w->tensor_scales)) & 3) ||
      (up != nullptr && (reinterpret_cast<uintptr_t>(up->tensor_scales) & 3)))
    return MSK_ERR_ALIGNMENT;
  int nsm = 0;
  s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  Experts4 a{};
  a.x_codes = x->packed, a.x_scales = x->scales, a.w_scales = w->scales, a.w_ts = w->tensor_scales;
  if (up != nullptr) a.up_scales = up->scales, a.up_ts = up->tensor_scales;
  a.offsets = offsets, a.slots = slots, a.y = y, a.y_stride = n > 1 ? y_stride : 0, a.x_rows = x->rows;
  a.n = (int)n, a.E = w->n_experts, a.rows = (int)w->rows, a.K = (int)w->cols, a.top_k = top_k, a.y_dtype = y_dtype;
  a.x_ts = x->tensor_scale;
  a.mblocks = (a.rows + 255) / 256;
  a.w_group = scale_group(w);
  a.withheld = g_withheld.load(std::memory_order_relaxed), a.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  const bool tiled = a.w_group == 1;
  const auto tiles_of = [&](int nt) { return a.mblocks * ((n + std::min<int64_t>(n, a.E) * (nt - 1)) / nt); };  // at most
  // Tiles of 256 tokens load weights less often: 32768 rows of 256 experts, 2048 x 1024, 73 us,
  // of 128 75, 65536 104 and 116; fewer rows no worse.  Of 128: where all tiles run at once (256 x
  // 6144 x 4096 9.5 us, of 256 11.4), where threads load scales and experts have no more on
  // average (16384 rows of 256, 2048 x 1088, 65.6 and 70), and where gate and up or gathered
  // tokens' scales need the room.
  const bool half = up != nullptr || slots != nullptr || tiles_of(kMaxN / 2) <= nsm / 2 || (!tiled && n <= 128ll * w->n_experts);
  a.nt = (int)std::min<int64_t>(half ? kMaxN / 2 : kMaxN, (n + kStepN - 1) / kStepN * kStepN);
  const long long tiles = tiles_of(a.nt);
  if (tiles > (1ll << 31) - 1 - 65536) return MSK_ERR_SHAPE;
  const int mats = up != nullptr ? 2 : 1;
  const int slot = mats * (kACodes + weight_scales_bytes(a.w_group)) + a.nt / 2 * (kStageK / 2) + (a.nt > 128 ? 2 : 1) * 512 * kSteps;
  a.stages = std::min(kMaxStages, (kRing - (slots != nullptr && tiled ? kQuads : 0)) / slot);  // (4 at least)
  s = weight_maps(w, &a.w_map, &a.ws_map);
  if (s == MSK_OK && up != nullptr) s = weight_maps(up, &a.up_map, &a.us_map);
  if (s != MSK_OK) return s;
  // (a map takes the host 0.13 us: only those that some tile may take)
  const auto codes_by = [&](CUtensorMap* m, int box, bool taken) { return !taken || codes_map(m, x->packed, x->rows, a.K, box); };
  const auto scales_by = [&](CUtensorMap* m, int box, bool taken) { return !taken || scales_map(m, x->scales, x->rows, a.K, box, 1); };
  if (slots == nullptr && (!codes_by(&a.x_map, 64, a.nt >= 128) || !codes_by(&a.x16_map, 16, n > 8) || !codes_by(&a.x8_map, 8, true) ||
                           !scales_by(&a.xs_map, a.nt, tiled && a.nt > 64) || !scales_by(&a.xs32_map, 32, tiled && n > 8) ||
                           !scales_by(&a.xs8_map, 8, tiled)))
    return MSK_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto launch = [&](auto t) {
    constexpr bool kTiled = decltype(t)::value;
    if (up != nullptr) return slots != nullptr ? launch_products<true, true, kTiled>(a, tiles, st) : launch_products<true, false, kTiled>(a, tiles, st);
    return slots != nullptr ? launch_products<false, true, kTiled>(a, tiles, st) : launch_products<false, false, kTiled>(a, tiles, st);
  };
  const cudaError_t e = tiled ? launch(std::true_type()) : launch(std::false_type());
  return e == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}
