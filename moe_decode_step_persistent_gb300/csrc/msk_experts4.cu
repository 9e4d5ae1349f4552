// 4-bit matrices: rows quantised and read back, and products of quantised rows,
// sorted by expert, with each expert's 4-bit weights.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>

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
  long long rows, x_stride;
  int pieces;  // of a row
  float ts;
};

// A block of 16 elements a thread, as in the 4-bit cache's writer.
template <int DT>
__global__ void __launch_bounds__(256) quantize_kernel(const Rows4 a) {
  grid_dep_wait();
  grid_dep_launch();
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, r = i / a.pieces;
  if (r >= a.rows) return;
  float x[16];
  load16<DT>(a.x, r * a.x_stride + (i - r * a.pieces) * 16, x);
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
  const long long i0 = (long long)blockIdx.x * (256 * U) + threadIdx.x, n = a.rows * a.pieces;
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
    const long long r = i / a.pieces, off = r * a.x_stride + (i - r * a.pieces) * E;
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
  a.rows = rows, a.x_stride = rows > 1 ? stride : 0, a.ts = ts;
  const int piece = write ? 16 : dtype == MSK_FP32 ? 4 : 8, per = write ? 256 : 256 * kReadUnroll;
  a.pieces = (int)(cols / piece);
  const OpsLaunch l(dim3((unsigned)((rows * a.pieces + per - 1) / per)), 256, 0, static_cast<cudaStream_t>(stream));
  auto launch = [&](void (*q)(Rows4), void (*d)(Rows4)) { return cudaLaunchKernelEx(&l.cfg, write ? q : d, a); };
  const cudaError_t e = dtype == MSK_BF16   ? launch(quantize_kernel<MSK_BF16>, dequantize_kernel<MSK_BF16>)
                        : dtype == MSK_FP16 ? launch(quantize_kernel<MSK_FP16>, dequantize_kernel<MSK_FP16>)
                                            : launch(quantize_kernel<MSK_FP32>, dequantize_kernel<MSK_FP32>);
  return e == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

constexpr int kM = 128;            // weight rows of a tile (the MMA's M)
constexpr int kStageK = 256;       // columns of a stage
constexpr int kSteps = kStageK / 64;  // MMAs of a stage
constexpr int kMaxN = 224;         // tokens of a tile at most (the MMA's N): two accumulators and the scales fill tensor memory
constexpr int kMaxStages = 10;
constexpr int kMaxE = 1024;
constexpr int kScaleWarps = 4, kEpiWarps = 8;
constexpr int kWarps = 2 + kScaleWarps + kEpiWarps;
constexpr int kProductThreads = 32 * kWarps;
constexpr int kAhead = 4;          // stages whose scales are on their way in registers
constexpr int kACodes = kM * kStageK / 2;
constexpr int kRing = 204 * 1024;  // (dynamic shared memory: beside it 12 KB for the experts' tables and what aligns the ring)
constexpr int kTables = (3 * kMaxE + 4) * 4;
constexpr int kSmem = 1024 + kRing + kTables;
// tensor memory columns: two accumulators, then the scales of a stage's rows and tokens
constexpr int kAccCols = kMaxN, kSfA = 2 * kAccCols, kSfB = kSfA + 4 * kSteps;
static_assert(kSfB + 8 * kSteps <= 512, "tensor memory");

static __device__ uint32_t g_error;  // nonzero once a wait has run out

struct Experts4 {
  CUtensorMap w_map, up_map;  // [E rows][cols / 2] bytes, boxes of 128 x 128 (GLU: of 16 x 128)
  CUtensorMap x_map;          // [x_rows][cols / 2] bytes, boxes of 16 x 128 (gathered: of one row)
  const uint8_t *x_scales, *w_scales, *up_scales;
  const float *w_ts, *up_ts;
  const int32_t *offsets, *slots;
  void* y;
  long long y_stride, x_rows;
  int n, E, rows, K, top_k, y_dtype, nt, stages, mblocks;
  float x_ts;
  bool vec;  // scales in pieces of 16 bytes
};

struct Bars {
  uint64_t full[kMaxStages], sfull[kMaxStages], empty[kMaxStages];
  uint64_t accf[2], acce[2];
  uint64_t done;
};

// Four rows of a 2-D tensor map, one after the other.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int x, const int (&r)[4], uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(dst),
      "l"(map), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A tile: 128 weight rows of an expert and up to nt of its tokens' rows.
struct Tile {
  int e, m;       // expert, block of weight rows
  int p0, count;  // first place and number of places
  int n;          // count, up to the MMA's next N
};

// y^T = W x^T by block-scaled NVFP4 on the fifth-generation tensor cores: M =
// 128 weight rows, N = up to 224 tokens of one expert, K = 64 a step.  Weights
// and tokens come by tiled copies (gathered ones, four rows each, where tokens
// are named by slots), both with the 128-byte swizzle; the scales, row-major in
// memory, by plain loads some stages ahead, written as the tensor cores want
// them.  Tiles run over experts, then blocks of weight rows, then tokens, so that
// neighbouring blocks share weights in L2; a block takes every grid-th one.
// GLU: a tile's rows are 64 gate and 64 up rows, 16 and 16 in turn, so that a
// lane's partner 16 lanes on holds the up value of its gate value.
//
// Roles: a warp that copies, one that issues, four that write scales, eight that
// end the tiles from one of two accumulators while the other fills.
template <bool GLU>
__global__ void __launch_bounds__(kProductThreads, 1) experts4_kernel(const __grid_constant__ Experts4 a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_base;
  __shared__ int abort, never, tiles_all;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // (dynamic shared memory starts at a multiple of 1024 in the shared window)
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t ring = smem_u32(smem);
  int* starts = reinterpret_cast<int*>(smem + kRing);  // [E]: first place of each expert
  int* counts = starts + kMaxE;                         // [E]
  int* ends = counts + kMaxE;                           // [E]: tiles up to and with each expert
  const int chunks = a.nt > 128 ? 2 : 1;                // of tokens' scales, 128 rows each
  const int slot_a = kACodes, slot_b = a.nt * (kStageK / 2), slot_sfa = kM * kStageK / 16;
  const int slot_bytes = slot_a + slot_b + slot_sfa + chunks * 512 * kSteps;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&a.w_map);
    prefetch_tensormap(&a.x_map);
    if (GLU) prefetch_tensormap(&a.up_map);
  }
  if (tid == 32) {
    abort = 0, never = 0;
    for (int i = 0; i < a.stages; ++i)
      mbar_init(bar(bars.full[i]), 1), mbar_init(bar(bars.sfull[i]), kScaleWarps), mbar_init(bar(bars.empty[i]), 1);
    for (int i = 0; i < 2; ++i) mbar_init(bar(bars.accf[i]), 1), mbar_init(bar(bars.acce[i]), kEpiWarps);
    mbar_init(bar(bars.done), 1);
    mbar_fence_init();
    fence_proxy_async_shared();
  }
  if (warp == 2) tmem_alloc(smem_u32(&tmem_base), 512);
  grid_dep_wait();
  grid_dep_launch();

  // The experts' places (whatever the offsets hold, ranges in [0, n] that do not
  // overlap) and tiles.
  if (warp == 0) {
    int at = 0, tiles = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      int first = 0, last = 0;
      if (e < a.E) {
        first = max(0, min(a.n, __ldg(a.offsets + e)));
        last = max(0, min(a.n, __ldg(a.offsets + e + 1)));
      }
      int end = max(first, last);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, end, o);
        if (lane >= o) end = max(end, v);
      }
      const int before = __shfl_up_sync(0xFFFFFFFFu, end, 1);
      first = max(first, lane > 0 ? max(at, before) : at);
      end = max(end, at);
      const int count = max(0, last - first);
      int t = (count + a.nt - 1) / a.nt * a.mblocks;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, t, o);
        if (lane >= o) t += v;
      }
      if (e < a.E) starts[e] = first, counts[e] = count, ends[e] = tiles + t;
      tiles += __shfl_sync(0xFFFFFFFFu, t, 31);
      at = __shfl_sync(0xFFFFFFFFu, end, 31);
    }
    if (lane == 0) tiles_all = tiles;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const int mine = (int)blockIdx.x < tiles_all ? (tiles_all - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x : 0;
  const int kst = (a.K + kStageK - 1) / kStageK;  // stages of a tile
  const uint64_t deadline = gtimer() + kOpsWaitNs + (uint64_t)mine * kst * kOpsStepNs;
  const volatile int* ab = &abort;
  auto wait = [&](uint64_t& b, uint32_t parity) {
    if (mbar_wait(bar(b), parity, deadline, ab)) return true;
    abort = 1;
    return false;
  };
  auto wait_warp = [&](uint64_t& b, uint32_t parity) { return (bool)__all_sync(0xFFFFFFFFu, wait(b, parity)); };
  auto tile_at = [&](int i) {
    const int t = (int)blockIdx.x + i * (int)gridDim.x;
    int lo = 0, hi = a.E - 1;  // the first expert whose tiles go beyond t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ends[mid] > t) hi = mid;
      else lo = mid + 1;
    }
    const int count = counts[lo], nb = (count + a.nt - 1) / a.nt;
    const int local = t - (lo > 0 ? ends[lo - 1] : 0);
    const int m = local / nb, j = local - m * nb;
    const int step = ((count + nb - 1) / nb + 15) & ~15;  // tokens of a tile, the same for all but the last
    Tile r;
    r.e = lo, r.m = m, r.p0 = starts[lo] + j * step, r.count = min(step, count - j * step), r.n = (r.count + 15) & ~15;
    return r;
  };
  // The row of x at a place.
  auto source = [&](int p) {
    if (a.slots == nullptr) return p;
    const int s = __ldg(a.slots + p);
    return max(0, min((int)a.x_rows - 1, (int)((unsigned)max(s, 0) / (unsigned)a.top_k)));
  };

  if (warp == 0) {
    // --- copies ---------------------------------------------------------------
    int st = 0;
    uint32_t ph = 1;  // (a fresh barrier passes a wait for phase 1)
    bool ok = true;
    for (int i = 0; i < mine && ok; ++i) {
      const Tile t = tile_at(i);
      int r[2][4];
      if (a.slots != nullptr) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = 4 * (lane + 32 * u) + j;
            r[u][j] = k < t.count ? source(t.p0 + k) : 0;
          }
      }
      const int wrow = t.e * a.rows + t.m * (GLU ? 64 : kM);
      for (int s = 0; s < kst && ok; ++s) {
        ok = wait_warp(bars.empty[st], ph);
        if (!ok) break;
        const uint32_t dst = ring + st * slot_bytes, b = bar(bars.full[st]);
        const int x = s * (kStageK / 2);
        if (lane == 0) mbar_arrive_expect_tx(b, (uint32_t)(slot_a + t.n * (kStageK / 2)));
        __syncwarp();
        if (GLU) {
          if (lane < 8) tma_load_2d(dst + lane * 2048, lane & 1 ? &a.up_map : &a.w_map, x, wrow + (lane >> 1) * 16, b);
        } else if (lane == 0) {
          tma_load_2d(dst, &a.w_map, x, wrow, b);
        }
        if (a.slots != nullptr) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (4 * (lane + 32 * u) < t.n) tma_gather4(dst + slot_a + (lane + 32 * u) * 512, &a.x_map, x, r[u], b);
        } else if (16 * lane < t.n) {
          tma_load_2d(dst + slot_a + lane * 2048, &a.x_map, x, t.p0 + 16 * lane, b);
        }
        if (++st == a.stages) st = 0, ph ^= 1;
      }
    }
  } else if (warp == 1) {
    // --- MMAs -----------------------------------------------------------------
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int i = 0; i < mine && ok; ++i) {
        const Tile t = tile_at(i);
        const int d = i & 1;
        ok = wait(bars.acce[d], ((i >> 1) & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc = tmem + d * kAccCols, idesc = idesc_mxf4nvf4(t.n);
        const int nc = t.n > 128 ? 2 : 1;
        for (int s = 0; s < kst; ++s) {
          ok = wait(bars.full[st], ph) && wait(bars.sfull[st], ph);
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = ring + st * slot_bytes, sfa = at + slot_a + slot_b, sfb = sfa + slot_sfa;
          const uint64_t ad = umma_desc(at, 16, 1024) | kSwizzle128, bd = umma_desc(at + slot_a, 16, 1024) | kSwizzle128;
          const int steps = min(kSteps, (a.K - s * kStageK) / 64);
          for (int k = 0; k < steps; ++k) {
            tc_cp_sf(tmem + kSfA + 4 * k, umma_desc(sfa + 512 * k, 128, 128));
            tc_cp_sf(tmem + kSfB + 8 * k, umma_desc(sfb + 512 * chunks * k, 128, 128));
            if (nc == 2) tc_cp_sf(tmem + kSfB + 8 * k + 4, umma_desc(sfb + 512 * chunks * k + 512, 128, 128));
            mma_mxf4nvf4(acc, ad + 2 * k, bd + 2 * k, idesc, tmem + kSfA + 4 * k, tmem + kSfB + 8 * k, s > 0 || k > 0);
          }
          tc_commit(bar(bars.empty[st]));
          if (++st == a.stages) st = 0, ph ^= 1;
        }
        if (ok) tc_commit(bar(bars.accf[d]));
      }
      // what is still in flight ends before the block does
      tc_commit(bar(bars.done));
      mbar_wait(bar(bars.done), 0, gtimer() + kOpsWaitNs, &never);
    }
  } else if (warp < 2 + kScaleWarps) {
    // --- scales ---------------------------------------------------------------
    // A thread has a row of the tile and up to two tokens.  Four lanes of a
    // quarter warp's rows, 32 apart, make the 16 bytes that follow each other.
    const int r32 = (warp - 2) * 8 + (lane >> 2), r4 = lane & 3, row = 32 * r4 + r32;
    const int total = mine * kst, pitch = a.K / 16;
    const uint8_t *pa = nullptr, *pb[2] = {nullptr, nullptr};
    int fi = 0, fs = 0;  // tile and stage of the next loads
    uint4 va[kAhead], vb[kAhead][2];
    auto load = [&](const uint8_t* p, int s) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (p == nullptr) return v;
      if (a.vec) return __ldg(reinterpret_cast<const uint4*>(p) + s);
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p) + 4 * s;
      const int left = a.K / 64 - 4 * s;
      v.x = __ldg(q);
      if (left > 1) v.y = __ldg(q + 1);
      if (left > 2) v.z = __ldg(q + 2);
      if (left > 3) v.w = __ldg(q + 3);
      return v;
    };
    auto fetch = [&](uint4& ra, uint4 (&rb)[2]) {
      if (fi >= mine) return;
      if (fs == 0) {
        const Tile t = tile_at(fi);
        int wr = t.m * kM + row;  // the row of the matrix
        const uint8_t* base = a.w_scales;
        if (GLU) {
          wr = t.m * 64 + (row >> 5) * 16 + (row & 15);
          if (row & 16) base = a.up_scales;
        }
        pa = wr < a.rows ? base + ((long long)t.e * a.rows + wr) * pitch : nullptr;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int k = row + 128 * c;
          pb[c] = k < t.count ? a.x_scales + (long long)source(t.p0 + k) * pitch : nullptr;
        }
      }
      ra = load(pa, fs);
      rb[0] = load(pb[0], fs);
      rb[1] = load(pb[1], fs);
      if (++fs == kst) fs = 0, ++fi;
    };
#pragma unroll
    for (int d = 0; d < kAhead; ++d) fetch(va[d], vb[d]);
    int st = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int n0 = 0; n0 < total && ok; n0 += kAhead) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        if (n0 + d >= total || !ok) break;
        ok = wait_warp(bars.empty[st], ph);
        if (!ok) break;
        const uint32_t sfa = ring + st * slot_bytes + slot_a + slot_b + 16 * r32 + 4 * r4, sfb = sfa + slot_sfa;
        const uint32_t wa[4] = {va[d].x, va[d].y, va[d].z, va[d].w};
#pragma unroll
        for (int k = 0; k < kSteps; ++k) sts32(sfa + 512 * k, wa[k]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c >= chunks) break;
          const uint32_t wb[4] = {vb[d][c].x, vb[d][c].y, vb[d][c].z, vb[d][c].w};
#pragma unroll
          for (int k = 0; k < kSteps; ++k) sts32(sfb + 512 * (chunks * k + c), wb[k]);
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bars.sfull[st]));
        fetch(va[d], vb[d]);
        if (++st == a.stages) st = 0, ph ^= 1;
      }
    }
  } else {
    // --- epilogue -------------------------------------------------------------
    const int quad = warp & 3, half = (warp - 2 - kScaleWarps) >> 2;
    bool ok = true;
    for (int i = 0; i < mine && ok; ++i) {
      const Tile t = tile_at(i);
      const int d = i & 1;
      // The tensors' scales: a significand and two halves of a power of two, so
      // that no product leaves fp32's range unless the result does.
      float f[2][2];
#pragma unroll
      for (int u = 0; u < (GLU ? 2 : 1); ++u) {
        const float* p = u ? a.up_ts : a.w_ts;
        const double ts = (double)(p != nullptr ? __ldg(p + t.e) : 1.f) * (double)a.x_ts;
        const int ex = (int)((__double2hiint(ts) >> 20) & 0x7FF);
        if (ex == 0 || ex == 0x7FF) {  // (zero, infinite or NaN)
          f[u][0] = (float)ts, f[u][1] = 1.f;
        } else {
          const int e2 = max(-250, min(250, ex - 1023)), h = e2 / 2;
          f[u][0] = (float)(__hiloint2double((__double2hiint(ts) & 0x800FFFFF) | 0x3FF00000, __double2loint(ts))) * exp2i(h);
          f[u][1] = exp2i(e2 - h);
        }
      }
      ok = wait_warp(bars.accf[d], (i >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16) + d * kAccCols;
      auto store = [&](int c, int row, float v) {
        const long long o = (long long)(t.p0 + c) * a.y_stride + row;
        if (a.y_dtype == MSK_FP32) static_cast<float*>(a.y)[o] = v;
        else if (a.y_dtype == MSK_FP16) static_cast<__half*>(a.y)[o] = __float2half_rn(v);
        else static_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(v);
      };
      for (int c0 = 16 * half; c0 < t.n; c0 += 32) {
        float v[16];
        tmem_ld16(at + c0, v);
        if (!GLU) {
          const int row = t.m * kM + quad * 32 + lane;
          if (row < a.rows) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c0 + j < t.count) store(c0 + j, row, v[j] * f[0][0] * f[0][1]);
          }
        } else {
          // lane l < 16 ends column j, lane l + 16 column j + 1
          const bool up = lane >= 16;
          const int row = t.m * 64 + quad * 16 + (lane & 15);
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const float mine_v = up ? v[j + 1] : v[j], other = __shfl_xor_sync(0xFFFFFFFFu, up ? v[j] : v[j + 1], 16);
            const float g = (up ? other : mine_v) * f[0][0] * f[0][1], u = (up ? mine_v : other) * f[1][0] * f[1][1];
            // silu(g) = g / (1 + e^-g), from e^-|g|, which does not overflow
            const float ex = expf(-fabsf(g)), s = g * ((g >= 0.f ? 1.f : ex) / (1.f + ex));
            if (row < a.rows && c0 + j + up < t.count) store(c0 + j + up, row, s * u);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.acce[d]));
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && abort) {
    atomicExch(&g_error, 1u);
    // copies end before the block does: a slot's newest may be a use ahead of what was waited for
    for (uint32_t q = 0; q < 2; ++q)
      for (int k = 0; k < a.stages; ++k) mbar_wait(bar(bars.full[k]), q, gtimer() + kOpsWaitNs / 100, &never);
  }
}

bool check_experts(const msk_fp4_experts* w, msk_status& s) {
  s = MSK_OK;
  if (w->n_experts < 1 || w->n_experts > kMaxE || w->rows < 0 || w->rows > (1 << 24) || w->cols < 64 || w->cols > (1 << 17) ||
      w->cols % 64 || (int64_t)w->n_experts * w->rows > (1ll << 31) - 256)
    s = MSK_ERR_SHAPE;
  return s == MSK_OK;
}

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

extern "C" msk_status msk_experts_fp4(const msk_nvfp4_desc* x, const int32_t* slots, int32_t top_k, int64_t n,
                                      const int32_t* offsets, const msk_fp4_experts* w, const msk_fp4_experts* up, void* y,
                                      int32_t y_dtype, int64_t y_stride, void* stream) {
  if (x == nullptr || w == nullptr || !dtype_ok(y_dtype) || n < 0) return MSK_ERR_INVALID_ARG;
  msk_status s;
  if (!check_experts(w, s) || (up != nullptr && !check_experts(up, s))) return s;
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
      reinterpret_cast<uintptr_t>(y) % dtype_bytes(y_dtype) ||
      ((reinterpret_cast<uintptr_t>(slots) | reinterpret_cast<uintptr_t>(offsets) | reinterpret_cast<uintptr_t>(w->tensor_scales)) & 3) ||
      (up != nullptr && (reinterpret_cast<uintptr_t>(up->tensor_scales) & 3)))
    return MSK_ERR_ALIGNMENT;
  int nsm = 0;
  s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  Experts4 a{};
  a.x_scales = x->scales, a.w_scales = w->scales, a.w_ts = w->tensor_scales;
  if (up != nullptr) a.up_scales = up->scales, a.up_ts = up->tensor_scales;
  a.offsets = offsets, a.slots = slots, a.y = y, a.y_stride = n > 1 ? y_stride : 0, a.x_rows = x->rows;
  a.n = (int)n, a.E = w->n_experts, a.rows = (int)w->rows, a.K = (int)w->cols, a.top_k = top_k, a.y_dtype = y_dtype;
  a.x_ts = x->tensor_scale;
  a.vec = a.K % kStageK == 0;
  a.mblocks = (a.rows + (up != nullptr ? 64 : kM) - 1) / (up != nullptr ? 64 : kM);
  a.nt = (int)std::min<int64_t>(kMaxN, (n + 15) / 16 * 16);
  const long long tiles = (long long)a.mblocks * ((n + a.nt - 1) / a.nt + std::min<int64_t>(n, a.E));  // at most
  if (tiles > (1ll << 31) - 1 - 65536) return MSK_ERR_SHAPE;
  const int slot = kACodes + a.nt * (kStageK / 2) + kM * kStageK / 16 + (a.nt > 128 ? 2 : 1) * 512 * kSteps;
  a.stages = std::min(kMaxStages, kRing / slot);
  const CUtensorMapDataType bytes = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const long long wrows = (long long)a.E * a.rows;
  const int box = up != nullptr ? 16 : kM;
  if (!matrix_map(&a.w_map, bytes, w->packed, wrows, a.K / 2, a.K / 2, box, kStageK / 2, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (up != nullptr && !matrix_map(&a.up_map, bytes, up->packed, wrows, a.K / 2, a.K / 2, box, kStageK / 2, CU_TENSOR_MAP_SWIZZLE_128B)) ||
      !matrix_map(&a.x_map, bytes, x->packed, x->rows, a.K / 2, a.K / 2, slots != nullptr ? 1 : 16, kStageK / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return MSK_ERR_CUDA;
  static std::atomic<bool> ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MSK_ERR_CUDA;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(experts4_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
        cudaFuncSetAttribute(experts4_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
      return MSK_ERR_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  const OpsLaunch l(dim3((unsigned)std::min<long long>(nsm, tiles)), kProductThreads, kSmem, static_cast<cudaStream_t>(stream));
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, up != nullptr ? experts4_kernel<true> : experts4_kernel<false>, a);
  return e == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}
