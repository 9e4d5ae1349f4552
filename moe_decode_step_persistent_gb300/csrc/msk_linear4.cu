// Products of up to 16 rows of 16-bit activations with NVFP4 weights.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "msk_internal.h"
#include "msk_ops.cuh"
#include "msk_tc.cuh"

namespace msk {
namespace {

constexpr int kGroup = 256;        // columns of a stage
constexpr int kRows = 128;         // weight rows of a tile (the MMA's M)
constexpr int kTeams = 4;          // take the stages in turn; 4 warps of 32 rows each
constexpr int kDeqWarps = 4 * kTeams;
constexpr int kThreads = 32 * (kDeqWarps + kTeams);  // ... and a warp a team that issues its MMAs
constexpr int kABufs = 3;          // decoded operands of a team in tensor memory
constexpr int kMaxStages = 2 * kTeams;  // kTeams or twice as many: a slot is a team's own, so that the team sees each of its phases
// x in shared memory: for every 64 columns NG groups of 8 tokens x 128 bytes,
// swizzled.
template <int NG>
constexpr int kXBytes = NG * 1024;
constexpr int kChunks = kGroup / 64;  // decoded operands of a stage
constexpr int kCodeBytes = kRows * kGroup / 2, kScaleBytes = kRows * kGroup / 16, kStageBytes = kCodeBytes + kScaleBytes;
constexpr int kMaxKs = 8;          // blocks of a cluster along the columns
constexpr int kSmem = 224 * 1024;  // (dynamic; 3 KB of the block's 227 are static or aligned away)
// Partial sums from the cluster's blocks, two tiles: units of a token's 32 rows
// that this block adds up, a slot for each block.
constexpr int kUnits = 16 * kRows / 32, kPartFloats = (kUnits + kMaxKs) * 32, kPartBytes = 2 * kPartFloats * 4;
// tensor memory columns: decoded operands, then two sets of accumulators
constexpr int kACols = 32, kDCols = 16, kD0 = kTeams * kABufs * kACols;

static __device__ uint32_t g_error;  // nonzero once a wait has run out

struct Lin4 {
  CUtensorMap codes_map;   // [rows][cols / 2] bytes, boxes of 128 x 128
  CUtensorMap scales_map;  // [rows][cols / 16] bytes, boxes of 128 x 16 (cols a multiple of 256)
  CUtensorMap x_map;       // [cols / 64][tokens][64], boxes of 4 x 8 NG x 64
  const uint8_t* scales;
  void* y;
  long long x_stride, y_stride, N;
  int K, T, y_dtype, groups, ks, stages;
  bool fp16, scales_tma;
  float ts;    // the tensor's scale: its significand ...
  int ts_exp;  // ... and the power of two that it is multiplied with
};

struct Bars {  // mbarriers of a block
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t afull[kTeams][kABufs], aempty[kTeams][kABufs];
  uint64_t dfull[2], dempty[2];
  uint64_t parts[2], pfree[2];  // the cluster's partial sums of a tile are there; have been read in every block
  uint64_t xfull;
  uint64_t done[kTeams];  // an issuer's MMAs are complete
};

// y^T = W x^T on the fifth-generation tensor cores: M = 128 weight rows, N =
// 16 tokens, fp16 operands, fp32 accumulators.  The weights stream through
// shared memory by tiled copies and are decoded, exactly, into the A operand
// in tensor memory: a thread takes 64 columns of a row, a conversion and a
// multiply by the block scale for two weights.  x lies in shared memory as
// the B operand for the block's life.
//
// Roles: 16 decoding warps in four teams that take the stages in turn (a
// thread has a row's 256 columns of a stage, 64 at a time) and for each team a
// warp that issues its MMAs and refills the slots that it has read.
// (One thread issues an MMA in 55 cycles, four threads one in 16 each; a
// stage's bytes leave 49 for each of its 16.)  Everything between the roles is
// an mbarrier; a team's sums lie in an accumulator of their own and are added
// in the epilogue, which reads tile i while tile i + 1 is decoded.
//
// 131072 x 4096: 60 us for 16 tokens, 58 for one (5.1 TB/s, 76% of what a copy
// reaches).  Bound by the decoding and DRAM alike: issue slots are 64% in use,
// the ALU that converts 55%.  On mma.sync the decoding and the MMAs together
// take longer than the bytes (88 us for 16 tokens).
//
// With too few tiles for the GPU, or more columns than x has room for, a
// cluster of `ks` blocks shares a tile's columns and adds its sums up in rank
// order, each block a share of the tile that the others store into its shared
// memory (reading them there instead, behind fences: 1 us more for one tile).
// NG: 8-token groups that x has room for; CL: blocks share tiles in clusters.
template <int NG, bool CL>
__global__ void __launch_bounds__(kThreads, 1) linear4_kernel(const __grid_constant__ Lin4 a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ uint32_t amaxs[16];  // each token's largest magnitude, as an fp32 number's bits
  // undo each token's scaling and apply the tensor's: two factors, a half of the
  // power of two each, so that no product leaves fp32's range unless the result does
  __shared__ float2 back[16];
  __shared__ uint32_t tmem_base;
  __shared__ int abort, never;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ks = CL ? a.ks : 1;
  const int rank = blockIdx.x % ks, clusters = gridDim.x / ks, cluster = blockIdx.x / ks;
  const int ga = a.groups * rank / ks, gb = a.groups * (rank + 1) / ks, ng = gb - ga;  // (at most 128 groups)
  const int tiles = (int)((a.N + kRows - 1) / kRows);
  const int mine = cluster < tiles ? (tiles - cluster + clusters - 1) / clusters : 0;
  uint64_t deadline;
  // (dynamic shared memory starts at a multiple of 1024 in the shared window)
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t ring = smem_u32(smem);
  uint8_t* xs = smem + a.stages * kStageBytes;
  float* parts = reinterpret_cast<float*>(xs + ((a.groups + ks - 1) / ks) * kChunks * kXBytes<NG>);  // clusters only
  auto bar = [](uint64_t& b) { return smem_u32(&b); };

  // (what the cluster's blocks have stored)
  auto wait_parts = [&](uint64_t& b, uint32_t parity) {
    bool ok = false;
    for (uint32_t spins = 1; !(ok = mbar_try_wait_cluster(bar(b), parity)); ++spins)
      if (spins % 64 == 0 && (*(const volatile int*)&abort || gtimer() > deadline)) break;
    if (!ok) abort = 1;
    return (bool)__all_sync(0xFFFFFFFFu, ok);
  };

  if (warp == kDeqWarps && lane == 0) {
    prefetch_tensormap(&a.x_map);
    prefetch_tensormap(&a.codes_map);
    if (a.scales_tma) prefetch_tensormap(&a.scales_map);
    for (int i = 0; i < a.stages; ++i) mbar_init(bar(bars.full[i]), 1), mbar_init(bar(bars.empty[i]), 4);
    mbar_init(bar(bars.xfull), 1);
    mbar_fence_init();
    fence_proxy_async_shared();
  }
  if (tid == 0) {
    abort = 0, never = 0;
    for (int t = 0; t < kTeams; ++t) {
      for (int i = 0; i < kABufs; ++i) mbar_init(bar(bars.afull[t][i]), 4), mbar_init(bar(bars.aempty[t][i]), 1);
      mbar_init(bar(bars.done[t]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(bars.dfull[i]), kTeams), mbar_init(bar(bars.dempty[i]), kDeqWarps);
      mbar_init(bar(bars.parts[i]), 1), mbar_init(bar(bars.pfree[i]), kDeqWarps * ks);
    }
    mbar_fence_init();
  }
  if (tid < 16) amaxs[tid] = 0;
  if (warp == 0) tmem_alloc(smem_u32(&tmem_base), 512);
  grid_dep_wait();
  grid_dep_launch();
  deadline = gtimer() + kOpsWaitNs + (uint64_t)mine * ng * kOpsStepNs;

  // --- copies ---------------------------------------------------------------
  const int total = mine * ng;  // stages in all
  auto load = [&](int st, int ti, int g) {
    const uint32_t dst = ring + st * kStageBytes, b = bar(bars.full[st]);
    const int row = (cluster + ti * clusters) * kRows;
    mbar_arrive_expect_tx(b, a.scales_tma ? kStageBytes : kCodeBytes);
    tma_load_2d(dst, &a.codes_map, (ga + g) * (kGroup / 2), row, b);
    if (a.scales_tma) tma_load_2d(dst + kCodeBytes, &a.scales_map, (ga + g) * (kGroup / 16), row, b);
  };
  if (warp == kDeqWarps && lane == 0) {  // under way before the block has met
    // x first: behind the ring's copies it would wait for all of them
    mbar_arrive_expect_tx(bar(bars.xfull), ng * kChunks * kXBytes<NG>);
    for (int g = 0; g < ng; ++g)
      asm volatile(
          "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
              smem_u32(xs) + g * kChunks * kXBytes<NG>),
          "l"(&a.x_map), "r"(0), "r"(0), "r"((ga + g) * kChunks), "r"(bar(bars.xfull))
          : "memory");
    for (int i = 0; i < min(total, a.stages); ++i) load(i, i / ng, i % ng);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (CL) cluster_arrive();  // (waited for below: the others' barriers are set up)
  const uint32_t tmem = tmem_base;
  const volatile int* ab = &abort;
  auto wait = [&](uint64_t& b, uint32_t parity) {
    if (mbar_wait(bar(b), parity, deadline, ab)) return true;
    abort = 1;
    return false;
  };

  auto wait_warp = [&](uint64_t& b, uint32_t parity) { return (bool)__all_sync(0xFFFFFFFFu, wait(b, parity)); };

  // --- x in place: scaled by a power of two for each token, fp16 ---------------
  if (warp < kDeqWarps && total > 0) {
    wait_warp(bars.xfull, 0);
    // items: 256 columns of a token, token by token; a warp takes a run of them
    const int items = a.T * ng, per = (items + kDeqWarps - 1) / kDeqWarps, i1 = min(items, (warp + 1) * per);
    auto piece = [&](int t, int g) {  // this lane's 8 columns
      const int k8 = g * 32 + lane;
      return reinterpret_cast<uint4*>(xs + (k8 >> 3) * kXBytes<NG> + t * 128 + (((k8 ^ t) & 7) << 4));
    };
    if (!a.fp16) {
      for (int it = warp * per; it < i1;) {
        const int t = it / ng, g0 = it - t * ng, n = min(ng - g0, i1 - it);
        uint32_t m = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
          const uint4 v = *piece(t, g0 + j);
          asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(v.x & 0x7FFF7FFFu));
          asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(v.y & 0x7FFF7FFFu));
          asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(v.z & 0x7FFF7FFFu));
          asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(v.w & 0x7FFF7FFFu));
        }
        const uint32_t f = __float_as_uint(fmaxf(fmaxf(bf16_lo(m), bf16_hi(m)), 0.f));  // (a NaN does not count)
        const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, f);
        if (lane == 0) atomicMax(&amaxs[t], w);
        it += n;
      }
      named_bar(1, 32 * kDeqWarps);
      for (int it = warp * per; it < i1;) {
        const int t = it / ng, g0 = it - t * ng, n = min(ng - g0, i1 - it);
        const float mul = exp2i(row_shift(__uint_as_float(amaxs[t])));
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
          uint4* p = piece(t, g0 + j);
          const uint4 v = *p;
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = pack_f16x2(bf16_lo(w[i]) * mul, bf16_hi(w[i]) * mul);
          *p = make_uint4(w[0], w[1], w[2], w[3]);
        }
        it += n;
      }
      fence_proxy_async_shared();
    }
    if (tid < 16) {
      // (below -252 every sum, at most 2^41, ends in 0 all the same)
      const int e = max(a.ts_exp - (a.fp16 ? 0 : row_shift(__uint_as_float(amaxs[tid]))), -252), half = e / 2;
      back[tid] = make_float2(a.ts * exp2i(half), exp2i(e - half));
    }
  }
  __syncthreads();
  if (CL) cluster_wait();

  if (warp < kDeqWarps) {
    // --- decoding and epilogue ----------------------------------------------
    const int team = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t tlane = tmem + ((uint32_t)(quad * 32) << 16);
    // adds the teams' sums up for four tokens of this warp's rows and stores them
    auto epilogue = [&](int i) {
      const int d = i & 1;
      if (!wait_warp(bars.dfull[d], (i >> 1) & 1)) return false;
      tc_fence_after();
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < kTeams; ++t) {
        if (((t - i * ng) & (kTeams - 1)) >= ng) continue;  // (this team had none of the tile's stages)
        float v[4];
        tmem_ld4(tlane + kD0 + (d * kTeams + t) * kDCols + team * 4, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] += v[j];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.dempty[d]));
      const long long n0 = (long long)(cluster + (long long)i * clusters) * kRows;
      auto store = [&](int t, long long n, float v) {
        const long long o = t * a.y_stride + n;
        if (a.y_dtype == MSK_FP32) static_cast<float*>(a.y)[o] = v;
        else if (a.y_dtype == MSK_FP16) static_cast<__half*>(a.y)[o] = __float2half_rn(v);
        else static_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(v);
      };
      if (!CL) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = team * 4 + j;
          if (t < a.T && n0 + r < a.N) store(t, n0 + r, s[j] * back[t].x * back[t].y);
        }
        return true;
      }
      // Unit u = 4 token + quarter of the rows is added up by block u mod ks.
      // The sums go there by asynchronous stores that its barrier counts.
      const int units = 4 * a.T, owned = units > rank ? (units - rank + ks - 1) / ks : 0;
      if (tid == 0 && owned > 0) mbar_arrive_expect_tx(bar(bars.parts[d]), (uint32_t)(owned * ks * 128));
      if (i >= 2 && !wait_warp(bars.pfree[d], ((i >> 1) - 1) & 1)) return false;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = team * 4 + j, u = 4 * t + quad, to = u % ks;
        if (t < a.T)
          st_async(mapa(smem_u32(parts + d * kPartFloats + (u / ks * ks + rank) * 32 + lane), to), s[j] * back[t].x * back[t].y,
                   mapa(bar(bars.parts[d]), to));
      }
      if (owned > 0 && !wait_parts(bars.parts[d], (i >> 1) & 1)) return false;
      for (int k = warp; k < owned; k += kDeqWarps) {
        const int u = k * ks + rank, rr = (u & 3) * 32 + lane;
        const float* f = parts + d * kPartFloats + k * ks * 32 + lane;
        float v = 0.f;
        for (int b = 0; b < ks; ++b) v += f[b * 32];
        if (n0 + rr < a.N) store(u >> 2, n0 + rr, v);
      }
      if (i + 2 < mine) {  // the place is written again for tile i + 2
        __syncwarp();
        if (lane < ks) mbar_arrive_cluster(mapa(bar(bars.pfree[d]), lane));
      }
      return true;
    };

    int buf = 0, tile = 0, g = team, done = 0;  // (g: the team's next stage, counted from the tile's first one)
    uint32_t aph = 1;                           // (a fresh barrier passes a wait for phase 1)
    bool ok = true;
    int st = team;
    uint32_t ph = 0;
    for (int n = team; n < total && ok; n += kTeams) {
      for (; g >= ng; g -= ng) ++tile;
      // a tile behind: its MMAs are over by now, and the next but one tile's
      // wait for nothing else
      while (ok && done + 1 < tile) ok = epilogue(done++);
      uint4 e = make_uint4(0, 0, 0, 0);
      if (!a.scales_tma) {
        const long long row = (long long)(cluster + (long long)tile * clusters) * kRows + r;
        const int col = (ga + g) * kGroup;
        const uint2* p = reinterpret_cast<const uint2*>(a.scales + row * (a.K / 16) + col / 16);
        if (row < a.N) {
          const uint2 lo = __ldg(p);
          e.x = lo.x, e.y = lo.y;
          if (col + 128 < a.K) {
            const uint2 hi = __ldg(p + 1);
            e.z = hi.x, e.w = hi.y;
          }
        }
      }
      ok = ok && wait_warp(bars.full[st], ph);
      if (!ok) break;
      const uint32_t s = ring + st * kStageBytes;
      uint4 c[8];  // this thread's row: 256 codes, piece p of 16 bytes at p ^ (row mod 8)
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = lds128(s + r * 128 + ((j ^ (r & 7)) << 4));
      if (a.scales_tma) e = lds128(s + kCodeBytes + r * 16);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.empty[st]));
      const uint32_t es[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const uint32_t w[8] = {c[2 * k].x, c[2 * k].y, c[2 * k].z, c[2 * k].w, c[2 * k + 1].x, c[2 * k + 1].y, c[2 * k + 1].z, c[2 * k + 1].w};
        uint32_t v[32];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t f = f16x2_bcast(e4m3_pair_to_f16x2(es[k], b >> 1), b & 1);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[b * 8 + j] = hmul2(e2m1_byte_to_f16x2(w[2 * b + (j >> 2)], j & 3), f);
        }
        ok = ok && wait_warp(bars.aempty[team][buf], aph);
        if (!ok) break;
        tc_fence_after();
        tmem_st32(tlane + (team * kABufs + buf) * kACols, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bars.afull[team][buf]));
        if (++buf == kABufs) buf = 0, aph ^= 1;
      }
      g += kTeams;
      st += kTeams;
      if (st >= a.stages) st = team, ph ^= 1;
    }
    while (ok && done < mine) ok = epilogue(done++);
  } else if (lane == 0) {
    // --- a team's MMAs, and the copies into the slots that it leaves ---------------
    const int team = warp - kDeqWarps;
    // (8 tokens: the MMA's second group of 8 reads the first one again)
    const uint64_t b0 = umma_desc(smem_u32(xs), 16, NG == 2 ? 1024 : 0) | kSwizzle128;
    int buf = 0, tile = 0, g = team, st = team;
    int rt = (team + a.stages) / ng, rg = (team + a.stages) % ng;  // the stage that goes where the team's next one was
    uint32_t ph = 0, sph = 0;
    constexpr uint32_t idesc = (1u << 4) | ((16u / 8) << 17) | ((128u / 16) << 24);  // fp32 += fp16 fp16, N = 16, M = 128
    const uint32_t afull = bar(bars.afull[team][0]), aempty = bar(bars.aempty[team][0]);
    const uint32_t at0 = tmem + team * kABufs * kACols;
    bool ok = wait(bars.dempty[0], 1), fresh = true;  // (fresh: the tile's sums start from nothing)
    for (int n = team; n < total && ok; n += kTeams) {
      for (; g >= ng && ok; g -= ng) {
        tc_commit(bar(bars.dfull[tile & 1]));
        ++tile, fresh = true;
        ok = wait(bars.dempty[tile & 1], ((tile >> 1) & 1) ^ 1);
      }
      if (ok && n + a.stages < total) {  // as soon as the team has read the stage: its next one
        ok = wait(bars.empty[st], sph);
        if (ok) load(st, rt, rg);
      }
      if (!ok) break;
      const uint32_t dt = tmem + kD0 + ((tile & 1) * kTeams + team) * kDCols;
      const uint64_t b = b0 + g * (kChunks * kXBytes<NG> >> 4);
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        if (!mbar_try_wait(afull + buf * 8, ph) && !(ok = wait(bars.afull[team][buf], ph))) break;
        tc_fence_after();
        const uint32_t at = at0 + buf * kACols;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_f16_ts(dt, at + j * 8, b + k * (kXBytes<NG> >> 4) + j * 2, idesc, k > 0 || j > 0 || !fresh);
        tc_commit(aempty + buf * 8);
        buf = buf == kABufs - 1 ? 0 : buf + 1;
        ph ^= buf == 0;
      }
      fresh = false;
      g += kTeams;
      st += kTeams;
      if (st >= a.stages) st = team, sph ^= 1;
      for (rg += kTeams; rg >= ng; rg -= ng) ++rt;
    }
    for (; tile < mine && ok; ++tile) {
      if (tile > 0 && g < 0) ok = wait(bars.dempty[tile & 1], ((tile >> 1) & 1) ^ 1);
      if (ok) tc_commit(bar(bars.dfull[tile & 1]));
      g = -1;
    }
    // what is still in flight ends before the block does
    tc_commit(bar(bars.done[team]));
    mbar_wait(bar(bars.done[team]), 0, gtimer() + kOpsWaitNs, &never);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && abort) {
    atomicExch(&g_error, 1u);
    // copies too (no issuer starts one any more): a slot's newest may be a use ahead
    // of what was waited for
    for (uint32_t q = 0; q < 2; ++q) {
      mbar_wait(bar(bars.xfull), q, gtimer() + kOpsWaitNs / 100, &never);
      for (int k = 0; k < a.stages; ++k) mbar_wait(bar(bars.full[k]), q, gtimer() + kOpsWaitNs / 100, &never);
    }
  }
  if (CL) {
    __syncwarp();
    cluster_sync();  // (no block leaves while others may store into it)
    if (tid == 0 && abort)  // (sums that this block has not waited for may still be on their way)
      for (const uint64_t end = gtimer() + kOpsWaitNs / 100; gtimer() < end;) __nanosleep(1000);
  }
}

// What the kernel's launches go by, looked up once a device: clusters of each
// size that run at a time.
struct Setup {
  std::once_flag once;
  bool ok = false;
  int active[kMaxKs + 1] = {};
};

template <int NG, bool CL>
bool look_up(Setup& s, int from, int to) {
  if (cudaFuncSetAttribute(linear4_kernel<NG, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return false;
  for (int ks = from; ks <= to; ++ks) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3((unsigned)ks), cfg.blockDim = dim3(kThreads), cfg.dynamicSmemBytes = kSmem;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)ks, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at, cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&s.active[ks], linear4_kernel<NG, CL>, &cfg) != cudaSuccess || s.active[ks] < 1) return false;
  }
  return true;
}

template <int NG>
const Setup* setup() {
  static Setup devices[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  Setup& s = devices[dev];
  std::call_once(s.once, [&s] { s.ok = look_up<NG, false>(s, 1, 1) && look_up<NG, true>(s, 2, kMaxKs); });
  return s.ok ? &s : nullptr;
}

template <int NG>
msk_status launch_linear(Lin4& a, const void* x, long long x_stride, cudaStream_t st) {
  const Setup* su = setup<NG>();
  if (su == nullptr) return MSK_ERR_CUDA;
  // Blocks along the columns: as many as x's room asks for, and more while
  // all of a wave's clusters still run at once (two stages or more a block):
  // 1 x 4096 x 4096 8.9 us, with one block a tile 13.0 (both before early starts).
  const int room = (kSmem - 1024 - kPartBytes - kTeams * kStageBytes) / (kChunks * kXBytes<NG>);  // groups of a block
  const int tiles = (int)((a.N + kRows - 1) / kRows);
  a.ks = (a.groups + room - 1) / room;
  while (a.ks < kMaxKs && tiles <= su->active[a.ks + 1] && a.groups >= 2 * (a.ks + 1)) ++a.ks;
  const int per = (a.groups + a.ks - 1) / a.ks;
  // x as [cols / 64][tokens][64]; a box is a stage's columns
  const cuuint64_t xd[3] = {64, (cuuint64_t)a.T, (cuuint64_t)a.K / 64}, xp[2] = {(cuuint64_t)(a.T > 1 ? x_stride : a.K) * 2, 128};
  const cuuint32_t xb[3] = {64, 8 * NG, kChunks}, es[3] = {1, 1, 1};
  if (tensor_map_encoder()(&a.x_map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(x), xd, xp, xb, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return MSK_ERR_CUDA;
  const int xbytes = per * kChunks * kXBytes<NG>, pbytes = a.ks > 1 ? kPartBytes : 0;
  // (two slots a team where there is room: 8 x 65536 x 4096 36.5 us, with one 37.5)
  a.stages = (kSmem - 1024 - pbytes - xbytes) / kStageBytes >= kMaxStages ? kMaxStages : kTeams;
  const OpsLaunch l(dim3((unsigned)(std::min(tiles, su->active[a.ks]) * a.ks)), kThreads, 1024 + a.stages * kStageBytes + xbytes + pbytes, st,
                    a.ks);
  const cudaError_t e = a.ks > 1 ? cudaLaunchKernelEx(&l.cfg, linear4_kernel<NG, true>, a) : cudaLaunchKernelEx(&l.cfg, linear4_kernel<NG, false>, a);
  return e == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}

}  // namespace

cudaError_t kv4_error(uint32_t* e);       // (msk_kv4.cu)
cudaError_t experts4_error(uint32_t* e);  // (msk_experts4.cu)

cudaError_t linear4_error(uint32_t* e) {
  cudaError_t r = cudaMemcpyFromSymbol(e, g_error, sizeof(*e));
  const uint32_t zero = 0;
  if (r == cudaSuccess && *e != 0) r = cudaMemcpyToSymbol(g_error, &zero, sizeof(zero));
  return r;
}

}  // namespace msk

using namespace msk;

extern "C" msk_status msk_linear_fp4(const void* x, int32_t x_dtype, int64_t x_stride, const msk_nvfp4_desc* w,
                                     int32_t tokens, void* y, int32_t y_dtype, int64_t y_stride, void* stream) {
  if (w == nullptr || (x_dtype != MSK_BF16 && x_dtype != MSK_FP16) || !dtype_ok(y_dtype)) return MSK_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > kMaxT || w->rows < 0 || w->rows > (1ll << 31) - kRows || w->cols <= 0 || w->cols % 128 ||
      w->cols > 32768)
    return MSK_ERR_SHAPE;
  if (tokens == 0 || w->rows == 0) return MSK_OK;
  if (x == nullptr || y == nullptr || w->packed == nullptr || w->scales == nullptr) return MSK_ERR_INVALID_ARG;
  if (tokens > 1 && (x_stride < w->cols || y_stride < w->rows)) return MSK_ERR_INVALID_ARG;
  if (!ops_aligned16(x) || x_stride % 8 || !ops_aligned16(w->packed) || !ops_aligned16(w->scales) ||
      reinterpret_cast<uintptr_t>(y) % dtype_bytes(y_dtype))
    return MSK_ERR_ALIGNMENT;
  int nsm = 0;
  const msk_status s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  Lin4 a{};
  a.scales = w->scales, a.y = y;
  a.y_stride = y_stride, a.N = w->rows, a.K = (int)w->cols, a.T = tokens;
  a.y_dtype = y_dtype, a.fp16 = x_dtype == MSK_FP16;
  a.ts = w->tensor_scale;
  if (std::isfinite(a.ts) && a.ts != 0.f) a.ts = 2.f * std::frexp(a.ts, &a.ts_exp), --a.ts_exp;  // [1, 2)
  a.groups = (a.K + kGroup - 1) / kGroup;
  // (a tiled copy's rows lie a multiple of 16 bytes apart: with an odd
  // multiple of 128 columns the scales' do not, and are loaded one by one)
  a.scales_tma = a.K % kGroup == 0;
  const CUtensorMapDataType bytes = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!matrix_map(&a.codes_map, bytes, w->packed, a.N, a.K / 2, a.K / 2, kRows, kGroup / 2, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (a.scales_tma && !matrix_map(&a.scales_map, bytes, w->scales, a.N, a.K / 16, a.K / 16, kRows, kGroup / 16,
                                   CU_TENSOR_MAP_SWIZZLE_NONE)))
    return MSK_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // (up to 8 tokens x takes half the room: 8 x 65536 x 4096 36.5 us, with room for 16 38.2)
  return tokens <= 8 ? launch_linear<1>(a, x, x_stride, st) : launch_linear<2>(a, x, x_stride, st);
}

extern "C" msk_status msk_ops_check(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return MSK_ERR_CUDA;
  uint32_t e = 0, f = 0, g = 0;
  if (linear4_error(&e) != cudaSuccess || kv4_error(&f) != cudaSuccess || experts4_error(&g) != cudaSuccess) return MSK_ERR_CUDA;
  return e || f || g ? MSK_ERR_TIMEOUT : MSK_OK;
}
