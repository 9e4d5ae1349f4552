// A prompt's tokens to their experts and back: the router's choice, the slots
// sorted by expert, and the experts' outputs weighted and summed at their tokens.
#include <algorithm>
#include <atomic>

#include "msk_internal.h"
#include "msk_ops.cuh"

namespace msk {
namespace {

// ---------------------------------------------------------------------------
// route: the top_k greatest of logits + bias, and their softmax
// ---------------------------------------------------------------------------

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;

struct Route {
  const void* logits;
  const float* bias;
  int32_t* experts;
  float* gates;
  long long tokens, ld;
  int E, top_k;
};

// An fp32 number's bits in an order that unsigned comparison follows, and back.
// Two zeros of either sign are one (x + 0 is +0), a NaN is below everything.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  if (x != x) return 0u;
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float ordered_value(uint32_t k) {
  return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k);
}
constexpr uint32_t kMinusInf = 0x007FFFFFu;  // ordered(-inf): an expert up to here is barred

template <int DT>
__device__ __forceinline__ float element(const void* p, long long i) {
  if (DT == MSK_FP32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t v = __ldg(static_cast<const uint16_t*>(p) + i);
  return DT == MSK_FP16 ? __half2float(__ushort_as_half(v)) : __uint_as_float((uint32_t)v << 16);
}

// A warp a token, C candidates a lane: lane l's are experts C l .. C l + C - 1,
// so that of equal logits the lowest lane, and in a lane the first, is the lowest
// index.  A round takes the warp's greatest key; its lane goes on to its next, of
// which it has three at hand (that a lane has a fourth among 8 chosen ones of 256
// happens once in 700 tokens).  Which of a lane's candidates they were is
// found out at the end, for all ranks at once.
template <int DT, int C, bool VEC>
__global__ void __launch_bounds__(128) route_kernel(const Route a) {
  constexpr int S = DT == MSK_FP32 ? 4 : 2;
  const int lane = threadIdx.x & 31, e0 = lane * C;
  grid_dep_wait();
  grid_dep_launch();
  float bias[C];
#pragma unroll
  for (int j = 0; j < C; ++j) bias[j] = a.bias != nullptr && e0 + j < a.E ? __ldg(a.bias + e0 + j) : 0.f;
  for (long long t = (long long)blockIdx.x * 4 + (threadIdx.x >> 5); t < a.tokens; t += (long long)gridDim.x * 4) {
    uint32_t key[C];
    if (VEC && e0 + C <= a.E) {
      constexpr int W = C * S / 4;  // 32-bit words
      uint32_t w[W];
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(a.logits) + (t * a.ld + e0) * S);
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const uint4 u = __ldg(p + i);
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
      }
#pragma unroll
      for (int j = 0; j < C; ++j) {
        float x;
        if (DT == MSK_FP32) x = __uint_as_float(w[j % W]);
        else {
          const float2 f = unpack16(w[j / 2], DT == MSK_FP16);
          x = j & 1 ? f.y : f.x;
        }
        key[j] = ordered(x + bias[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j) key[j] = e0 + j < a.E ? ordered(element<DT>(a.logits, t * a.ld + e0 + j) + bias[j]) : 0u;
    }
    uint32_t best[3] = {0u, 0u, 0u};
    auto enter = [&](uint32_t k) {
      const uint32_t x = min(best[0], k), y = min(best[1], x);
      best[0] = max(best[0], k), best[1] = max(best[1], x), best[2] = max(best[2], y);
    };
#pragma unroll
    for (int j = 0; j < C; ++j) enter(key[j]);
    uint32_t mine = 0u;      // lane r: the key of rank r,
    int from = 0, skip = 0;  // the lane that has it, and which of its keys like that
    uint32_t last = 0u;      // this lane's last key that has won,
    int won = 0, same = 0;   // ranks of this lane's, of those like that
    int ranks = a.top_k;
    for (int r = 0; r < a.top_k; ++r) {
      const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best[0]);
      if (m <= kMinusInf) {  // (uniform: none is left)
        ranks = r;
        break;
      }
      const int win = __ffs(__ballot_sync(0xFFFFFFFFu, best[0] == m)) - 1;
      const int next = m == last ? same + 1 : 0, of = __shfl_sync(0xFFFFFFFFu, next, win);
      if (lane == r) mine = m, from = win, skip = of;
      if (lane == win) {
        last = m, same = next, ++won;
        best[0] = best[1], best[1] = best[2], best[2] = 0u;
        if (won % 3 == 0) {  // three are used up: those behind the ones that have won
          int like = same + 1;  // of the keys like the last, this many have
          best[0] = 0u;
#pragma unroll
          for (int j = 0; j < C; ++j) {
            if (key[j] < m || (key[j] == m && --like < 0)) enter(key[j]);
          }
        }
      }
    }
    // lane r: which of lane `from`'s keys; of several like it, the one behind those of earlier ranks
    const bool in = lane < ranks;
    int chosen = -1;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t k = __shfl_sync(0xFFFFFFFFu, key[j], from);
      if (k == mine && skip-- == 0) chosen = from * C + j;
    }
    if (!in) chosen = -1;
    // the softmax of the chosen, in their order of rank
    const float v = ordered_value(mine), v0 = __shfl_sync(0xFFFFFFFFu, v, 0);
    float e = in ? expf(v - v0) : 0.f, sum = e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane < a.top_k) {
      a.experts[t * a.top_k + lane] = chosen;
      a.gates[t * a.top_k + lane] = in ? e / sum : 0.f;
    }
  }
}

template <int DT, int C>
cudaError_t launch_route(const Route& a, bool aligned, int nsm, cudaStream_t st) {
  // (as many blocks as run at once: a warp goes on with its bias in registers)
  const OpsLaunch l(dim3((unsigned)std::min<long long>((a.tokens + 3) / 4, nsm * 16)), 128, 0, st);
  if (C * (DT == MSK_FP32 ? 4 : 2) % 16 == 0 && aligned)
    return cudaLaunchKernelEx(&l.cfg, route_kernel<DT, C, C * (DT == MSK_FP32 ? 4 : 2) % 16 == 0>, a);
  return cudaLaunchKernelEx(&l.cfg, route_kernel<DT, C, false>, a);
}

template <int DT>
cudaError_t launch_route(const Route& a, bool aligned, int nsm, cudaStream_t st) {
  const int c = (a.E + 31) / 32;
  return c <= 2    ? launch_route<DT, 2>(a, aligned, nsm, st)
         : c <= 4  ? launch_route<DT, 4>(a, aligned, nsm, st)
         : c <= 8  ? launch_route<DT, 8>(a, aligned, nsm, st)
         : c <= 16 ? launch_route<DT, 16>(a, aligned, nsm, st)
                   : launch_route<DT, 32>(a, aligned, nsm, st);
}

// ---------------------------------------------------------------------------
// sort: a stable counting sort of the slots by expert
// ---------------------------------------------------------------------------

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 16, kSortClusters = 4;

struct Sort {
  const int32_t* experts;
  int32_t *offsets, *slots, *places;
  long long n;
  long long per_warp;  // slots of a warp, a multiple of 32
  int E, blocks;       // blocks of a cluster
};

// The lanes whose expert is this lane's, e in [-1, 2^bits): a ballot a bit (the
// match instruction takes its time for each expert of 32).
__device__ __forceinline__ uint32_t same_expert(int e, int bits) {
  uint32_t m = __ballot_sync(0xFFFFFFFFu, e >= 0);
  if (e < 0) m = ~m;
  for (int b = 0; b < bits; ++b) {
    const uint32_t s = __ballot_sync(0xFFFFFFFFu, (e >> b) & 1);
    m &= (e >> b) & 1 ? s : ~s;
  }
  return m;
}

// The slots are split into runs, one a warp, in their order, the runs over the
// blocks of a cluster (one block for few slots) and, of many slots, over several
// clusters.  Each warp counts its run's experts, in shared memory, the lanes with the
// same expert as one; the block sums its warps' counts, the cluster its blocks', and
// the experts' are scanned.  A slot's place is its warp's first one of its expert
// and its number among the warp's.  Clusters do not wait for one another: each
// counts the slots of the others too, where the order in which counts are added
// does not matter.  One launch, no workspace; the places do not depend on an order
// of arrival.
// 131072 slots of 256 experts: 9.5 us (issue of the 64 SMs at work 44 %, then barriers, single
// stores and the counting of others' slots), 2^20 slots 32.7, 2^24 438; few slots: a chain of
// latencies, 3.1.
constexpr int kHeld = 8;
__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const Sort a) {
  extern __shared__ __align__(16) int32_t sort_smem[];
  int32_t* count = sort_smem;                 // [warps][E], then each warp's next place
  // [E] each, of this block (the cluster reads them): its runs' slots, and its share of those of
  // the clusters before and of all the others
  int32_t *total = count + kSortWarps * a.E, *earlier = total + a.E, *others = earlier + a.E;
  __shared__ int32_t warp_sum[kSortWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % a.blocks, cluster = blockIdx.x / a.blocks, clusters = gridDim.x / a.blocks;
  for (int i = tid; i < (kSortWarps + 3) * a.E; i += kSortThreads) count[i] = 0;
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  const long long s0 = ((long long)blockIdx.x * kSortWarps + warp) * a.per_warp, s1 = min(a.n, s0 + a.per_warp);
  int32_t* mine = count + warp * a.E;
  const int bits = 32 - __clz(a.E - 1 | 1);
  // a step's experts, and its slots' numbers among those of their expert in the run: of a
  // run of up to kHeld steps here, of a longer one in `places`, where each thread reads its own
  int held[kHeld], number[kHeld];
  const bool longer = a.per_warp > 32 * kHeld;
  auto load = [&](long long s) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int e = s + 32 * j + lane < s1 ? __ldg(a.experts + s + 32 * j + lane) : -1;
      held[j] = e >= 0 && e < a.E ? e : -1;
    }
  };
  for (long long s = s0; s < s1; s += 32 * kHeld) {
    load(s);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (s + 32 * j >= s1) break;
      const int e = held[j];
      const uint32_t same = same_expert(e, bits), less = same & ((1u << lane) - 1);
      const int before = e >= 0 ? mine[e] : 0;
      __syncwarp();
      if (e >= 0 && less == 0) mine[e] = before + __popc(same);
      __syncwarp();
      number[j] = before + __popc(less);
      if (longer && s + 32 * j + lane < s1) a.places[s + 32 * j + lane] = number[j];
    }
  }
  if (clusters > 1) {
    // the other clusters' slots, every blocks-th 4096 of them here
    const long long c0 = (long long)cluster * a.blocks * kSortWarps * a.per_warp, c1 = min(a.n, c0 + a.blocks * kSortWarps * a.per_warp);
    for (long long s = (long long)rank * 4 * kSortThreads; s < a.n; s += (long long)a.blocks * 4 * kSortThreads) {
      int e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long slot = s + j * kSortThreads + tid;
        e[j] = slot < a.n && (slot < c0 || slot >= c1) ? __ldg(a.experts + slot) : -1;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (e[j] < 0 || e[j] >= a.E) continue;
        atomicAdd(others + e[j], 1);
        if (s + j * kSortThreads + tid < c0) atomicAdd(earlier + e[j], 1);
      }
    }
  }
  __syncthreads();
  // (E <= the threads of a block: thread e has expert e)
  int32_t sum = 0, before = 0;
  if (tid < a.E) {
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) sum += count[w * a.E + tid];
    total[tid] = sum;
  }
  if (a.blocks > 1) {
    cluster_sync();
    if (tid < a.E) {
      const uint32_t at = smem_u32(total + tid);
      int32_t v[kSortCluster];
#pragma unroll
      for (int b = 0; b < kSortCluster; ++b) {
        v[b] = 0;
        if (b < a.blocks) asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[b]) : "r"(mapa(at, b)) : "memory");
      }
      sum = 0;
#pragma unroll
      for (int b = 0; b < kSortCluster; ++b) before += b < rank ? v[b] : 0, sum += v[b];
      if (clusters > 1) {
        const uint32_t ae = smem_u32(earlier + tid), ao = smem_u32(others + tid);
#pragma unroll
        for (int b = 0; b < kSortCluster; ++b) {
          v[b] = 0;
          if (b < a.blocks) asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[b]) : "r"(mapa(ae, b)) : "memory");
        }
#pragma unroll
        for (int b = 0; b < kSortCluster; ++b) before += v[b];
#pragma unroll
        for (int b = 0; b < kSortCluster; ++b) {
          v[b] = 0;
          if (b < a.blocks) asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[b]) : "r"(mapa(ao, b)) : "memory");
        }
#pragma unroll
        for (int b = 0; b < kSortCluster; ++b) sum += v[b];
      }
    }
    cluster_arrive();  // (waited for at the end: its totals have been read)
  }
  int32_t scan = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  int32_t all = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    const int32_t v = warp_sum[w];
    scan += w < warp ? v : 0, all += v;
  }
  if (tid < a.E) {
    int32_t place = scan - sum + before;
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const int32_t c = count[w * a.E + tid];
      count[w * a.E + tid] = place, place += c;
    }
    if (blockIdx.x == 0) {
      a.offsets[tid + 1] = scan;
      if (tid == 0) a.offsets[0] = 0;
    }
  }
  __syncthreads();
  for (long long s = s0; s < s1; s += 32 * kHeld) {
    if (longer) {
      load(s);
#pragma unroll
      for (int j = 0; j < kHeld; ++j) number[j] = s + 32 * j + lane < s1 ? a.places[s + 32 * j + lane] : 0;
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const long long slot = s + 32 * j + lane;
      if (slot >= s1) break;
      const int e = held[j];
      const int32_t place = e >= 0 ? mine[e] + number[j] : -1;
      a.places[slot] = place;
      if (place >= 0) a.slots[place] = (int32_t)slot;
    }
  }
  for (long long p = all + (long long)blockIdx.x * kSortThreads + tid; p < a.n; p += (long long)gridDim.x * kSortThreads) a.slots[p] = -1;
  if (a.blocks > 1) cluster_wait();
}

// ---------------------------------------------------------------------------
// combine: out[t] = sum over ranks of gate * y[place]
// ---------------------------------------------------------------------------

struct Combine {
  const void* y;
  const int32_t* places;
  const float* gates;
  void* out;
  long long tokens, y_rows, y_stride, out_stride, pieces;  // pieces of a token
  int cols, top_k;
};

__device__ __forceinline__ long long token_of(const Combine& a, long long i) {
  // (a division of 64 bits is some 40 instructions)
  return a.tokens * a.pieces <= 0xFFFFFFFFll ? (long long)((uint32_t)i / (uint32_t)a.pieces) : i / a.pieces;
}

// V sums as V elements of type ODT (an address aligned to 16 bytes or to V elements).
template <int ODT, int V>
__device__ __forceinline__ void store_sums(void* out, long long at, const float (&s)[V]) {
  if constexpr (V == 1) {
    if (ODT == MSK_FP32) static_cast<float*>(out)[at] = s[0];
    else if (ODT == MSK_FP16) static_cast<__half*>(out)[at] = __float2half_rn(s[0]);
    else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(s[0]);
  } else if constexpr (ODT == MSK_FP32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int j = 0; j < V / 4; ++j) p[j] = make_float4(s[4 * j], s[4 * j + 1], s[4 * j + 2], s[4 * j + 3]);
  } else {
    uint32_t x[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) x[j] = pack16(s[2 * j], s[2 * j + 1], ODT == MSK_FP16);
    uint16_t* p = static_cast<uint16_t*>(out) + at;
    if constexpr (V == 4) {
      *reinterpret_cast<uint2*>(p) = make_uint2(x[0], x[1]);
    } else {
#pragma unroll
      for (int j = 0; j < V / 8; ++j) reinterpret_cast<uint4*>(p)[j] = make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
    }
  }
}

// A thread has B bytes of a token's columns (V elements; B = 0: one element, where
// rows are not aligned), its ranks' rows all loaded before they are summed, eight at
// a time.  Sums in fp32, by rank.  8192 tokens x 8 x 2048 columns of 16 bits: 50 us, bound by
// DRAM; of 2047, one element a thread, 176 (loads of two bytes and a position for each).
template <int DT, int ODT, int B>
__global__ void __launch_bounds__(256) combine_kernel(const Combine a) {
  constexpr int S = DT == MSK_FP32 ? 4 : 2, V = B ? B / S : 1, U = 8, W = B ? B / 4 : 1;
  grid_dep_wait();
  grid_dep_launch();
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.tokens * a.pieces) return;
  const long long t = token_of(a, i);
  const int c = (int)(i - t * a.pieces) * V;
  float sum[V] = {};
  for (int r0 = 0; r0 < a.top_k; r0 += U) {
    uint32_t w[U][W];
    float g[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long slot = t * a.top_k + r0 + u;
      const int p = r0 + u < a.top_k ? __ldg(a.places + slot) : -1;
      const bool in = p >= 0 && p < a.y_rows;  // (a dropped slot's row is not read)
      g[u] = !in ? 0.f : a.gates != nullptr ? __ldg(a.gates + slot) : 1.f;
#pragma unroll
      for (int j = 0; j < W; ++j) w[u][j] = 0u;
      if (!in) continue;
      const long long at = p * a.y_stride + c;
      const char* from = static_cast<const char*>(a.y) + at * S;
      if constexpr (B == 32) {
        ldg256(from, w[u]);
      } else if constexpr (B == 16) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(from));
        w[u][0] = v.x, w[u][1] = v.y, w[u][2] = v.z, w[u][3] = v.w;
      } else {
        w[u][0] = __float_as_uint(element<DT>(a.y, at));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (B == 0 || DT == MSK_FP32) {
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] = fmaf(g[u], __uint_as_float(w[u][j]), sum[j]);
      } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const float2 f = unpack16(w[u][j], DT == MSK_FP16);
          sum[2 * j] = fmaf(g[u], f.x, sum[2 * j]), sum[2 * j + 1] = fmaf(g[u], f.y, sum[2 * j + 1]);
        }
      }
    }
  }
  store_sums<ODT, V>(a.out, t * a.out_stride + c, sum);
}

template <int DT, int ODT>
cudaError_t launch_combine(Combine& a, cudaStream_t st) {
  constexpr int S = DT == MSK_FP32 ? 4 : 2, O = ODT == MSK_FP32 ? 4 : 2;
  auto fits = [&](int bytes) {  // rows of y in pieces of `bytes`, of out in what they become, 16 at most
    const int v = bytes / S, o = std::min(16, v * O);
    return a.cols % v == 0 && reinterpret_cast<uintptr_t>(a.y) % bytes == 0 && a.y_stride * S % bytes == 0 &&
           reinterpret_cast<uintptr_t>(a.out) % o == 0 && a.out_stride * O % o == 0;
  };
  // (32 bytes where 4M outputs and more fill the GPU all the same: 8192 tokens x 8 x 2048
  // columns 50.4 us, with 16 52.6; fewer have the more threads for it)
  const int b = fits(32) && a.tokens * a.cols >= 1 << 22 ? 32 : fits(16) ? 16 : 0;
  a.pieces = b ? a.cols / (b / S) : a.cols;
  const OpsLaunch l(dim3((unsigned)((a.tokens * a.pieces + 255) / 256)), 256, 0, st);
  return cudaLaunchKernelEx(&l.cfg, b == 32 ? combine_kernel<DT, ODT, 32> : b == 16 ? combine_kernel<DT, ODT, 16> : combine_kernel<DT, ODT, 0>, a);
}

template <int DT>
cudaError_t launch_combine(Combine& a, int odt, cudaStream_t st) {
  return odt == MSK_BF16   ? launch_combine<DT, MSK_BF16>(a, st)
         : odt == MSK_FP16 ? launch_combine<DT, MSK_FP16>(a, st)
                           : launch_combine<DT, MSK_FP32>(a, st);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr long long kMaxSlots = 1ll << 30;  // places are 32-bit

}  // namespace
}  // namespace msk

using namespace msk;

extern "C" msk_status msk_moe_route(const void* logits, int32_t dtype, int64_t tokens, int32_t n_experts, int64_t ld,
                                    const float* bias, int32_t top_k, int32_t* experts, float* gates, void* stream) {
  if (!dtype_ok(dtype) || tokens < 0) return MSK_ERR_INVALID_ARG;
  if (n_experts < 1 || n_experts > kMaxExperts || top_k < 1 || top_k > kMaxTopK || top_k > n_experts) return MSK_ERR_SHAPE;
  if (tokens > kMaxSlots / top_k) return MSK_ERR_SHAPE;
  if (tokens == 0) return MSK_OK;
  if (logits == nullptr || experts == nullptr || gates == nullptr || (tokens > 1 && ld < n_experts)) return MSK_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % dtype_bytes(dtype) || !aligned4(bias) || !aligned4(experts) || !aligned4(gates))
    return MSK_ERR_ALIGNMENT;
  int nsm = 0;
  const msk_status s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  Route a{};
  a.logits = logits, a.bias = bias, a.experts = experts, a.gates = gates;
  a.tokens = tokens, a.ld = ld, a.E = n_experts, a.top_k = top_k;
  const bool aligned = ops_aligned16(logits) && (tokens == 1 || ld * dtype_bytes(dtype) % 16 == 0);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MSK_BF16   ? launch_route<MSK_BF16>(a, aligned, nsm, st)
                        : dtype == MSK_FP16 ? launch_route<MSK_FP16>(a, aligned, nsm, st)
                                            : launch_route<MSK_FP32>(a, aligned, nsm, st);
  return e == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}

extern "C" msk_status msk_moe_sort(const int32_t* experts, int64_t n, int32_t n_experts, int32_t* offsets, int32_t* slots,
                                   int32_t* places, void* stream) {
  if (n < 0) return MSK_ERR_INVALID_ARG;
  if (n_experts < 1 || n_experts > kMaxExperts || n > kMaxSlots) return MSK_ERR_SHAPE;
  if (offsets == nullptr || (n > 0 && (experts == nullptr || slots == nullptr || places == nullptr))) return MSK_ERR_INVALID_ARG;
  if (!aligned4(experts) || !aligned4(offsets) || !aligned4(slots) || !aligned4(places)) return MSK_ERR_ALIGNMENT;
  int nsm = 0;
  const msk_status s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  Sort a{};
  a.experts = experts, a.offsets = offsets, a.slots = slots, a.places = places, a.n = n, a.E = n_experts;
  // (a block goes through 4096 slots, 4 steps a warp, in the time that a cluster's barriers take;
  // with four clusters of 16 65536 slots take 8.0 us, 131072 9.6, 2^20 32.7, 2^24 438, with one 9.1,
  // 13.2, 77 and 1119, with two 8.7, 11.4, 50 and 703, with eight, which do not all run at once,
  // 8.0, 16.5, 44 and 618)
  a.blocks = n <= 4096 ? 1 : n <= 8 * 4096 ? 8 : kSortCluster;
  const int clusters = a.blocks < kSortCluster ? 1 : (int)std::min<int64_t>(kSortClusters, (n + 16383) / 16384);
  const long long warps = (long long)a.blocks * clusters * kSortWarps;
  a.per_warp = ((n + warps - 1) / warps + 31) / 32 * 32;
  const int smem = (kSortWarps + 3) * n_experts * 4;
  static std::atomic<bool> ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MSK_ERR_CUDA;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kSortWarps + 3) * kMaxExperts * 4) != cudaSuccess ||
        cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return MSK_ERR_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  const OpsLaunch l(dim3((unsigned)(a.blocks * clusters)), kSortThreads, smem, static_cast<cudaStream_t>(stream), a.blocks);
  return cudaLaunchKernelEx(&l.cfg, sort_kernel, a) == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}

extern "C" msk_status msk_moe_combine(const void* y, int32_t y_dtype, int64_t y_rows, int64_t y_stride, const int32_t* places,
                                      const float* gates, int64_t tokens, int32_t top_k, int64_t cols, void* out,
                                      int32_t out_dtype, int64_t out_stride, void* stream) {
  if (!dtype_ok(y_dtype) || !dtype_ok(out_dtype) || tokens < 0 || y_rows < 0) return MSK_ERR_INVALID_ARG;
  if (top_k < 1 || cols < 0 || cols > (1ll << 30) || tokens > kMaxSlots / top_k || y_rows > kMaxSlots) return MSK_ERR_SHAPE;
  if (tokens * cols >= (1ll << 38)) return MSK_ERR_SHAPE;  // (the grid)
  if (tokens == 0 || cols == 0) return MSK_OK;
  if ((y == nullptr && y_rows > 0) || places == nullptr || out == nullptr) return MSK_ERR_INVALID_ARG;
  if ((y_rows > 1 && y_stride < cols) || (tokens > 1 && out_stride < cols)) return MSK_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(y) % dtype_bytes(y_dtype) || reinterpret_cast<uintptr_t>(out) % dtype_bytes(out_dtype) ||
      !aligned4(places) || !aligned4(gates))
    return MSK_ERR_ALIGNMENT;
  int nsm = 0;
  const msk_status s = ops_device(&nsm);
  if (s != MSK_OK) return s;
  Combine a{};
  a.y = y, a.places = places, a.gates = gates, a.out = out;
  a.tokens = tokens, a.y_rows = y_rows, a.y_stride = y_rows > 1 ? y_stride : 0, a.out_stride = tokens > 1 ? out_stride : 0;
  a.cols = (int)cols, a.top_k = top_k;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = y_dtype == MSK_BF16   ? launch_combine<MSK_BF16>(a, out_dtype, st)
                        : y_dtype == MSK_FP16 ? launch_combine<MSK_FP16>(a, out_dtype, st)
                                              : launch_combine<MSK_FP32>(a, out_dtype, st);
  return e == cudaSuccess ? MSK_OK : MSK_ERR_CUDA;
}
