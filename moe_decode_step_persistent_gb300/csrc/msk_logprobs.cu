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

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
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

// A row's aligned vectors, and the single logits before and behind them.
template <int DT>
struct Row {
  const char* xv;  // first vector of this block's segment
  int nv;          // vectors of the segment
  int first;       // logits of the row before them
  int head, tail;  // single logits of the row's ends, 0 unless this block's
  __device__ __forceinline__ Row(const LogProbs& a, long long row, int S, int part) {
    constexpr int es = DT == MSK_FP32 ? 4 : 2;
    const char* x = static_cast<const char*>(a.logits) + row * a.ld * es;
    head = (int)min(a.V, (long long)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / es);
    const int n = (int)((a.V - head) / Vec<DT>::N);
    tail = (int)(a.V - head) - n * Vec<DT>::N;
    const int v0 = (int)((long long)n * part / S);
    nv = (int)((long long)n * (part + 1) / S) - v0;
    first = head + v0 * Vec<DT>::N;
    xv = x + (long long)first * es;
    if (part != 0) head = 0;
    if (part != S - 1) tail = 0;
  }
  __device__ __forceinline__ const char* row() const { return xv - (long long)first * (DT == MSK_FP32 ? 4 : 2); }
  // The index of thread t's single logit, or -1.
  __device__ __forceinline__ int single(int t, const LogProbs& a) const {
    return t < head ? t : t >= 32 && t < 32 + tail ? (int)a.V - tail + (t - 32) : -1;
  }
};

__device__ __forceinline__ float clamp_reach(float c) {
  // the clamp's distance below the maximum: at least 300 powers of two, and
  // enough steps of the type (|m| / 64; fp16's smallest) that rounding it keeps
  // more than 260 of them
  return fmaxf(300.f / c, 0x1p-20f);
}

// One thread's share of a row: a single logit perhaps, and every NT-th vector,
// four a step, so that the sums are rescaled once for 16 or 32 logits.  Returns
// the statistics; key: the greatest logit's (0 without one), above: how many
// are greater than xg; steps: where that logit is and what the other steps hold.
struct Steps {
  float second;  // the greatest logit outside the step with the greatest one (NaN: unknown)
  int left;      // vectors from that step's first on, 0: it is not in a vector
};
template <int DT, int NT, bool STEPS>
__device__ __forceinline__ Stat thread_stats(const Row<DT>& x, const LogProbs& a, int tid, float c, float reach, float xg,
                                             uint32_t& key, int& above, Steps& steps) {
  constexpr int U = 4;
  const int mine = x.single(tid, a);
  Stat q = {-INFINITY, 0.f, 0.f};
  above = 0;
  steps = {-INFINITY, 0};
  if (mine >= 0) {
    const float v = load1<DT>(x.row(), mine);
    above += v > xg;
    q.m = max_nan(q.m, v);
    q.s = v == -INFINITY ? 0.f : ex2((v - v) * c);  // (NaN for what is no number)
  }
  unsigned long long s2 = pair(q.s, 0.f), u2 = pair(0.f, 0.f);
  const uint32_t xg2 = DT == MSK_FP32 ? __float_as_uint(xg) : pack16(xg, xg, DT == MSK_FP16);
  const char* at = x.xv + (long long)tid * 16;
  for (int left = x.nv - tid; left > 0; left -= U * NT, at += U * NT * 16) {
    Vec<DT> w[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (k * NT < left) w[k].u = load_stream(at + k * (NT * 16));
      else w[k].none();
    }
    const float bm = vec_max<DT, U>(w), mn = max_nan(q.m, bm), r = anchor(mn);
    if (STEPS) {
      steps.second = max_nan(steps.second, min_nan(bm, q.m));
      if (bm > q.m) steps.left = left;
    }
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
  float s0, s1, u0, u1;
  unpair(s2, s0, s1);
  unpair(u2, u0, u1);
  key = tid < x.nv || mine >= 0 ? ordered(q.m) : 0u;
  return {q.m, s0 + s1, u0 + u1};
}

// The warp's statistics, all relative to its maximum.
__device__ __forceinline__ Stat warp_stats(const Stat& q, uint32_t key, float c) {
  const uint32_t wk = __reduce_max_sync(0xFFFFFFFFu, key);
  const float m = wk == 0u ? -INFINITY : key_value((unsigned long long)wk << 32);
  const float d = (q.m - anchor(m)) * c, f = ex2(d);
  float s = f * q.s, u = f * (q.u + fmaxf(d, -300.f) * q.s);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
  }
  return {m, s, u};
}

// The logits of the lanes' vectors that reach `lo` (few), into the warp's list of
// the 32 greatest.
// in: whether a lane has a vector; first, step: the index of lane 0's first
// logit, and from one lane's to the next.
template <int DT>
__device__ __forceinline__ void list_vectors(unsigned long long& list, const Vec<DT>& w, bool in, int first, int step,
                                             float lo, int lane) {
  constexpr int VN = Vec<DT>::N;
  const Vec<DT> one[1] = {w};
  const float most = vec_max<DT, 1>(one);
  // (a vector none of whose keys passes the list's last one is left out: ties)
  const unsigned long long bound = ((unsigned long long)ordered(most) << 32) | (0xFFFFFFFFu - (uint32_t)(first + lane * step));
  const unsigned long long last = __shfl_sync(0xFFFFFFFFu, list, 31);
  uint32_t lanes = __ballot_sync(0xFFFFFFFFu, in && !(most < lo) && bound > last);
  while (lanes) {
    const int src = __ffs(lanes) - 1;
    lanes &= lanes - 1;
    // a lane for each of the vector's logits
    const uint32_t u[4] = {__shfl_sync(0xFFFFFFFFu, w.u.x, src), __shfl_sync(0xFFFFFFFFu, w.u.y, src),
                           __shfl_sync(0xFFFFFFFFu, w.u.z, src), __shfl_sync(0xFFFFFFFFu, w.u.w, src)};
    const int i = DT == MSK_FP32 ? lane & 3 : lane >> 1 & 3;
    const uint32_t p = i < 2 ? (i == 0 ? u[0] : u[1]) : (i == 2 ? u[2] : u[3]);
    float y = __uint_as_float(p);
    if (DT != MSK_FP32) {
      const float2 f = unpack16(p, DT == MSK_FP16);
      y = lane & 1 ? f.y : f.x;
    }
    const unsigned long long key =
        ((unsigned long long)ordered(y) << 32) | (0xFFFFFFFFu - (uint32_t)(first + src * step + lane));
    const unsigned long long least = __shfl_sync(0xFFFFFFFFu, list, 31);
    uint32_t hit = __ballot_sync(0xFFFFFFFFu, lane < VN && !(y < lo) && key > least);
    while (hit) {
      const int from = __ffs(hit) - 1;
      hit &= hit - 1;
      list_insert(list, __shfl_sync(0xFFFFFFFFu, key, from), lane);
    }
  }
}

// A row's results from its statistics and sorted alternatives (a lane's each).
__device__ __forceinline__ void put_row(const LogProbs& a, long long row, const Stat& z, int above, int tok, float xg, float c,
                                        unsigned long long alt, int lane) {
  const bool given = tok >= 0 && tok < a.V, bad = !(z.s > 0.f && z.s < INFINITY);
  // in log2 units, then nats
  constexpr float kLn2 = 0.6931471805599453f;
  const float log_s = bad ? NAN : log2f(z.s);
  if (lane == 0) {
    if (a.logprob) a.logprob[row] = given ? ((xg - z.m) * c - log_s) * kLn2 : 0.f;
    if (a.rank) a.rank[row] = given ? above : -1;
    if (a.entropy) a.entropy[row] = bad ? NAN : (log_s - z.u / z.s) * kLn2;
  }
  if (lane < a.top) {
    if (a.top_ids) a.top_ids[row * a.top + lane] = (int32_t)(0xFFFFFFFFu - (uint32_t)alt);
    if (a.top_logprobs) a.top_logprobs[row * a.top + lane] = bad ? NAN : ((key_value(alt) - z.m) * c - log_s) * kLn2;
  }
}

__device__ __forceinline__ int row_token(const LogProbs& a, long long row) {
  return a.tokens && row < a.rows ? a.tokens[row] : -1;
}
template <int DT>
__device__ __forceinline__ float row_logit(const LogProbs& a, long long row, int tok) {
  if (tok < 0 || tok >= a.V) return INFINITY;
  return load1<DT>(static_cast<const char*>(a.logits) + row * a.ld * (DT == MSK_FP32 ? 4 : 2), tok);
}

// The n-th greatest (1 <= n <= 64) of the warp's 64 numbers, two a lane: the
// greatest left, n times (fewer with ties).
__device__ __forceinline__ uint32_t greatest(uint32_t g0, uint32_t g1, int n) {
  for (;;) {
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(g0, g1));
    n -= __popc(__ballot_sync(0xFFFFFFFFu, g0 == m)) + __popc(__ballot_sync(0xFFFFFFFFu, g1 == m));
    if (n <= 0 || m == 0u) return m;
    g0 = g0 == m ? 0u : g0, g1 = g1 == m ? 0u : g1;
  }
}

// Alternatives cost no second pass: if `top` groups of threads have maxima that
// reach a bound, so do `top` logits, and all of those lie in the (few) threads
// whose own maxima reach it.  Those threads' logits are looked at again.

// Many long rows.  Blocks take rows blockIdx.x, + gridDim.x, ...: 16 warps read
// one row after the other without a stop, and two more end the rows (join the
// warps' sums, find the alternatives, write the results) in turn while the 16
// read on.  Each of the two has a place for a row's statistics, which it gives
// back once it has read them (named barriers, one each way).
// 1024 x 131072 with 20 alternatives: bf16 56 us (4.8 TB/s), fp32 91 (5.9); a
// block a row, all warps at its end: 67 and 115.  Issue slots bound it in 16 bits
// (62% in use; eight instructions for two logits), DRAM in fp32.
constexpr int kStreamThreads = 512, kFetch = 16, kHits = 128;
enum { kFull0 = 1, kFree0 = 3 };  // barriers; + 1 for the second place
template <int ID>
__device__ __forceinline__ void place_sync(int place) {
  if (place == 0) asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(kStreamThreads + 32) : "memory");
  else asm volatile("bar.sync %0, %1;" ::"n"(ID + 1), "n"(kStreamThreads + 32) : "memory");
}
template <int ID>
__device__ __forceinline__ void place_arrive(int place) {
  if (place == 0) asm volatile("bar.arrive %0, %1;" ::"n"(ID), "n"(kStreamThreads + 32) : "memory");
  else asm volatile("bar.arrive %0, %1;" ::"n"(ID + 1), "n"(kStreamThreads + 32) : "memory");
}

template <int DT>
__global__ void __launch_bounds__(kStreamThreads + 64, 2) logprobs_stream_kernel(const __grid_constant__ LogProbs a) {
  constexpr int NT = kStreamThreads, NW = NT / 32, PER = NT / 32, VN = Vec<DT>::N;
  __shared__ Stat st[2][NW];
  __shared__ int cnt[2][NW];
  __shared__ uint32_t keys[2][NT];
  __shared__ float second[2][NT];  // (see Steps)
  __shared__ int where[2][NT];
  __shared__ uint16_t owners[2][NT], scan[2][NT];
  __shared__ uint4 fetched[2][kFetch][32];
  __shared__ unsigned long long hits[2][kHits];
  __shared__ int n_hits[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float c = a.inv_t * 1.4426950408889634f, reach = clamp_reach(c);
  grid_dep_wait();  // (and the next kernel does not start early: its blocks would come to lie unevenly, 65 us for 56)
  if (warp < NW) {
    int place = 0;
    int tok = row_token(a, blockIdx.x);
    float xg = row_logit<DT>(a, blockIdx.x, tok);
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
      tok = row_token(a, row + gridDim.x);
      uint32_t key;
      int above;
      Steps steps;
      const Stat t = thread_stats<DT, NT, true>(Row<DT>(a, row, 1, 0), a, tid, c, reach, xg, key, above, steps);
      xg = row_logit<DT>(a, row + gridDim.x, tok);
      const Stat q = warp_stats(t, key, c);
      above = __reduce_add_sync(0xFFFFFFFFu, above);
      if (row >= 2ll * gridDim.x) place_sync<kFree0>(place);
      keys[place][tid] = key, second[place][tid] = steps.second, where[place][tid] = steps.left;
      if (lane == 0) st[place][warp] = q, cnt[place][warp] = above;
      __syncwarp();
      place_arrive<kFull0>(place);
      place ^= 1;
    }
    return;
  }
  const int end = warp - NW;
  for (long long row = blockIdx.x + (long long)end * gridDim.x; row < a.rows; row += 2ll * gridDim.x) {
    const int tok = row_token(a, row);
    const float xg = row_logit<DT>(a, row, tok);
    const Row<DT> x(a, row, 1, 0);
    __syncwarp();
    place_sync<kFull0>(end);
    Stat z = lane < NW ? st[end][lane] : Stat{-INFINITY, 0.f, 0.f};
    const int above = __reduce_add_sync(0xFFFFFFFFu, lane < NW ? cnt[end][lane] : 0);
    uint32_t k[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) k[i] = keys[end][i * 32 + lane];
    const bool more = row + 2ll * gridDim.x < a.rows;
    __syncwarp();
    if (more && a.top == 0) place_arrive<kFree0>(end);
#pragma unroll
    for (int o = 16; o; o >>= 1) z = stat_join(z, stat_shfl(z, o), c);
    unsigned long long list = 0ull;
    if (a.top > 0) {
      // the bound: the `top`-th greatest maximum of 64 groups of threads, two a lane
      uint32_t g0 = 0, g1 = 0;
#pragma unroll
      for (int i = 0; i < PER; i += 2) g0 = max(g0, k[i]), g1 = max(g1, k[i + 1]);
      const uint32_t lo = greatest(g0, g1, a.top);
      const float lo_value = lo == 0u ? -INFINITY : key_value((unsigned long long)lo << 32);
      int n = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const uint32_t has = __ballot_sync(0xFFFFFFFFu, k[i] >= lo);
        if (k[i] >= lo) owners[end][n + __popc(has & ((1u << lane) - 1))] = (uint16_t)(i * 32 + lane);
        n += __popc(has);
      }
      if (lane == 0) n_hits[end] = 0;
      __syncwarp();
      // Logits that reach the bound go to `hits`, in any order.
      auto hit = [&](float y, int index) {
        const int at = atomicAdd(&n_hits[end], 1);
        if (at < kHits) hits[end][at] = ((unsigned long long)ordered(y) << 32) | (0xFFFFFFFFu - (uint32_t)index);
      };
      // A lane for each of the threads: most have them in one step of their
      // vectors only.  The others' vectors are all looked at, below.
      int n_scan = 0;
      for (int i = 0; i < n; i += 32) {
        const int o = owners[end][min(i + lane, n - 1)];
        const int left = where[end][o];
        const bool one = second[end][o] < lo_value, rest = i + lane < n && !one;
        const uint32_t some = __ballot_sync(0xFFFFFFFFu, rest);
        if (rest) scan[end][n_scan + __popc(some & ((1u << lane) - 1))] = (uint16_t)o;
        n_scan += __popc(some);
        if (i + lane < n && one) {
          constexpr int U = 4;
          Vec<DT> w[U];
#pragma unroll
          for (int k = 0; k < U; ++k) {
            w[k].none();
            if (k * NT < left) w[k].u = load_stream(x.xv + (long long)(x.nv - left + k * NT) * 16);
          }
#pragma unroll
          for (int k = 0; k < U; ++k) {
            float y[VN];
            w[k].get(y);
#pragma unroll
            for (int j = 0; j < VN; ++j)
              if (k * NT < left && !(y[j] < lo_value)) hit(y[j], x.first + (x.nv - left + k * NT) * VN + j);
          }
        }
      }
      __syncwarp();
      if (more) place_arrive<kFree0>(end);
      // The hits are ranked; should there be more than the place holds (ties), the
      // list is made one by one instead.
      for (int way = 0; way < 2; ++way) {
        const uint16_t* look = way == 0 ? scan[end] : owners[end];
        const int n_look = way == 0 ? n_scan : n;
        if (x.head + x.tail > 0) {  // single logits
          for (int i = 0; i < n; i += 32) {
            const int single = i + lane < n ? x.single(owners[end][i + lane], a) : -1;
            const float v = single >= 0 ? load1<DT>(x.row(), single) : 0.f;
            const bool in = single >= 0 && !(v < lo_value);
            if (way == 0 && in) hit(v, single);
            const unsigned long long key = ((unsigned long long)ordered(v) << 32) | (0xFFFFFFFFu - (uint32_t)single);
            uint32_t lanes = __ballot_sync(0xFFFFFFFFu, way == 1 && in);
            while (lanes) {
              const int src = __ffs(lanes) - 1;
              lanes &= lanes - 1;
              list_insert(list, __shfl_sync(0xFFFFFFFFu, key, src), lane);
            }
          }
        }
        // vectors, a lane for each, several loads under way
        const uint32_t mine = smem_u32(&fetched[end][0][lane]);
        for (int i = 0, v = n_look > 0 ? look[0] : 0; i < n_look;) {
          int m = 0, my_v = 0;  // this batch's; the first of the 32 vectors of its item `lane`
          for (; m < kFetch && i < n_look; ++m) {
            if (m == lane) my_v = v;
            if (v + lane * NT < x.nv) cp_async16(mine + m * 512, x.xv + (long long)(v + lane * NT) * 16);
            v += 32 * NT;
            if (v >= x.nv) v = ++i < n_look ? look[i] : 0;
          }
          cp_async_wait_all();
          uint32_t which = 0;  // of the lane's vectors
#pragma unroll 4
          for (int j = 0; j < m; ++j) {
            Vec<DT> w[1];
            w[0].u = lds128(mine + j * 512);
            const int v0 = __shfl_sync(0xFFFFFFFFu, my_v, j);
            const bool in = v0 + lane * NT < x.nv;
            if (way == 1) list_vectors<DT>(list, w[0], in, x.first + v0 * VN, NT * VN, lo_value, lane);
            else if (in && !(vec_max<DT, 1>(w) < lo_value)) which |= 1u << j;
          }
          while (way == 0 && __any_sync(0xFFFFFFFFu, which != 0)) {
            const int j = which ? __ffs(which) - 1 : 0;
            const int first = x.first + (__shfl_sync(0xFFFFFFFFu, my_v, j) + lane * NT) * VN;
            if (which) {
              Vec<DT> w;
              w.u = lds128(mine + j * 512);
              float y[VN];
              w.get(y);
#pragma unroll
              for (int k = 0; k < VN; ++k)
                if (!(y[k] < lo_value)) hit(y[k], first + k);
              which &= which - 1;
            }
            __syncwarp();
          }
          if (way == 0 && __any_sync(0xFFFFFFFFu, n_hits[end] > kHits)) break;
        }
        __syncwarp();
        const int have = n_hits[end];
        if (way == 1 || have > kHits) continue;
        constexpr int H = kHits / 32;
        unsigned long long h[H];
        int rank[H];
#pragma unroll
        for (int i = 0; i < H; ++i) h[i] = lane + 32 * i < have ? hits[end][lane + 32 * i] : 0ull, rank[i] = 0;
#pragma unroll 2
        for (int j = 0; j < have; ++j) {
          const unsigned long long other = hits[end][j];
#pragma unroll
          for (int i = 0; i < H; ++i) rank[i] += other > h[i];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < H; ++i)
          if (h[i] != 0ull) hits[end][rank[i]] = h[i];
        __syncwarp();
        list = lane < have ? hits[end][lane] : 0ull;
        break;
      }
      __syncwarp();
    }
    put_row(a, row, z, above, tok, xg, c, list, lane);
  }
}

// Few rows, or short ones: a block for a row, or a cluster of blocks for
// `gridDim.x` segments of it.  All warps take part in the row's end, each with a
// sorted list of the alternatives that it has found.  Latency bounds it: 16 x
// 131072 with 8 alternatives 7.7 us.
template <int DT, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) logprobs_kernel(const __grid_constant__ LogProbs a) {
  constexpr int VN = Vec<DT>::N, NW = NT / 32;
  __shared__ Stat st[NW];
  __shared__ int cnt[NW];
  __shared__ int owners[NT];
  __shared__ int n_owners, n_cand;
  __shared__ uint32_t group_max[64], bound;  // (a thread without a logit: 0)
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
  const float c = a.inv_t * 1.4426950408889634f;
  grid_dep_wait();
  grid_dep_launch();
  const int tok = row_token(a, row);
  const float xg = row_logit<DT>(a, row, tok);
  const Row<DT> x(a, row, S, part);
  uint32_t key;
  int above;
  Steps steps;
  const Stat t = thread_stats<DT, NT, false>(x, a, tid, c, clamp_reach(c), xg, key, above, steps);
  Stat q = warp_stats(t, key, c);
  above = __reduce_add_sync(0xFFFFFFFFu, above);
  if (lane == 0) st[warp] = q, cnt[warp] = above;
  if (tid == 0) n_owners = 0, n_cand = 0;
  if (tid < kMaxTop) best[tid] = 0ull;
  if (a.top > 0) {
    uint32_t gm = key;
#pragma unroll
    for (int o = 1; o < NT / 64; o <<= 1) gm = max(gm, __shfl_xor_sync(0xFFFFFFFFu, gm, o));
    if (lane % (NT / 64) == 0) group_max[tid / (NT / 64)] = gm;
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
    const uint32_t lo = greatest(group_max[lane], group_max[lane + 32], a.top);
    if (lane == 0) bound = lo;
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
      const int single = x.single(o, a);
      if (single >= 0) {
        const uint32_t k = ordered(load1<DT>(x.row(), single));
        if (k >= lo) list_insert(list, ((unsigned long long)k << 32) | (0xFFFFFFFFu - (uint32_t)single), lane);
      }
      for (int vb = o; vb < x.nv; vb += 32 * NT) {
        const int v = vb + lane * NT;
        Vec<DT> w;
        w.none();
        if (v < x.nv) w.u = load_stream(x.xv + (long long)v * 16);
        list_vectors<DT>(list, w, v < x.nv, x.first + vb * VN, NT * VN, lo_value, lane);
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
  if (warp == 0) put_row(a, row, S > 1 ? joined : seg, S > 1 ? joined_above : seg_above, tok, xg, c, best[lane], lane);
}

template <int DT>
cudaError_t launch_logprobs(const LogProbs& a, int nsm, cudaStream_t st) {
  // Few rows: 2 segments a row while all blocks are resident at once, 4 and 8
  // (portable cluster sizes) while each has an SM of its own, and if a segment
  // is worth a block.  131072 logits, 20 alternatives: 16 rows in 8 segments
  // 7.6 us; 76 rows in 2 segments 11.2 us, in 4 17.0; 152 rows in 2 14.1, whole
  // 16.0; 304 rows whole 23.7, in 2 29.0.
  int S = 1;
  while (S < 8 && a.rows * S * 2 <= (S == 1 ? 2ll : 1ll) * nsm && a.V / (S * 2) >= 4096) S *= 2;
  // Rows of up to 64 KB take blocks of 128 threads, eight an SM (2048 x 8192 bf16
  // 14.5 us, the warps that read on 24.1; 2048 x 32768 33.3 and 38.6; 400 x 50021
  // 17.0 and 14.2; 400 x 20000 fp32 13.9 and 11.8).
  if (S == 1 && a.V * (DT == MSK_FP32 ? 4 : 2) > 65536) {
    const OpsLaunch l(dim3((unsigned)std::min<long long>(a.rows, 2 * nsm)), kStreamThreads + 64, 0, st);
    return cudaLaunchKernelEx(&l.cfg, logprobs_stream_kernel<DT>, a);
  }
  const unsigned gy = (unsigned)std::min<long long>(a.rows, 65535);
  const OpsLaunch l(dim3((unsigned)S, gy, (unsigned)((a.rows + gy - 1) / gy)), S == 1 ? 128 : 512, 0, st, S);
  return S == 1 ? cudaLaunchKernelEx(&l.cfg, logprobs_kernel<DT, 128>, a) : cudaLaunchKernelEx(&l.cfg, logprobs_kernel<DT, 512>, a);
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
