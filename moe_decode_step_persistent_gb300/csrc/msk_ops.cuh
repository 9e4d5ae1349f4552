// Shared by the operators beside the step (4-bit cache, 4-bit products, log
// probabilities): element types, the device check of their entry points, and
// small device helpers.
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "../../include/msk.h"
#include "msk_device.cuh"

namespace msk {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // (msk_api.cu)

inline bool ops_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int dtype_bytes(int32_t t) { return t == MSK_FP32 ? 4 : 2; }
inline bool dtype_ok(int32_t t) { return t == MSK_BF16 || t == MSK_FP16 || t == MSK_FP32; }

// Whether the current device is one these kernels are compiled for; its SM
// count.  (Attributes are looked up by the runtime without a device call.)
inline msk_status ops_device(int* nsm) {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MSK_ERR_CUDA;
  return major == 10 && minor == 3 ? MSK_OK : MSK_ERR_UNSUPPORTED_DEVICE;
}

// Bound of every wait on an mbarrier (linear4_kernel and kv4_tc_kernel have
// them); after it a kernel records an error (msk_ops_check), ends its copies and
// MMAs, and returns.  Barriers of a block's threads and of a cluster's blocks have
// no limit: all of them come to each, also after a wait that ran out.
constexpr uint64_t kOpsWaitNs = 200ull * 1000 * 1000;
// ... and more for each step of a block's work, many times what it takes.
constexpr uint64_t kOpsStepNs = 20ull * 1000;

// The launches' attributes: a cluster, and that the kernel may start before the
// one in front of it has ended: it sets itself up, and touches global memory
// only behind grid_dep_wait().
struct OpsLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  OpsLaunch(dim3 grid, int threads, int smem, cudaStream_t st, int cluster = 1) {
    cfg.gridDim = grid, cfg.blockDim = dim3((unsigned)threads), cfg.dynamicSmemBytes = (size_t)smem, cfg.stream = st;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at, cfg.numAttrs = 2;
  }
};

// The SM count the workspace sizes are made for when there is no device to
// ask; kernels never use more blocks than a workspace has room for.
constexpr int kOpsSms = 152;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// Two 16-bit elements of a 32-bit word as floats.
__device__ __forceinline__ float2 unpack16(uint32_t w, bool fp16) {
  return fp16 ? unpack_f16x2(w) : make_float2(bf16_lo(w), bf16_hi(w));
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool fp16) {
  return fp16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

// Pairs of fp32 numbers and operations on them.
__device__ __forceinline__ unsigned long long pair(float x, float y) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(unsigned long long v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// The power of two by which a row of 16-bit floats with largest magnitude
// `amax` is multiplied before it is written as fp16, as an exponent: amax
// lands in [2^14, 2^15) of fp16's 65504, so that every element above 2^-31
// amax is exact in fp16 (bf16 has 8 significant bits; 2^-17 and above lie in
// steps of 2^-24 or wider), and smaller ones are off by at most 2^-25, that is
// 2^-39 amax.  An fp32 sum keeps less than that where amax has a part in it;
// where amax meets zeros, elements that small are what a caller loses.  The
// factor and its inverse stay normal fp32 numbers; at its limit even bf16's
// subnormals arrive exactly.
__device__ __forceinline__ int row_shift(float amax) {
  const int e = (int)(__float_as_uint(amax) >> 23) - 127;  // floor(log2), -127 for zero and subnormals
  return e < -112 ? 126 : (e > 127 ? -113 : 14 - e);
}

// 8-byte global -> shared copy.
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(dst), "l"(src) : "memory");
}

// --- thread-block clusters ---------------------------------------------------

// The address of block `rank`'s counterpart of a shared-memory address.
__device__ __forceinline__ uint32_t mapa(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
// A store into another block's shared memory that its mbarrier counts (4 bytes).
__device__ __forceinline__ void st_async(uint32_t addr, float v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(addr), "f"(v), "r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() { cluster_arrive(), cluster_wait(); }

// --- tensor cores: 16-bit operands (beside msk_tc.cuh's 4-bit ones) -------------

// Shared-memory descriptor bits of the 128-byte swizzle (16-byte piece p of
// row r at p ^ (r mod 8)).
constexpr uint64_t kSwizzle128 = 2ull << 61;

// D (tensor memory) = [D +] A B^T, 16-bit operands with fp32 accumulators: A
// from tensor memory (ts) or shared memory (ss), B from shared memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// 32 consecutive columns of the warp's 32 lanes, written and read.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

}  // namespace msk
