// Device helpers shared by the serving kernels (packed prefill, page tables, 8-bit cache).
#pragma once

#include <atomic>
#include <utility>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {

// further status details (dsa_common.cuh holds the first ones)
enum : unsigned {
  DETAIL_CAP_PAGES = 23, DETAIL_CAP_TOKENS = 24, DETAIL_CAP_TABLE = 25,
  DETAIL_BAD_SEQ = 37, DETAIL_BAD_LEN = 38, DETAIL_BAD_PAGE = 39, DETAIL_BAD_SLOT = 40, DETAIL_BAD_SCALE = 41,
  DETAIL_HELD = 42,
};

// launch_pdl_cluster with dynamic shared memory.
template <typename... KArgs, typename... Args>
inline cudaError_t serve_launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, int cluster, size_t smem,
                                        cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// SMs of the current device, looked up once per device (an attribute costs a driver call).
inline cudaError_t serve_sms(int* dev, int* sms) {
  static std::atomic<int> known[64];
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>* k = *dev < 64 ? &known[*dev] : nullptr;
  *sms = k ? k->load(std::memory_order_relaxed) : 0;
  if (*sms == 0) {
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
    if (e == cudaSuccess && k) k->store(*sms, std::memory_order_relaxed);
  }
  return e;
}

// Lets a kernel use `bytes` of dynamic shared memory on device `dev`, once per device.
template <auto Kernel>
inline cudaError_t serve_allow_smem(int dev, int bytes) {
  static std::atomic<uint64_t> done;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A dimension of a strided array: its size, and the distance of its neighbours.
struct ServeDim {
  int64_t n, stride;
};
// Whether the array's rows of `row` units are apart: with the dimensions in order of their strides, each steps over all
// that the smaller ones span.  (Layouts that interleave rows in any other way are taken for overlapping ones.)
template <int N>
inline bool serve_apart(int64_t row, ServeDim (&dims)[N]) {
  for (int i = 1; i < N; ++i)
    for (int j = i; j > 0 && dims[j].stride < dims[j - 1].stride; --j) std::swap(dims[j], dims[j - 1]);
  __int128 span = row;
  for (const ServeDim& d : dims) {
    if (d.n < 2) continue;
    if (d.stride < span) return false;
    span += (__int128)(d.n - 1) * d.stride;
  }
  return true;
}

inline bool serve_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16 (bf16 inputs, fp32 accumulate).
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Waits for a phase, bounded by the default limit whatever the launch's own and ignoring
// the abort flag: used to let copies and MMAs in flight finish before a CTA ends.
static __device__ __noinline__ void serve_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) return;
  }
}

// Waits for a phase, bounded like mbar_wait.  With `poll` the thread keeps asking; without it, the hardware
// suspends it, which leaves the issue slots to others but wakes it some hundred cycles later.
static __device__ __noinline__ bool serve_wait_loop(uint64_t* bar, uint32_t parity, uint64_t limit, unsigned* status,
                                                    unsigned detail, volatile int* abort_flag, bool poll) {
  const uint64_t t0 = globaltimer_ns();
  uint32_t spins = 0;
  while (true) {
    if (poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if (((++spins) & 7u) == 0u) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > limit) {
        report_timeout(status, detail, abort_flag);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool serve_wait(uint64_t* bar, uint32_t parity, uint64_t limit, unsigned* status, unsigned detail,
                                           volatile int* abort_flag, bool poll = false) {
  if (mbar_test_wait(bar, parity)) return true;
  return serve_wait_loop(bar, parity, limit, status, detail, abort_flag, poll);
}
// One lane waits, the whole warp learns the outcome.
__device__ __forceinline__ bool serve_warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit, unsigned* status,
                                                unsigned detail, volatile int* abort_flag, bool poll = false) {
  if (__builtin_expect(__all_sync(0xffffffffu, mbar_test_wait(bar, parity)), 1)) return true;
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = serve_wait_loop(bar, parity, limit, status, detail, abort_flag, poll) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

// serve_warp_wait without any call: for threads with so many live registers that a call would spill them.
__device__ __forceinline__ bool serve_warp_wait_inline(uint64_t* bar, uint32_t parity, uint64_t limit, unsigned* status,
                                                       unsigned detail, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  int ok = 1;
  if ((threadIdx.x & 31) == 0) {
    const uint64_t t0 = globaltimer_ns();
    uint32_t spins = 0;
    while (!mbar_test_wait(bar, parity)) {
      if (((++spins) & 63u) != 0u) continue;
      if (*abort_flag) { ok = 0; break; }
      if (globaltimer_ns() - t0 > limit) {
        report(status, DSA_ERR_TIMEOUT, detail);
        *abort_flag = 1;
        ok = 0;
        break;
      }
    }
  }
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

__device__ __forceinline__ float serve_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float serve_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// (x0, x1) = (a0, a1) * b + c as one packed multiply-add
__device__ __forceinline__ void serve_fma2(float a0, float a1, float b, float c, float& x0, float& x1) {
  uint64_t av, bv, cv, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(av) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(bv) : "f"(b), "f"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(cv) : "f"(c), "f"(c));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(av), "l"(bv), "l"(cv));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(r));
}

// (x0, x1) = (a0, a1) * (b0, b1) + (c0, c1) as one packed multiply-add
__device__ __forceinline__ void serve_fma2v(float a0, float a1, float b0, float b1, float c0, float c1, float& x0, float& x1) {
  uint64_t av, bv, cv, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(av) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(bv) : "f"(b0), "f"(b1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(cv) : "f"(c0), "f"(c1));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(av), "l"(bv), "l"(cv));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(r));
}

// (s0, s1) += (a, b) as one packed add
__device__ __forceinline__ void serve_add2(float& s0, float& s1, float a, float b) {
  uint64_t sv, av;
  asm("mov.b64 %0, {%1, %2};" : "=l"(sv) : "f"(s0), "f"(s1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(av) : "f"(a), "f"(b));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sv) : "l"(av));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(s0), "=f"(s1) : "l"(sv));
}

// (2^x0, 2^x1) on the multiply-add pipe, for x <= 100: 2^x = 2^n 2^f with n the nearest integer and a polynomial of
// degree 5 in f (|f| <= 1/2, fitted for a small largest relative error: 1.55e-7 with the coefficients below, 1.2e-7 at
// f = 0; 2.1e-7 with its roundings).
// Below -127 the result is 0, for -infinity too; NaN stays NaN.
__device__ __forceinline__ void serve_ex2_poly2(float x0, float x1, float& p0, float& p1) {
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x0));  // -127
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x1));
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: the sum's low bits are n
  float t0 = kRound, t1 = kRound, r0, r1, f0, f1;
  serve_add2(t0, t1, x0, x1);
  r0 = t0;
  r1 = t1;
  serve_add2(r0, r1, -kRound, -kRound);
  serve_fma2v(r0, r1, -1.f, -1.f, x0, x1, f0, f1);
  float y0 = 0.0013276472454890609f, y1 = y0;
  constexpr float c[5] = {1.0000001192092896f, 0.6931469440460205f, 0.24022120237350464f, 0.05550713092088699f, 0.009675540961325169f};
#pragma unroll
  for (int i = 4; i >= 0; --i) serve_fma2v(y0, y1, f0, f1, c[i], c[i], y0, y1);
  const float s0 = __int_as_float((__float_as_int(t0) << 23) + 0x3f800000);
  const float s1 = __int_as_float((__float_as_int(t1) << 23) + 0x3f800000);
  serve_fma2v(y0, y1, s0, s1, 0.f, 0.f, p0, p1);
}

// 16 consecutive 32-bit columns of this thread's TMEM lane
__device__ __forceinline__ void serve_tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void serve_tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// 32 bytes to global memory in one store (address 32-byte aligned)
__device__ __forceinline__ void serve_st_v8(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

}  // namespace dsa
