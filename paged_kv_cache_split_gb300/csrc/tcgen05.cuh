// tcgen05.cuh — the fifth-generation tensor-core instructions the latent kernels use
// (one CTA per tile, cta_group::1): shared-memory operand descriptors, the bf16 MMA
// with FP32 accumulators in tensor memory (TMEM), commits, and TMEM loads and stores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "pkv_internal.cuh"

namespace pkv {

// Operand in shared memory as boxes of rows of 128 bytes under the 128-byte swizzle
// (what a TMA copy with that swizzle writes), eight rows to a 1024-byte atom.
// K-major (a row holds 64 consecutive k of one m or n): atoms follow one another at
// `sbo` bytes along m or n; `lbo` is not used.  MN-major (a row holds 64 consecutive m
// of one k): atoms follow at `sbo` along k and at `lbo` along m.  Sixteen k further is
// 32 bytes on (K-major), or sixteen rows, 2048 bytes, on (MN-major).
__device__ __forceinline__ uint64_t tc_desc(uint32_t smem_addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: bf16 (or fp16) A and B, FP32 D; a_mn: A is MN-major, b_mn: B is.
__host__ __device__ constexpr uint32_t tc_idesc(int M, int N, bool a_mn, bool b_mn, bool fp16 = false) {
  return (1u << 4) | (fp16 ? 0u : (1u << 7) | (1u << 10)) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A B for one k-step of 16 (A and B in shared memory); one thread issues.
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// The same with A in tensor memory (bf16 pairs, one row per lane).
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// Arrive on `bar` once every MMA this thread issued so far has completed.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Writes of this thread to shared memory become visible to the asynchronous proxy
// (MMA operands, TMA).
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Allocation of TMEM columns (a power of two, at least 32) by one converged warp.
__device__ __forceinline__ void tc_alloc(uint32_t* smem_out, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_out)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}

#define PKV_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), \
                     "=r"(r[o + 6]), "=r"(r[o + 7])
#define PKV_W8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), \
                     "r"(r[o + 6]), "r"(r[o + 7])

// One lane per row, N consecutive 32-bit columns (the warp's 32 lanes).
template <int N>
__device__ __forceinline__ void tc_ld_rows(uint32_t addr, uint32_t (&r)[N]) {
  static_assert(N == 16 || N == 32, "columns per load");
  if constexpr (N == 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : PKV_R8(r, 0), PKV_R8(r, 8)
        : "r"(addr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : PKV_R8(r, 0), PKV_R8(r, 8), PKV_R8(r, 16), PKV_R8(r, 24)
        : "r"(addr));
}
template <int N>
__device__ __forceinline__ void tc_st_rows(uint32_t addr, const uint32_t (&r)[N]) {
  static_assert(N == 16 || N == 32, "columns per store");
  if constexpr (N == 16)
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::PKV_W8(
            r, 0),
        PKV_W8(r, 8), "r"(addr)
        : "memory");
  else
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::PKV_W8(r, 0),
        PKV_W8(r, 8), PKV_W8(r, 16), PKV_W8(r, 24), "r"(addr)
        : "memory");
}

// The warp's first 16 lanes, N columns, as N / 8 fragments of 16 rows x 8 columns: lane
// t holds rows t / 4 (r[4j], r[4j+1]) and t / 4 + 8 (r[4j+2], r[4j+3]) at columns
// 8j + 2 (t % 4) and the next.
template <int N>
__device__ __forceinline__ void tc_ld_frag16(uint32_t addr, uint32_t (&r)[N / 2]) {
  static_assert(N == 16 || N == 32 || N == 64, "columns");
  if constexpr (N == 16)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : PKV_R8(r, 0) : "r"(addr));
  else if constexpr (N == 32)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : PKV_R8(r, 0), PKV_R8(r, 8)
        : "r"(addr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : PKV_R8(r, 0), PKV_R8(r, 8), PKV_R8(r, 16), PKV_R8(r, 24)
        : "r"(addr));
}

// Waits are bounded.  The first one to give up sets the error word and `dead`; after that
// no wait blocks and nothing more is issued, so every thread still meets every barrier.
// Called by whole warps, which leave it converged.
__device__ __forceinline__ void wait_or_die(uint64_t* bar, uint32_t parity, volatile int* dead, int32_t* err) {
  if (!mbar_try_wait(bar, parity)) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
      if ((it & 63u) == 0) {
        if (*dead) break;
        if (global_timer_ns() - t0 > 1000000000ull) {
          atomicOr(err, ERR_TIMEOUT);
          *dead = 1;
          break;
        }
      }
    }
  }
  __syncwarp();
}

// The same for a whole converged warp, with warp-uniform control flow: the instructions
// that issue MMAs and copies take their operands from uniform registers, and a loop the
// compiler cannot prove uniform moves every operand there one by one (measured: 90 cycles
// per MMA issued by one diverged thread).  False when the wait gave up or the CTA is dead.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* dead, int32_t* err) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((it & 63u) == 0) {
      if (__any_sync(0xffffffffu, *dead)) return false;
      if (__any_sync(0xffffffffu, global_timer_ns() - t0 > 1000000000ull)) {
        atomicOr(err, ERR_TIMEOUT);
        *dead = 1;
        return false;
      }
    }
  }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}

// A value every lane holds, known to the compiler as warp-uniform.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ int64_t uniform(int64_t x) { return __shfl_sync(0xffffffffu, (long long)x, 0); }
__device__ __forceinline__ const uint8_t* lane_ptr(const uint8_t* p, int lane) {
  return reinterpret_cast<const uint8_t*>(
      (uintptr_t)__shfl_sync(0xffffffffu, (unsigned long long)(uintptr_t)p, lane));
}

// 2^x with the hardware approximation (relative error below 2^-22; tiny results flush to 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^e, e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ uint32_t fp16x2(float lo, float hi) {
  const __half2 t = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}

// Launch with programmatic dependence on the stream's previous kernel (the kernels wait
// for it before they touch global memory, and read that memory with ordinary loads: the
// previous kernel may write it while they are resident, which a non-coherent load does not
// allow).  The shared-memory limit of a kernel is raised
// once per device.
template <typename P>
inline cudaError_t tc_launch(void (*kernel)(P), dim3 grid, int threads, size_t smem, cudaStream_t stream, const P& p,
                             int device, std::atomic<uint64_t>* raised) {
  if (smem > 48 * 1024 && !(device < 64 && (raised->load(std::memory_order_relaxed) >> device & 1))) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (device < 64) raised->fetch_or(1ull << device);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace pkv
