// Device helpers of the paged history: block scales, unpacking, time buckets.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace hstu {

// The kernels of the paged history are launched while the kernel before them in the stream
// ends, and wait here, every thread and before any access to global memory, until that
// kernel and all it wrote are complete: the launch and the set-up of the blocks no longer lie
// between two calls (16 users of up to 4096 rows, d 512, e4m3 12.3 us a call without
// it and 10.4 with; 1 of 100003 28.7 and 26.6; 8 of 8192, d 1024, bf16 51.5 and 50.0).
__device__ __forceinline__ void wait_for_earlier_kernels() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Lets the next such kernel take the places of blocks that end.
__device__ __forceinline__ void let_next_kernel_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Behind that wait the caller's memory is read by ordinary loads (and bulk copies), never
// by __ldg: the read-only path takes what it reads for constant while the kernel runs, may
// keep lines that an SM read for the kernel before last, and its loads are not ordered behind
// the wait; the kernel before this one, which may still run when this one starts, writes pages,
// scales, times and rows.  Only the handle's own tables are constant.
template <class T>
__device__ __forceinline__ T fetch(const T* p) {
  return *p;
}
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned blocks, int threads, int smem,
                         cudaStream_t st, const A&... args) {
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(blocks);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = size_t(smem);
  c.stream = st;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

constexpr int kMinExponent = -126, kMaxExponent = 120;

// The smallest e with m <= 448 * 2^e (448 = 1.75 * 2^8), held in
// [kMinExponent, kMaxExponent]; 0 when m = 0.  m is finite and >= 0.
__device__ __forceinline__ int block_exponent(float m) {
  if (m == 0.f) return 0;
  const uint32_t bits = __float_as_uint(m);
  int e = int(bits >> 23) - 127 - 8;                    // m in [2^k, 2^(k + 1)): k - 8 ...
  if ((bits & 0x7FFFFFu) > 0x600000u) e += 1;           // ... or k - 7 above 1.75 * 2^k
  return e < kMinExponent ? kMinExponent : (e > kMaxExponent ? kMaxExponent : e);
}

// 2^(byte - 127) for the bytes a write makes (1 .. 247).
__device__ __forceinline__ float block_scale(uint8_t byte) {
  return __uint_as_float(uint32_t(byte) << 23);
}

__device__ __forceinline__ void unpack_bf16(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void unpack_e4m3(uint32_t v, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(v >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// bucket(dt) = #{k >= 1 : dt >= thr[k]}, gaps below zero count as zero.
__device__ __forceinline__ int time_bucket(const int64_t* thr, int nb, int64_t dt) {
  int lo = 0, hi = nb - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (dt >= thr[mid]) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace hstu
