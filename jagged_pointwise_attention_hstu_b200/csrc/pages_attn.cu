// Pointwise attention of new rows over a paged history.
//
// Row r of user b (n = lengths[b] cached rows) and head h:
//   s_j = q_r . k_j + rab_pos[min(n - j, clamp)] + rab_time[t(ts_r - ts_j)],  0 <= j < n
//   s_r = q_r . k_r + rab_pos[0] + rab_time[0]                               (the row itself)
//   O_r = (sum_j SiLU(s_j) v_j + SiLU(s_r) v_r) / n_norm
// A new action and an M-FALCON candidate are the same case: both sit at
// position n and see the cached rows and themselves.  There is no softmax, so
// parts of a history join by a plain sum.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "internal.h"
#include "pages.cuh"

namespace hstu {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int FMT>
__device__ __forceinline__ float page_value(const PagesArgs& a, int64_t block, int c) {
  if (FMT == HSTU_PAGES_FP32) return static_cast<const float*>(a.kv)[block * a.hd + c];
  if (FMT == HSTU_PAGES_BF16)
    return __uint_as_float(uint32_t(static_cast<const uint16_t*>(a.kv)[block * a.hd + c]) << 16);
  const uint8_t q = static_cast<const uint8_t*>(a.kv)[block * a.hd + c];
  const __half_raw h = __nv_cvt_fp8_to_halfraw(q, __NV_E4M3);
  return __half2float(__half(h)) * block_scale(a.scales[block]);
}

template <int FMT>
__device__ __forceinline__ float row_value(const PagesArgs& a, int64_t i) {
  if (FMT == HSTU_PAGES_FP32) return static_cast<const float*>(a.uvqk)[i];
  return __uint_as_float(uint32_t(static_cast<const uint16_t*>(a.uvqk)[i]) << 16);
}

// One warp per (user, head): the user's rows one after the other, the keys in
// order, a lane per dimension.
template <int FMT, int E>   // head_dim = 32 * E
__global__ void __launch_bounds__(256) pages_attention_kernel(const PagesArgs a) {
  __shared__ int64_t s_thr[256];
  for (int k = threadIdx.x; k < a.time_buckets; k += blockDim.x) s_thr[k] = a.thresholds[k];
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int64_t wid = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (wid >= int64_t(a.B) * a.H) return;
  const int b = int(wid / a.H), h = int(wid % a.H);
  const int64_t r0 = a.offsets[b], r1 = a.offsets[b + 1];
  int err = 0;
  if (r0 < 0 || r1 < r0 || r1 > a.R || (b == 0 && r0 != 0)) err = HSTU_DEVERR_OFFSETS;
  int64_t n = a.lengths[b];
  if (n < 0 || n > (int64_t(a.width) << a.page_shift)) err |= HSTU_DEVERR_PAGES;
  if (err != 0) {
    if (lane == 0) atomicOr(a.error, err);
    return;
  }
  for (int64_t r = r0; r < r1; ++r) {
    const int64_t base = r * 4 * a.d + h * a.hd + lane;
    float q[E], o[E];
    float self = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[e] = row_value<FMT>(a, base + 2 * a.d + 32 * e);
      o[e] = 0.f;
      self = fmaf(q[e], row_value<FMT>(a, base + 3 * a.d + 32 * e), self);
    }
    const int64_t ts = a.ts[r];
    if (ts < 0 || ts >= kMaxTimestamp) err |= HSTU_DEVERR_TIMESTAMPS;
    for (int64_t j = 0; j < n; ++j) {
      const int32_t page = a.table[int64_t(b) * a.width + (j >> a.page_shift)];
      if (page < 0 || page >= a.num_pages) {
        err |= HSTU_DEVERR_PAGES;
        continue;
      }
      const int64_t slot = j & ((1 << a.page_shift) - 1);
      const int64_t block = ((int64_t(page) * a.H + h) * 2 << a.page_shift) + slot;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q[e], page_value<FMT>(a, block, lane + 32 * e), s);
      s = warp_sum(s);
      const int64_t dp = n - j;
      s += a.rab_pos[dp > a.pos_clamp ? a.pos_clamp : dp];
      const int64_t then = a.page_ts[(int64_t(page) << a.page_shift) + slot];
      s += a.rab_time[time_bucket(s_thr, a.time_buckets, ts - then)];
      const float p = s / (1.0f + expf(-s));
#pragma unroll
      for (int e = 0; e < E; ++e)
        o[e] = fmaf(p, page_value<FMT>(a, block + (int64_t(1) << a.page_shift), lane + 32 * e), o[e]);
    }
    self = warp_sum(self) + a.rab_pos[0] + a.rab_time[0];
    const float p = self / (1.0f + expf(-self));
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e] = fmaf(p, row_value<FMT>(a, base + a.d + 32 * e), o[e]);
      a.av[r * a.d + h * a.hd + lane + 32 * e] = o[e] / float(a.n_norm);
    }
  }
  if (err != 0 && lane == 0) atomicOr(a.error, err);
}

}  // namespace

cudaError_t launch_pages_attention(const PagesArgs& a, cudaStream_t st) {
  if (a.R <= 0 || a.B <= 0) return cudaSuccess;
  const unsigned blocks = unsigned((int64_t(a.B) * a.H + 7) / 8);
#define HSTU_PAGES_ATTN(F, E) pages_attention_kernel<F, E><<<blocks, 256, 0, st>>>(a)
  if (a.format == HSTU_PAGES_FP32) {
    switch (a.hd) {
      case 32: HSTU_PAGES_ATTN(HSTU_PAGES_FP32, 1); break;
      case 64: HSTU_PAGES_ATTN(HSTU_PAGES_FP32, 2); break;
      case 96: HSTU_PAGES_ATTN(HSTU_PAGES_FP32, 3); break;
      case 128: HSTU_PAGES_ATTN(HSTU_PAGES_FP32, 4); break;
      default: return cudaErrorInvalidValue;
    }
  } else if (a.format == HSTU_PAGES_BF16) {
    if (a.hd == 64) HSTU_PAGES_ATTN(HSTU_PAGES_BF16, 2);
    else if (a.hd == 128) HSTU_PAGES_ATTN(HSTU_PAGES_BF16, 4);
    else return cudaErrorInvalidValue;
  } else {
    if (a.hd == 64) HSTU_PAGES_ATTN(HSTU_PAGES_E4M3, 2);
    else if (a.hd == 128) HSTU_PAGES_ATTN(HSTU_PAGES_E4M3, 4);
    else return cudaErrorInvalidValue;
  }
#undef HSTU_PAGES_ATTN
  return cudaGetLastError();
}

}  // namespace hstu
