// Paged history: rows of SiLU(f1(X)) kept in pages, written (and quantised) a
// row at a time and read back.
//
// A user's history grows by single actions and users come and go, so the keys
// and values of one layer live in pages of page_size rows
//   kv [num_pages, H, 2, page_size, head_dim]      plane 0 keys, plane 1 values
// and position j of user b is row j % page_size of page table[b][j / page_size].
// One head's keys of a page are one contiguous run of page_size * head_dim
// elements, its values the next: what the attention of one head reads.
//
// E4M3 pages hold a block (one head's key or value of one row) x as codes times
// a power of two: with m = max |x_i| over the finite x_i and e the smallest
// integer with m <= 448 * 2^e (held in [-126, 120]; 0 when m = 0), code_i is
// x_i * 2^-e rounded to the nearest e4m3, ties to even.  A power of two and not
// m / 448: x * 2^-e and code * 2^e are then exact, so e4m3's own rounding (2^-4
// relative at most in its normal range) is the only one, reading back into bf16
// is exact, and e4m3 being a floating type a finer scale would not make the
// codes more precise.  Codes are held to 448, at e = 120 to 240: code * 2^e stays
// finite.  Infinities and NaN become NaN codes, e4m3's only non-finite value.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "pages.cuh"

namespace hstu {
namespace {

constexpr int kRowWarps = 8;   // rows (warps) per block of the write and read kernels

// The largest b with offs[b] <= r, for 0 <= r < offs[B], found by the whole
// warp: 32 probes a step, so one step for up to 32 users and two for 1024.
__device__ __forceinline__ int32_t user_of_row(const int32_t* __restrict__ offs, int32_t B,
                                               int64_t r, int lane) {
  int32_t lo = 0, n = B;   // the answer is in [lo, lo + n)
  while (n > 1) {
    const int32_t step = (n + 31) >> 5;
    const int32_t k = lane * step;
    const bool le = k < n && int64_t(__ldg(offs + lo + k)) <= r;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int32_t top = m == 0 ? 0 : 31 - __clz(m);
    lo += top * step;
    n = n - top * step < step ? n - top * step : step;
  }
  return lo;
}

struct Place {
  int64_t row;   // (page * H) * 2 * page_size + slot: the block of plane 0 of head 0
  int64_t ts;    // index into the page timestamps
  int err;
  bool ok;
};

// What place_of does not see, by the first block: an offsets table that does not
// start at zero, falls, or ends behind the rows.
__device__ __forceinline__ void check_offsets(const PagesArgs& a) {
  if (blockIdx.x != 0) return;
  bool bad = false;
  for (int32_t i = threadIdx.x; i < a.B; i += blockDim.x) {
    const int32_t lo = __ldg(a.offsets + i), hi = __ldg(a.offsets + i + 1);
    bad |= lo > hi || (i == 0 && lo != 0) || (i == a.B - 1 && hi > a.R);
  }
  if (bad) atomicOr(a.error, HSTU_DEVERR_OFFSETS);
}

// Where row r of the call lives, by the whole warp; `ok` false: nowhere (a row
// behind the last sequence, or an error).
__device__ __forceinline__ Place place_of(const PagesArgs& a, int64_t r, int lane) {
  Place p;
  p.ok = false;
  p.err = 0;
  p.row = 0;
  p.ts = 0;
  const int32_t b = user_of_row(a.offsets, a.B, r, lane);
  const int64_t r0 = __ldg(a.offsets + b), r1 = __ldg(a.offsets + b + 1);
  if (r < r0 || r >= r1 || r0 < 0 || r1 > a.R) {
    // behind the last sequence, or a table that check_offsets reports
    return p;
  }
  if (a.one_row && r1 - r0 > 1) {
    p.err = HSTU_DEVERR_PAGES;
    return p;
  }
  const int64_t pos = (a.lengths != nullptr ? int64_t(__ldg(a.lengths + b)) : 0) + (r - r0);
  if (pos < 0 || (pos >> a.page_shift) >= a.width) {
    p.err = HSTU_DEVERR_PAGES;
    return p;
  }
  const int32_t page = __ldg(a.table + int64_t(b) * a.width + (pos >> a.page_shift));
  if (page < 0 || page >= a.num_pages) {
    p.err = HSTU_DEVERR_PAGES;
    return p;
  }
  const int32_t slot = int32_t(pos & ((1 << a.page_shift) - 1));
  p.row = ((int64_t(page) * a.H * 2) << a.page_shift) + slot;
  p.ts = (int64_t(page) << a.page_shift) + slot;
  p.ok = true;
  return p;
}

// Quantises eight values of one block whose finite maximum is m; 2^-e exact.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float m, int& e) {
  e = block_exponent(m);
  const float inv = __int_as_float((127 - e) << 23);
  const float top = e == kMaxExponent ? 240.f : 448.f;
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float u = x[2 * i] * inv, v = x[2 * i + 1] * inv;
    // fminf and fmaxf drop a NaN: a non-finite value is put back as NaN
    u = fabsf(x[2 * i]) < INFINITY ? fminf(fmaxf(u, -top), top) : NAN;
    v = fabsf(x[2 * i + 1]) < INFINITY ? fminf(fmaxf(v, -top), top) : NAN;
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(u, v), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// One warp per row: the row's keys and values in chunks of 16 bytes, a lane a
// chunk, straight into the row's blocks.  Bound by memory: a row reads
// 2d elements and writes them (or their codes) once.
template <int FMT>
__global__ void __launch_bounds__(kRowWarps * 32) pages_write_kernel(const PagesArgs a) {
  constexpr int kElems = FMT == HSTU_PAGES_FP32 ? 4 : 8;   // elements of a chunk
  check_offsets(a);
  const int lane = threadIdx.x & 31;
  const int64_t r = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (r >= a.R) return;
  const Place p = place_of(a, r, lane);
  if (!p.ok) {
    if (p.err != 0 && lane == 0) atomicOr(a.error, p.err);
    return;
  }
  const uint4* src = static_cast<const uint4*>(a.uvqk) + r * (4 * a.d / kElems);
  const int per_plane = a.d / kElems, per_head = a.hd / kElems;
  const int chunks = 2 * per_plane;
  if (lane == 0 && a.ts != nullptr) {
    const int64_t t = a.ts[r];
    if (t < 0 || t >= kMaxTimestamp) atomicOr(a.error, HSTU_DEVERR_TIMESTAMPS);
    a.page_ts[p.ts] = t;
  }
  for (int c0 = 0; c0 < chunks; c0 += 32) {
    const int c = c0 + lane;
    const bool on = c < chunks;
    const int plane = c >= per_plane ? 1 : 0;
    const int k = c - plane * per_plane;              // chunk of the plane
    const int h = on ? k / per_head : 0;
    const int64_t block = p.row + ((int64_t(2 * h + plane)) << a.page_shift);
    // input columns: U | V | Q | K
    const uint4 v = on ? __ldg(src + (plane == 0 ? 3 : 1) * per_plane + k)
                       : make_uint4(0u, 0u, 0u, 0u);
    if (FMT != HSTU_PAGES_E4M3) {
      if (on) static_cast<uint4*>(a.kv)[block * per_head + (k - h * per_head)] = v;
    } else {
      float x[8];
      unpack_bf16(v, x);
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
      // the lanes of one block are neighbours: 8 (head dim 64) or 16 (128)
      for (int o = per_head >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      int e;
      const uint2 q = quantise8(x, m, e);
      if (on) {
        static_cast<uint2*>(a.kv)[block * per_head + (k - h * per_head)] = q;
        if (k == h * per_head) a.scales[block] = uint8_t(e + 127);
      }
    }
  }
}

// The way back: a warp per row, pages into the K and V columns of U|V|Q|K.
template <int FMT>
__global__ void __launch_bounds__(kRowWarps * 32) pages_read_kernel(const PagesArgs a) {
  constexpr int kElems = FMT == HSTU_PAGES_FP32 ? 4 : 8;
  check_offsets(a);
  const int lane = threadIdx.x & 31;
  const int64_t r = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (r >= a.R) return;
  const Place p = place_of(a, r, lane);
  if (!p.ok) {
    if (p.err != 0 && lane == 0) atomicOr(a.error, p.err);
    return;
  }
  uint4* dst = static_cast<uint4*>(a.out) + r * (4 * a.d / kElems);
  const int per_plane = a.d / kElems, per_head = a.hd / kElems;
  const int chunks = 2 * per_plane;
  if (lane == 0 && a.ts_out != nullptr) a.ts_out[r] = a.page_ts[p.ts];
  for (int c = lane; c < chunks; c += 32) {
    const int plane = c >= per_plane ? 1 : 0;
    const int k = c - plane * per_plane;
    const int h = k / per_head;
    const int64_t block = p.row + ((int64_t(2 * h + plane)) << a.page_shift);
    uint4 v;
    if (FMT != HSTU_PAGES_E4M3) {
      v = __ldg(static_cast<const uint4*>(a.kv) + block * per_head + (k - h * per_head));
    } else {
      const uint2 q = __ldg(static_cast<const uint2*>(a.kv) + block * per_head + (k - h * per_head));
      const float s = block_scale(__ldg(a.scales + block));
      float x[8];
      unpack_e4m3(q.x, x);
      unpack_e4m3(q.y, x + 4);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // exact: 4 significant bits
        const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i] * s, x[2 * i + 1] * s);
        w[i] = *reinterpret_cast<const uint32_t*>(&t);
      }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    dst[(plane == 0 ? 3 : 1) * per_plane + k] = v;
  }
}

}  // namespace

cudaError_t launch_pages_write(const PagesArgs& a, cudaStream_t st) {
  if (a.R <= 0 || a.B <= 0) return cudaSuccess;
  const unsigned blocks = unsigned((a.R + kRowWarps - 1) / kRowWarps);
  switch (a.format) {
    case HSTU_PAGES_BF16: pages_write_kernel<HSTU_PAGES_BF16><<<blocks, kRowWarps * 32, 0, st>>>(a); break;
    case HSTU_PAGES_FP32: pages_write_kernel<HSTU_PAGES_FP32><<<blocks, kRowWarps * 32, 0, st>>>(a); break;
    case HSTU_PAGES_E4M3: pages_write_kernel<HSTU_PAGES_E4M3><<<blocks, kRowWarps * 32, 0, st>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_pages_read(const PagesArgs& a, cudaStream_t st) {
  if (a.R <= 0 || a.B <= 0) return cudaSuccess;
  const unsigned blocks = unsigned((a.R + kRowWarps - 1) / kRowWarps);
  switch (a.format) {
    case HSTU_PAGES_BF16: pages_read_kernel<HSTU_PAGES_BF16><<<blocks, kRowWarps * 32, 0, st>>>(a); break;
    case HSTU_PAGES_FP32: pages_read_kernel<HSTU_PAGES_FP32><<<blocks, kRowWarps * 32, 0, st>>>(a); break;
    case HSTU_PAGES_E4M3: pages_read_kernel<HSTU_PAGES_E4M3><<<blocks, kRowWarps * 32, 0, st>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace hstu
