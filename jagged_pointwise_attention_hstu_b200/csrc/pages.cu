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
  // a length is an int32, and the rows of a user fewer than 2^30: no overflow past int64
  const int64_t pos = (a.lengths != nullptr ? int64_t(__ldg(a.lengths + b)) : 0) + (r - r0);
  if (pos < 0 || (pos >> a.page_shift) >= a.width) {
    p.err = HSTU_DEVERR_PAGES;
    return p;
  }
  const int32_t page = __ldg(a.table + (int64_t(b) * a.width + (pos >> a.page_shift)));
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

// Four codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t four_codes(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(w) : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}

constexpr uint32_t kAbs = 0x7fff7fffu;
// Two maxima of bf16; a NaN stays one.
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Codes of a lane's eight bf16 of a block that kLanes neighbouring lanes hold,
// and the block's scale byte; by the whole warp.
//
// The maximum is taken of two bf16 at a time, and nothing is clamped, since
// |x| <= 448 * 2^e by the choice of e.  Values that are not finite, and the
// exponent that is held at 120, sit above 448 * 2^119 = bits 0x7F60: a warp
// that has one takes the long way.
template <int kLanes>
__device__ __forceinline__ uint2 quantise8(const uint4& v, int& scale) {
  uint32_t top = max2(max2(v.x & kAbs, v.y & kAbs), max2(v.z & kAbs, v.w & kAbs));
#pragma unroll
  for (int o = kLanes >> 1; o > 0; o >>= 1) top = max2(top, __shfl_xor_sync(0xffffffffu, top, o));
  top = max(top & 0xffffu, top >> 16);
  float x[8];
  unpack_bf16(v, x);
  uint2 c;
  if (!__any_sync(0xffffffffu, top > 0x7F60u)) {
    // e + 127 with e = k - 8 for top in (1.75 * 2^(k - 1), 1.75 * 2^k]: 0x1F carries above it
    scale = max(int((top + 0x1Fu) >> 7) - 8, kMinExponent + 127);
    scale = top == 0 ? 127 : scale;
    const float inv = __int_as_float((254 - scale) << 23);
    c.x = four_codes(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    c.y = four_codes(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
  } else {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
#pragma unroll
    for (int o = kLanes >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int e = block_exponent(m);
    const float inv = __int_as_float((127 - e) << 23), most = e == kMaxExponent ? 240.f : 448.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)   // fminf and fmaxf would drop a NaN
      x[i] = fabsf(x[i]) < INFINITY ? fminf(fmaxf(x[i] * inv, -most), most) : NAN;
    c.x = four_codes(x[0], x[1], x[2], x[3]);
    c.y = four_codes(x[4], x[5], x[6], x[7]);
    scale = e + 127;
  }
  return c;
}

// A row's keys and values in chunks of 16 bytes, heads of the keys first: lane
// `lane` has the chunks lane, lane + 32, ..., which are the same place of a
// block's kPerHead whatever the block (96, fp32 only: heads of 24 chunks).
template <int FMT, int HD>
struct Chunks {
  static constexpr int kElems = FMT == HSTU_PAGES_FP32 ? 4 : 8;   // elements of a chunk
  static constexpr int kPerHead = HD / kElems;
  static constexpr int kBatch = 4;                                // of a lane, loaded at once
  int lane, H, shift;
  __device__ __forceinline__ Chunks(const PagesArgs& a)
      : lane(threadIdx.x & 31), H(a.H), shift(a.page_shift) {}
  __device__ __forceinline__ int all() const { return 2 * H * kPerHead; }
  // of U | V | Q | K: K (the first half), then V
  __device__ __forceinline__ int column(int c) const { return c + (c < H * kPerHead ? 3 * H * kPerHead : 0); }
  __device__ __forceinline__ int in(int c) const {
    return 32 % kPerHead == 0 ? lane % kPerHead : c % kPerHead;
  }
  // of the block, from the row's first: head h's keys are block 2h, its values 2h + 1
  __device__ __forceinline__ int block(int c) const {
    const int b = c / kPerHead;
    return (2 * b - (b < H ? 0 : 2 * H - 1)) << shift;
  }
};

// One warp per row, a lane a chunk, straight into the row's blocks.  Bound by
// memory: a row reads 2d elements and writes them (or their codes) once.  All
// of a lane's loads (d 1024: 8) are on their way before the row's place is
// looked up.  What it took to get there were fewer instructions, about 75 a
// chunk of e4m3 (65536 rows of d 1024: 137 us at 205).
template <int FMT, int HD>
__global__ void __launch_bounds__(kRowWarps * 32) pages_write_kernel(const PagesArgs a) {
  using C = Chunks<FMT, HD>;
  check_offsets(a);
  const int64_t r = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (r >= a.R) return;
  const C ch(a);
  const int all = ch.all();
  const uint4* src = static_cast<const uint4*>(a.uvqk) + r * (2 * all);
  uint4 v[C::kBatch];
  auto load = [&](int c0) {
#pragma unroll
    for (int i = 0; i < C::kBatch; ++i) {
      const int c = c0 + 32 * i + ch.lane;
      v[i] = c < all ? __ldg(src + ch.column(c)) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  load(0);
  const Place p = place_of(a, r, ch.lane);
  if (!p.ok) {
    if (p.err != 0 && ch.lane == 0) atomicOr(a.error, p.err);
    return;
  }
  if (ch.lane == 0 && a.ts != nullptr) {
    const int64_t t = a.ts[r];
    if (t < 0 || t >= kMaxTimestamp) atomicOr(a.error, HSTU_DEVERR_TIMESTAMPS);
    a.page_ts[p.ts] = t;
  }
  uint4* to = static_cast<uint4*>(a.kv) + p.row * C::kPerHead;
  uint2* codes = static_cast<uint2*>(a.kv) + p.row * C::kPerHead;
  uint8_t* scales = a.scales + p.row;
  for (int c0 = 0;;) {
#pragma unroll
    for (int i = 0; i < C::kBatch; ++i) {
      if (c0 + 32 * i >= all) break;
      const int c = c0 + 32 * i + ch.lane;
      const int block = ch.block(c), in = ch.in(c);
      if constexpr (FMT != HSTU_PAGES_E4M3) {
        if (c < all) to[block * C::kPerHead + in] = v[i];
      } else {
        int scale;
        const uint2 q = quantise8<C::kPerHead>(v[i], scale);
        if (c < all) {
          codes[block * C::kPerHead + in] = q;
          if (in == 0) scales[block] = uint8_t(scale);
        }
      }
    }
    c0 += 32 * C::kBatch;
    if (c0 >= all) break;
    load(c0);
  }
}

// The way back: a warp per row, pages into the K and V columns of U|V|Q|K.
template <int FMT, int HD>
__global__ void __launch_bounds__(kRowWarps * 32) pages_read_kernel(const PagesArgs a) {
  using C = Chunks<FMT, HD>;
  check_offsets(a);
  const int64_t r = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (r >= a.R) return;
  const C ch(a);
  const int all = ch.all();
  const Place p = place_of(a, r, ch.lane);
  if (!p.ok) {
    if (p.err != 0 && ch.lane == 0) atomicOr(a.error, p.err);
    return;
  }
  uint4* dst = static_cast<uint4*>(a.out) + r * (2 * all);
  const uint4* from = static_cast<const uint4*>(a.kv) + p.row * C::kPerHead;
  const uint2* codes = static_cast<const uint2*>(a.kv) + p.row * C::kPerHead;
  const uint8_t* scales = a.scales + p.row;
  if (ch.lane == 0 && a.ts_out != nullptr) a.ts_out[r] = a.page_ts[p.ts];
  for (int c0 = ch.lane; c0 < all; c0 += 32 * C::kBatch) {
    uint4 v[C::kBatch];
    float s[C::kBatch];
#pragma unroll
    for (int i = 0; i < C::kBatch; ++i) {
      const int c = c0 + 32 * i;
      if (c >= all) continue;
      const int block = ch.block(c), at = block * C::kPerHead + ch.in(c);
      if constexpr (FMT != HSTU_PAGES_E4M3) {
        v[i] = __ldg(from + at);
      } else {
        const uint2 q = __ldg(codes + at);
        v[i].x = q.x;
        v[i].y = q.y;
        s[i] = block_scale(__ldg(scales + block));
      }
    }
#pragma unroll
    for (int i = 0; i < C::kBatch; ++i) {
      const int c = c0 + 32 * i;
      if (c >= all) continue;
      if constexpr (FMT == HSTU_PAGES_E4M3) {
        float x[8];
        unpack_e4m3(v[i].x, x);
        unpack_e4m3(v[i].y, x + 4);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {   // exact: 4 significant bits
          const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * e] * s[i], x[2 * e + 1] * s[i]);
          w[e] = *reinterpret_cast<const uint32_t*>(&t);
        }
        v[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      dst[ch.column(c)] = v[i];
    }
  }
}

}  // namespace

#define HSTU_PAGES_ROWS(KERNEL, F, D) \
  KERNEL<F, D><<<blocks, kRowWarps * 32, 0, st>>>(a); \
  return cudaGetLastError()
#define HSTU_PAGES_DISPATCH(KERNEL)                                                 \
  if (a.R <= 0 || a.B <= 0) return cudaSuccess;                                     \
  const unsigned blocks = unsigned((a.R + kRowWarps - 1) / kRowWarps);              \
  switch (a.format * 256 + a.hd) {                                                  \
    case HSTU_PAGES_BF16 * 256 + 64: HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_BF16, 64);   \
    case HSTU_PAGES_BF16 * 256 + 128: HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_BF16, 128); \
    case HSTU_PAGES_E4M3 * 256 + 64: HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_E4M3, 64);   \
    case HSTU_PAGES_E4M3 * 256 + 128: HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_E4M3, 128); \
    case HSTU_PAGES_FP32 * 256 + 32: HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_FP32, 32);   \
    case HSTU_PAGES_FP32 * 256 + 64: HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_FP32, 64);   \
    case HSTU_PAGES_FP32 * 256 + 96: HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_FP32, 96);   \
    case HSTU_PAGES_FP32 * 256 + 128: HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_FP32, 128); \
    default: return cudaErrorInvalidValue;                                          \
  }

cudaError_t launch_pages_write(const PagesArgs& a, cudaStream_t st) {
  HSTU_PAGES_DISPATCH(pages_write_kernel)
}

cudaError_t launch_pages_read(const PagesArgs& a, cudaStream_t st) {
  HSTU_PAGES_DISPATCH(pages_read_kernel)
}

}  // namespace hstu
