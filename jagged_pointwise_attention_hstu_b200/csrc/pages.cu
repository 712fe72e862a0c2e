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

constexpr int kRowWarps = 8;   // warps per block of the write and read kernels

// The largest b with offs[b] <= r, for 0 <= r < offs[B], found by the whole
// warp: 32 probes a step, so one step for up to 32 users and two for 1024.
__device__ __forceinline__ int32_t user_of_row(const int32_t* offs, int32_t B, int64_t r, int lane) {
  int32_t lo = 0, n = B;   // the answer is in [lo, lo + n)
  while (n > 1) {
    const int32_t step = (n + 31) >> 5;
    const int32_t k = lane * step;
    const bool le = k < n && fetch(offs + lo + k) <= r;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int32_t top = m == 0 ? 0 : 31 - __clz(m);
    lo += top * step;
    n = n - top * step < step ? n - top * step : step;
  }
  return lo;
}

struct Place {         // 32 bits: a pool has fewer rows than 2^31
  int32_t row;         // (page * H) * 2 * page_size + slot: the block of plane 0 of head 0
  int32_t ts;          // index into the page timestamps
  int err;
  bool ok;
};

// What place_of does not see, by the first block: an offsets table that does not
// start at zero, falls, or ends behind the rows.
__device__ __forceinline__ void check_offsets(const PagesArgs& a) {
  if (blockIdx.x != 0) return;
  bool bad = false;
  for (int32_t i = threadIdx.x; i < a.B; i += blockDim.x) {
    const int32_t lo = fetch(a.offsets + i), hi = fetch(a.offsets + i + 1);
    bad |= lo > hi || (i == 0 && lo != 0) || (i == a.B - 1 && hi > a.R);
  }
  if (bad) atomicOr(a.error, HSTU_DEVERR_OFFSETS);
}

// The same for a lane's own row, r >= the row that user b has.
__device__ __forceinline__ int32_t user_from(const int32_t* offs, int32_t B, int32_t r, int32_t b) {
  if (b + 1 >= B || fetch(offs + b + 1) > r) return b;
  int32_t lo = b + 1, hi = B;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (fetch(offs + mid) <= r) lo = mid; else hi = mid;
  }
  return lo;
}

// Where rows r .. r + ROWS - 1 of the call live, by the whole warp, lane i row r + i (ROWS
// = 1: every lane row r); `ok` false: nowhere (a row behind the last sequence, or an error).
template <int ROWS>
__device__ __forceinline__ Place place_of(const PagesArgs& a, int32_t r, int lane) {
  Place p;
  p.ok = false;
  p.err = 0;
  p.row = 0;
  p.ts = 0;
  int32_t b = user_of_row(a.offsets, a.B, r, lane);
  if (ROWS > 1) {
    r += lane;
    if (lane >= ROWS || r >= a.R) return p;
    b = user_from(a.offsets, a.B, r, b);
  }
  const int32_t r0 = fetch(a.offsets + b), r1 = fetch(a.offsets + b + 1);
  // behind the last sequence, or a table that check_offsets reports
  if (r < r0 || r >= r1 || r0 < 0 || r1 > a.R) return p;
  p.err = HSTU_DEVERR_PAGES;
  if (a.one_row && r1 - r0 > 1) return p;
  const int32_t first = a.lengths != nullptr ? fetch(a.lengths + b) : 0;
  if (first < 0 || first >= (1 << 30)) return p;       // positions end at 2^30, rows too
  const int32_t pos = first + (r - r0), k = pos >> a.page_shift;
  if (k >= int32_t(a.width)) return p;
  const int32_t page = fetch(a.table + (int64_t(b) * int32_t(a.width) + k));
  if (page < 0 || page >= a.num_pages) return p;
  const int32_t slot = pos & ((1 << a.page_shift) - 1);
  p.row = ((page * a.H * 2) << a.page_shift) + slot;
  p.ts = (page << a.page_shift) + slot;
  p.err = 0;
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

__device__ __forceinline__ uint32_t times2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
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
  uint2 c;
  if (!__any_sync(0xffffffffu, top > 0x7F60u)) {
    // e + 127 with e = k - 8 for top in (1.75 * 2^(k - 1), 1.75 * 2^k]: 0x1F carries above it
    scale = max(int((top + 0x1Fu) >> 7) - 8, kMinExponent + 127);
    scale = top == 0 ? 127 : scale;
    // x * 2^-e in bf16: exact, or so small that its code is zero either way
    const uint32_t inv = uint32_t(254 - scale) * 0x00800080u;
    float x[8];
    unpack_bf16(make_uint4(times2(v.x, inv), times2(v.y, inv), times2(v.z, inv), times2(v.w, inv)), x);
    c.x = four_codes(x[0], x[1], x[2], x[3]);
    c.y = four_codes(x[4], x[5], x[6], x[7]);
  } else {
    float x[8], m = 0.f;
    unpack_bf16(v, x);
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

// A row's keys, and its values, in chunks of 16 bytes: lane `lane` has the chunks lane,
// lane + 32, ... of both, which are the same place of a block's kPerHead whatever the
// block (but for heads of 96, fp32 only, of 24 chunks).
template <int FMT, int HD>
struct Chunks {
  static constexpr int kElems = FMT == HSTU_PAGES_FP32 ? 4 : 8;   // elements of a chunk
  static constexpr int kPerHead = HD / kElems;
  static constexpr int kBatch = 4;                                // of each, loaded at once: of
                                                                  // one row, or of 2 or 4
  int lane, each, step;     // chunks of the keys; blocks from a head to the next
  __device__ __forceinline__ explicit Chunks(const PagesArgs& a)
      : lane(threadIdx.x & 31), each(a.H * kPerHead), step(2 << a.page_shift) {}
  // chunk c of the keys, from the row's first block: its block, and its place there
  __device__ __forceinline__ int block(int c) const { return c / kPerHead * step; }
  __device__ __forceinline__ int in(int c) const {
    return 32 % kPerHead == 0 ? lane % kPerHead : c % kPerHead;
  }
};

// A warp has ROWS neighbouring rows, a lane their chunks, straight into the rows'
// blocks.  Bound by memory, a row reads 2d elements and writes them (or their codes) once,
// and nearly by its instructions.  All of a lane's loads (8, whatever d is) are on their
// way before the rows' places are looked up; the scale bytes of eight rows are
// gathered and stored as one where they are neighbours, since a store of one byte
// costs as much as one of 32.  65536 rows of d 1024 to e4m3 pages: 73 us, 5.6 TB/s (149
// with one load at a time and 25 instructions a value, 12 now; 78 with a store a scale
// byte; 65.6 with nothing to compute).
template <int FMT, int HD, int ROWS>
__global__ void __launch_bounds__(kRowWarps * 32) pages_write_kernel(const PagesArgs a) {
  using C = Chunks<FMT, HD>;
  constexpr bool kScaled = FMT == HSTU_PAGES_E4M3;
  constexpr int kBatch = C::kBatch / ROWS, kAll = kRowWarps * ROWS;
  static_assert(kRowWarps == 8, "scales of eight rows are eight bytes");
  __shared__ __align__(8) uint8_t s_scale[kScaled ? 32 : 1][kAll];   // at most 16 heads
  __shared__ int32_t s_row[kAll];
  let_next_kernel_start();
  wait_for_earlier_kernels();
  check_offsets(a);
  const int first = (threadIdx.x >> 5) * ROWS;                       // the warp's, of the block's
  const int32_t r = int32_t(blockIdx.x) * kAll + first;              // fewer than 2^30
  const C ch(a);
  const int lane = ch.lane, plane = 1 << a.page_shift;
  uint4 v[2][ROWS][kBatch];
  auto load = [&](int c0) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      // U | V | Q | K
      const uint4* vals = static_cast<const uint4*>(a.uvqk) + (int64_t(r + j) * 4 + 1) * ch.each;
      const uint4* keys = vals + 2 * ch.each;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = c0 + 32 * i + lane;
        const bool on = r + j < a.R && c < ch.each;
        v[0][j][i] = on ? fetch(keys + c) : make_uint4(0u, 0u, 0u, 0u);
        v[1][j][i] = on ? fetch(vals + c) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  load(0);
  Place mine;
  mine.ok = false;
  if (r < a.R) {
    mine = place_of<ROWS>(a, r, lane);
    if (lane < ROWS && mine.err != 0) atomicOr(a.error, mine.err);
    if (lane < ROWS && mine.ok && a.ts != nullptr) {
      const int64_t t = a.ts[r + lane];
      if (t < 0 || t >= kMaxTimestamp) atomicOr(a.error, HSTU_DEVERR_TIMESTAMPS);
      a.page_ts[mine.ts] = t;
    }
  }
  const unsigned there = ROWS == 1 ? (mine.ok ? 1 : 0) : __ballot_sync(0xffffffffu, mine.ok);
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    const int32_t row = ROWS == 1 ? mine.row : __shfl_sync(0xffffffffu, mine.row, j);
    if (!(there >> j & 1)) continue;
    uint4* to = static_cast<uint4*>(a.kv) + int64_t(row) * C::kPerHead;
    uint2* codes = static_cast<uint2*>(a.kv) + int64_t(row) * C::kPerHead;
    for (int c0 = 0;;) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (c0 + 32 * i >= ch.each) break;
        const int c = c0 + 32 * i + lane;
        const bool on = c < ch.each;
        const int at = ch.block(c) * C::kPerHead + ch.in(c);
#pragma unroll
        for (int x = 0; x < 2; ++x) {                 // keys, values
          if constexpr (!kScaled) {
            if (on) to[at + x * plane * C::kPerHead] = v[x][j][i];
          } else {
            int scale;
            const uint2 q = quantise8<C::kPerHead>(v[x][j][i], scale);
            if (on) {
              codes[at + x * plane * C::kPerHead] = q;
              if (ch.in(c) == 0) s_scale[2 * (c / C::kPerHead) + x][first + j] = uint8_t(scale);
            }
          }
        }
      }
      c0 += 32 * kBatch;
      if (ROWS > 1 || c0 >= ch.each) break;           // several rows: no more chunks than a batch
      load(c0);
    }
  }
  if constexpr (kScaled) {
    if (lane < ROWS) s_row[first + lane] = mine.ok ? mine.row : -1;
    __syncthreads();
    const int b = threadIdx.x % 32, e = threadIdx.x / 32 * 8;   // a thread a block of eight rows
    if (b < 2 * a.H && e < kAll) {
      const int32_t row = s_row[e];
      bool together = row >= 0 && row % 8 == 0;
#pragma unroll
      for (int i = 1; i < 8; ++i) together = together && s_row[e + i] == row + i;
      uint8_t* to = a.scales + (int64_t(b) << a.page_shift);
      if (together) {
        *reinterpret_cast<uint2*>(to + row) = *reinterpret_cast<const uint2*>(&s_scale[b][e]);
      } else {
        for (int i = 0; i < 8; ++i)
          if (s_row[e + i] >= 0) to[s_row[e + i]] = s_scale[b][e + i];
      }
    }
  }
}

// The way back: pages into the K and V columns of U|V|Q|K, a warp's rows as above.
template <int FMT, int HD, int ROWS>
__global__ void __launch_bounds__(kRowWarps * 32) pages_read_kernel(const PagesArgs a) {
  using C = Chunks<FMT, HD>;
  constexpr int kBatch = C::kBatch / ROWS;
  let_next_kernel_start();
  wait_for_earlier_kernels();
  check_offsets(a);
  const int32_t r = (int32_t(blockIdx.x) * kRowWarps + int32_t(threadIdx.x >> 5)) * ROWS;   // fewer than 2^30
  if (r >= a.R) return;
  const C ch(a);
  const int lane = ch.lane, plane = 1 << a.page_shift;
  const Place mine = place_of<ROWS>(a, r, lane);
  if (lane < ROWS && mine.err != 0) atomicOr(a.error, mine.err);
  const unsigned there = ROWS == 1 ? (mine.ok ? 1 : 0) : __ballot_sync(0xffffffffu, mine.ok);
  if (there == 0) return;
  if (lane < ROWS && mine.ok && a.ts_out != nullptr) a.ts_out[r + lane] = a.page_ts[mine.ts];
  int32_t row[ROWS];
#pragma unroll
  for (int j = 0; j < ROWS; ++j)
    row[j] = ROWS == 1 ? mine.row : __shfl_sync(0xffffffffu, mine.row, j);
  for (int c0 = lane; c0 < ch.each; c0 += 32 * kBatch) {
    uint4 v[2][ROWS][kBatch];
    float s[2][ROWS][kBatch];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const uint4* from = static_cast<const uint4*>(a.kv) + int64_t(row[j]) * C::kPerHead;
      const uint2* codes = static_cast<const uint2*>(a.kv) + int64_t(row[j]) * C::kPerHead;
      const uint8_t* scales = a.scales + row[j];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = c0 + 32 * i;
        if (c >= ch.each || !(there >> j & 1)) continue;
        const int block = ch.block(c), at = block * C::kPerHead + ch.in(c);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if constexpr (FMT != HSTU_PAGES_E4M3) {
            v[x][j][i] = fetch(from + at + x * plane * C::kPerHead);
          } else {
            const uint2 q = fetch(codes + at + x * plane * C::kPerHead);
            v[x][j][i].x = q.x;
            v[x][j][i].y = q.y;
            s[x][j][i] = block_scale(fetch(scales + block + x * plane));
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      uint4* vals = static_cast<uint4*>(a.out) + (int64_t(r + j) * 4 + 1) * ch.each;
      uint4* keys = vals + 2 * ch.each;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = c0 + 32 * i;
        if (c >= ch.each || !(there >> j & 1)) continue;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if constexpr (FMT == HSTU_PAGES_E4M3) {
            float f[8];
            unpack_e4m3(v[x][j][i].x, f);
            unpack_e4m3(v[x][j][i].y, f + 4);
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {   // exact: 4 significant bits
              const __nv_bfloat162 t =
                  __floats2bfloat162_rn(f[2 * e] * s[x][j][i], f[2 * e + 1] * s[x][j][i]);
              w[e] = *reinterpret_cast<const uint32_t*>(&t);
            }
            v[x][j][i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          (x == 0 ? keys : vals)[c] = v[x][j][i];
        }
      }
    }
  }
}

}  // namespace

// Rows of a warp: one, or as many as a batch of loads covers once there are more rows than
// warps the GPU holds (64 an SM): 64 users of up to 1024 rows, d 256, e4m3 are written in
// 6.8 us (10.1 with one row a warp) and read in 6.1 (8.7), 191 of up to 293, d 64, fp32 in 4.0
// (7.4) and 5.1 (7.0); with fewer rows than warps the latency of a row counts, 16 users of up
// to 1024, d 256, bf16 3.8 us to read with four rows a warp and 3.1 with one.  Heads of 96 have
// 96 chunks a row at least.
#define HSTU_PAGES_ROWS(KERNEL, F, D)                                                      \
  const int each = a.d / Chunks<F, D>::kElems;                                              \
  const int rows = a.R <= 64 * int64_t(a.num_sms) || each > 64 ? 1 : each > 32 ? 2 : 4;     \
  const unsigned blocks = unsigned((a.R + kRowWarps * rows - 1) / (kRowWarps * rows));      \
  return launch_early(rows == 1 ? KERNEL<F, D, 1> : rows == 2 ? KERNEL<F, D, D == 96 ? 1 : 2> \
                                                              : KERNEL<F, D, D == 96 ? 1 : 4>, \
                      blocks, kRowWarps * 32, 0, st, a)
#define HSTU_PAGES_DISPATCH(KERNEL)                                                 \
  if (a.R <= 0 || a.B <= 0) return cudaSuccess;                                     \
  switch (a.format * 256 + a.hd) {                                                  \
    case HSTU_PAGES_BF16 * 256 + 64: { HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_BF16, 64); }\
    case HSTU_PAGES_BF16 * 256 + 128: { HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_BF16, 128); }\
    case HSTU_PAGES_E4M3 * 256 + 64: { HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_E4M3, 64); }\
    case HSTU_PAGES_E4M3 * 256 + 128: { HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_E4M3, 128); }\
    case HSTU_PAGES_FP32 * 256 + 32: { HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_FP32, 32); }\
    case HSTU_PAGES_FP32 * 256 + 64: { HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_FP32, 64); }\
    case HSTU_PAGES_FP32 * 256 + 96: { HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_FP32, 96); }\
    case HSTU_PAGES_FP32 * 256 + 128: { HSTU_PAGES_ROWS(KERNEL, HSTU_PAGES_FP32, 128); }\
    default: return cudaErrorInvalidValue;                                          \
  }

cudaError_t launch_pages_write(const PagesArgs& a, cudaStream_t st) {
  HSTU_PAGES_DISPATCH(pages_write_kernel)
}

cudaError_t launch_pages_read(const PagesArgs& a, cudaStream_t st) {
  HSTU_PAGES_DISPATCH(pages_read_kernel)
}

}  // namespace hstu
