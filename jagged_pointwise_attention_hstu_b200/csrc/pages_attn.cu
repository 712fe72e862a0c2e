// Pointwise attention of new rows over a paged history.
//
// Row r of user b (n = lengths[b] cached rows) and head h:
//   s_j = q_r . k_j + rab_pos[min(n - j, clamp)] + rab_time[t(ts_r - ts_j)],  0 <= j < n
//   s_r = q_r . k_r + rab_pos[0] + rab_time[0]                               (the row itself)
//   O_r = (sum_j SiLU(s_j) v_j + SiLU(s_r) v_r) / n_norm
// A new action and an M-FALCON candidate are the same case: both sit at
// position n and see the cached rows and themselves.  There is no softmax, so
// parts of a history join by a plain sum.
//
// What bounds it: every cached key and value is read once for one or a few
// rows, 4 flops a pair of elements, so memory does.  The kernel is built to
// keep that stream going on every SM whatever the lengths:
//  * work is cut in units of kUnit keys of one segment (a user, a group of its
//    rows, a head); every block takes an equal run of consecutive units, found
//    from the lengths on the device (the host never knows them, so a captured
//    call follows them).  A segment cut between blocks is joined by the last
//    of them to arrive, in the order of the blocks: same bits every time, no
//    block waits for another, and one launch does it all.
//  * a producer warp walks the block's units, looks their pages up and fetches
//    them with bulk copies into a ring of stages in shared memory (a page's
//    keys and values of a head are one contiguous run), units and segments
//    ahead of the four warps that compute.
//  * products on mma.sync, whose N = 8 fits a few rows (a tcgen05 tile has 64
//    rows at least, for work that is bound by the loads).  Scores: the 16 rows
//    of the first operand are 8 keys twice, with the even and the odd pairs of
//    their dimensions, and a row of q takes two columns, so that the 16 bytes a
//    lane reads of a key are its operand as they are; key g and query t meet in
//    one lane.
//  * from the scores to P a lane has a key: bias, scales, SiLU and the split
//    are done once a key and row.  P goes through 16-bit shared memory into the
//    second operand of the output product (rows = columns of P, M = dimensions).
//  * fp32 results from 16-bit operands: q, k and v are exact in bf16 (bf16
//    pages) or fp16 (e4m3 codes, and q times a power of two), and P is split
//    into pieces that go through the product as columns of their own: three
//    bf16 pieces (8 + 8 + 8 bits) or two fp16 ones (11 + 11).
// fp32 pages (the fp32 path, small models) take the same units with loads
// straight into registers and fp32 arithmetic.
//
// Measured (B200, warm calls, a call's share of a graph of 21): 8 users of 8192 rows, d 1024,
// bf16 49.3 us (5.5 TB/s); 256 of 4096, d 512, e4m3 183 to 201 us (5.5 to 6.0 TB/s; 175
// with the arithmetic left out); 168 of 2080, d 768, bf16 167 us (6.4 TB/s); 1 of 100003,
// d 512, e4m3 26.1 us (4.0 TB/s: the start takes 4 us, the join 3); 1 of 37, d 256 5.3 us.
// What bounds e4m3 at head dim 64 besides memory is the latency of the 12 warps an SM holds
// (a step of 32 keys is 382 instructions: 146 are waits and book-keeping, 236 the arithmetic,
// 67 of those conversions).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "pages.cuh"
#include "sm100.cuh"

namespace hstu {
namespace {

constexpr int kWarps = 4;       // that compute
constexpr int kFold = 16;       // matrix products chained before the fp32 sums take over

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// s / (1 + exp(-s)); exp(-s) above fp32 gives -0, below it s.
// The approximate exp2 and reciprocal are off by a few steps of fp32, as a score's own sum is;
// outputs stay within 5e-7 of 64 bits, relative to their norm.
__device__ __forceinline__ float silu(float s) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(s * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return s * r;
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes as fp16, exactly.
__device__ __forceinline__ void halves_of_e4m3(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What a variant of the kernel is made of.  NT: tiles of 8 columns of P (fp32 pages: rows).
// Row 4i + t of q has its pieces in columns that lane t of a quad holds: 0 and 1 in tile i at
// 2t and 2t + 1; a third one in tile 2 at 2t + i, or, with one tile for two rows, at
// 2t + 4, which is two lanes on.
template <int FMT, int HD, int NT>
struct Shape {
  static constexpr bool kF32 = FMT == HSTU_PAGES_FP32;
  static constexpr bool kF16 = FMT == HSTU_PAGES_E4M3;
  static constexpr int kPieces = kF32 ? 1 : (kF16 ? 2 : 3);
  // rows of q of a segment (4 would fit a tile of e4m3 at head dim 128, but not three blocks an SM)
  static constexpr int kGroup = kF32 ? NT : NT > 1 ? 8 : kF16 && HD == 64 ? 4 : 2;
  static constexpr int kTiles = (kGroup + 3) / 4;               // of 4 rows of q, for the scores
  static constexpr int kColumns = 8 * NT;                       // of P
  static constexpr int kRows = kF32 ? 4 : kGroup;               // of the sums
  static __device__ __forceinline__ int column(int row, int piece) {
    if (piece < 2) return 2 * row + piece;
    return NT == 1 ? 4 + 2 * row : 16 + 2 * (row & 3) + (row >> 2);
  }
  static constexpr int kRow = HD * (kF32 ? 4 : (kF16 ? 1 : 2)); // bytes of a key
  // blocks of 16 keys, a warp's step: two where a step of one would be 2 KB, and for several
  // rows of q, whose work a lane a key is
  static constexpr int kBlocks = !kF32 && (kRow == 64 || (kRow == 128 && NT > 1)) ? 2 : 1;
  static constexpr int kStep = 16 * kBlocks;                    // keys of a warp's step
  static constexpr int kUnit = kWarps * kStep;                  // keys of a unit
  static constexpr int kPad = HD + 8;                           // row stride of the sums
  static constexpr int kThreads = 32 * (kWarps + (kF32 ? 0 : 1));
  // the ring: the stages' keys and values, then their times and scales
  static constexpr bool kSwizzle = !kF32 && kRow >= 128;        // rows of 128 bytes, TMA's swizzle
  static constexpr int kHalves = kSwizzle ? kRow / 128 : 1;     // boxes of 128 bytes of a row
  static constexpr int kDataBytes = 2 * kUnit * kRow;
  static constexpr int kSideBytes = 8 * kUnit + (kF16 ? 2 * kUnit : 0);
  static constexpr int kRowsBytes = 3 * kGroup * HD * 2;        // a part's q, k and v
  static constexpr int kRingBytes(int stages) { return stages * (kDataBytes + kSideBytes + kRowsBytes); }
  // blocks an SM and stages a block: as many blocks as registers allow, for parts that end at
  // different times, and what is left for stages (bf16 at head dim 64: 4 blocks of 2 stages;
  // 3 of 3 are 0 to 3 us slower)
  static constexpr bool kBig = kRow == 256 || NT > 1;
  static constexpr int kStages = kF16 && !kBig ? 3 : 2;
  static constexpr int kPerSm = kF32 ? (HD == 128 ? 2 : 3) : kBig ? 2 : (kF16 ? 3 : 4);
};

struct User {
  int64_t r0;
  int32_t rows, n, nu;   // rows of the call, cached rows, units of one segment
  int32_t segments;      // groups of rows * heads; none for an ill-formed user (err says why)
};

// A user's share of the work.  The units of a call are fewer than 2^31: the entry point sees
// to that.
template <class S>
__device__ __forceinline__ User user_of(const PagesArgs& a, int32_t b, int& err) {
  User u;
  const int32_t r0 = fetch(a.offsets + b), r1 = fetch(a.offsets + b + 1);
  u.n = fetch(a.lengths + b);
  if (r0 < 0 || r1 < r0 || r1 > a.R || (b == 0 && r0 != 0)) err |= HSTU_DEVERR_OFFSETS;
  if (u.n < 0 || u.n > (a.width << a.page_shift)) err |= HSTU_DEVERR_PAGES;
  u.r0 = r0;
  u.rows = err == 0 ? r1 - r0 : 0;
  u.nu = err == 0 && u.n > 0 ? (u.n + S::kUnit - 1) / S::kUnit : 1;
  u.segments = (u.rows + S::kGroup - 1) / S::kGroup * a.H;
  return u;
}

// The block's work.  share: the units of a block if all had as many.
//
// Parts, if every block can have one part of one segment, of at most `share`
// units: then it does, the segments cut into equal parts.  Else runs: block c has
// the units from c * share on, whatever segments they belong to; but a segment of
// at most share / 8 units is not cut, the block it ends in takes it whole.  A cut
// costs the join of its parts (2 to 3 us: the parts' way to memory, a ticket, the
// parts' way back), as much as a few units, and a block with the ends of two
// segments pays for two.  (16 users of up to 4096 rows, d 512: runs 15.9 us,
// parts 13.8; 1 of 100003: 32.9 and 30.7.  Longer segments left whole put two on some
// blocks and none on others: 109 users of up to 3698 rows, d 256, 39 us where
// segments up to 4 units longer than the share were.)
constexpr int32_t kWarpUsers = 64;   // with more users all threads plan, not one warp

struct Plan {
  int32_t sums[8];
  int32_t start, share, u0, u1;   // runs: the first user's first unit, the run
  int32_t user;                   // of the part, or the first of the run
  int32_t item, pieces;           // parts: the user's part, parts of a segment (0: runs)
};

// The threads that make the plan: one warp, or all kAll of the block.
template <int kAll>
struct Team {
  static __device__ __forceinline__ int rank() { return kAll == 32 ? threadIdx.x & 31 : threadIdx.x; }
  static __device__ __forceinline__ void sync() {
    if (kAll == 32) __syncwarp();
    else __syncthreads();
  }
  static __device__ __forceinline__ bool any(bool x) {
    return kAll == 32 ? __any_sync(0xffffffffu, x) : __syncthreads_or(x) != 0;
  }
  // Sum of each thread's x, and that of the threads before; `sums` may be used again behind a sync.
  static __device__ __forceinline__ int32_t scan(int32_t x, int32_t* sums, int32_t& before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    before = inc - x;
    if (kAll == 32) return __shfl_sync(0xffffffffu, inc, 31);
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int32_t total = 0;
#pragma unroll
    for (int w = 0; w < kAll / 32; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    return total;
  }
};

// By the whole team; `pl` is the team's own.  False: nothing to do.  Small code
// (loops that are not unrolled, 32 bits): every instruction of it is new to the SM.
template <class S, int kAll>
__device__ __forceinline__ bool make_plan(const PagesArgs& a, Plan& pl) {
  using T = Team<kAll>;
  const int tid = T::rank();
  const int32_t per = (a.B + kAll - 1) / kAll, b0 = tid * per, b1 = min(b0 + per, a.B);
  int err = 0;
  int32_t mine = 0, before;
#pragma unroll 1
  for (int32_t b = b0; b < b1; ++b) {
    int e = 0;
    const User x = user_of<S>(a, b, e);
    mine += x.segments * x.nu;
    err |= e;
  }
  const int32_t total = T::scan(mine, pl.sums, before);
  if (blockIdx.x == 0 && err != 0) atomicOr(a.error, err);   // by every team alike
  // users whose rows overlap could have more units than 32 bits count
  if (T::any((err & HSTU_DEVERR_OFFSETS) != 0) || total == 0) return false;
  const int32_t share = (total + gridDim.x - 1) / gridDim.x;
  T::sync();
  int32_t items = 0, items_before;
#pragma unroll 1
  for (int32_t b = b0; b < b1; ++b) {
    int e = 0;
    const User x = user_of<S>(a, b, e);
    items += x.segments * ((x.nu + share - 1) / share);
  }
  const int32_t parts = T::scan(items, pl.sums, items_before);
  const bool runs = parts > int32_t(gridDim.x);
  const int32_t c = blockIdx.x;
  const int32_t c0 = c * share, c1 = total - c0 > share ? c0 + share : total;
  if (runs ? c0 >= total : c >= parts) return false;
  if (tid == 0) {
    pl.share = share;
    if (runs) pl.pieces = 0;
    if (c1 == total) pl.u1 = total;
  }
  // the threads that have the block's part, or the users of the two ends of its run
#pragma unroll 1
  for (int end = 0; end < (runs ? 2 : 1); ++end) {
    const int32_t u = runs ? (end == 0 ? c0 : c1) : c;
    int32_t at = runs ? before : items_before;
    if (u < at || u >= at + (runs ? mine : items)) continue;
#pragma unroll 1
    for (int32_t b = b0; b < b1; ++b) {
      int e = 0;
      const User x = user_of<S>(a, b, e);
      const int32_t pieces = runs ? x.nu : (x.nu + share - 1) / share;
      const int32_t k = x.segments * pieces;
      if (u < at + k) {
        const int32_t rel = u - at;
        const int32_t cut = x.nu <= share / 8 ? u - rel % x.nu : u;
        if (end == 1) {
          pl.u1 = cut;
        } else {
          pl.user = b;
          pl.start = at;
          pl.u0 = cut;
          pl.item = rel;
          if (!runs) pl.pieces = pieces;
        }
        break;
      }
      at += k;
    }
  }
  T::sync();
  return !runs || pl.u0 < pl.u1;
}

// A block's part of one segment: tiles (units) [tile0, tile1) of row group
// `first` .. `first` + nq - 1 of a user, head h.
struct Part {
  int64_t row0;          // the group's first row
  int32_t h, nq, n;
  int32_t b;
  int32_t tile0, tile1;
  int32_t c0, c1;        // the first and last block that have a part
};

// Walks the block's work part by part (one warp, or all alike).
template <class S>
struct Walk {
  int32_t u, u1, start, share, b, item, pieces;
  User user;
  __device__ __forceinline__ Walk(const PagesArgs& a, const Plan& pl, bool any)
      : u(pl.u0), u1(pl.u1), start(pl.start), share(pl.share), b(pl.user), item(pl.item),
        pieces(pl.pieces) {
    int e = 0;
    if (any) user = user_of<S>(a, b, e);
  }
  __device__ __forceinline__ bool next(const PagesArgs& a, Part& p) {
    int32_t seg;
    p.c0 = p.c1 = int32_t(blockIdx.x);
    if (pieces != 0) {                    // one part of one segment
      if (item < 0) return false;
      seg = item / pieces;
      const int32_t k = item - seg * pieces;
      p.tile0 = int32_t(int64_t(k) * user.nu / pieces);
      p.tile1 = int32_t(int64_t(k + 1) * user.nu / pieces);
      p.c0 -= k;
      p.c1 = p.c0 + pieces - 1;
      item = -1;
    } else {
      if (u >= u1) return false;
      if (u >= start + user.segments * user.nu) {   // the next user that has rows
        start += user.segments * user.nu;
        for (;;) {
          const int32_t c = b + 1 + int32_t(threadIdx.x & 31);
          int e = 0;
          const bool has = c < a.B && user_of<S>(a, c, e).segments > 0;
          const unsigned m = __ballot_sync(0xffffffffu, has);
          if (m != 0) {
            b += __ffs(m);
            break;
          }
          b += 32;
          if (b >= a.B) return false;     // cannot happen: u < total
        }
        int e = 0;
        user = user_of<S>(a, b, e);
      }
      const int32_t rel = u - start;
      seg = rel / user.nu;
      p.tile0 = rel - seg * user.nu;
      p.tile1 = min(user.nu, p.tile0 + (u1 - u));
      if (p.tile0 != 0 || p.tile1 != user.nu) {
        const int32_t seg0 = u - p.tile0;   // the segment's first unit
        p.c0 = seg0 / share;
        p.c1 = (seg0 + user.nu - 1) / share;
      }
      u += p.tile1 - p.tile0;
    }
    const int32_t first = seg / a.H * S::kGroup;
    p.b = b;
    p.h = seg % a.H;
    p.nq = min(user.rows - first, S::kGroup);
    p.n = user.n;
    p.row0 = user.r0 + first;
    return true;
  }
};

// rab_time's bins: next threshold, the two table entries it decides between.
__device__ __forceinline__ void fill_time(const PagesArgs& a, int4* s_time, int k) {
  const int cand = __ldg(a.time_lut + k);
  const int next = cand + 1 < a.time_buckets ? cand + 1 : a.time_buckets - 1;
  s_time[k] = make_int4(cand + 1 < a.time_buckets ? __ldg(a.thr32 + cand + 1) : 0x7FFFFFFF,
                        __float_as_int(fetch(a.rab_time + cand)),
                        __float_as_int(fetch(a.rab_time + next)), 0);
}

// rab_pos for key j of the n cached, with pos_far what most have.
__device__ __forceinline__ float pos_bias(const PagesArgs& a, float pos_far, int32_t n, int32_t j) {
  return n - j < a.pos_clamp ? fetch(a.rab_pos + (j < n ? n - j : 0)) : pos_far;
}

// Whether the bins serve a gap (from 0 to 2^31 - 3 s), and what they say: bin 4e + m of
// gap + 1 has the exponent and the first two bits of the mantissa.
__device__ __forceinline__ bool bin_gap(const PagesArgs& a, int64_t gap) {
  return a.lut_exact && uint32_t(uint64_t(gap) >> 32) == 0 && uint32_t(gap) < 0x7FFFFFFEu;
}
__device__ __forceinline__ float bin_bias(const int4* s_time, uint32_t gap) {
  const int4 bin = s_time[(__float_as_uint(__uint2float_rz(gap + 1u)) >> 21) - 4 * 127];
  return __int_as_float(gap >= uint32_t(bin.x) ? bin.z : bin.y);
}
__device__ __forceinline__ float time_bias(const PagesArgs& a, const int4* s_time, int64_t gap) {
  return bin_gap(a, gap) ? bin_bias(s_time, uint32_t(gap))
                         : fetch(a.rab_time + time_bucket(a.thresholds, a.time_buckets, gap));
}
__device__ __forceinline__ int64_t gap_of(int64_t now, int64_t then) {
  return int64_t(uint64_t(now) - uint64_t(then));   // any two timestamps: no signed overflow
}

// What each row adds of itself, SiLU(s_r) v_r: a warp a row, its q, k and v by load(which, row,
// dimension), which = 0, 1, 2.
template <int HD, class Load, class Self>
__device__ __forceinline__ void self_terms(int nq, float bias, Load load, Self& self) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int q = warp; q < nq; q += kWarps) {
    float s = 0.f, v[HD / 32];
#pragma unroll
    for (int e = 0; e < HD / 32; ++e) {
      v[e] = load(2, q, lane + 32 * e);
      s = fmaf(load(0, q, lane + 32 * e), load(1, q, lane + 32 * e), s);
    }
    s = silu(warp_sum(s) + bias);
#pragma unroll
    for (int e = 0; e < HD / 32; ++e) self[q][lane + 32 * e] = s * v[e];
  }
}

// The warps' sums of a part, by the 128 threads that compute: written out, or
// left for the last block of the segment, which joins the parts in block order.
// sync() is a barrier of these threads; it returns false to give up.
template <class S, int HD, class Sum, class Self, class Sync>
__device__ __forceinline__ bool finish(const PagesArgs& a, const Part& p, Sum& sum,
                                       const Self& self, int32_t* last, Sync sync) {
  constexpr int kAll = kWarps * 32;
  const int tid = threadIdx.x;
  const bool whole = p.c0 == p.c1;
  float* part = a.partial + (int64_t(blockIdx.x) * 2 + (p.tile0 == 0 ? 1 : 0)) * (S::kGroup * HD);
  for (int i = tid; i < p.nq * HD; i += kAll) {
    const int q = i / HD, c = i % HD;
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x += sum[w][q][c];
    if (p.tile0 == 0) x += self[q][c];
    if (whole) a.av[(p.row0 + q) * a.d + p.h * HD + c] = x / float(a.n_norm);
    else part[i] = x;
  }
  if (!whole) {
    if (!sync()) return false;
    if (tid == 0) {
      int32_t k;                                   // behind the barrier: releases all threads' parts
      asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                   : "=r"(k) : "l"(a.tickets + p.c0) : "memory");
      *last = k == p.c1 - p.c0 ? 1 : 0;
      if (*last) a.tickets[p.c0] = 0;              // as the next call expects it
    }
    if (!sync()) return false;
    if (*last) {
      // A thread has four columns of a row in every slots-th part (a segment over the whole GPU
      // has hundreds, and one after the other their latency was the call's); the slots are
      // added in order, through the shared memory of the sums.
      const int32_t quads = p.nq * (HD / 4), slots = quads < kAll ? kAll / quads : 1;
      float* all = &sum[0][0][0];
      static_assert(sizeof(sum) >= size_t(kAll) * 16, "slots");
      auto out = [&](int32_t i, float x) {
        a.av[(p.row0 + i / HD) * a.d + p.h * HD + i % HD] = x / float(a.n_norm);
      };
      for (int32_t i = tid; i < quads * slots; i += slots > 1 ? kAll * 2 : kAll) {
        const int32_t quad = i % quads;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int32_t c = p.c0 + i / quads; c <= p.c1; c += slots) {
          const float4 y = __ldcg(reinterpret_cast<const float4*>(
              a.partial + (int64_t(c) * 2 + (c == p.c0 ? 1 : 0)) * (S::kGroup * HD)) + quad);
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        if (slots > 1) {
          *reinterpret_cast<float4*>(all + 4 * i) = x;
        } else {
          out(4 * quad, x.x), out(4 * quad + 1, x.y), out(4 * quad + 2, x.z), out(4 * quad + 3, x.w);
        }
      }
      if (slots > 1) {
        if (!sync()) return false;
        for (int32_t i = tid; i < 4 * quads; i += kAll) {
          float x = 0.f;
          for (int32_t k = 0; k < slots; ++k) x += all[k * 4 * quads + i];
          out(i, x);
        }
      }
    }
  }
  return sync();
}

// fp32 pages: 8 lanes a key, 4 keys at once, fp32 throughout.
template <int HD, int NT>
__global__ void __launch_bounds__(kWarps * 32, (Shape<HSTU_PAGES_FP32, HD, NT>::kPerSm))
    pages_attention_f32_kernel(const PagesArgs a) {
  using S = Shape<HSTU_PAGES_FP32, HD, NT>;
  constexpr int E = HD / 32;
  __shared__ Plan plans[kWarps];
  __shared__ int4 s_time[128];
  __shared__ __align__(16) float s_sum[kWarps][S::kRows][S::kPad];
  __shared__ float s_self[NT][HD];
  __shared__ int32_t s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int k4 = lane >> 3, t8 = lane & 7;
  let_next_kernel_start();
  wait_for_earlier_kernels();
  fill_time(a, s_time, tid);
  const bool alone = a.B <= kWarpUsers;      // a warp plans for itself
  Plan& plan = plans[alone ? warp : 0];
  if (!(alone ? make_plan<S, 32>(a, plan) : make_plan<S, S::kThreads>(a, plan))) return;
  __syncthreads();
  Walk<S> walk(a, plan, true);
  const float pos_far = fetch(a.rab_pos + a.pos_clamp);
  const float self_bias = fetch(a.rab_pos) + fetch(a.rab_time);
  const int32_t slot_mask = (1 << a.page_shift) - 1;
  const int64_t plane = int64_t(1) << a.page_shift;
  int err = 0;
  Part p;
  while (walk.next(a, p)) {
    const int32_t n = p.n;
    const int32_t* table = a.table + int64_t(p.b) * a.width;
    if (p.tile0 == 0) {
      const float* rows = static_cast<const float*>(a.uvqk) + p.row0 * 4 * a.d + p.h * HD;
      self_terms<HD>(p.nq, self_bias, [&](int which, int q, int c) {
        return rows[(int64_t(q) * 4 + (which == 0 ? 2 : which == 1 ? 3 : 1)) * a.d + c];
      }, s_self);
    }
    float q[NT][4 * E], o[NT][4 * E];
    int64_t now[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int64_t r = p.row0 + (i < p.nq ? i : 0);
      now[i] = fetch(a.ts + r);
      if (now[i] < 0 || now[i] >= kMaxTimestamp) err |= HSTU_DEVERR_TIMESTAMPS;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float4 v = fetch(reinterpret_cast<const float4*>(static_cast<const float*>(a.uvqk) +
                               r * 4 * a.d + 2 * a.d + p.h * HD + 32 * e) + t8);
        q[i][4 * e] = v.x, q[i][4 * e + 1] = v.y, q[i][4 * e + 2] = v.z, q[i][4 * e + 3] = v.w;
        o[i][4 * e] = o[i][4 * e + 1] = o[i][4 * e + 2] = o[i][4 * e + 3] = 0.f;
      }
    }
    float (*sum)[S::kPad] = s_sum[warp];
    bool folded = false;
    for (int32_t tile = p.tile0; tile < p.tile1; ++tile) {
      const int32_t j0 = tile * S::kUnit + warp * S::kStep, jl = j0 + (lane & 15);
      if (j0 < n) {
        const int32_t page = fetch(table + (j0 >> a.page_shift));
        if (page < 0 || page >= a.num_pages) {
          err |= HSTU_DEVERR_PAGES;
        } else {
          const int64_t then = fetch(a.page_ts + (int64_t(page) << a.page_shift) + (jl & slot_mask));
          float bias[NT];                // of the lane's key
#pragma unroll
          for (int i = 0; i < NT; ++i)
            bias[i] = pos_bias(a, pos_far, n, jl) + time_bias(a, s_time, gap_of(now[i], then));
          const float* base = static_cast<const float*>(a.kv) +
              ((((int64_t(page) * a.H + p.h) * 2) << a.page_shift) + (j0 & slot_mask)) * HD;
          float4 k[4][E], v[4][E];
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const float* at = base + int64_t(4 * s + k4) * HD + 32 * e + 4 * t8;
              k[s][e] = fetch(reinterpret_cast<const float4*>(at));
              v[s][e] = fetch(reinterpret_cast<const float4*>(at + plane * HD));
            }
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const bool ok = j0 + 4 * s + k4 < n;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              float x = 0.f;
#pragma unroll
              for (int e = 0; e < E; ++e) {
                x = fmaf(q[i][4 * e], k[s][e].x, x);
                x = fmaf(q[i][4 * e + 1], k[s][e].y, x);
                x = fmaf(q[i][4 * e + 2], k[s][e].z, x);
                x = fmaf(q[i][4 * e + 3], k[s][e].w, x);
              }
              x += __shfl_xor_sync(0xffffffffu, x, 1);
              x += __shfl_xor_sync(0xffffffffu, x, 2);
              x += __shfl_xor_sync(0xffffffffu, x, 4);
              const float y = silu(x + __shfl_sync(0xffffffffu, bias[i], 4 * s + k4));
              if (ok) {                  // no memory behind the history may reach the sum
#pragma unroll
                for (int e = 0; e < E; ++e) {
                  o[i][4 * e] = fmaf(y, v[s][e].x, o[i][4 * e]);
                  o[i][4 * e + 1] = fmaf(y, v[s][e].y, o[i][4 * e + 1]);
                  o[i][4 * e + 2] = fmaf(y, v[s][e].z, o[i][4 * e + 2]);
                  o[i][4 * e + 3] = fmaf(y, v[s][e].w, o[i][4 * e + 3]);
                }
              }
            }
          }
        }
      }
      if ((tile - p.tile0) % kFold == kFold - 1 || tile + 1 == p.tile1) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4 * E; ++e) {
            float x = o[i][e] + __shfl_xor_sync(0xffffffffu, o[i][e], 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            float* at = &sum[i][(e >> 2) * 32 + 4 * t8 + (e & 3)];
            if (k4 == 0) *at = folded ? *at + x : x;
            o[i][e] = 0.f;
          }
        folded = true;
      }
    }
    __syncthreads();
    finish<S, HD>(a, p, s_sum, s_self, &s_last, [] {
      __syncthreads();
      return true;
    });
  }
  if (err != 0) atomicOr(a.error, err);
}

// One unit on its way through the ring.
struct Unit {
  int4 what;             // tile, runs (below) whose page index is none, Flag, cached rows
  Part part;
  int64_t now[8];        // of a part's first unit: the rows' times
};
enum Flag { kLast = 1, kStop = 2 };   // of its part; no more units

// untiled bulk copy global -> shared; all of dst, src and bytes multiples of 16
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar)) : "memory");
}

// Waits for a phase for at most `limit` cycles.  The bound is looked at before the first
// try_wait, which may sleep for longer than a copy takes: a bound of a few cycles gives up.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, long long limit) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(sm100::smem_u32(bar)), "r"(parity) : "memory");
  if (ok) return true;
  const long long t0 = clock64();
  do {
    if (clock64() - t0 > limit) return false;
  } while (!sm100::mbar_try_wait(bar, parity));
  return true;
}

// The same by a whole warp, which gives up as one: lanes look at the clock at different
// moments, and a lane that left alone would be missing from the warp's next vote.
__device__ __forceinline__ bool wait_by_all(uint64_t* bar, uint32_t parity, long long limit) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, limit)) != 0;
}

__device__ __forceinline__ uint2 lds8(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

template <class S>
struct Ring {
  uint64_t full[S::kStages], empty[S::kStages], turn;
  Unit unit[S::kStages];
  int32_t last;
};

// A unit's keys lie in runs of run = min(page_size, kUnit) keys, a page each:
// [run][plane][key] in the stage, as in the pool; its scales [run][plane][key],
// its times [key].  Rows of 64 bytes come as they are, by untiled copies.  The
// rows of 128 and 256 bytes would meet in the same banks: they come through a
// tensor map, [run][plane][half][key] of 128 bytes with TMA's swizzle (16-byte
// chunk c of row r at c ^ (r & 7)), in boxes of a run or of 16 keys.
template <int FMT, int HD, int NT>
__global__ void __launch_bounds__((Shape<FMT, HD, NT>::kThreads), (Shape<FMT, HD, NT>::kPerSm))
    pages_attention_kernel(const PagesArgs a, const __grid_constant__ CUtensorMap map_run,
                           const __grid_constant__ CUtensorMap map_16) {
  using S = Shape<FMT, HD, NT>;
  using namespace sm100;
  constexpr int NB = S::kBlocks;
  extern __shared__ __align__(1024) uint8_t stages[];
  __shared__ Plan plan;
  __shared__ Ring<S> ring;
  __shared__ int4 s_time[128];
  __shared__ __align__(16) float s_sum[kWarps][S::kRows][S::kPad];
  __shared__ float s_self[S::kGroup][HD];
  __shared__ int64_t s_now[kWarps][S::kGroup];   // the rows' times, a copy a warp
  // P of a warp's step, a row per column of the operand
  __shared__ __align__(16) uint16_t s_p[kWarps][S::kColumns][S::kStep + 8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long limit = a.wait_limit > 0 ? a.wait_limit : kWaitLimit;
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&ring.full[s], 1);
      mbar_init(&ring.empty[s], kWarps);
    }
    mbar_init(&ring.turn, kWarps);
    fence_mbarrier_init();
  }
  let_next_kernel_start();
  __syncthreads();
  wait_for_earlier_kernels();
  // what there is to do is the producer's to know; with many users all threads plan
  const bool alone = a.B <= kWarpUsers;
  if (!alone && !make_plan<S, S::kThreads>(a, plan)) return;
  const int32_t run_shift = (1 << a.page_shift) < S::kUnit ? a.page_shift : 31 - __clz(S::kUnit);
  const int32_t run = 1 << run_shift;
  int err = 0;

  if (warp == kWarps) {
    // ---- the producer
    const bool any = !alone || make_plan<S, 32>(a, plan);
    Walk<S> walk(a, plan, any);
    Part p;
    uint32_t issued = 0;                 // units put into the ring
    bool ok = true;
    while (ok && any && walk.next(a, p)) {
      const int32_t* table = a.table + int64_t(p.b) * a.width;
      auto page_of = [&](int32_t tile) { // of the lane's run; -1: no key there, -2: no such page
        const int64_t j = int64_t(tile) * S::kUnit + (int64_t(lane) << run_shift);
        if (tile >= p.tile1 || (lane << run_shift) >= S::kUnit || j >= p.n) return -1;
        const int32_t x = fetch(table + (j >> a.page_shift));
        return x >= 0 && x < a.num_pages ? x : -2;
      };
      const int64_t now = lane < p.nq ? fetch(a.ts + p.row0 + lane) : 0;
      if (now < 0 || now >= kMaxTimestamp) err |= HSTU_DEVERR_TIMESTAMPS;
      int32_t page_next = page_of(p.tile0);
      for (int32_t tile = p.tile0; tile < p.tile1; ++tile) {
        const int32_t page = page_next;
        page_next = page_of(tile + 1);
        const int s = issued % S::kStages;
        ok = wait_by_all(&ring.empty[s], ((issued / S::kStages) & 1) ^ 1, limit);
        if (!ok) break;
        const int32_t j = tile * S::kUnit + (lane << run_shift);
        // whole blocks of 16 keys: what lies behind the history in the last one is not used
        int32_t keys = page >= 0 ? (p.n - j < run ? (p.n - j + 15) & ~15 : run) : 0;
        const uint32_t per_key = 2 * S::kRow + (S::kF16 ? 2 : 0) + 8;
        // with a part's first unit come its rows of q, and of k and v where it is a segment's first
        const int32_t rows = tile == p.tile0 ? p.nq * (tile == 0 ? 3 : 1) : 0;
        const uint32_t bytes = __reduce_add_sync(0xffffffffu, uint32_t(keys) * per_key +
                                                                 (lane < rows ? HD * 2 : 0));
        const unsigned bad = __ballot_sync(0xffffffffu, page == -2);
        if (bad != 0) err |= HSTU_DEVERR_PAGES;
        if (lane == 0) {
          ring.unit[s].part = p;
          ring.unit[s].what = make_int4(tile, int(bad), tile + 1 == p.tile1 ? kLast : 0, p.n);
        }
        if (rows > 0 && lane < S::kGroup) ring.unit[s].now[lane] = now;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&ring.full[s], bytes);
        __syncwarp();
        if (lane < rows) {
          const int32_t which = lane / p.nq, q = lane - which * p.nq;
          const char* from = static_cast<const char*>(a.uvqk) +
              (((p.row0 + q) * 4 + (which == 0 ? 2 : which == 1 ? 3 : 1)) * a.d + p.h * HD) * 2;
          bulk_load(smem_u32(stages) + S::kStages * (S::kDataBytes + S::kSideBytes) +
                        s * S::kRowsBytes + (which * S::kGroup + q) * (HD * 2),
                    from, HD * 2, &ring.full[s]);
        }
        if (keys > 0) {
          uint64_t* bar = &ring.full[s];
          const uint32_t data = smem_u32(stages) + s * S::kDataBytes;
          const uint32_t side = smem_u32(stages) + S::kStages * S::kDataBytes + s * S::kSideBytes;
          const int32_t slot = j & ((1 << a.page_shift) - 1);
          const int64_t block = (((int64_t(page) * a.H + p.h) * 2) << a.page_shift) + slot;
          const uint32_t first = lane << (run_shift + 1);       // of the stage's blocks
          const int32_t plane = 1 << a.page_shift;
          bulk_load(side + (lane << run_shift) * 8,
                    a.page_ts + (int64_t(page) << a.page_shift) + slot, keys * 8, bar);
          const bool both = keys == plane;                      // a whole page: planes at once
          if constexpr (S::kSwizzle) {
            const int32_t y = int32_t(block), step = keys == run ? run : 16;
            const CUtensorMap* map = keys == run ? &map_run : &map_16;
            uint8_t* to = stages + s * S::kDataBytes + first * S::kRow;
            for (int32_t r = 0; r < keys; r += step)
#pragma unroll
              for (int x = 0; x < S::kHalves; ++x) {
                tma_load_2d(to + (x * run + r) * 128, map, bar, 128 * x, y + r);
                tma_load_2d(to + (x * run + r) * 128 + run * S::kRow, map, bar, 128 * x,
                            y + plane + r);
              }
          } else {
            const char* kv = static_cast<const char*>(a.kv) + block * S::kRow;
            bulk_load(data + first * S::kRow, kv, (both ? 2 : 1) * keys * S::kRow, bar);
            if (!both)
              bulk_load(data + (first + run) * S::kRow, kv + int64_t(plane) * S::kRow,
                        keys * S::kRow, bar);
          }
          if constexpr (S::kF16) {
            const uint32_t at = side + 8 * S::kUnit + first;
            bulk_load(at, a.scales + block, (both ? 2 : 1) * keys, bar);
            if (!both) bulk_load(at + run, a.scales + block + plane, keys, bar);
          }
        }
        ++issued;
      }
    }
    const int s = issued % S::kStages;
    if (ok) ok = wait_by_all(&ring.empty[s], ((issued / S::kStages) & 1) ^ 1, limit);
    if (ok && lane == 0) {
      ring.unit[s].what = make_int4(0, 0, kStop, 0);
      mbar_arrive(&ring.full[s]);
    }
    if (!ok) err |= HSTU_DEVERR_TIMEOUT;
    // no copy may land after the block has gone, whoever gave up (the stage of the stop has
    // been given back: its copies have landed)
    for (uint32_t k = issued > S::kStages ? issued - S::kStages : 0; k < issued; ++k)
      if (!ok || k % S::kStages != s) mbar_wait(&ring.full[k % S::kStages], (k / S::kStages) & 1);
    if (err != 0) atomicOr(a.error, err);
    return;
  }

  // ---- the warps that compute
  constexpr int KC = S::kRow / 64;             // 16-byte chunks a lane has of a key
  constexpr int VW = S::kRow / 32;             // words a lane has of a value
  constexpr int KS = HD / 32;                  // products a tile of scores takes
  constexpr int MT = HD / 16;                  // tiles of 16 dimensions of the output
  constexpr int QT = S::kTiles;
  constexpr int kQ = S::kGroup < 4 ? S::kGroup : 4;   // rows of a tile
  const int g = lane >> 2, t = lane & 3;
  const float pos_far = fetch(a.rab_pos + a.pos_clamp);
  const float self_bias = fetch(a.rab_pos) + fetch(a.rab_time);
  float (*sum)[S::kPad] = s_sum[warp];
  uint16_t (*ps)[S::kStep + 8] = s_p[warp];
  uint32_t turn = 0;
  auto sync = [&]() {                          // of the warps that compute
    __syncwarp();
    if (lane == 0) mbar_arrive(&ring.turn);
    const bool ok = wait_by_all(&ring.turn, turn, limit);
    turn ^= 1;
    return ok;
  };
  // the 16-byte chunks of a key that are the lane's, and which of its rows a lane's key is
  auto chunk = [&](int y) { return S::kSwizzle ? 2 * t + (y & 1) + 8 * (y >> 1) : t; };
  auto key_of = [&](int i) { return S::kSwizzle ? 2 * t + (i & 1) + 8 * (i >> 1) : t + 4 * i; };
  const int spot = (lane & 16) + (S::kSwizzle ? 4 * (lane >> 1 & 3) + (lane & 1) + 2 * (lane >> 3 & 1)
                                              : 4 * (lane & 3) + (lane >> 2 & 3));
  // byte offsets that do not change: of the warp's blocks in a stage, of the lane's chunks of a
  // block's keys, and of its rows and chunks of the values (b: the low bit of chunk or row)
  uint32_t block_at[NB], k_at[2], v_at[2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int32_t kb = warp * S::kStep + 16 * nb;
    block_at[nb] = ((kb >> run_shift) << (run_shift + 1)) * S::kRow +
                   (kb & (run - 1)) * (S::kSwizzle ? 128 : S::kRow);
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    k_at[b] = S::kSwizzle ? g * 128 + (((2 * t + b) ^ g) << 4) : g * S::kRow + 16 * t;
    v_at[b] = S::kSwizzle ? (2 * t + b) * 128 + ((g ^ (2 * t + b)) << 4) : t * S::kRow + 8 * g;
  }
  const uint32_t half_at = run * 128, plane_at = run * S::kRow;
  const int32_t kl = warp * S::kStep + (lane & (S::kStep - 1));   // the lane's own key of a unit
  // its scales: [run][plane][key]
  const int32_t scale_at = 8 * S::kUnit + ((kl >> run_shift) << (run_shift + 1)) + (kl & (run - 1));
  uint32_t qb[QT][KS][2];
  // e4m3: the rows' scales of q, and what keeps their P within fp16
  float q_scale[S::kGroup], inv[S::kGroup], acc[MT][NT][4];
  int nq = 1, folds = 0, chain = 0;
  fill_time(a, s_time, tid);
  bool up = sync(), done = false;

  bool fresh = true;                           // the next unit begins a part, or there is none
  uint32_t parity = 0;
  for (int st = 0; up;) {
    if (!wait_by_all(&ring.full[st], parity, limit)) break;
    const int4 what = ring.unit[st].what;
    if (what.z & kStop) {
      done = true;
      break;
    }
    const int32_t tile = what.x, n = what.w;

    if (fresh) {
      // ---- a new part: q, and nothing summed
      const __nv_bfloat16* rows = reinterpret_cast<const __nv_bfloat16*>(
          stages + S::kStages * (S::kDataBytes + S::kSideBytes) + st * S::kRowsBytes);
      nq = ring.unit[st].part.nq;
      __syncwarp();
      if (lane < S::kGroup) s_now[warp][lane] = ring.unit[st].now[lane < nq ? lane : nq - 1];
      // Columns 2i and 2i + 1 of the score product are query i, with the even and the odd
      // pairs of its dimensions: what the lane's g is, at its t's dimensions.
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        const int q = 4 * i + (g >> 1) < nq ? 4 * i + (g >> 1) : nq - 1;
        const bool odd = (g & 1) != 0;
        const uint4* src = reinterpret_cast<const uint4*>(rows + q * HD);
        if constexpr (!S::kF16) {
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const uint4 v = src[chunk(c)];
            qb[i][c][0] = odd ? v.y : v.x;
            qb[i][c][1] = odd ? v.w : v.z;
          }
        } else {
          // fp16 of q * 2^-e with |q| below 2^15: bf16's 8 bits are exact down to 2^-32 of the
          // largest element, and 2^-40 of it is what the others lose
          float x[KC][16];
          float m = 0.f;
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            unpack_bf16(src[2 * chunk(c)], x[c]);
            unpack_bf16(src[2 * chunk(c) + 1], x[c] + 8);
#pragma unroll
            for (int y = 0; y < 16; ++y) m = fmaxf(m, fabsf(x[c][y]));
          }
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          int e = int(__float_as_uint(m) >> 23) - 127 - 14;
          e = e < -126 ? -126 : (e > 112 ? 112 : e);
          const float qs = __int_as_float((e + 127) << 23), f = __int_as_float((127 - e) << 23);
#pragma unroll
          for (int c = 0; c < kQ; ++c) q_scale[4 * i + c] = __shfl_sync(0xffffffffu, qs, 8 * c);
#pragma unroll
          for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const int at = 8 * y + 4 * w;
                qb[i][2 * c + y][w] = pack_half((odd ? x[c][at + 2] : x[c][at]) * f,
                                                (odd ? x[c][at + 3] : x[c][at + 1]) * f);
              }
        }
      }
      __syncwarp();
      for (int i = lane; i < S::kColumns * (S::kStep + 8) / 2; i += 32)
        reinterpret_cast<uint32_t*>(&ps[0][0])[i] = 0u;   // columns without a piece
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.f;
      // fp16 pieces: P times a power of two of its row, inv, stays below 2^15
#pragma unroll
      for (int i = 0; i < S::kGroup; ++i) inv[i] = __int_as_float((127 + 126) << 23);
      folds = chain = 0;
      if (tile == 0)
        self_terms<HD>(nq, self_bias, [&](int which, int q, int c) {
          return __bfloat162float(rows[(which * S::kGroup + q) * HD + c]);
        }, s_self);
    }

    const int32_t k0 = warp * S::kStep, j0 = tile * S::kUnit + k0;   // the warp's keys
    if (j0 < n) {
      const uint32_t data = smem_u32(stages) + st * S::kDataBytes;
      const int32_t jl = tile * S::kUnit + kl;
      bool mine = jl < n;
      if (what.y != 0) mine = mine && !(uint32_t(what.y) >> (kl >> run_shift) & 1);
      const uint8_t* side = stages + S::kStages * S::kDataBytes + st * S::kSideBytes;
      const int64_t then = *reinterpret_cast<const int64_t*>(side + 8 * kl);
      // The key's scale in two factors, one of them 1, with q's between them: a product that fp32
      // holds is reached without a step beyond it, whichever of the two scales is large.
      float ks_down = 1.f, ks_up = 1.f, vs = 1.f;
      if constexpr (S::kF16) {
        const float ks = block_scale(side[scale_at]);
        ks_down = fminf(ks, 1.f), ks_up = fmaxf(ks, 1.f);
        vs = block_scale(side[scale_at + run]);
      }
      float s[NB][2][QT];                // of key 16 nb + 8 x + g and row 4i + t
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float c[QT][4];
#pragma unroll
          for (int i = 0; i < QT; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
#pragma unroll
          for (int y = 0; y < KC; ++y) {
            const uint4 v = lds16(data + block_at[nb] + k_at[y & 1] + (y >> 1) * half_at +
                                  8 * x * (S::kSwizzle ? 128 : S::kRow));
            if constexpr (S::kF16) {
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                uint32_t a0, a1, a2, a3;
                halves_of_e4m3(w[2 * z], a0, a1);
                halves_of_e4m3(w[2 * z + 1], a2, a3);
#pragma unroll
                for (int i = 0; i < QT; ++i)
                  mma<true>(c[i], a0, a1, a2, a3, qb[i][2 * y + z][0], qb[i][2 * y + z][1]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < QT; ++i)
                mma<false>(c[i], v.x, v.y, v.z, v.w, qb[i][y][0], qb[i][y][1]);
            }
          }
#pragma unroll
          for (int i = 0; i < QT; ++i) s[nb][x][i] = c[i][0] + c[i][3];
        }
      }
      const float pos = j0 + S::kStep > n - a.pos_clamp ? pos_bias(a, pos_far, n, jl) : pos_far;
      // ---- a lane a key: N rows of q at once, from row 4i on (those behind nq are copies of
      // the last, in columns that nobody reads)
      auto score = [&](auto count, int i) {
        constexpr int N = decltype(count)::value;
        float y[N];
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const int src = 4 * (lane & 7) + c;
          const float y0 = __shfl_sync(0xffffffffu, s[0][0][i], src);
          const float y1 = __shfl_sync(0xffffffffu, s[0][1][i], src);
          y[c] = lane & 8 ? y1 : y0;
          if constexpr (NB == 2) {
            const float y2 = __shfl_sync(0xffffffffu, s[1][0][i], src);
            const float y3 = __shfl_sync(0xffffffffu, s[1][1][i], src);
            const float z = lane & 8 ? y3 : y2;
            y[c] = lane & 16 ? z : y[c];
          }
          if constexpr (S::kF16) y[c] = y[c] * ks_down * q_scale[4 * i + c] * ks_up;
        }
        // lanes without a key take gap 0
        int64_t gap[N];
        bool bins = true;
#pragma unroll
        for (int c = 0; c < N; ++c) {
          gap[c] = mine ? gap_of(s_now[warp][4 * i + c], then) : 0;
          bins = bins && bin_gap(a, gap[c]);
        }
        float tb[N];
        if (__all_sync(0xffffffffu, bins)) {
#pragma unroll
          for (int c = 0; c < N; ++c) tb[c] = bin_bias(s_time, uint32_t(gap[c]));
        } else {
#pragma unroll
          for (int c = 0; c < N; ++c) tb[c] = time_bias(a, s_time, gap[c]);
        }
#pragma unroll
        for (int c = 0; c < N; ++c) {
          y[c] = silu(y[c] + (pos + tb[c]));
          if constexpr (S::kF16) y[c] *= vs;
          y[c] = mine ? y[c] : 0.f;      // no key here: what memory holds must not reach the sum
        }
        if constexpr (S::kF16) {         // four rows a tile of scores, and a tile of P
          bool over = false;
#pragma unroll
          for (int c = 0; c < N; ++c) over |= fabsf(y[c]) * inv[4 * i + c] > 32768.f;
          if (__any_sync(0xffffffffu, over)) {                       // raise a row's power
#pragma unroll
            for (int c = 0; c < N; ++c) {
              float m = fabsf(y[c]);
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
              if (!(m * inv[4 * i + c] > 32768.f)) continue;
              int e = int(__float_as_uint(m) >> 23) - 127 - 6;       // to [2^6, 2^7): room to grow
              e = e > 126 ? 126 : (e < -126 ? -126 : e);
              const float f = __int_as_float((127 - e) << 23);
              const float ratio = t == c ? f / inv[4 * i + c] : 1.f;   // columns 2t, 2t + 1: row t
              inv[4 * i + c] = f;
#pragma unroll
              for (int m2 = 0; m2 < MT; ++m2) {
                acc[m2][i][0] *= ratio, acc[m2][i][1] *= ratio;
                acc[m2][i][2] *= ratio, acc[m2][i][3] *= ratio;
              }
            }
          }
#pragma unroll
          for (int c = 0; c < N; ++c) {
            y[c] *= inv[4 * i + c];
            const __half hi = __float2half_rn(y[c]);
            const __half lo = __float2half_rn(y[c] - __half2float(hi));
            if (S::kStep == 32 || lane < S::kStep) {
              ps[S::column(4 * i + c, 0)][spot] = __half_as_ushort(hi);
              ps[S::column(4 * i + c, 1)][spot] = __half_as_ushort(lo);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const __nv_bfloat16 hi = __float2bfloat16_rn(y[c]);
            y[c] -= __bfloat162float(hi);
            const __nv_bfloat16 mid = __float2bfloat16_rn(y[c]);
            const __nv_bfloat16 lo = __float2bfloat16_rn(y[c] - __bfloat162float(mid));
            if (S::kStep == 32 || lane < S::kStep) {
              ps[S::column(4 * i + c, 0)][spot] = __bfloat16_as_ushort(hi);
              ps[S::column(4 * i + c, 1)][spot] = __bfloat16_as_ushort(mid);
              ps[S::column(4 * i + c, 2)][spot] = __bfloat16_as_ushort(lo);
            }
          }
        }
      };
      __syncwarp();                      // the last step's P has been read
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        if (nq == 4 * i + 1) score(std::integral_constant<int, 1>{}, i);
        else if (nq > 4 * i) score(std::integral_constant<int, kQ>{}, i);
      }
      __syncwarp();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (j0 + 16 * nb >= n) continue;           // nothing was loaded there
        uint2 pb[NT];                  // P of the lane's four keys, column g
#pragma unroll
        for (int i = 0; i < NT; ++i)
          pb[i] = *reinterpret_cast<const uint2*>(&ps[8 * i + g][16 * nb + 4 * t]);
        uint32_t v[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t row = data + block_at[nb] + plane_at + v_at[i & (S::kSwizzle ? 1 : 0)] +
                               (S::kSwizzle ? (i >> 1) * 1024 : i * 4 * S::kRow);
          if constexpr (VW == 2) {
            const uint2 x = lds8(row);
            v[i][0] = x.x, v[i][1] = x.y;
          } else {
#pragma unroll
            for (int c = 0; c < VW / 4; ++c) {
              const uint4 x = lds16(row + half_at * c);
              v[i][4 * c] = x.x, v[i][4 * c + 1] = x.y, v[i][4 * c + 2] = x.z, v[i][4 * c + 3] = x.w;
            }
          }
        }
        if (j0 + 16 * nb + 16 > n) {               // rows behind the history: 0 * NaN
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (j0 + 16 * nb + key_of(i) >= n)
#pragma unroll
              for (int w = 0; w < VW; ++w) v[i][w] = 0u;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {             // 16 dimensions: a lane's two neighbours
          uint32_t a0, a1, a2, a3;
          if constexpr (S::kF16) {
            const uint32_t sel = m & 1 ? 0x7362u : 0x5140u;
            halves_of_e4m3(__byte_perm(v[0][m >> 1], v[1][m >> 1], sel), a0, a1);
            halves_of_e4m3(__byte_perm(v[2][m >> 1], v[3][m >> 1], sel), a2, a3);
          } else {
            a0 = __byte_perm(v[0][m], v[1][m], 0x5410);
            a1 = __byte_perm(v[0][m], v[1][m], 0x7632);
            a2 = __byte_perm(v[2][m], v[3][m], 0x5410);
            a3 = __byte_perm(v[2][m], v[3][m], 0x7632);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i)
            mma<S::kF16>(acc[m][i], a0, a1, a2, a3, pb[i].x, pb[i].y);
        }
      }
    }
    // ---- the chain of products into the warp's fp32 sums
    ++chain;
    if (chain == kFold || (what.z & kLast)) {
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        float scale = 1.f;                         // of row 4i + t
        if constexpr (S::kF16) {
          float f = t & 1 ? inv[4 * i + 1] : inv[4 * i];
          if constexpr (kQ == 4) f = t & 2 ? (t & 1 ? inv[4 * i + 3] : inv[4 * i + 2]) : f;
          scale = 1.f / f;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int dim = (S::kF16 ? g * (HD / 8) + 2 * m : 64 * (m >> 2) + 8 * g + 2 * (m & 3));
          float2 x = make_float2(acc[m][i][0] + acc[m][i][1], acc[m][i][2] + acc[m][i][3]);
          if constexpr (S::kF16) {
            x.x *= scale, x.y *= scale;
          } else if constexpr (NT > 1) {
            x.x += acc[m][2][i], x.y += acc[m][2][2 + i];
          } else {
            x.x += __shfl_xor_sync(0xffffffffu, acc[m][0][0], 2);
            x.y += __shfl_xor_sync(0xffffffffu, acc[m][0][2], 2);
          }
          if (4 * i + t < S::kGroup) {
            float2* at = reinterpret_cast<float2*>(&sum[4 * i + t][dim]);
            if (folds > 0) {
              const float2 y = *at;
              x.x += y.x, x.y += y.y;
            }
            *at = x;
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.f;
      ++folds;
      chain = 0;
    }
    if (what.z & kLast) {
      const Part part = ring.unit[st].part;        // the stage goes back before the join
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.empty[st]);
      up = sync() && finish<S, HD>(a, part, s_sum, s_self, &ring.last, sync);
    } else {
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.empty[st]);
    }
    fresh = (what.z & kLast) != 0;
    if (++st == S::kStages) st = 0, parity ^= 1;
  }
  if (!done) err |= HSTU_DEVERR_TIMEOUT;
  if (err != 0) atomicOr(a.error, err);
}

// No more blocks than there can be units.
template <class S>
unsigned grid_of(const PagesArgs& a) {
  const int64_t most = a.R * a.H * ((a.width << a.page_shift) / S::kUnit + 1);
  const int64_t grid = int64_t(a.num_sms) * S::kPerSm;
  return unsigned(grid < most ? grid : most);
}

template <int FMT, int HD, int NT>
cudaError_t launch(const PagesArgs& a, cudaStream_t st) {
  using S = Shape<FMT, HD, NT>;
  static_assert(S::kPerSm <= kPagesBlocksPerSm, "workspace");
  static_assert(S::kGroup * HD <= kPagesPartial && S::kGroup <= 8, "workspace");
  static_assert(S::kTiles * 4 >= S::kGroup && S::kGroup * S::kPieces <= S::kColumns, "operand");
  static_assert(S::kF32 || NT == 1 || NT == (FMT == HSTU_PAGES_BF16 ? 3 : 2), "columns");
  static_assert(S::kHalves * 128 >= S::kRow || !S::kSwizzle, "boxes");
  static_assert(S::kF32 || S::kRingBytes(S::kStages) <= 128 * 1024, "ring");
  if constexpr (S::kF32) {
    return launch_early(pages_attention_f32_kernel<HD, NT>, grid_of<S>(a), S::kThreads, 0, st, a);
  } else {
    static std::atomic<uint64_t> done{0};
    constexpr int bytes = S::kRingBytes(S::kStages);
    cudaError_t e = smem_opt_in(pages_attention_kernel<FMT, HD, NT>, bytes, done);
    if (e != cudaSuccess) return e;
    CUtensorMap run, block;
    memset(&run, 0, sizeof(run));
    memset(&block, 0, sizeof(block));
    if (S::kSwizzle) {
      const int page = 1 << a.page_shift;
      const uint64_t rows = uint64_t(a.num_pages) * a.H * 2 * page;
      if (!make_tmap_2d_u8_sw128(&run, a.kv, S::kRow, rows, page < S::kUnit ? page : S::kUnit) ||
          !make_tmap_2d_u8_sw128(&block, a.kv, S::kRow, rows, 16))
        return cudaErrorInvalidValue;
    }
    return launch_early(pages_attention_kernel<FMT, HD, NT>, grid_of<S>(a), S::kThreads, bytes, st,
                        a, run, block);
  }
}

}  // namespace

cudaError_t launch_pages_attention(const PagesArgs& a, cudaStream_t st) {
  if (a.R <= 0 || a.B <= 0) return cudaSuccess;
  // More rows than users: some user has several, so the variants that take more rows of a user
  // at once.  Users without rows hide that, as the host knows R and B but no counts.  16
  // candidates each of 3 users of 8192 rows, in a call of those users (wide) and of 64 (narrow):
  // bf16 63 and 90 us (heads of 64, d 512), 129 and 157 (128, d 1024), e4m3 80 and 128 (128, d
  // 1024), but 68 and 56 (64, d 512), fp32 146 and 205 (64, d 512).  With two rows a user, 8
  // users of 2048: bf16 19 and 16 (d 512), 32 and 21 (d 1024), e4m3 24 and 20 (d 1024), fp32
  // 19 and 25.  Callers leave idle users out where it counts, as runtime.PagedHistory.score does.
  const bool wide = a.R > a.B;
#define HSTU_PAGES_ATTN(F, D) \
  return wide ? launch<F, D, (F == HSTU_PAGES_BF16 ? 3 : 2)>(a, st) : launch<F, D, 1>(a, st)
  if (a.format == HSTU_PAGES_FP32) {
    switch (a.hd) {
      case 32: HSTU_PAGES_ATTN(HSTU_PAGES_FP32, 32);
      case 64: HSTU_PAGES_ATTN(HSTU_PAGES_FP32, 64);
      case 96: HSTU_PAGES_ATTN(HSTU_PAGES_FP32, 96);
      case 128: HSTU_PAGES_ATTN(HSTU_PAGES_FP32, 128);
      default: return cudaErrorInvalidValue;
    }
  }
  if (a.format == HSTU_PAGES_BF16) {
    if (a.hd == 64) HSTU_PAGES_ATTN(HSTU_PAGES_BF16, 64);
    if (a.hd == 128) HSTU_PAGES_ATTN(HSTU_PAGES_BF16, 128);
  } else {
    if (a.hd == 64) HSTU_PAGES_ATTN(HSTU_PAGES_E4M3, 64);
    if (a.hd == 128) HSTU_PAGES_ATTN(HSTU_PAGES_E4M3, 128);
  }
#undef HSTU_PAGES_ATTN
  return cudaErrorInvalidValue;
}

}  // namespace hstu
