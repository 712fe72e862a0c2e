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
//  * a warp takes 16 keys at a time straight from global memory into the
//    operand layout of the matrix instructions: the next block's keys are
//    loaded as soon as the scores of this one have used theirs, its values as
//    soon as the product has.  Nothing is staged in shared memory.
//  * products on mma.sync, whose N = 8 fits a few rows (a tcgen05 tile has 64
//    rows at least and wants its operands in shared memory, for work that is
//    bound by the loads).  Scores: the 16 rows of the first operand are 8 keys
//    twice, with the even and the odd pairs of their dimensions, and a row of
//    q takes two columns, so that the 16 bytes a lane loads of a key are its
//    operand as they are; key g and query t meet in one lane.
//  * from the scores to P a lane has a key: bias, scales, SiLU and the split
//    are done once a key and row.  P goes through 16-bit shared memory into the
//    second operand of the output product (rows = columns of P, M = dimensions).
//  * fp32 results from 16-bit operands: q, k and v are exact in bf16 (bf16
//    pages) or fp16 (e4m3 codes, and q times a power of two), and P is split
//    into pieces that go through the product as columns of their own: three
//    bf16 pieces (8 + 8 + 8 bits) or two fp16 ones (11 + 11).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "internal.h"
#include "pages.cuh"

namespace hstu {
namespace {

constexpr int kWarps = 4;
constexpr int kFold = 16;       // matrix products chained before the fp32 sums take over

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// s / (1 + exp(-s)); exp(-s) above fp32 gives -0, below it s.
__device__ __forceinline__ float silu(float s) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(s * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return s * r;
}

__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
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
// What a variant of the kernel is made of.  NT: tiles of 8 columns of P.
template <int FMT, int HD, int NT>
struct Shape {
  static constexpr bool kF32 = FMT == HSTU_PAGES_FP32;
  static constexpr bool kF16 = FMT == HSTU_PAGES_E4M3;
  static constexpr int kPieces = kF32 ? 1 : (kF16 ? 2 : 3);
  static constexpr int kGroup = kF32 ? NT : (kF16 ? 4 * NT : 2 * NT);   // rows of q of a segment
  static constexpr int kTiles = (kGroup + 3) / 4;               // of 4 rows of q, for the scores
  static constexpr int kRows = kF32 ? NT : 8 * NT;              // columns of P, rows of the sums
  static constexpr int kBlocks = (kF32 || (HD == 128 && !kF16)) ? 1 : 2;   // of 16 keys, a warp's step
  static constexpr int kStep = 16 * kBlocks;                    // keys of a warp's step
  static constexpr int kUnit = kWarps * kStep;                  // keys of a unit
  static constexpr int kElem = kF32 ? 4 : (kF16 ? 1 : 2);
  static constexpr int kPerSm = HD == 128 ? (NT == 2 ? 2 : 3) : (NT == 2 ? 3 : 4);
  static constexpr int kPad = HD + 8;                           // row stride of the sums
};

struct User {
  int64_t r0, units;
  int32_t rows, n, nu;   // rows of the call, cached rows, units of one segment
};

// A user's share of the work; an ill-formed user has none (err says why).
template <class S>
__device__ __forceinline__ User user_of(const PagesArgs& a, int32_t b, int& err) {
  User u;
  const int64_t r0 = __ldg(a.offsets + b), r1 = __ldg(a.offsets + b + 1);
  const int64_t n = __ldg(a.lengths + b);
  u.r0 = r0;
  u.units = 0;
  u.rows = 0;
  u.n = 0;
  u.nu = 1;
  if (r0 < 0 || r1 < r0 || r1 > a.R || (b == 0 && r0 != 0)) {
    err |= HSTU_DEVERR_OFFSETS;
    return u;
  }
  if (n < 0 || n > (a.width << a.page_shift)) {
    err |= HSTU_DEVERR_PAGES;
    return u;
  }
  u.rows = int32_t(r1 - r0);
  u.n = int32_t(n);
  u.nu = n == 0 ? 1 : int32_t((n + S::kUnit - 1) / S::kUnit);
  u.units = int64_t((u.rows + S::kGroup - 1) / S::kGroup) * a.H * u.nu;
  return u;
}

struct Shared {
  int64_t scan[kWarps];
  int64_t start;         // first unit of the block's first user
  int32_t user;
  int32_t last;
  float self[8];         // SiLU of each row's score with itself
};

template <int FMT, int HD, int NT>
__global__ void __launch_bounds__(kWarps * 32, (Shape<FMT, HD, NT>::kPerSm))
    pages_attention_kernel(const PagesArgs a) {
  using S = Shape<FMT, HD, NT>;
  constexpr int NB = S::kBlocks;
  static_assert(S::kTiles * 4 >= S::kGroup && S::kGroup * S::kPieces <= S::kRows, "operand");
  __shared__ Shared sh;
  __shared__ int4 s_time[128];                       // per bin: next threshold, two table entries
  __shared__ float s_sum[kWarps][S::kRows][S::kPad];
  // P of a warp's step, a row per column of the operand
  __shared__ __align__(16) uint16_t s_p[S::kF32 ? 1 : kWarps][S::kRows][S::kStep + 8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;

  // ---- the block's units [u0, u1) of all units
  const int32_t per = (a.B + kWarps * 32 - 1) / (kWarps * 32);
  int err = 0;
  int64_t mine = 0;
  for (int32_t b = tid * per; b < (tid + 1) * per && b < a.B; ++b) mine += user_of<S>(a, b, err).units;
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) sh.scan[warp] = inc;
  if (tid < 128) {
    const int cand = __ldg(a.time_lut + tid);
    const int next = cand + 1 < a.time_buckets ? cand + 1 : a.time_buckets - 1;
    s_time[tid] = make_int4(cand + 1 < a.time_buckets ? __ldg(a.thr32 + cand + 1) : 0x7FFFFFFF,
                            __float_as_int(__ldg(a.rab_time + cand)),
                            __float_as_int(__ldg(a.rab_time + next)), 0);
  }
  __syncthreads();
  int64_t before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh.scan[w];
    total += sh.scan[w];
  }
  if (blockIdx.x == 0 && err != 0) atomicOr(a.error, err);
  err = 0;
  // equal runs, but at least min_units: a cut costs a join (see launch)
  int64_t share = (total + gridDim.x - 1) / gridDim.x;
  if (share < a.min_units) share = a.min_units;
  int64_t u0 = int64_t(blockIdx.x) * share;
  if (u0 >= total) return;
  const int64_t u1 = u0 + share < total ? u0 + share : total;
  if (u0 >= before && u0 < before + mine) {
    int64_t at = before;
    int32_t b = tid * per;
    for (;; ++b) {
      int e = 0;
      const int64_t k = user_of<S>(a, b, e).units;
      if (u0 < at + k) break;
      at += k;
    }
    sh.start = at;
    sh.user = b;
  }
  __syncthreads();
  int32_t b = sh.user;
  int64_t start = sh.start;
  User user = user_of<S>(a, b, err);

  const float pos_far = __ldg(a.rab_pos + a.pos_clamp);
  const float self_bias = __ldg(a.rab_pos) + __ldg(a.rab_time);

  while (u0 < u1) {
    while (u0 >= start + user.units) {   // the next user that has rows
      start += user.units;
      for (;;) {
        const int32_t c = b + 1 + lane;
        int e = 0;
        const bool has = c < a.B && user_of<S>(a, c, e).units > 0;
        const unsigned m = __ballot_sync(0xffffffffu, has);
        if (m != 0) {
          b += __ffs(m);
          break;
        }
        b += 32;
        if (b >= a.B) return;            // cannot happen: u0 < total
      }
      user = user_of<S>(a, b, err);
    }
    const int64_t rel = u0 - start;
    const int32_t seg = int32_t(rel / user.nu), tile0 = int32_t(rel - int64_t(seg) * user.nu);
    const int h = seg % a.H, first = seg / a.H * S::kGroup;
    const int nq = user.rows - first < S::kGroup ? user.rows - first : S::kGroup;
    const int64_t row0 = user.r0 + first;
    const int32_t tile1 = int64_t(user.nu - tile0) < u1 - u0 ? user.nu : int32_t(tile0 + (u1 - u0));
    const int64_t seg0 = u0 - tile0;     // the segment's first unit
    const int32_t n = user.n;
    const int32_t* table = a.table + int64_t(b) * a.width;

    // the rows' scores with themselves go with the segment's first unit
    if (tile0 == 0) {
      for (int q = warp; q < nq; q += kWarps) {
        const int64_t at = (row0 + q) * 4 * a.d + 2 * a.d + h * HD + lane;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) {
          if (S::kF32)
            s = fmaf(static_cast<const float*>(a.uvqk)[at + 32 * e],
                     static_cast<const float*>(a.uvqk)[at + a.d + 32 * e], s);
          else
            s = fmaf(__bfloat162float(static_cast<const __nv_bfloat16*>(a.uvqk)[at + 32 * e]),
                     __bfloat162float(static_cast<const __nv_bfloat16*>(a.uvqk)[at + a.d + 32 * e]), s);
        }
        s = warp_sum(s) + self_bias;
        const int64_t ts = __ldg(a.ts + row0 + q);
        if (ts < 0 || ts >= kMaxTimestamp) err |= HSTU_DEVERR_TIMESTAMPS;
        if (lane == 0) sh.self[q] = silu(s);
      }
    }

    const int64_t ts0 = __ldg(a.ts + row0);
    // the two biases of a row of the group at key j, whose time is `then`
    auto bias_of = [&](int q, int32_t j, int64_t then) {
      const float pos = n - j < a.pos_clamp ? __ldg(a.rab_pos + (j < n ? n - j : 0)) : pos_far;
      const uint64_t now = uint64_t(q == 0 ? ts0 : __ldg(a.ts + row0 + q));
      const int64_t gap = int64_t(now - uint64_t(then));
      if (a.lut_exact && gap < 0x7FFFFFFE) {
        const uint32_t x = gap > 0 ? uint32_t(gap) + 1u : 1u;
        const int z = __clz(x);
        const int4 bin = s_time[(31 - z) * 4 + ((x << z) >> 29 & 3)];
        return pos + __int_as_float(gap >= bin.x ? bin.z : bin.y);
      }
      return pos + __ldg(a.rab_time + time_bucket(a.thresholds, a.time_buckets, gap));
    };
    auto page_of = [&](int32_t tile) {   // of the lane's key; -1: no key there
      const int32_t j = tile * S::kUnit + warp * S::kStep + (lane & (S::kStep - 1));
      if (tile >= tile1 || j >= n) return -1;
      const int32_t p = __ldg(table + (j >> a.page_shift));
      if (p >= 0 && p < a.num_pages) return p;
      err |= HSTU_DEVERR_PAGES;
      return -1;
    };
    const int32_t slot_mask = (1 << a.page_shift) - 1;
    // block of plane 0 of this head at the first of the 16 keys from j on
    auto block_at = [&](int32_t page, int32_t j) {
      return ((((int64_t(page) * a.H + h) * 2) << a.page_shift) + (j & slot_mask));
    };
    const int64_t plane = int64_t(1) << a.page_shift;

    int64_t then = 0;
    float (*sum)[S::kPad] = s_sum[warp];
    bool folded = false;

    if constexpr (S::kF32) {
      // 8 lanes a key, 4 keys at once, fp32 throughout
      constexpr int E = HD / 32;
      const int k4 = lane >> 3, t8 = lane & 7;
      float q[NT][4 * E], o[NT][4 * E];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int64_t r = row0 + (i < nq ? i : 0);
          const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.uvqk) +
                                 r * 4 * a.d + 2 * a.d + h * HD + 32 * e) + t8);
          q[i][4 * e] = v.x, q[i][4 * e + 1] = v.y, q[i][4 * e + 2] = v.z, q[i][4 * e + 3] = v.w;
          o[i][4 * e] = o[i][4 * e + 1] = o[i][4 * e + 2] = o[i][4 * e + 3] = 0.f;
        }
      for (int32_t tile = tile0; tile < tile1; ++tile) {
        const int32_t j0 = tile * S::kUnit + warp * S::kStep;
        const int32_t mine_p = page_of(tile), page = __shfl_sync(0xffffffffu, mine_p, 0);
        if (page >= 0) {                 // else no keys here, or a page that is none
          const int32_t jl = j0 + (lane & 15);
          if (mine_p >= 0) then = __ldg(a.page_ts + (int64_t(page) << a.page_shift) + (jl & slot_mask));
          float bias[NT];                // of the lane's key
#pragma unroll
          for (int i = 0; i < NT; ++i) bias[i] = bias_of(i < nq ? i : 0, jl, then);
          const float* base = reinterpret_cast<const float*>(
              static_cast<const char*>(a.kv) + block_at(page, j0) * (HD * S::kElem));
          float4 k[4][E], v[4][E];
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const float* at = base + int64_t(4 * s + k4) * HD + 32 * e + 4 * t8;
              k[s][e] = __ldg(reinterpret_cast<const float4*>(at));
              v[s][e] = __ldg(reinterpret_cast<const float4*>(at + plane * HD));
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
              const float p = silu(x + __shfl_sync(0xffffffffu, bias[i], 4 * s + k4));
              if (!ok) continue;           // no memory behind the history may reach the sum
#pragma unroll
              for (int e = 0; e < E; ++e) {
                o[i][4 * e] = fmaf(p, v[s][e].x, o[i][4 * e]);
                o[i][4 * e + 1] = fmaf(p, v[s][e].y, o[i][4 * e + 1]);
                o[i][4 * e + 2] = fmaf(p, v[s][e].z, o[i][4 * e + 2]);
                o[i][4 * e + 3] = fmaf(p, v[s][e].w, o[i][4 * e + 3]);
              }
            }
          }
        }
        if ((tile - tile0) % kFold == kFold - 1 || tile + 1 == tile1) {
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
      if (!folded)
        for (int i = lane; i < NT * HD; i += 32) sum[i / HD][i % HD] = 0.f;
    } else {
      constexpr int KC = HD * S::kElem / 64;     // 16-byte chunks a lane has of a key
      constexpr int VW = HD * S::kElem / 32;     // words a lane has of a value
      constexpr int KS = HD / 32;                // products a tile of scores takes
      constexpr int MT = HD / 16;                // tiles of 16 dimensions of the output
      constexpr int QT = S::kTiles;
      // Columns 2i and 2i + 1 of the score product are query i, with the even and the odd
      // pairs of its dimensions: what the lane's g is, at its t's dimensions.
      uint32_t qb[QT][KS][2];
      float q_scale[QT];
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        const int q = 4 * i + (g >> 1) < nq ? 4 * i + (g >> 1) : nq - 1;
        const bool odd = (g & 1) != 0;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(a.uvqk) + (row0 + q) * 4 * a.d + 2 * a.d + h * HD);
        q_scale[i] = 1.f;
        if constexpr (!S::kF16) {
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const uint4 v = __ldg(src + t + 4 * c);
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
            unpack_bf16(__ldg(src + 2 * (t + 4 * c)), x[c]);
            unpack_bf16(__ldg(src + 2 * (t + 4 * c) + 1), x[c] + 8);
#pragma unroll
            for (int k = 0; k < 16; ++k) m = fmaxf(m, fabsf(x[c][k]));
          }
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          int e = int(__float_as_uint(m) >> 23) - 127 - 14;
          e = e < -126 ? -126 : (e > 112 ? 112 : e);
          q_scale[i] = __int_as_float((e + 127) << 23);
          const float inv = __int_as_float((127 - e) << 23);
#pragma unroll
          for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const int at = 8 * k + 4 * w;
                qb[i][2 * c + k][w] = pack_half((odd ? x[c][at + 2] : x[c][at]) * inv,
                                                (odd ? x[c][at + 3] : x[c][at + 1]) * inv);
              }
        }
      }
      uint16_t (*ps)[S::kStep + 8] = s_p[warp];
      __syncwarp();
      for (int i = lane; i < S::kRows * (S::kStep + 8) / 2; i += 32)
        reinterpret_cast<uint32_t*>(&ps[0][0])[i] = 0u;   // columns without a piece
      float acc[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.f;
      // fp16 pieces: P times a power of two of its row stays below 2^15; inv is that of the row
      // whose two pieces are the lane's columns (row t of the tile)
      float inv[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) inv[i] = __int_as_float((127 + 126) << 23);

      uint4 kr[NB][2][KC];
      uint32_t vr[NB][4][VW];
      float ks = 0.f, vs = 0.f;
      const char* kv = static_cast<const char*>(a.kv);
      // keys g and g + 8 of each block; the lane's own key's time and scales
      auto load_k = [&](int32_t tile, int32_t p) {
        const int32_t j0 = tile * S::kUnit + warp * S::kStep;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int32_t page = __shfl_sync(0xffffffffu, p, 16 * nb);
          if (page < 0) continue;
          const char* at = kv + (block_at(page, j0 + 16 * nb) + g) * (HD * S::kElem) + 16 * t;
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            kr[nb][0][c] = load16(at + 64 * c);
            kr[nb][1][c] = load16(at + 8 * HD * S::kElem + 64 * c);
          }
        }
        if (p >= 0) {
          const int32_t j = j0 + (lane & (S::kStep - 1));
          then = __ldg(a.page_ts + (int64_t(p) << a.page_shift) + (j & slot_mask));
          if (S::kF16) {
            const uint8_t* sc = a.scales + block_at(p, j);
            ks = block_scale(__ldg(sc));
            vs = block_scale(__ldg(sc + plane));
          }
        }
      };
      // values of the keys 4t .. 4t + 3 of each block: the lane's rows of P
      auto load_v = [&](int32_t tile, int32_t p) {
        const int32_t j0 = tile * S::kUnit + warp * S::kStep;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int32_t page = __shfl_sync(0xffffffffu, p, 16 * nb);
          if (page < 0) continue;
          const char* at = kv + (block_at(page, j0 + 16 * nb) + plane + 4 * t) * (HD * S::kElem) +
                           (VW == 2 ? 8 : 16) * g;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const char* row = at + i * (HD * S::kElem);
            if constexpr (VW == 2) {
              const uint2 v = load8(row);
              vr[nb][i][0] = v.x, vr[nb][i][1] = v.y;
            } else {
#pragma unroll
              for (int c = 0; c < VW / 4; ++c) {
                const uint4 v = load16(row + 128 * c);
                vr[nb][i][4 * c] = v.x, vr[nb][i][4 * c + 1] = v.y;
                vr[nb][i][4 * c + 2] = v.z, vr[nb][i][4 * c + 3] = v.w;
              }
            }
          }
          if (j0 + 16 * nb + 16 > n) {             // rows behind the history: 0 * NaN
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (j0 + 16 * nb + 4 * t + i >= n)
#pragma unroll
                for (int w = 0; w < VW; ++w) vr[nb][i][w] = 0u;
          }
        }
      };
      // acc into the warp's fp32 sums
      auto fold = [&]() {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float scale = S::kF16 ? 1.f / inv[i] : 1.f;
          const int r = 8 * i + 2 * t;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const int dim = (S::kF16 ? g * (HD / 8) + 2 * m : 64 * (m >> 2) + 8 * g + 2 * (m & 3));
            float2* p0 = reinterpret_cast<float2*>(&sum[r][dim]);
            float2* p1 = reinterpret_cast<float2*>(&sum[r + 1][dim]);
            float2 x0 = make_float2(acc[m][i][0] * scale, acc[m][i][2] * scale);
            float2 x1 = make_float2(acc[m][i][1] * scale, acc[m][i][3] * scale);
            if (folded) {
              const float2 y0 = *p0, y1 = *p1;
              x0.x += y0.x, x0.y += y0.y, x1.x += y1.x, x1.y += y1.y;
            }
            *p0 = x0;
            *p1 = x1;
            acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.f;
          }
        }
        folded = true;
      };

      int32_t p_now = page_of(tile0);
      load_k(tile0, p_now);
      load_v(tile0, p_now);
      int32_t p_next = page_of(tile0 + 1);
      for (int32_t tile = tile0; tile < tile1; ++tile) {
        const int32_t j0 = tile * S::kUnit + warp * S::kStep;
        const int32_t jl = j0 + (lane & (S::kStep - 1));      // the lane's key
        int32_t page[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) page[nb] = __shfl_sync(0xffffffffu, p_now, 16 * nb);
        const float ks_now = ks, vs_now = vs;
        const int64_t then_now = then;
        float s[NB][2][QT];              // of key 16 nb + 8 x + g and row 4i + t
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int i = 0; i < QT; ++i) s[nb][x][i] = 0.f;
            if (page[nb] < 0) continue;
            float c[QT][4];
#pragma unroll
            for (int i = 0; i < QT; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
#pragma unroll
            for (int k = 0; k < KC; ++k) {
              const uint4 v = kr[nb][x][k];
              if constexpr (S::kF16) {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  uint32_t a0, a1, a2, a3;
                  halves_of_e4m3(w[2 * y], a0, a1);
                  halves_of_e4m3(w[2 * y + 1], a2, a3);
#pragma unroll
                  for (int i = 0; i < QT; ++i)
                    mma<true>(c[i], a0, a1, a2, a3, qb[i][2 * k + y][0], qb[i][2 * k + y][1]);
                }
              } else {
#pragma unroll
                for (int i = 0; i < QT; ++i)
                  mma<false>(c[i], v.x, v.y, v.z, v.w, qb[i][k][0], qb[i][k][1]);
              }
            }
#pragma unroll
            for (int i = 0; i < QT; ++i) s[nb][x][i] = c[i][0] + c[i][3];
          }
        }
        load_k(tile + 1, p_next);
        const int32_t p_then = page_of(tile + 2);
        __syncwarp();                    // the last step's P has been read
        for (int q = 0; q < nq; ++q) {   // a lane a key
          float y = 0.f;
#pragma unroll
          for (int i = 0; i < QT; ++i) {
            if (QT > 1 && (q >> 2) != i) continue;
            const int src = 4 * (lane & 7) + (q & 3);
            const float y0 = __shfl_sync(0xffffffffu, s[0][0][i], src);
            const float y1 = __shfl_sync(0xffffffffu, s[0][1][i], src);
            y = lane & 8 ? y1 : y0;
            if constexpr (NB == 2) {
              const float y2 = __shfl_sync(0xffffffffu, s[1][0][i], src);
              const float y3 = __shfl_sync(0xffffffffu, s[1][1][i], src);
              const float z = lane & 8 ? y3 : y2;
              y = lane & 16 ? z : y;
            }
            if constexpr (S::kF16)
              y = y * __shfl_sync(0xffffffffu, q_scale[i], 8 * (q & 3)) * ks_now;
          }
          y = silu(y + bias_of(q, jl, then_now));
          if constexpr (S::kF16) y *= vs_now;
          y = p_now >= 0 ? y : 0.f;      // no key here: what memory holds must not reach the sum
          if constexpr (S::kF16) {
            float f = 1.f;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              if (NT > 1 && (q >> 2) != i) continue;
              f = __shfl_sync(0xffffffffu, inv[i], q & 3);
              if (__any_sync(0xffffffffu, fabsf(y) * f > 32768.f)) {   // raise the row's power
                float m = fabsf(y);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                int e = int(__float_as_uint(m) >> 23) - 127 - 6;       // to [2^6, 2^7): room to grow
                e = e > 126 ? 126 : (e < -126 ? -126 : e);
                const float now = __int_as_float((127 - e) << 23);
                const float ratio = now / f;
                f = now;
                if (t == (q & 3)) {
                  inv[i] = now;
#pragma unroll
                  for (int k = 0; k < MT; ++k) {
                    acc[k][i][0] *= ratio, acc[k][i][1] *= ratio;
                    acc[k][i][2] *= ratio, acc[k][i][3] *= ratio;
                  }
                }
              }
            }
            y *= f;
            const __half hi = __float2half_rn(y);
            const __half lo = __float2half_rn(y - __half2float(hi));
            if (S::kStep == 32 || lane < S::kStep) {
              ps[2 * q][lane] = __half_as_ushort(hi);
              ps[2 * q + 1][lane] = __half_as_ushort(lo);
            }
          } else {
            const __nv_bfloat16 hi = __float2bfloat16_rn(y);
            y -= __bfloat162float(hi);
            const __nv_bfloat16 mid = __float2bfloat16_rn(y);
            const __nv_bfloat16 lo = __float2bfloat16_rn(y - __bfloat162float(mid));
            if (S::kStep == 32 || lane < S::kStep) {
              ps[3 * q][lane] = __bfloat16_as_ushort(hi);
              ps[3 * q + 1][lane] = __bfloat16_as_ushort(mid);
              ps[3 * q + 2][lane] = __bfloat16_as_ushort(lo);
            }
          }
        }
        __syncwarp();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (page[nb] < 0) continue;
          uint2 pb[NT];                  // P of the keys 4t .. 4t + 3, column g
#pragma unroll
          for (int i = 0; i < NT; ++i)
            pb[i] = *reinterpret_cast<const uint2*>(&ps[8 * i + g][16 * nb + 4 * t]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {           // 16 dimensions: a lane's two neighbours
            uint32_t a0, a1, a2, a3;
            if constexpr (S::kF16) {
              const uint32_t sel = m & 1 ? 0x7362u : 0x5140u;
              halves_of_e4m3(__byte_perm(vr[nb][0][m >> 1], vr[nb][1][m >> 1], sel), a0, a1);
              halves_of_e4m3(__byte_perm(vr[nb][2][m >> 1], vr[nb][3][m >> 1], sel), a2, a3);
            } else {
              a0 = __byte_perm(vr[nb][0][m], vr[nb][1][m], 0x5410);
              a1 = __byte_perm(vr[nb][0][m], vr[nb][1][m], 0x7632);
              a2 = __byte_perm(vr[nb][2][m], vr[nb][3][m], 0x5410);
              a3 = __byte_perm(vr[nb][2][m], vr[nb][3][m], 0x7632);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
              mma<S::kF16>(acc[m][i], a0, a1, a2, a3, pb[i].x, pb[i].y);
          }
        }
        load_v(tile + 1, p_next);
        p_now = p_next;
        p_next = p_then;
        if ((tile - tile0) % kFold == kFold - 1) fold();
      }
      if (!folded || (tile1 - tile0) % kFold != 0) fold();
    }
    __syncthreads();

    // ---- the warps' sums, and the other blocks' where the segment is cut
    const int32_t c0 = int32_t(seg0 / share), c1 = int32_t((seg0 + user.nu - 1) / share);
    const bool whole = c0 == c1;
    float* part = a.partial + (int64_t(blockIdx.x) * 2 + (tile0 == 0 ? 1 : 0)) * (S::kGroup * HD);
    for (int i = tid; i < nq * HD; i += kWarps * 32) {
      const int q = i / HD, c = i % HD;
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int k = 0; k < S::kPieces; ++k) x += s_sum[w][q * S::kPieces + k][c];
      if (tile0 == 0) {
        const int64_t at = (row0 + q) * 4 * a.d + a.d + h * HD + c;
        const float v = S::kF32 ? static_cast<const float*>(a.uvqk)[at]
                                : __bfloat162float(static_cast<const __nv_bfloat16*>(a.uvqk)[at]);
        x = fmaf(sh.self[q], v, x);
      }
      if (whole) a.av[(row0 + q) * a.d + h * HD + c] = x / float(a.n_norm);
      else part[i] = x;
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int32_t k = atomicAdd(a.tickets + c0, 1);
        sh.last = k == c1 - c0 ? 1 : 0;
        if (sh.last) a.tickets[c0] = 0;            // as the next call expects it
      }
      __syncthreads();
      if (sh.last) {
        __threadfence();
        for (int i = tid; i < nq * HD; i += kWarps * 32) {
          float x = 0.f;
          for (int32_t c = c0; c <= c1; ++c)
            x += __ldcg(a.partial + (int64_t(c) * 2 + (c == c0 ? 1 : 0)) * (S::kGroup * HD) + i);
          a.av[(row0 + i / HD) * a.d + h * HD + i % HD] = x / float(a.n_norm);
        }
      }
    }
    __syncthreads();
    u0 += tile1 - tile0;
  }
  if (err != 0) atomicOr(a.error, err);
}

template <int FMT, int HD, int NT>
cudaError_t launch(const PagesArgs& a, cudaStream_t st) {
  using S = Shape<FMT, HD, NT>;
  // no more blocks than there can be units
  const int64_t keys = (a.width << a.page_shift) / S::kUnit + 1;
  const int64_t most = (a.R < INT32_MAX / (a.H * keys) ? a.R * a.H * keys : INT32_MAX);
  const int64_t grid = int64_t(a.num_sms) * S::kPerSm;
  static_assert(S::kPerSm <= kPagesBlocksPerSm && S::kGroup * HD <= kPagesPartial, "workspace");
  pages_attention_kernel<FMT, HD, NT>
      <<<unsigned(grid < most ? grid : most), kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pages_attention(const PagesArgs& args, cudaStream_t st) {
  if (args.R <= 0 || args.B <= 0) return cudaSuccess;
  PagesArgs a = args;
  a.min_units = 2;
  // more rows than users: candidates, so the variants that take more rows of a user at once
  const bool wide = a.R > a.B;
#define HSTU_PAGES_ATTN(F, D) return wide ? launch<F, D, 2>(a, st) : launch<F, D, 1>(a, st)
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
