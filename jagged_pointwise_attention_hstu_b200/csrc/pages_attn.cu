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
//    bound by the loads).  Scores: rows of q (M) times keys (N); output:
//    values (M = dimensions) times P (N = rows); the score layout of a lane is
//    the operand layout of P, so P never leaves its registers.
//  * fp32 results from 16-bit operands: q, k and v are exact in bf16 (bf16
//    pages) or fp16 (e4m3 codes, and q times a power of two), and P is split
//    into pieces that go through the product as rows of their own: three bf16
//    pieces (8 + 8 + 8 bits) or two fp16 ones (11 + 11).  One row of the eight
//    would do for a single query; the pieces take the others.
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

__device__ __forceinline__ float silu(float s) { return __fdividef(s, 1.0f + __expf(-s)); }

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

__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t two) {   // exact
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(two), __NV_E4M3);
  return uint32_t(h.x) | (uint32_t(h.y) << 16);
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What a variant of the kernel is made of.  NT: tiles of 8 operand rows.
template <int FMT, int HD, int NT>
struct Shape {
  static constexpr bool kF32 = FMT == HSTU_PAGES_FP32;
  static constexpr bool kF16 = FMT == HSTU_PAGES_E4M3;
  static constexpr int kPieces = kF32 ? 1 : (kF16 ? 2 : 3);
  static constexpr int kGroup = kF32 ? NT : 8 * NT / kPieces;   // rows of q a segment holds
  static constexpr int kRows = kF32 ? NT : 8 * NT;              // rows of its sums
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
  __shared__ Shared sh;
  __shared__ int4 s_time[128];                       // per bin: next threshold, two table entries
  __shared__ float s_sum[kWarps][S::kRows][S::kPad];
  __shared__ float s_bias[kWarps][S::kGroup][S::kStep];
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

    // ---- the bias of the step's keys, a lane a key, for every row of the group
    float (*bias)[S::kStep] = s_bias[warp];
    const int64_t ts0 = __ldg(a.ts + row0);
    auto write_bias = [&](int32_t j, bool ok, int64_t then) {
      float pos = pos_far;
      if (n - j < a.pos_clamp) pos = __ldg(a.rab_pos + (ok ? n - j : 0));
      for (int q = 0; q < nq; ++q) {
        const uint64_t now = uint64_t(q == 0 ? ts0 : __ldg(a.ts + row0 + q));
        const int64_t gap = int64_t(now - uint64_t(then));
        float v;
        if (a.lut_exact && gap < 0x7FFFFFFE) {
          const uint32_t x = gap > 0 ? uint32_t(gap) + 1u : 1u;
          const int z = __clz(x);
          const int4 bin = s_time[(31 - z) * 4 + ((x << z) >> 29 & 3)];
          v = __int_as_float(gap >= bin.x ? bin.z : bin.y);
        } else {
          v = __ldg(a.rab_time + time_bucket(a.thresholds, a.time_buckets, gap));
        }
        if (S::kStep == 32 || lane < S::kStep) bias[q][lane & (S::kStep - 1)] = v + pos;
      }
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
          __syncwarp();
          write_bias(jl, mine_p >= 0, then);
          __syncwarp();
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
              if (!ok) continue;           // no memory behind the history may reach the sum
              const float p = silu(x + bias[i < nq ? i : 0][4 * s + k4]);
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
      constexpr int KS = HD / 16;                // steps of 16 dimensions
      constexpr int MT = HD / 16;                // tiles of 16 dimensions of the output
      // q: rows g and g + 8 of the operand; row r is piece r % kPieces of query r / kPieces
      uint32_t qa[KS][4];
      float q_scale[2];
      float mask1[2], mask2[2];                  // 1: the row's piece is behind the first / second
      int q_at[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = g + 8 * half;
        const int q = r / S::kPieces < nq ? r / S::kPieces : nq - 1;
        q_at[half] = q;
        mask1[half] = r % S::kPieces >= 1 ? 1.f : 0.f;
        mask2[half] = r % S::kPieces >= 2 ? 1.f : 0.f;
        q_scale[half] = 1.f;
        if (half >= NT) {
#pragma unroll
          for (int s = 0; s < KS; ++s) qa[s][1] = qa[s][3] = 0u;
          continue;
        }
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(a.uvqk) + (row0 + q) * 4 * a.d + 2 * a.d + h * HD);
        if constexpr (!S::kF16) {
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const uint4 v = __ldg(src + t + 4 * c);
            qa[2 * c][half] = v.x;
            qa[2 * c][half + 2] = v.y;
            qa[2 * c + 1][half] = v.z;
            qa[2 * c + 1][half + 2] = v.w;
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
            for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[c][i]));
          }
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          int e = int(__float_as_uint(m) >> 23) - 127 - 14;
          e = e < -126 ? -126 : (e > 112 ? 112 : e);
          q_scale[half] = __int_as_float((e + 127) << 23);
          const float inv = __int_as_float((127 - e) << 23);
#pragma unroll
          for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              qa[4 * c + w][half] = pack_half(x[c][4 * w] * inv, x[c][4 * w + 1] * inv);
              qa[4 * c + w][half + 2] = pack_half(x[c][4 * w + 2] * inv, x[c][4 * w + 3] * inv);
            }
        }
      }
      float acc[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.f;
      // fp16 pieces: P is kept below 2^15 by a power of two of its row (inv), raised when needed
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
      // values of the keys 2t, 2t + 1, 2t + 8, 2t + 9: the lane's columns of P
      auto load_v = [&](int32_t tile, int32_t p) {
        const int32_t j0 = tile * S::kUnit + warp * S::kStep;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int32_t page = __shfl_sync(0xffffffffu, p, 16 * nb);
          if (page < 0) continue;
          const char* at = kv + (block_at(page, j0 + 16 * nb) + plane) * (HD * S::kElem);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const char* row = at + (2 * t + (i & 1) + 8 * (i >> 1)) * (HD * S::kElem);
            if constexpr (VW == 2) {
              const uint2 v = load8(row + 8 * g);
              vr[nb][i][0] = v.x, vr[nb][i][1] = v.y;
            } else {
#pragma unroll
              for (int c = 0; c < VW / 4; ++c) {
                const uint4 v = load16(row + 16 * g + 128 * c);
                vr[nb][i][4 * c] = v.x, vr[nb][i][4 * c + 1] = v.y;
                vr[nb][i][4 * c + 2] = v.z, vr[nb][i][4 * c + 3] = v.w;
              }
            }
            if (j0 + 16 * nb + 16 > n && j0 + 16 * nb + 2 * t + (i & 1) + 8 * (i >> 1) >= n) {
#pragma unroll
              for (int w = 0; w < VW; ++w) vr[nb][i][w] = 0u;   // rows behind the history: 0 * NaN
            }
          }
        }
      };
      // acc into the warp's fp32 sums
      auto fold = [&]() {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float s0 = 1.f, s1 = 1.f;      // the scales of rows 2t and 2t + 1
          if constexpr (S::kF16) {
            s0 = 1.f / __shfl_sync(0xffffffffu, inv[i], 8 * t);
            s1 = 1.f / __shfl_sync(0xffffffffu, inv[i], 8 * t + 4);
          }
          const int r = 8 * i + 2 * t;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const int dim = (S::kF16 ? g * (HD / 8) + 2 * m : 64 * (m >> 2) + 8 * g + 2 * (m & 3));
            float2* p0 = reinterpret_cast<float2*>(&sum[r][dim]);
            float2* p1 = reinterpret_cast<float2*>(&sum[r + 1][dim]);
            float2 x0 = make_float2(acc[m][i][0] * s0, acc[m][i][2] * s0);
            float2 x1 = make_float2(acc[m][i][1] * s1, acc[m][i][3] * s1);
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
        int32_t page[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) page[nb] = __shfl_sync(0xffffffffu, p_now, 16 * nb);
        __syncwarp();
        write_bias(j0 + (lane & (S::kStep - 1)), p_now >= 0, then);
        const float ks_now = ks, vs_now = vs;
        float s[NB][2][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (page[nb] < 0) continue;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            s[nb][x][0] = s[nb][x][1] = s[nb][x][2] = s[nb][x][3] = 0.f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
              const uint4 k = kr[nb][x][c];
              if constexpr (S::kF16) {
                const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  mma<true>(s[nb][x], qa[4 * c + i][0], qa[4 * c + i][1], qa[4 * c + i][2],
                            qa[4 * c + i][3], half2_of_e4m3(w[i] & 0xffffu),
                            half2_of_e4m3(w[i] >> 16));
              } else {
                mma<false>(s[nb][x], qa[2 * c][0], qa[2 * c][1], qa[2 * c][2], qa[2 * c][3], k.x,
                           k.y);
                mma<false>(s[nb][x], qa[2 * c + 1][0], qa[2 * c + 1][1], qa[2 * c + 1][2],
                           qa[2 * c + 1][3], k.z, k.w);
              }
            }
          }
        }
        load_k(tile + 1, p_next);
        const int32_t p_then = page_of(tile + 2);
        __syncwarp();
        uint32_t pb[NB][NT][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (page[nb] < 0) continue;
#pragma unroll
          for (int x = 0; x < 2; ++x) {            // keys 8x + 2t, 8x + 2t + 1 of the block
            const int key = 16 * nb + 8 * x + 2 * t;
            float k0 = 1.f, k1 = 1.f, v0 = 1.f, v1 = 1.f;
            if constexpr (S::kF16) {
              k0 = __shfl_sync(0xffffffffu, ks_now, key);
              k1 = __shfl_sync(0xffffffffu, ks_now, key + 1);
              v0 = __shfl_sync(0xffffffffu, vs_now, key);
              v1 = __shfl_sync(0xffffffffu, vs_now, key + 1);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const float2 bb = *reinterpret_cast<const float2*>(&bias[q_at[i]][key]);
              float y0 = s[nb][x][2 * i], y1 = s[nb][x][2 * i + 1];
              if constexpr (S::kF16) y0 = y0 * q_scale[i] * k0, y1 = y1 * q_scale[i] * k1;
              y0 = silu(y0 + bb.x);
              y1 = silu(y1 + bb.y);
              if constexpr (S::kF16) y0 *= v0, y1 *= v1;
              if (j0 + 16 * nb + 16 > n) {         // the block that the history ends in
                y0 = j0 + key < n ? y0 : 0.f;
                y1 = j0 + key + 1 < n ? y1 : 0.f;
              }
              s[nb][x][2 * i] = y0;
              s[nb][x][2 * i + 1] = y1;
            }
          }
        }
        if constexpr (S::kF16) {                   // keep |P| * inv within fp16
          bool over = false;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < NT; ++i)
              if (page[nb] >= 0)
                over |= fmaxf(fmaxf(fabsf(s[nb][0][2 * i]), fabsf(s[nb][0][2 * i + 1])),
                              fmaxf(fabsf(s[nb][1][2 * i]), fabsf(s[nb][1][2 * i + 1]))) * inv[i] >
                        32768.f;
          if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              float m = 0.f;
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                if (page[nb] >= 0)
                  m = fmaxf(m, fmaxf(fmaxf(fabsf(s[nb][0][2 * i]), fabsf(s[nb][0][2 * i + 1])),
                                     fmaxf(fabsf(s[nb][1][2 * i]), fabsf(s[nb][1][2 * i + 1]))));
              // the row's four lanes, and both pieces of its query
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
              float ratio = 1.f;
              if (m * inv[i] > 32768.f) {          // to [2^6, 2^7): room to grow
                int e = int(__float_as_uint(m) >> 23) - 127 - 6;
                e = e > 126 ? 126 : (e < -126 ? -126 : e);
                const float now = __int_as_float((127 - e) << 23);
                ratio = now / inv[i];
                inv[i] = now;
              }
              const float r0 = __shfl_sync(0xffffffffu, ratio, 8 * t);
              const float r1 = __shfl_sync(0xffffffffu, ratio, 8 * t + 4);
#pragma unroll
              for (int k = 0; k < MT; ++k) {
                acc[k][i][0] *= r0, acc[k][i][2] *= r0;
                acc[k][i][1] *= r1, acc[k][i][3] *= r1;
              }
            }
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (page[nb] < 0) continue;
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {          // the row's piece of P
              float y0 = s[nb][x][2 * i], y1 = s[nb][x][2 * i + 1];
              if constexpr (S::kF16) {
                y0 *= inv[i], y1 *= inv[i];
                const uint32_t w = pack_half(y0, y1);
                const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&w));
                y0 = fmaf(-mask1[i], hi.x, y0), y1 = fmaf(-mask1[i], hi.y, y1);
                pb[nb][i][x] = pack_half(y0, y1);
              } else {
                uint32_t w = pack_bf16(y0, y1);
                y0 = fmaf(-mask1[i], __uint_as_float(w << 16), y0);
                y1 = fmaf(-mask1[i], __uint_as_float(w & 0xffff0000u), y1);
                w = pack_bf16(y0, y1);
                y0 = fmaf(-mask2[i], __uint_as_float(w << 16), y0);
                y1 = fmaf(-mask2[i], __uint_as_float(w & 0xffff0000u), y1);
                pb[nb][i][x] = pack_bf16(y0, y1);
              }
            }
#pragma unroll
          for (int m = 0; m < MT; ++m) {           // 16 dimensions: a lane's two neighbours
            uint32_t a0, a1, a2, a3;
            if constexpr (S::kF16) {
              const uint32_t sel = m & 1 ? 0x7362u : 0x5140u;
              const uint32_t x = __byte_perm(vr[nb][0][m >> 1], vr[nb][1][m >> 1], sel);
              const uint32_t y = __byte_perm(vr[nb][2][m >> 1], vr[nb][3][m >> 1], sel);
              a0 = half2_of_e4m3(x & 0xffffu), a1 = half2_of_e4m3(x >> 16);
              a2 = half2_of_e4m3(y & 0xffffu), a3 = half2_of_e4m3(y >> 16);
            } else {
              a0 = __byte_perm(vr[nb][0][m], vr[nb][1][m], 0x5410);
              a1 = __byte_perm(vr[nb][0][m], vr[nb][1][m], 0x7632);
              a2 = __byte_perm(vr[nb][2][m], vr[nb][3][m], 0x5410);
              a3 = __byte_perm(vr[nb][2][m], vr[nb][3][m], 0x7632);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
              mma<S::kF16>(acc[m][i], a0, a1, a2, a3, pb[nb][i][0], pb[nb][i][1]);
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
