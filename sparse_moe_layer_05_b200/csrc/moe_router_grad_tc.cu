// moe_router_grad_tc.cu -- gradients of the router product s = x W^T + b:
//   dW = ds^T x,  db = sum_t ds,  dx = bf16(ds W + dx_in)
// on the tensor cores (kind::f16, fp32 accumulators).
//
// Precision. x is bf16, or an 8-bit checkpoint row q 2^(s-127) r_t g_i whose
// q 2^(s-127) has four significant bits: both enter an UMMA exactly, the row's
// r_t moves to the other operand (ds r_t, one fp32 rounding) and g_i to the sum.
// The fp32 operands are split into terms hi, mid, lo, each the rounding of what the
// ones before leave:
//   dW  three bf16 terms of ds (24 bits: nothing is lost above 2^-110). The tensor
//       core's accumulator loses up to an fp32 step per addition (a sum over
//       1365 tokens was off by 1.6e-6 of its norm, one over 512 by 6e-7), so
//       every kFlush tokens the sums move to registers and start anew
//   dx  two fp16 terms of ds and of W (22 bits), products mid hi, hi mid and hi hi:
//       off by at most 3 2^-22 of each product. fp16's range is brought over each
//       token's gradients and over the weights of a tile of columns by powers of
//       two, which leave with the output's rounding; below 2^-29 of the largest of
//       those a value keeps fewer bits, 2^-39 of the largest being lost at most.
//       (Two bf16 terms, 16 bits, cost the same and changed the rounded output by
//       1.3e-4 of its norm where the order of an fp32 sum changes it by 3e-5, E = 128;
//       three would double the products.)
// A padded token's terms are zero, and its row of x is zeroed in shared memory
// (it may hold a NaN).
//
// Launches: the terms (with db's partial sums), dW, and dx with the sums of
// dW's parts. No operand is transposed in memory: tokens are K of the first product
// (both operands MN-major) and M of the second (ds K-major, W MN-major).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "moe_internal.h"
#include "moe_mx_convert.cuh"
#include "moe_ptx.cuh"

namespace moe {
namespace {

constexpr int kMD = 128;              // d columns of a dW tile (UMMA M)
constexpr int kMaxStages = 8;
constexpr int kFlush = 512;           // tokens per accumulation in TMEM
constexpr int kSplitTokens = 1 << 16; // tokens per running sum in registers: 128 additions
constexpr int kSmemLimit = 232448 - 1024;
constexpr int kFixed = 1024;          // barriers, TMEM address, flags
constexpr int kTermBlocks = 148 * 4;

// ------------------------------------------------------------- the terms ----

// The terms lie in panels of 64 columns, [panel][token][64]: one TMA box takes
// any number of panels, and a box's rows are one piece of memory.
struct Plan {
  int groups;      // experts in one or two groups of at most 128
  int eg, egp;     // experts of a group, rounded up to 16
  int accs;        // accumulators of a group: hi, mid, lo, or hi and mid + lo
  int lo;          // first column of the lo terms (hi at 0, mid at egp)
  int panels;      // panels of a group's three terms
  int ep;          // E rounded up to 16
  int dx_panel;    // first panel of the terms the dx product reads: mid, then hi
  int all;         // panels in all
  int bt;          // tokens per stage of the dW kernel
  int tiles_d, splits, term_blocks;
};

Plan make_plan(int E, int T, int d, bool scaled, int num_sms) {
  Plan p;
  p.groups = E > 128 ? 2 : 1;
  p.eg = (E + p.groups - 1) / p.groups;
  p.egp = (p.eg + 15) / 16 * 16;
  // two sets of accumulators have to fit TMEM's 512 columns; an UMMA's columns
  // start at a panel
  p.accs = 6 * p.egp <= 512 ? 3 : 2;
  p.lo = p.accs == 3 ? 2 * p.egp : (2 * p.egp + 63) / 64 * 64;
  p.panels = (p.lo + p.egp + 63) / 64;
  p.ep = (E + 15) / 16 * 16;
  p.dx_panel = p.groups * p.panels;
  p.all = p.dx_panel + (2 * p.ep + 63) / 64;
  // at least four stages fit; 8-bit rows need room as codes too
  p.bt = p.panels <= (scaled ? 3 : 5) ? 64 : 32;
  p.tiles_d = (d + kMD - 1) / kMD;
  // one CTA per SM, at least 256 tokens each
  int s = num_sms / (p.tiles_d * p.groups);
  if (s > T / 256) s = T / 256;
  const int least = (T + kSplitTokens - 1) / kSplitTokens;
  if (s < least) s = least;
  p.splits = s < 1 ? 1 : s;
  const int64_t tb = (static_cast<int64_t>(T) + 15) / 16;
  p.term_blocks = tb < kTermBlocks ? (tb < 1 ? 1 : static_cast<int>(tb)) : kTermBlocks;
  return p;
}

__device__ __forceinline__ uint32_t pack2(__nv_bfloat16 a, __nv_bfloat16 b) {
  return __bfloat16_as_ushort(a) | (static_cast<uint32_t>(__bfloat16_as_ushort(b)) << 16);
}

struct Terms {
  __nv_bfloat16 hi, mid, lo;
};
__device__ __forceinline__ Terms split3(float v) {
  Terms t;
  t.hi = __float2bfloat16_rn(v);
  const float r = v - __bfloat162float(t.hi);
  t.mid = __float2bfloat16_rn(r);
  t.lo = __float2bfloat16_rn(r - __bfloat162float(t.mid));
  return t;
}

// Two values' fp16 terms, the first in the lower halves.
__device__ __forceinline__ void split2h(float a, float b, uint32_t& hi, uint32_t& mid) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 m = __floats2half2_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  mid = *reinterpret_cast<const uint32_t*>(&m);
}
// |v|, or 0 for what is no finite number: infinities and NaNs set no scale.
__device__ __forceinline__ float finite_size(float v) {
  const float a = fabsf(v);
  return a < __int_as_float(0x7F800000) ? a : 0.f;
}
__device__ __forceinline__ float exp2_int(int k) { return __int_as_float((k + 127) << 23); }   // -126 .. 127
// k that brings 2^k times the largest value into [2^14, 2^15), fp16's upper end, as
// far as 2^k is a normal fp32 number with a normal inverse: -113 .. 126.
__device__ __forceinline__ int half_scale(float largest) {
  const int k = 141 - static_cast<int>(__float_as_uint(largest) >> 23);
  return k > 126 ? 126 : k;
}

// Tokens of a tile's scale words: a stage's words are one aligned piece.
__host__ __device__ constexpr int64_t padded_tokens(int T) { return (static_cast<int64_t>(T) + 63) / 64 * 64; }

// Rows [t0, t1) of the terms per block; a thread holds one pair of experts, so
// its sum for db stays in registers. Blocks sum consecutive tokens. The `lanes`
// threads of a row join its largest value over shuffles, above 64 experts over
// shared memory too.
constexpr int kTermRows = 4;          // rows a thread loads at a time

__global__ void __launch_bounds__(256) router_terms_kernel(const float* __restrict__ dl,
                                                           const float* __restrict__ rstd,
                                                           const uint8_t* __restrict__ scales,
                                                           const uint8_t* __restrict__ mask, int E,
                                                           int T, int d, const Plan p, int lanes, bool dw,
                                                           uint16_t* __restrict__ terms,
                                                           uint16_t* __restrict__ words,
                                                           int8_t* __restrict__ exps,
                                                           float* __restrict__ db_part, int* status) {
  pdl_wait_and_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  __shared__ float2 sum[256];
  __shared__ uint32_t tops[2][kTermRows][8];   // a warp's largest values, two rounds in turn
  const int64_t t0 = static_cast<int64_t>(T) * blockIdx.x / gridDim.x;
  const int64_t t1 = static_cast<int64_t>(T) * (blockIdx.x + 1) / gridDim.x;
  const int pair = threadIdx.x % lanes, row = threadIdx.x / lanes, rows = 256 / lanes;
  const int e = 2 * pair, warp = threadIdx.x >> 5;
  const bool even = (E & 1) == 0, stores = e < p.ep;
  const size_t panel = static_cast<size_t>(T) * 64;
  // address of column c for token 0
  auto column = [&](int first, int c) { return terms + (first + (c >> 6)) * panel + (c & 63); };
  float sa = 0.f, sb = 0.f;
  const bool together = p.groups == 1;
  // the pair's places among dW's columns (a group may start at an odd expert)
  const int ga = e / p.eg, gb = (e + 1) / p.eg, ca = e - ga * p.eg, cb = e + 1 - gb * p.eg;
  uint16_t* const hi_a = column(together ? 0 : ga * p.panels, together ? e : ca);
  uint16_t* const mid_a = column(together ? 0 : ga * p.panels, p.egp + (together ? e : ca));
  uint16_t* const lo_a = column(together ? 0 : ga * p.panels, p.lo + (together ? e : ca));
  uint16_t* const hi_b = column(gb * p.panels, cb);
  uint16_t* const mid_b = column(gb * p.panels, p.egp + cb);
  uint16_t* const lo_b = column(gb * p.panels, p.lo + cb);
  uint16_t* const mid_x = column(p.dx_panel, e);
  uint16_t* const hi_x = column(p.dx_panel, p.ep + e);
  int round = 0;
  for (int64_t base = t0; base < t1; base += rows * kTermRows, round ^= 1) {   // the block as one
    float a[kTermRows], b[kTermRows], r[kTermRows];
#pragma unroll
    for (int k = 0; k < kTermRows; ++k) {
      const int64_t t = base + row + k * rows;
      a[k] = b[k] = 0.f;
      r[k] = 1.f;
      if (t < t1 && e < E && (mask == nullptr || mask[t] != 0)) {
        if (even) {
          const float2 v = __ldg(reinterpret_cast<const float2*>(dl + t * E + e));
          a[k] = v.x;
          b[k] = v.y;
        } else {
          a[k] = __ldg(dl + t * E + e);
          if (e + 1 < E) b[k] = __ldg(dl + t * E + e + 1);
        }
        if (rstd) r[k] = __ldg(rstd + t);
      }
    }
    if (exps) {
      // sizes compare as their bits do
      uint32_t top[kTermRows];
#pragma unroll
      for (int k = 0; k < kTermRows; ++k)
        top[k] = __float_as_uint(fmaxf(finite_size(a[k]), finite_size(b[k])));
      if (lanes < 32) {
        for (int off = lanes >> 1; off > 0; off >>= 1)
#pragma unroll
          for (int k = 0; k < kTermRows; ++k) top[k] = max(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], off));
      } else {
#pragma unroll
        for (int k = 0; k < kTermRows; ++k) top[k] = __reduce_max_sync(0xFFFFFFFFu, top[k]);
      }
      if (lanes > 32) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
          for (int k = 0; k < kTermRows; ++k) tops[round][k][warp] = top[k];
        __syncthreads();
        const int first = warp & ~((lanes >> 5) - 1);
        for (int w = first; w < first + (lanes >> 5); ++w)
#pragma unroll
          for (int k = 0; k < kTermRows; ++k) top[k] = max(top[k], tops[round][k][w]);
      }
#pragma unroll
      for (int k = 0; k < kTermRows; ++k) {
        const int64_t t = base + row + k * rows;
        if (t >= t1 || !stores) continue;
        const int ex = half_scale(__uint_as_float(top[k]));
        const float up = exp2_int(ex);
        uint32_t hi, mid;
        split2h(a[k] * up, b[k] * up, hi, mid);
        const size_t at = static_cast<size_t>(t) * 64;
        *reinterpret_cast<uint32_t*>(mid_x + at) = mid;
        *reinterpret_cast<uint32_t*>(hi_x + at) = hi;
        if (pair == 0) exps[t] = static_cast<int8_t>(ex);
      }
    }
#pragma unroll
    for (int k = 0; k < kTermRows; ++k) {
      const int64_t t = base + row + k * rows;
      if (t >= t1) continue;
      sa += a[k];
      sb += b[k];
      if (!dw || !stores) continue;
      const size_t at = static_cast<size_t>(t) * 64;
      // r is 1 where the rows are bf16
      const Terms u = split3(a[k] * r[k]), v = split3(b[k] * r[k]);
      if (together) {
        *reinterpret_cast<uint32_t*>(hi_a + at) = pack2(u.hi, v.hi);
        *reinterpret_cast<uint32_t*>(mid_a + at) = pack2(u.mid, v.mid);
        *reinterpret_cast<uint32_t*>(lo_a + at) = pack2(u.lo, v.lo);
      } else {
        if (e < E) {
          hi_a[at] = __bfloat16_as_ushort(u.hi);
          mid_a[at] = __bfloat16_as_ushort(u.mid);
          lo_a[at] = __bfloat16_as_ushort(u.lo);
        }
        if (e + 1 < E) {
          hi_b[at] = __bfloat16_as_ushort(v.hi);
          mid_b[at] = __bfloat16_as_ushort(v.mid);
          lo_b[at] = __bfloat16_as_ushort(v.lo);
        }
      }
    }
  }
  if (words) {
    // the 8-bit rows' scales as the dW kernel takes them: [tile of 128 columns]
    // [token][4] 16-bit words, bit 8 set for rows that count as zeros: a padded token's,
    // past the last one, and where the inverse root is 0 (the codes of an infinity are
    // bf16's infinity, which the term's zero does not undo)
    const int G = d / 32;
    const int64_t end = blockIdx.x + 1 == gridDim.x ? padded_tokens(T) : t1;
    uint2* const to = reinterpret_cast<uint2*>(words) + t0;
    const int64_t pitch = padded_tokens(T);
    // neighbouring threads: neighbouring tiles of a token (the scales' order)
    for (int64_t b0 = t0; b0 < end; b0 += 1024) {
      const int items = static_cast<int>(end - b0 < 1024 ? end - b0 : 1024) * p.tiles_d;
#pragma unroll 4
      for (int v = threadIdx.x; v < items; v += 256) {
        const int i = v / p.tiles_d, tile = v - i * p.tiles_d;
        const int64_t t = b0 + i;
        const bool row = t < T;
        const uint8_t* const from = scales + t * G + tile * 4;
        const uint32_t dead = !row || __ldg(rstd + t) == 0.f || (mask && __ldg(mask + t) == 0) ? 0x100u : 0u;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = dead | (row && tile * 4 + k < G ? __ldg(from + k) : 127u);
        to[tile * pitch + (t - t0)] = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
      }
    }
  }
  sum[threadIdx.x] = make_float2(sa, sb);
  __syncthreads();
  if (row == 0 && e < E) {
    for (int r = 1; r < rows; ++r) {
      const float2 v = sum[r * lanes + pair];
      sa += v.x;
      sb += v.y;
    }
    db_part[static_cast<size_t>(blockIdx.x) * E + e] = sa;
    if (e + 1 < E) db_part[static_cast<size_t>(blockIdx.x) * E + e + 1] = sb;
  }
}

// ---------------------------------------------------------- descriptors ----

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzled
// layout: rows of K hold 64 MN elements (128 bytes), 8 rows 1024 bytes apart,
// the next 64 MN elements `mn_stride` bytes on. 16 of K are 2048 bytes.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t mn_stride) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(mn_stride >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
constexpr uint32_t kAMnMajor = 1u << 15, kBMnMajor = 1u << 16;

// True in one lane of a converged warp, the same lane each time. Instructions
// that take their operands from uniform registers (UMMAs, TMA) are issued under
// it from warp-uniform loops: from a loop that one lane runs alone, each took
// over 100 cycles.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "elect.sync _|P, 0xFFFFFFFF;\n\t"
      "selp.b32 %0, 1, 0, P;\n\t}"
      : "=r"(p));
  return p != 0;
}
// mbar_wait by a whole warp, the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, int* status) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort, status));
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) return;
}

// A descriptor's start address may be advanced by adding bytes / 16 (the sums
// stay within its 14 bits: shared memory ends below 2^18). One thread issues
// all of a CTA's UMMAs, and rebuilding both descriptors for each took it longer
// (about 200 cycles) than the tensor core needs for one.
__device__ __forceinline__ uint64_t advance(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }

__device__ __forceinline__ void tma_load_panels(uint32_t dst, const CUtensorMap* m, int token, int panel,
                                                uint32_t bar) {
  tma_load_3d(dst, m, 0, token, panel, bar);
}

// 16 E4M3 codes times the scale 2^(s - 127) as bf16, exactly. A code placed in
// bf16 bits as sign | exponent and mantissa << 4 is 2^-120 of its value, subnormal
// codes included, so one bf16 product with 2^(s - 7) does it (two where that
// exceeds bf16's range). NaN codes (which only NaN rows have) become NaN.
__device__ __forceinline__ void e4m3x16_to_bf16(uint4 q, uint32_t s, uint32_t (&o)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  const uint32_t e = s > 134u ? 254u : s + 120u;   // biased exponent of the first factor
  const uint32_t m = (e << 7) | (e << 23);
  uint32_t nan = s == 255u ? 0x80u : 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = __byte_perm(w[k], 0, 0x1404), b = __byte_perm(w[k], 0, 0x3424);
    o[2 * k] = bf16x2_mul((a & 0x80008000u) | ((a >> 4) & 0x07F007F0u), m);
    o[2 * k + 1] = bf16x2_mul((b & 0x80008000u) | ((b >> 4) & 0x07F007F0u), m);
    nan |= ((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  }
  if (s > 134u || nan) {
    const uint32_t r = s > 134u ? s - 134u + 127u : 127u, m2 = (r << 7) | (r << 23);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[2 * k] = bf16x2_mul(o[2 * k], m2);
      o[2 * k + 1] = bf16x2_mul(o[2 * k + 1], m2);
      if ((w[k] & 0x7Fu) == 0x7Fu || s == 255u) o[2 * k] |= 0x7FFFu;
      if ((w[k] & 0x7F00u) == 0x7F00u || s == 255u) o[2 * k] |= 0x7FFF0000u;
      if ((w[k] & 0x7F0000u) == 0x7F0000u || s == 255u) o[2 * k + 1] |= 0x7FFFu;
      if ((w[k] & 0x7F000000u) == 0x7F000000u || s == 255u) o[2 * k + 1] |= 0x7FFF0000u;
    }
  }
}

// ----------------------------------------------------------------- dW ----

struct DwArgs {
  const uint8_t* mask;
  const uint16_t* words;   // the 8-bit rows' scales
  int E, T, d;
  Plan p;
  int stages, stage_bytes, tmem_cols;
  float* part;     // [splits][E][d]
  int* status;
};

// Warp 0 loads the stages (TMA), warps 1 and 2 issue the UMMAs: a commit and
// the wait for the next stage take an issuer some 300 cycles, so the two take
// stages in turn, each with its own accumulators. Warp 3 zeroes the rows of
// padded tokens (bf16 rows), warps 4..11 move the accumulators to registers
// (warp w the lanes of quarter w % 4, chunks of 16 experts in turn with warp
// w +- 4). 8-bit rows arrive as codes and scale words and are converted into the
// stage's bf16 rows by warps 12..15 and 16..19, a stage each in turn. (Rows held in
// registers ahead of their turn did not work: the loads of the stage after the
// next were waited for with those of the next, 780 cycles a stage of 32 tokens.)
constexpr int kSumWarps = 8, kConvWarps = 8;
constexpr int kSumChunks = 4;         // chunks of 16 experts a warp sums
constexpr int kConvGroup = 4;         // warps that convert a stage

template <bool Q8, int BT>
__global__ void __launch_bounds__(128 + 32 * (kSumWarps + (Q8 ? kConvWarps : 0)), 1)
    router_dw_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmD,
                     const DwArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = threadIdx.x & 31;
  const int S = a.stages;
  constexpr uint32_t xhalf = BT * 128;   // 64 columns of a stage's rows
  uint8_t* fixed = smem + S * a.stage_bytes;
  const uint32_t bar0 = smem_u32(fixed);
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_ready = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto bar_empty = [&](int s) { return bar0 + 8u * (2 * kMaxStages + s); };
  auto bar_acc = [&](int b) { return bar0 + 8u * (3 * kMaxStages + b); };
  auto bar_free = [&](int b) { return bar0 + 8u * (3 * kMaxStages + 2 + b); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(fixed + 8 * (3 * kMaxStages + 4));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);

  const int tile = blockIdx.x % a.p.tiles_d;
  const int group = blockIdx.x / a.p.tiles_d % a.p.groups;
  const int split = blockIdx.x / (a.p.tiles_d * a.p.groups);
  const int i0 = tile * kMD;
  const int nblk = (a.T + BT - 1) / BT;
  const int b0 = static_cast<int>(static_cast<int64_t>(nblk) * split / a.p.splits);
  const int b1 = static_cast<int>(static_cast<int64_t>(nblk) * (split + 1) / a.p.splits);
  constexpr int per = kFlush / BT;
  const int n = b1 - b0;
  // accumulations of the even and the odd stages: they end in turn
  const int flushes = ((n + 1) / 2 + per - 1) / per + (n / 2 + per - 1) / per;
  const bool fix = !Q8 && a.mask != nullptr;
  const bool second = Q8 || fix;        // a stage is complete with bar_ready too

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    misc[2] = misc[3] = misc[4] = 0;
    for (int s = 0; s < S; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_ready(s), Q8 ? kConvGroup : 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_acc(b), 1);
      mbar_init(bar_free(b), kSumWarps);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmD);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(misc), static_cast<uint32_t>(a.tmem_cols));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait_and_trigger();               // no global memory was touched before
  const uint32_t tmem = misc[0];

  if (warp == 0) {
    int s = 0, ph = 0, issued = 0;
    for (int i = 0; i < n; ++i) {
      if (!warp_wait(bar_empty(s), ph ^ 1, abort_flag, a.status)) break;
      const uint32_t st = sbase + s * a.stage_bytes, bar = bar_full(s);
      const int t = (b0 + i) * BT;
      if (elect_one()) {
        const uint32_t terms = static_cast<uint32_t>(a.p.panels) * xhalf;
        mbar_expect_tx(bar, terms + (Q8 ? BT * 128 + BT * 8 : 2 * xhalf));
        if (Q8) {
          tma_load_2d(st + 2 * xhalf + terms, &tmX, i0, t, bar);
          bulk_load(st + 2 * xhalf + terms + BT * 128,
                    a.words + (tile * padded_tokens(a.T) + t) * 4, BT * 8, bar);
        } else {
          tma_load_2d(st, &tmX, i0, t, bar);
          tma_load_2d(st + xhalf, &tmX, i0 + 64, t, bar);
        }
        tma_load_panels(st + 2 * xhalf, &tmD, t, group * a.p.panels, bar);
      }
      __syncwarp();
      issued = i + 1;
      if (++s == S) { s = 0; ph ^= 1; }
    }
    if (lane == 0) misc[2] = static_cast<uint32_t>(issued);
  } else if (warp < 3) {
    const uint32_t egp = static_cast<uint32_t>(a.p.egp), set = egp * a.p.accs;
    const uint32_t major = kAMnMajor | kBMnMajor;
    const uint32_t idesc = idesc_bf16_f32(kMD, static_cast<int>(set)) | major;
    const uint32_t idesc_lo = idesc_bf16_f32(kMD, static_cast<int>(egp)) | major;
    const uint64_t a0 = sdesc_mn_sw128(sbase, xhalf), d0 = advance(a0, 2 * xhalf);
    const uint32_t lo_bytes = static_cast<uint32_t>(a.p.lo) / 64 * xhalf;
    const bool two = a.p.accs == 2;
    // issuer w: stages w, w + 2, ... into accumulator set w
    const int w = warp - 1;
    const uint32_t acc = tmem + w * set;
    int consumed = 0, f = 0, at = 0;
    for (int i = w; i < n; i += 2) {
      const int s = i % S, ph = i / S & 1;
      if (at == 0 && !warp_wait(bar_free(w), (f & 1) ^ 1, abort_flag, a.status)) break;
      if (!warp_wait(bar_full(s), ph, abort_flag, a.status)) break;
      if (second && !warp_wait(bar_ready(s), ph, abort_flag, a.status)) break;
      consumed = i + 1;
      tc_fence_after();
      const uint64_t ad = advance(a0, static_cast<uint32_t>(s * a.stage_bytes));
      const uint64_t bd = advance(d0, static_cast<uint32_t>(s * a.stage_bytes));
      const bool last = ++at == per || i + 2 >= n;
      if (elect_one()) {
        const uint32_t on = at != 1;
#pragma unroll
        for (int u = 0; u < BT / 16; ++u) {
          umma_bf16(acc, advance(ad, u * 2048), advance(bd, u * 2048), idesc, on | (u != 0));
          if (two)
            umma_bf16(acc + egp, advance(ad, u * 2048), advance(bd, lo_bytes + u * 2048), idesc_lo, 1u);
        }
        umma_commit(bar_empty(s));
        if (last) umma_commit(bar_acc(w));
      }
      __syncwarp();
      if (last) {
        ++f;
        at = 0;
      }
    }
    if (lane == 0) misc[3 + w] = static_cast<uint32_t>(consumed);
  } else if (warp == 3) {
    if (fix) {
      int s = 0, ph = 0;
      uint32_t next[BT / 32];               // the stage's mask bytes, loaded a stage ahead
      auto load = [&](int i) {
#pragma unroll
        for (int h = 0; h < BT / 32; ++h) {   // rows past T are zero already
          const int64_t t = static_cast<int64_t>(b0 + i) * BT + 32 * h + lane;
          next[h] = i < n && t < a.T ? __ldg(a.mask + t) : 1u;
        }
      };
      load(0);
      for (int i = 0; i < n; ++i) {
        uint32_t live[BT / 32];
#pragma unroll
        for (int h = 0; h < BT / 32; ++h) live[h] = next[h];
        load(i + 1);
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar_full(s), ph, abort_flag, a.status))) break;
        // a row per lane; eight lanes a full 128 bytes at a time (one row after
        // another by the whole warp held the UMMAs up: T = 16384, E = 32, d = 2880,
        // 67 us against 61)
#pragma unroll
        for (int h = 0; h < BT / 32; ++h)
          if (live[h] == 0) {
            uint8_t* row = smem + s * a.stage_bytes + (32 * h + lane) * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              *reinterpret_cast<uint4*>(row + ((c ^ (lane & 7)) << 4)) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(row + xhalf + ((c ^ (lane & 7)) << 4)) = make_uint4(0, 0, 0, 0);
            }
          }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_ready(s));
        if (++s == S) { s = 0; ph ^= 1; }
      }
    }
  } else if (warp < 4 + kSumWarps) {
    // lane = d column, TMEM columns = experts; acc set f & 1 holds flush f
    const int quad = warp & 3, half = (warp - 4) >> 2, i = i0 + quad * 32 + lane;
    const int egp = a.p.egp, chunks = egp / 16;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    float sum[kSumChunks][16];
#pragma unroll
    for (int c = 0; c < kSumChunks; ++c)
#pragma unroll
      for (int j = 0; j < 16; ++j) sum[c][j] = 0.f;
    bool ok = true;
    for (int f = 0; f < flushes && ok; ++f) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_acc(f & 1), (f >> 1) & 1, abort_flag, a.status));
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + lanes + (f & 1) * egp * a.p.accs;
#pragma unroll
      for (int c = 0; c < kSumChunks; ++c) {
        const int ch = 2 * c + half;
        if (ch >= chunks) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t u[8], v[8], w[8];
          const uint32_t at = acc + ch * 16 + h * 8;
          tmem_ld8x2_sync(at, at + egp, u, v);
          if (a.p.accs == 3) {
            tmem_ld8_sync(at + 2 * egp, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(w[j]));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            sum[c][8 * h + j] += __uint_as_float(u[j]) + __uint_as_float(v[j]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_free(f & 1));
    }
    const int e0 = group * a.p.eg, ne = a.E - e0 < a.p.eg ? a.E - e0 : a.p.eg;
    float* out = a.part + (static_cast<size_t>(split) * a.E + e0) * a.d + i;
    if (ok && i < a.d)
#pragma unroll
      for (int c = 0; c < kSumChunks; ++c)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int e = (2 * c + half) * 16 + j;
          if (e < ne) out[static_cast<size_t>(e) * a.d] = sum[c][j];
        }
  } else {
    // 8-bit rows: 16 columns of tokens tr, tr + 16, ... of every second stage
    const int cw = warp - 4 - kSumWarps;
    const int ct = (cw % kConvGroup) * 32 + lane, tr = ct >> 3, c = ct & 7;
    for (int i = cw / kConvGroup; i < n; i += 2) {
      const int s = i % S;
      if (!warp_wait(bar_full(s), i / S & 1, abort_flag, a.status)) break;
      uint8_t* const st = smem + s * a.stage_bytes;
      const uint8_t* const codes = st + (2 + a.p.panels) * xhalf;
      const uint16_t* const words = reinterpret_cast<const uint16_t*>(codes + BT * 128);
      uint8_t* const xa = st + (c >> 2) * xhalf;
      const int ch = (c & 3) * 2;
#pragma unroll
      for (int u = 0; u < BT / 16; ++u) {
        const int row = 16 * u + tr;
        uint4 q = *reinterpret_cast<const uint4*>(codes + row * 128 + ((c ^ (row & 7)) << 4));
        uint32_t w = words[row * 4 + (c >> 1)];
        if (w > 255u) {      // a row that counts as zeros
          q = make_uint4(0, 0, 0, 0);
          w = 127u;
        }
        uint32_t o[8];
        e4m3x16_to_bf16(q, w, o);
        *reinterpret_cast<uint4*>(xa + row * 128 + ((ch ^ (row & 7)) << 4)) =
            make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(xa + row * 128 + (((ch + 1) ^ (row & 7)) << 4)) =
            make_uint4(o[4], o[5], o[6], o[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ready(s));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // a wait gave up: the loads in flight land and the issued UMMAs finish before
    // the memory is given back (each wait here is bounded too)
    const uint32_t issued = misc[2], done = misc[3] > misc[4] ? misc[3] : misc[4];
    for (uint32_t i = issued > static_cast<uint32_t>(S) ? issued - S : 0; i < issued; ++i)
      drain_wait(bar_full(static_cast<int>(i % S)), (i / S) & 1u);
    for (uint32_t i = done > static_cast<uint32_t>(S) ? done - S : 0; i < done; ++i)
      drain_wait(bar_empty(static_cast<int>(i % S)), (i / S) & 1u);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, static_cast<uint32_t>(a.tmem_cols));
  }
}

// dW = sum of the parts in order (times g), db = sum of the term blocks' sums.
struct SumArgs {
  const float* part;
  const float* g;        // [d] or null
  const float* db_part;
  int splits, term_blocks, E, d, blocks;
  bool accumulate;
  float* dW;             // null: not wanted
  float* db;
};

// The share of block blk's `threads` threads (whole warps), thread tid.
__device__ __forceinline__ void router_sums(const SumArgs& a, int blk, int tid, int threads) {
  const size_t n4 = a.dW ? static_cast<size_t>(a.E) * a.d / 4 : 0;
  const size_t stride = static_cast<size_t>(a.blocks) * threads;
  for (size_t v = static_cast<size_t>(blk) * threads + tid; v < n4; v += stride) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 6
    for (int k = 0; k < a.splits; ++k) {
      const float4 b = __ldg(reinterpret_cast<const float4*>(a.part) + k * n4 + v);
      s.x += b.x;
      s.y += b.y;
      s.z += b.z;
      s.w += b.w;
    }
    if (a.g) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(a.g) + v % (a.d / 4));
      s.x *= w.x;
      s.y *= w.y;
      s.z *= w.z;
      s.w *= w.w;
    }
    float4* o = reinterpret_cast<float4*>(a.dW) + v;
    if (a.accumulate) {
      const float4 b = *o;
      s.x += b.x;
      s.y += b.y;
      s.z += b.z;
      s.w += b.w;
    }
    *o = s;
  }
  if (!a.db) return;
  // db: one warp per expert
  const int lane = tid & 31, warps = threads >> 5;
  for (int e = blk * warps + (tid >> 5); e < a.E; e += a.blocks * warps) {
    float s = 0.f;
    for (int b = lane; b < a.term_blocks; b += 32)
      s += __ldg(a.db_part + static_cast<size_t>(b) * a.E + e);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    if (lane == 0) a.db[e] = a.accumulate ? a.db[e] + s : s;
  }
}

__global__ void __launch_bounds__(256) router_sums_kernel(const SumArgs a) {
  pdl_wait_and_trigger();
  router_sums(a, blockIdx.x, threadIdx.x, blockDim.x);
}

// ----------------------------------------------------------------- dx ----

constexpr int kTM = 128;              // tokens per tile (UMMA M)
constexpr int kBoxBytes = kTM * 128;  // 64 term columns of a token tile
constexpr int kMaxRing = 8, kMaxStaging = 8;

struct DxArgs {
  const float* W;
  const uint8_t* mask;
  const int8_t* exps;                 // [T]: a token's terms are 2^exps[t] ds
  int E, T, d;
  Plan p;
  int n_tile;                         // columns per tile
  int full, splits, last_splits;      // whole tiles along d; CTAs per tile, and of the part tile
  int boxes, ring, staging;
  int off_ring, off_staging, off_fixed;
  int tmem_cols;
  bool has_in;
  SumArgs sums;
  int* status;
};

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// One CTA keeps the two terms of W's tile columns in shared memory and takes
// every splits-th token tile (128 tokens). Warp 0 loads ds terms, warp 1 issues
// the UMMAs, the tiles into two accumulators in turn (two issuers, one to each
// accumulator, ran in step and both waited for their outputs at the same time:
// 2850 cycles a tile where the UMMAs take 1540). A tile leaves in units of 64
// columns: warps 4..7 and 8..11 (one per lane quarter each) take the units in
// turn, add dx_in and round; warp 2 moves them: a staging buffer receives dx_in by
// TMA, is updated in place and stored by TMA (each thread storing its token's
// columns itself, 32 bytes at a time, took 25 us where this takes 20, T = 8192,
// E = 32, d = 2880). A store reads its buffer for 1200 cycles under load, so two
// are in flight. Wide tiles, because ds's terms are read once per tile column:
// with 128 columns the 128-expert layer's reads (200 MB from L2 at T = 16384) and
// not the tensor core set the time. Warps 12..15 sum dW's parts meanwhile.
constexpr int kOutWarps = 8;
constexpr int kSumsWarps = 4;
constexpr int kUnitBytes = kTM * 128;
constexpr int kDxThreads = 128 + 32 * (kOutWarps + kSumsWarps);
// eight weights at a time: a thread's share of a tile, at most 384 experts times
// 64-column units (launch_router_backward_tc's choice of n_tile)
constexpr int kDxWeights = 384;
constexpr int kDxChunks = kDxWeights * 8 / kDxThreads;
constexpr int kDxTops = 8;            // misc words of the warps' largest weights

template <bool MASKED>
__global__ void __launch_bounds__(kDxThreads, 1)
    router_dx_kernel(const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmIn,
                     const __grid_constant__ CUtensorMap tmOut, const DxArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = threadIdx.x & 31;
  uint8_t* fixed = smem + a.off_fixed;
  const uint32_t bar0 = smem_u32(fixed);
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (kMaxRing + s); };
  auto bar_acc = [&](int b) { return bar0 + 8u * (2 * kMaxRing + b); };
  auto bar_free = [&](int b) { return bar0 + 8u * (2 * kMaxRing + 2 + b); };
  auto bar_in = [&](int s) { return bar0 + 8u * (2 * kMaxRing + 4 + s); };
  auto bar_out = [&](int s) { return bar0 + 8u * (2 * kMaxRing + 4 + kMaxStaging + s); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(fixed + 8 * (2 * kMaxRing + 4 + 2 * kMaxStaging));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);

  // CTAs of the whole tiles first, then those of the part tile
  const bool whole = static_cast<int>(blockIdx.x) < a.full * a.splits;
  const int nt = whole ? static_cast<int>(blockIdx.x) % a.full : a.full;
  const int split = whole ? static_cast<int>(blockIdx.x) / a.full
                          : static_cast<int>(blockIdx.x) - a.full * a.splits;
  const int splits = whole ? a.splits : a.last_splits;
  const int i0 = nt * a.n_tile;
  const int units = whole ? a.n_tile / 64 : (a.d - i0 + 63) / 64;   // of a tile
  const int cols = units * 64;
  const int ttiles = (a.T + kTM - 1) / kTM;
  const int n = split < ttiles ? (ttiles - 1 - split) / splits + 1 : 0;
  auto tile_row = [&](int j) { return (split + j * splits) * kTM; };
  const uint32_t wblock = static_cast<uint32_t>(a.p.ep) * 256;   // 2 ep rows of 128 bytes

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    misc[2] = misc[3] = misc[4] = 0;
    for (int s = 0; s < a.ring; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_acc(b), 1);
      mbar_init(bar_free(b), units > 1 ? kOutWarps : kOutWarps / 2);
    }
    for (int s = 0; s < a.staging; ++s) {
      mbar_init(bar_in(s), 1);
      mbar_init(bar_out(s), kOutWarps / 2);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmD);
    tma_prefetch_desc(&tmOut);
    if (a.has_in) tma_prefetch_desc(&tmIn);
  }
  if (warp == 3) {
    tmem_alloc(smem_u32(misc), static_cast<uint32_t>(a.tmem_cols));
    tmem_relinquish();
  }
  // W's columns i0 .. i0 + cols - 1 times 2^kw as hi rows 0 .. ep - 1, mid rows
  // ep .. 2 ep - 1
  const int chunks = cols / 8;
  float w[kDxChunks][8], top = 0.f;
#pragma unroll
  for (int n = 0; n < kDxChunks; ++n) {
    const int v = threadIdx.x + n * kDxThreads;
    const int e = v / chunks, i = i0 + v % chunks * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[n][j] = 0.f;
    if (e < a.E && i < a.d) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(a.W + static_cast<size_t>(e) * a.d + i));
      const float4 y = __ldg(reinterpret_cast<const float4*>(a.W + static_cast<size_t>(e) * a.d + i) + 1);
      w[n][0] = x.x; w[n][1] = x.y; w[n][2] = x.z; w[n][3] = x.w;
      w[n][4] = y.x; w[n][5] = y.y; w[n][6] = y.z; w[n][7] = y.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_size(w[n][j]));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
  if (lane == 0) misc[kDxTops + warp] = __float_as_uint(top);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kDxThreads / 32; ++k) top = fmaxf(top, __uint_as_float(misc[kDxTops + k]));
  const int kw = half_scale(top);
  const float up = exp2_int(kw);
#pragma unroll
  for (int n = 0; n < kDxChunks; ++n) {
    const int v = threadIdx.x + n * kDxThreads;
    const int e = v / chunks, ch = v % chunks;
    if (e >= a.p.ep) continue;
    uint32_t hi[4], mid[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) split2h(w[n][2 * j] * up, w[n][2 * j + 1] * up, hi[j], mid[j]);
    uint8_t* blk = smem + (ch >> 3) * wblock;
    const uint32_t at = ((ch & 7) ^ (e & 7)) << 4;     // ep is a multiple of 8
    *reinterpret_cast<uint4*>(blk + e * 128 + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(blk + (a.p.ep + e) * 128 + at) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // W alone was read so far: it is no kernel's of this pass, and whatever wrote it
  // ended before the pass's first kernel began. All else waits for the launch before,
  // behind which dW's parts and the terms are complete. (Tiles begun without the wait,
  // on the grounds that the dW kernel's blocks had waited for the terms, were 4 us
  // earlier at T = 192, E = 248 and no earlier from T = 8192 on; but memory written by
  // earlier grids is visible only to a grid that waits itself.)
  pdl_wait_and_trigger();
  const uint32_t tmem = misc[0];

  if (warp == 0) {
    int s = 0, ph = 0, issued = 0;
    bool ok = true;
    for (int j = 0; j < n && ok; ++j)
      for (int x = 0; x < a.boxes; ++x) {
        if (!(ok = warp_wait(bar_empty(s), ph ^ 1, abort_flag, a.status))) break;
        if (elect_one()) {
          mbar_expect_tx(bar_full(s), kBoxBytes);
          tma_load_panels(sbase + a.off_ring + s * kBoxBytes, &tmD, tile_row(j), a.p.dx_panel + x,
                          bar_full(s));
        }
        __syncwarp();
        ++issued;
        if (++s == a.ring) { s = 0; ph ^= 1; }
      }
    if (lane == 0) misc[2] = static_cast<uint32_t>(issued);
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f16_f32(kTM, cols) | kBMnMajor;
    const int steps = a.p.ep / 16;                     // K steps of a term
    const uint64_t a0 = sdesc_k_sw128(sbase + a.off_ring), w0 = sdesc_mn_sw128(sbase, wblock);
    int s = 0, ph = 0, consumed = 0;
    bool ok = true;
    for (int j = 0; j < n && ok; ++j) {
      const int b = j & 1;
      if (!(ok = warp_wait(bar_free(b), ((j >> 1) & 1) ^ 1, abort_flag, a.status))) break;
      tc_fence_after();
      const uint32_t acc = tmem + b * a.n_tile;
      int step = 0;      // ds's mid steps, then its hi steps: small products come first
      for (int x = 0; x < a.boxes; ++x) {
        if (!(ok = warp_wait(bar_full(s), ph, abort_flag, a.status))) break;
        ++consumed;
        tc_fence_after();
        const uint64_t ad = advance(a0, static_cast<uint32_t>(s * kBoxBytes));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const int st = step + kk;
            if (st >= 2 * steps) break;
            const bool mid = st < steps;
            const uint64_t wd = advance(w0, static_cast<uint32_t>(mid ? st : st - steps) * 2048);
            if (!mid) umma_f16(acc, advance(ad, kk * 32), advance(wd, wblock / 2), idesc, 1u);
            umma_f16(acc, advance(ad, kk * 32), wd, idesc, st != 0);
          }
          umma_commit(bar_empty(s));
          if (x + 1 == a.boxes) umma_commit(bar_acc(b));
        }
        __syncwarp();
        step += 4;
        if (++s == a.ring) { s = 0; ph ^= 1; }
      }
    }
    if (lane == 0) misc[3] = static_cast<uint32_t>(consumed);
  } else if (warp == 2) {
    const int total = n * units;
    auto hand_out = [&](int q) {                       // the staging buffer of unit q
      const int s = q % a.staging;
      if (!a.has_in) {
        mbar_arrive(bar_in(s));
        return;
      }
      mbar_expect_tx(bar_in(s), kUnitBytes);
      tma_load_2d(sbase + a.off_staging + s * kUnitBytes, &tmIn, i0 + q % units * 64,
                  tile_row(q / units), bar_in(s));
    };
    int out = total < a.staging ? total : a.staging;   // units whose buffer was handed out
    if (elect_one())
      for (int q = 0; q < out; ++q) hand_out(q);
    __syncwarp();
    for (int q = 0; q < total; ++q) {
      const int s = q % a.staging;
      if (!warp_wait(bar_out(s), q / a.staging & 1, abort_flag, a.status)) break;
      const bool more = q > 0 && out < total;
      if (elect_one()) {
        tma_store_2d(&tmOut, sbase + a.off_staging + s * kUnitBytes, i0 + q % units * 64,
                     tile_row(q / units));
        bulk_commit();
        bulk_wait_read<1>();                           // unit q - 1 has left its buffer
        if (more) hand_out(out);
      }
      __syncwarp();
      out += more;
    }
    if (elect_one()) bulk_wait_read<0>();              // the lane that issued the stores
    __syncwarp();
    if (lane == 0) misc[4] = static_cast<uint32_t>(out);
  } else if (warp >= 4 && warp < 4 + kOutWarps) {
    const int quad = warp & 3, half = (warp - 4) >> 2, r = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    // the exponent and the mask's byte of the lane's token in tile j, loaded a tile ahead
    uint32_t next_live = 1;
    int next_k = 0;
    auto load_token = [&](int j) {
      const int64_t t = static_cast<int64_t>(tile_row(j)) + r;
      if (j >= n || t >= a.T) return;
      next_k = __ldg(a.exps + t);
      if (MASKED) next_live = __ldg(a.mask + t);
    };
    // the group's tiles: all, or with one unit a tile every second
    const int first = units > 1 ? 0 : half, stride = units > 1 ? 1 : 2;
    load_token(first);
    // this group's units, counted over all tiles: half, half + 2, ...
    int waited = -1, have = -1;
    bool live = true;
    float f0 = 1.f, f1 = 1.f;
    for (int q = half; q < n * units; q += 2) {
      const int j = q / units, u = q % units, b = j & 1, s = q % a.staging;
      if (j != have) {
        have = j;
        live = next_live != 0;
        // 2^-(the terms' exponents) as two factors: one alone may pass fp32's range
        const int k = -(next_k + kw);
        f0 = exp2_int(k >> 1);
        f1 = exp2_int(k - (k >> 1));
        load_token(j + stride);
      }
      for (; waited < j; ++waited)
        if ((units > 1 || ((waited + 1) & 1) == half) &&
            !warp_wait(bar_acc((waited + 1) & 1), (waited + 1) >> 1 & 1, abort_flag, a.status))
          break;
      if (waited < j) break;
      if (!warp_wait(bar_in(s), q / a.staging & 1, abort_flag, a.status)) break;
      tc_fence_after();
      uint8_t* row = smem + a.off_staging + s * kUnitBytes + r * 128;
      const uint32_t acc = tmem + b * a.n_tile + lanes + u * 64;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t v[16];
        tmem_ld16_sync(acc + 16 * c, v);
        if (c == 3) {
          tc_fence_before();
          __syncwarp();
          if (u + 2 >= units && lane == 0) mbar_arrive(bar_free(b));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4* o = reinterpret_cast<uint4*>(row + (((2 * c + h) ^ (r & 7)) << 4));
          uint32_t w[4] = {0, 0, 0, 0};
          if (a.has_in) {
            const uint4 x = *o;
            w[0] = x.x;
            w[1] = x.y;
            w[2] = x.z;
            w[3] = x.w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 y = make_float2(__uint_as_float(v[8 * h + 2 * k]), __uint_as_float(v[8 * h + 2 * k + 1]));
            const float2 sum = fma2(mul2(y, both(f0)), both(f1), bf16_pair(w[k]));
            const __nv_bfloat162 z = __floats2bfloat162_rn(sum.x, sum.y);
            w[k] = *reinterpret_cast<const uint32_t*>(&z);
          }
          // a padded token's row stays dx_in's (its sum may be zero times an infinity)
          if (!MASKED || live)
            *o = make_uint4(w[0], w[1], w[2], w[3]);
          else if (!a.has_in)
            *o = make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_out(s));
    }
  } else if (warp >= 4 && a.sums.blocks) {
    router_sums(a.sums, blockIdx.x, static_cast<int>(threadIdx.x) - 128 - 32 * kOutWarps,
                32 * kSumsWarps);
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // a wait gave up: loads in flight and issued UMMAs finish first (bounded)
    const int R = a.ring, issued = static_cast<int>(misc[2]), done = static_cast<int>(misc[3]);
    for (int k = issued > R ? issued - R : 0; k < issued; ++k) drain_wait(bar_full(k % R), k / R & 1);
    for (int k = done > R ? done - R : 0; k < done; ++k) drain_wait(bar_empty(k % R), k / R & 1);
    const int G = a.staging, out = static_cast<int>(misc[4]);
    for (int q = out > G ? out - G : 0; q < out; ++q) drain_wait(bar_in(q % G), q / G & 1);
  }
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, static_cast<uint32_t>(a.tmem_cols));
  }
}

int tmem_columns(int need) {
  int c = 32;
  while (c < need) c *= 2;
  return c;
}

struct Scratch {
  uint16_t* terms;
  uint16_t* words;
  int8_t* exps;
  float* db_part;
  float* part;
  size_t bytes;
};

Scratch scratch_of(void* base, const Plan& p, int E, int T, int d) {
  Scratch s;
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t o = off;
    off = (off + n + 255) & ~static_cast<size_t>(255);
    return o;
  };
  const size_t terms = take(static_cast<size_t>(T) * p.all * 128);
  const size_t words = take(static_cast<size_t>(padded_tokens(T)) * p.tiles_d * 8);
  const size_t exps = take(static_cast<size_t>(T));
  const size_t db = take(static_cast<size_t>(p.term_blocks) * E * 4);
  const size_t part = take(static_cast<size_t>(p.splits) * E * d * 4);
  s.terms = reinterpret_cast<uint16_t*>(b + terms);
  s.words = reinterpret_cast<uint16_t*>(b + words);
  s.exps = reinterpret_cast<int8_t*>(b + exps);
  s.db_part = reinterpret_cast<float*>(b + db);
  s.part = reinterpret_cast<float*>(b + part);
  s.bytes = off;
  return s;
}

constexpr int kPlanSms = 148;         // the workspace's size goes by the full part

}  // namespace

size_t router_grad_tc_scratch_bytes(int E, int T, int d) {
  // either form of the rows
  return scratch_of(nullptr, make_plan(E, T, d, true, kPlanSms), E, T, d).bytes;
}

template <class K>
static cudaError_t allow_smem(K kernel, bool (&done)[64]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

cudaError_t launch_router_backward_tc(const RouterGradProblem& g, cudaStream_t st) {
  const bool q8 = g.q != nullptr && g.dW != nullptr;
  const Plan p = make_plan(g.E, g.T, g.d, q8, kPlanSms);
  const Scratch sc = scratch_of(g.scratch, p, g.E, g.T, g.d);
  int lanes = 8;
  while (2 * lanes < p.ep) lanes *= 2;
  cudaError_t e = launch_kernel(router_terms_kernel, dim3(p.term_blocks), dim3(256), 0, st, g.dlogits,
                                q8 ? g.rstd : nullptr, g.scales, g.mask, g.E, g.T, g.d, p, lanes,
                                g.dW != nullptr, sc.terms, q8 ? sc.words : nullptr,
                                g.dx ? sc.exps : nullptr, sc.db_part, g.status);
  if (e != cudaSuccess) return e;
  pdl_launches() = true;
  auto encode_terms = [&](CUtensorMap* m, const cuuint32_t* box) {
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(g.T), static_cast<cuuint64_t>(p.all)};
    const cuuint64_t strides[2] = {128, static_cast<cuuint64_t>(g.T) * 128};
    return mx_encode_bf16_map(m, sc.terms, 3, dims, strides, box);
  };
  if (g.dW) {
    DwArgs a;
    a.mask = g.mask;
    a.words = sc.words;
    a.E = g.E;
    a.T = g.T;
    a.d = g.d;
    a.p = p;
    a.stage_bytes = p.bt * 128 * (2 + p.panels) + (q8 ? (p.bt * 136 + 1023) / 1024 * 1024 : 0);
    a.stages = (kSmemLimit - kFixed) / a.stage_bytes;
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    // an even number: a buffer's phases all belong to one issuer and one group of
    // converters, which have waited for each of them (a parity tells only
    // neighbouring phases apart)
    a.stages &= ~1;
    a.tmem_cols = tmem_columns(2 * p.accs * p.egp);
    a.part = sc.part;
    a.status = g.status;
    CUtensorMap tmX = {}, tmD;
    {
      const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.bt), static_cast<cuuint32_t>(p.panels)};
      if (!encode_terms(&tmD, box)) return cudaErrorInvalidValue;
    }
    if (q8) {
      const cuuint64_t dims[2] = {static_cast<cuuint64_t>(g.d), static_cast<cuuint64_t>(g.T)};
      const cuuint64_t strides[1] = {static_cast<cuuint64_t>(g.d)};
      const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(p.bt)};
      if (!mx_make_bytes_map(&tmX, g.q, 2, dims, strides, box)) return cudaErrorInvalidValue;
    } else {
      const cuuint64_t dims[2] = {static_cast<cuuint64_t>(g.d), static_cast<cuuint64_t>(g.T)};
      const cuuint64_t strides[1] = {static_cast<cuuint64_t>(g.d) * 2};
      const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(p.bt)};
      if (!mx_encode_bf16_map(&tmX, g.x, 2, dims, strides, box)) return cudaErrorInvalidValue;
    }
    static bool done[4][64] = {{false}};
    const dim3 grid(p.tiles_d * p.groups * p.splits);
    const dim3 block(128 + 32 * (kSumWarps + (q8 ? kConvWarps : 0)));
    const size_t smem = static_cast<size_t>(a.stages) * a.stage_bytes + kFixed + 1024;
    auto go = [&](auto kernel, bool (&set)[64]) {
      const cudaError_t err = allow_smem(kernel, set);
      return err != cudaSuccess ? err : launch_kernel(kernel, grid, block, smem, st, tmX, tmD, a);
    };
    if (q8)
      e = p.bt == 64 ? go(router_dw_kernel<true, 64>, done[0]) : go(router_dw_kernel<true, 32>, done[1]);
    else
      e = p.bt == 64 ? go(router_dw_kernel<false, 64>, done[2]) : go(router_dw_kernel<false, 32>, done[3]);
    if (e != cudaSuccess) return e;
  }
  SumArgs sums;
  sums.part = sc.part;
  sums.g = q8 ? g.g : nullptr;
  sums.db_part = sc.db_part;
  sums.splits = p.splits;
  sums.term_blocks = p.term_blocks;
  sums.E = g.E;
  sums.d = g.d;
  sums.accumulate = g.accumulate;
  sums.dW = g.dW;
  sums.db = g.db;
  const size_t items = g.dW ? static_cast<size_t>(g.E) * g.d / 4 : static_cast<size_t>(g.E) * 32;
  if (g.dx) {
    DxArgs a;
    a.W = g.W_r;
    a.mask = g.mask;
    a.exps = sc.exps;
    a.E = g.E;
    a.T = g.T;
    a.d = g.d;
    a.p = p;
    // the widest tile whose part of W leaves room for four boxes and four units
    a.n_tile = p.ep <= 96 ? 256 : p.ep <= 128 ? 192 : p.ep <= 192 ? 128 : 64;
    // few token tiles: narrow ones, so that W's conversion is spread over the SMs
    // (GPU time of a call, d = 2880, narrow against wide: T = 256 17.4 and 19.1 us at
    // E = 128, 15.0 and 17.1 at E = 64; T = 1024 24.0 and 23.1, 17.5 and 20.6; T = 2048,
    // E = 128 31.9 and 28.1)
    const int ttiles = (g.T + kTM - 1) / kTM;
    if (ttiles <= 8) a.n_tile = 64;
    a.full = g.d / a.n_tile;
    const int part = (g.d - a.full * a.n_tile + 63) / 64, per = a.n_tile / 64;
    // CTAs in proportion to the columns, one per SM where d allows
    a.splits = a.full ? kPlanSms * per / (a.full * per + part) : 0;
    if (a.splits > ttiles) a.splits = ttiles;
    if (a.full && a.splits < 1) a.splits = 1;
    a.last_splits = 0;
    if (part) {
      a.last_splits = a.full ? (a.splits * part + per - 1) / per : kPlanSms;
      const int left = kPlanSms - a.full * a.splits;
      if (a.last_splits > left) a.last_splits = left;
      if (a.last_splits > ttiles) a.last_splits = ttiles;
      if (a.last_splits < 1) a.last_splits = 1;
    }
    if (p.ep * per > kDxWeights) return cudaErrorInvalidValue;   // no choice above gives this
    a.boxes = (2 * p.ep + 63) / 64;
    const int wbytes = p.ep * 256 * per;
    const int room = kSmemLimit - kFixed - wbytes;
    a.ring = room / 2 / kBoxBytes;
    if (a.ring > 2 * a.boxes) a.ring = 2 * a.boxes;
    a.ring = a.ring < 4 ? 4 : a.ring > kMaxRing ? kMaxRing : a.ring;
    // an even number of units, so that a buffer's phases belong to one group of
    // warps, which has waited for each (a parity tells only neighbouring ones apart)
    a.staging = (room - a.ring * kBoxBytes) / kUnitBytes & ~1;
    if (a.staging > kMaxStaging) a.staging = kMaxStaging;
    a.off_ring = wbytes;
    a.off_staging = a.off_ring + a.ring * kBoxBytes;
    a.off_fixed = a.off_staging + a.staging * kUnitBytes;
    a.tmem_cols = tmem_columns(2 * a.n_tile);
    a.has_in = g.dx_in != nullptr;
    a.status = g.status;
    CUtensorMap tmD, tmIn = {}, tmOut;
    {
      const cuuint32_t box[3] = {64, kTM, 1};
      if (!encode_terms(&tmD, box)) return cudaErrorInvalidValue;
      const cuuint64_t dims[2] = {static_cast<cuuint64_t>(g.d), static_cast<cuuint64_t>(g.T)};
      const cuuint64_t strides[1] = {static_cast<cuuint64_t>(g.d) * 2};
      if (!mx_encode_bf16_map(&tmOut, g.dx, 2, dims, strides, box)) return cudaErrorInvalidValue;
      if (a.has_in && !mx_encode_bf16_map(&tmIn, g.dx_in, 2, dims, strides, box))
        return cudaErrorInvalidValue;
    }
    static bool done[2][64] = {{false}};
    const int blocks = a.full * a.splits + a.last_splits;
    a.sums = sums;
    // the sums are warps 12..15's where the tiles outlast them, else a launch of their own
    const bool apart = ttiles <= 16 && items > static_cast<size_t>(blocks) * 32 * kSumsWarps * 3;
    a.sums.blocks = (g.dW || g.db) && !apart ? blocks : 0;
    auto go = [&](auto kernel, bool (&set)[64]) {
      const cudaError_t err = allow_smem(kernel, set);
      return err != cudaSuccess ? err
                                : launch_kernel(kernel, dim3(blocks), dim3(kDxThreads),
                                                static_cast<size_t>(a.off_fixed) + kFixed + 1024, st, tmD,
                                                tmIn, tmOut, a);
    };
    e = g.mask ? go(router_dx_kernel<true>, done[0]) : go(router_dx_kernel<false>, done[1]);
    if (e != cudaSuccess || a.sums.blocks) return e;
  }
  if (!g.dW && !g.db) return cudaSuccess;
  const size_t want = (items + 255) / 256;
  sums.blocks = static_cast<int>(want < kPlanSms * 8 ? want : kPlanSms * 8);
  return launch_kernel(router_sums_kernel, dim3(sums.blocks), dim3(256), 0, st, sums);
}

}  // namespace moe
