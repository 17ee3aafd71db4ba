// moe_norm_ckpt.cu -- the pre-MoE RMSNorm for training: the forward that keeps
// its input as an 8-bit checkpoint, and the backward that reads it.
//
//   forward   r_t = 1 / sqrt(mean(h_t^2) + eps),  x = bf16((h r) g)
//             checkpoint: h as OCP MX blocks (E4M3 codes, one E8M0 scale per 32
//             elements, 1.03 bytes per element) and r_t in fp32
//   backward  n = h r;  dh = dh_in + r (g dx - n mean(n g dx)),  dg = sum_t dx n
//
// Field guide "gpt-oss 20B", "04 One decoder block" (RMSNorm before the MoE).
#include <cuda_bf16.h>
#include <stdint.h>

#include "moe_internal.h"
#include "moe_mx_convert.cuh"
#include "moe_ptx.cuh"

namespace moe {
namespace {

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void unpack2(uint32_t v, float* f) {
  f[0] = __uint_as_float(v << 16);
  f[1] = __uint_as_float(v & 0xFFFF0000u);
}

// a / b correctly rounded, y = 1 / b correctly rounded: q = a y is within an ulp
// of the quotient, a - b q is exact, and q + y (a - b q) rounds to the quotient
// (P. Markstein, IBM J. Res. Dev. 34, 1990), as long as nothing underflows or
// overflows: the caller keeps |a| and b between 2^-60 and 2^60. Three
// instructions; the division operator's dozen per element were a third of the
// kernel's.
__device__ __forceinline__ float2 quotient2(float2 a, float b, float y) {
  const float2 q = mul2(a, both(y));
  return fma2(fma2(both(-b), q, a), both(y), q);
}

__device__ __forceinline__ void async_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void async_copies_done() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

// One warp per row in turn, the row in shared memory. The sum of squares and the
// root are those of the norm without a checkpoint, in the same order, so x is the
// same bit for bit: lane l sums elements 4 l .. 4 l + 3 of each 128. Then each lane
// converts eight elements at a time (four lanes share a group's scale) and, as
// soon as it has read them, loads the next row's into their place.
constexpr int kCkptWarps = 4;

__global__ void __launch_bounds__(kCkptWarps * 32, 9) norm_ckpt_kernel(
    const uint16_t* __restrict__ h, const float* __restrict__ g, float eps, int T, int d,
    uint16_t* __restrict__ x, uint8_t* __restrict__ q, uint8_t* __restrict__ scales,
    float* __restrict__ rstd) {
  pdl_wait_and_trigger();
  extern __shared__ __align__(16) uint8_t rows[];
  constexpr float kLo = 8.673617379884035e-19f, kHi = 1.152921504606847e18f;   // 2^-60, 2^60
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kCkptWarps;
  const uint8_t* const row = rows + static_cast<size_t>(threadIdx.x >> 5) * d * 2;
  const uint32_t row_s = smem_u32(row);
  int64_t t = static_cast<int64_t>(blockIdx.x) * kCkptWarps + (threadIdx.x >> 5);
  if (t < T)
    for (int k = lane * 8; k < d; k += 256) async_copy16(row_s + k * 2, h + t * d + k);
  for (; t < T; t += step) {
    async_copies_done();
    __syncwarp();
    float ss = 0.f;
#pragma unroll 4
    for (int k = lane * 4; k < d; k += 128) {
      const uint2 v = *reinterpret_cast<const uint2*>(row + k * 2);
      float f[4];
      unpack2(v.x, f);
      unpack2(v.y, f + 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = fmaf(f[i], f[i], ss);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
    const float root = sqrtf(ss / (float)d + eps);
    const float y = 1.f / root;
    if (lane == 0) rstd[t] = y;
    const bool plain = root >= kLo && root <= kHi;
    uint8_t* const qr = q + t * d;
    uint8_t* const sr = scales + t * (d / 32);
    uint16_t* const xr = x + t * d;
    const uint16_t* const next = h + (t + step) * d;
    const bool more = t + step < T;
#pragma unroll 2
    for (int k0 = 0; k0 < d; k0 += 256) {
      const int k = k0 + lane * 8;
      const bool in = k < d;   // whole groups of four lanes: d is a multiple of 32
      uint4 v = make_uint4(0, 0, 0, 0);
      if (in) {
        v = *reinterpret_cast<const uint4*>(row + k * 2);
        if (more) async_copy16(row_s + k * 2, next + k);
      }
      float f[8];
      unpack2(v.x, f);
      unpack2(v.y, f + 2);
      unpack2(v.z, f + 4);
      unpack2(v.w, f + 6);
      float amax = fabsf(f[0]), amin = fabsf(f[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        amax = fmaxf(amax, fabsf(f[i]));
        amin = fminf(amin, fabsf(f[i]));
      }
      const bool fast = plain && amin >= kLo && amax <= kHi;
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      if (!in) continue;
      const int ex = mx_scale_exp<ACT_E4M3>(amax);
      const float inv = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
      float2 z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = mul2(make_float2(f[2 * i], f[2 * i + 1]), both(inv));
      *reinterpret_cast<uint2*>(qr + k) =
          make_uint2(f32x2_to_e4m3x2(z[0].x, z[0].y) | (f32x2_to_e4m3x2(z[1].x, z[1].y) << 16),
                     f32x2_to_e4m3x2(z[2].x, z[2].y) | (f32x2_to_e4m3x2(z[3].x, z[3].y) << 16));
      if ((lane & 3) == 0) sr[k / 32] = static_cast<uint8_t>(ex + 127);
      if (x) {
        const float4 g0 = __ldg(reinterpret_cast<const float4*>(g + k));
        const float4 g1 = __ldg(reinterpret_cast<const float4*>(g + k) + 1);
        const float2 gv[4] = {make_float2(g0.x, g0.y), make_float2(g0.z, g0.w),
                              make_float2(g1.x, g1.y), make_float2(g1.z, g1.w)};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = make_float2(f[2 * i], f[2 * i + 1]);
          const float2 n = mul2(fast ? quotient2(a, root, y) : make_float2(a.x / root, a.y / root), gv[i]);
          o[i] = pack_bf16(n.x, n.y);
        }
        *reinterpret_cast<uint4*>(xr + k) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// One block per row in turn, each thread eight columns per chunk: the gain's
// gradient of those columns stays in registers over the block's rows. The next
// row's loads run while this row's mean is formed.
constexpr int kNormThreads = 512;

struct NormRow {
  uint4 dx, h;         // h: 8 bf16, or 8 codes in .x and .y
  uint32_t scale;
};

template <bool Q8, int NC>
__global__ void __maxnreg__(NC == 1 ? 56 : 128) norm_backward_kernel(
    const uint16_t* dx, const uint16_t* __restrict__ h, const uint8_t* __restrict__ q,
    const uint8_t* __restrict__ scales, const float* __restrict__ rstd,
    const float* __restrict__ g, const uint8_t* __restrict__ mask, int T, int d,
    const uint16_t* dh_in, uint16_t* dh, float* __restrict__ partial) {
  pdl_wait_and_trigger();
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int vec = d / 8;
  float2 dg[NC][4];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) dg[c][i] = make_float2(0.f, 0.f);
  NormRow next[NC];
  uint4 in[NC];
  float next_r = 0.f;
  uint32_t next_live = 1;
  // whether or not the token is live: no load waits for the mask's
  auto load = [&](int t) {
    if (t >= T) return;
    next_r = __ldg(rstd + t);
    if (mask) next_live = __ldg(mask + t);
    const int64_t row = static_cast<int64_t>(t) * d;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int v = threadIdx.x + c * blockDim.x;
      if (v >= vec) continue;
      next[c].dx = *reinterpret_cast<const uint4*>(dx + row + v * 8);
      if (Q8) {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(q + row + v * 8));
        next[c].h.x = w.x;
        next[c].h.y = w.y;
        next[c].scale = __ldg(scales + (row >> 5) + (v >> 2));
      } else {
        next[c].h = __ldcs(reinterpret_cast<const uint4*>(h + row + v * 8));
      }
    }
  };
  auto load_in = [&](int t) {
    if (t >= T || !dh_in) return;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int v = threadIdx.x + c * blockDim.x;
      if (v < vec) in[c] = *reinterpret_cast<const uint4*>(dh_in + static_cast<int64_t>(t) * d + v * 8);
    }
  };
  const float inv_d = 1.f / static_cast<float>(d);
  int buf = 0;
  int t = blockIdx.x;
  load(t);
  load_in(t);
  for (; t < T; t += gridDim.x) {
    const bool live = next_live != 0;
    // a padded token's row: r = 0 and its values are not looked at
    const float r = live ? next_r : 0.f;
    float2 n[NC][4], u[NC][4];
    float2 dots = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int v = threadIdx.x + c * blockDim.x;
      if (v >= vec) continue;
      if (!live) {
#pragma unroll
        for (int i = 0; i < 4; ++i) n[c][i] = u[c][i] = make_float2(0.f, 0.f);
        continue;
      }
      const uint32_t dw[4] = {next[c].dx.x, next[c].dx.y, next[c].dx.z, next[c].dx.w};
      if (Q8) {
        const float2 s = both(e8m0_of_row(next[c].scale, r));
        const uint32_t hw[2] = {next[c].h.x, next[c].h.y};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          n[c][i] = mul2(mul2(e4m3x2_to_f32x2((hw[i >> 1] >> (16 * (i & 1))) & 0xFFFFu), s), both(r));
      } else {
        const uint32_t hw[4] = {next[c].h.x, next[c].h.y, next[c].h.z, next[c].h.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) n[c][i] = mul2(bf16_pair(hw[i]), both(r));
      }
      const float4 g0 = __ldg(reinterpret_cast<const float4*>(g) + 2 * v);
      const float4 g1 = __ldg(reinterpret_cast<const float4*>(g) + 2 * v + 1);
      const float2 gv[4] = {make_float2(g0.x, g0.y), make_float2(g0.z, g0.w), make_float2(g1.x, g1.y),
                            make_float2(g1.z, g1.w)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = bf16_pair(dw[i]);
        dg[c][i] = fma2(x, n[c][i], dg[c][i]);
        u[c][i] = mul2(x, gv[i]);
        dots = fma2(n[c][i], u[c][i], dots);
      }
    }
    float dot = dots.x + dots.y;
    load(t + gridDim.x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, off);
    if (lane == 0) red[buf][warp] = dot;
    __syncthreads();
    float m = lane < warps ? red[buf][lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m += __shfl_xor_sync(0xFFFFFFFFu, m, off);
    m *= -r * inv_d;
    buf ^= 1;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int v = threadIdx.x + c * blockDim.x;
      if (v >= vec) continue;
      // dh_in + r u - (r mean) n
      const uint32_t dw[4] = {in[c].x, in[c].y, in[c].z, in[c].w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 z = fma2(both(m), n[c][i], mul2(both(r), u[c][i]));
        if (dh_in) z = fma2(z, both(1.f), bf16_pair(dw[i]));
        o[i] = pack_bf16(z.x, z.y);
      }
      *reinterpret_cast<uint4*>(dh + static_cast<int64_t>(t) * d + v * 8) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
    load_in(t + gridDim.x);
  }
  float* pr = partial + static_cast<size_t>(blockIdx.x) * d;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int v = threadIdx.x + c * blockDim.x;
    if (v >= vec) continue;
    reinterpret_cast<float4*>(pr)[2 * v] =
        make_float4(dg[c][0].x, dg[c][0].y, dg[c][1].x, dg[c][1].y);
    reinterpret_cast<float4*>(pr)[2 * v + 1] =
        make_float4(dg[c][2].x, dg[c][2].y, dg[c][3].x, dg[c][3].y);
  }
}

// dg[i] (+)= sum over the blocks' rows, in block order within each of 32 shares,
// the shares in order.
__global__ void __launch_bounds__(1024) norm_dg_kernel(const float* __restrict__ partial, int rows,
                                                       int d, bool accumulate,
                                                       float* __restrict__ dg) {
  pdl_wait_and_trigger();
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;   // d is a multiple of 32
  float s = 0.f;
#pragma unroll 16
  for (int r = share; r < rows; r += 32) s += __ldg(partial + static_cast<size_t>(r) * d + i);
  sh[share][lane] = s;
  __syncthreads();
  // warp w: column w of the block's 32
  s = sh[lane][share];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
  if (lane == 0) {
    float* o = dg + blockIdx.x * 32 + share;
    *o = accumulate ? *o + s : s;
  }
}

struct NormBwdShape {
  int threads, chunks, blocks;
};

NormBwdShape norm_bwd_shape(int T, int d) {
  NormBwdShape s;
  const int vec = d / 8;                         // at most 2048
  s.chunks = vec <= kNormThreads ? 1 : vec <= 2 * kNormThreads ? 2 : 4;
  s.threads = ((vec + s.chunks - 1) / s.chunks + 31) / 32 * 32;
  // blocks of about 1152 threads per SM, at most eight: at d = 2880 three (two or
  // four took 50 us where three took 43, T = 8192). Each leaves a row of partial sums
  // to the launch after: at d = 96, T = 4096 sixteen took 10.7 us, eight 8.3; at
  // T = 16384 14.8 and 15.3, four 21.8. (Joining the rows of a cluster first was no
  // faster: its blocks have to find room together.)
  int per = 1152 / s.threads;
  per = per < 1 ? 1 : per > 8 ? 8 : per;
  s.blocks = T < 148 * per ? (T > 0 ? T : 1) : 148 * per;
  return s;
}

}  // namespace

cudaError_t launch_rms_norm_checkpoint(const uint16_t* h, const float* g, float eps, int T, int d,
                                       uint16_t* x, uint8_t* q, uint8_t* scales, float* rstd,
                                       cudaStream_t st) {
  // as many blocks as an SM holds (T = 8192, d = 2880: 47 us with 12 warps per SM, 37
  // with 20, 31 with 32), at most 36 warps of them
  const size_t smem = static_cast<size_t>(kCkptWarps) * d * 2;
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(norm_ckpt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kCkptWarps * 16384 * 2);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  int per = static_cast<int>(225 * 1024 / (smem + 1024));
  per = per < 1 ? 1 : per > 9 ? 9 : per;
  const int64_t b = (static_cast<int64_t>(T) + kCkptWarps - 1) / kCkptWarps;
  const int grid = static_cast<int>(b < 148 * per ? b : 148 * per);
  return launch_kernel(norm_ckpt_kernel, dim3(grid), dim3(kCkptWarps * 32), smem, st, h, g, eps, T, d,
                       x, q, scales, rstd);
}

size_t rms_norm_backward_scratch_bytes(int T, int d) {
  return static_cast<size_t>(norm_bwd_shape(T, d).blocks) * d * sizeof(float);
}

cudaError_t launch_rms_norm_backward(const uint16_t* dx, const uint16_t* h, const uint8_t* q,
                                     const uint8_t* scales, const float* rstd, const float* g,
                                     const uint8_t* mask, int T, int d, const uint16_t* dh_in,
                                     bool accumulate, uint16_t* dh, float* dg, void* scratch,
                                     cudaStream_t st) {
  const NormBwdShape s = norm_bwd_shape(T, d);
  float* partial = static_cast<float*>(scratch);
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, dim3(s.blocks), dim3(s.threads), 0, st, dx, h, q, scales, rstd, g,
                         mask, T, d, dh_in, dh, partial);
  };
  cudaError_t e;
  switch (s.chunks) {
    case 1: e = q ? go(norm_backward_kernel<true, 1>) : go(norm_backward_kernel<false, 1>); break;
    case 2: e = q ? go(norm_backward_kernel<true, 2>) : go(norm_backward_kernel<false, 2>); break;
    default: e = q ? go(norm_backward_kernel<true, 4>) : go(norm_backward_kernel<false, 4>);
  }
  if (e != cudaSuccess) return e;
  pdl_launches() = true;
  return launch_kernel(norm_dg_kernel, dim3(d / 32), dim3(1024), 0, st, partial, s.blocks, d,
                       accumulate, dg);
}

}  // namespace moe
