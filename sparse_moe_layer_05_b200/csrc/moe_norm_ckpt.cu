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

// One warp per row; sum of squares, root and division are those of the norm
// without a checkpoint, in the same order, so x is the same bit for bit.
__global__ void __launch_bounds__(256) norm_ckpt_kernel(const uint16_t* __restrict__ h,
                                                        const float* __restrict__ g, float eps,
                                                        int T, int d, uint16_t* __restrict__ x,
                                                        uint8_t* __restrict__ q,
                                                        uint8_t* __restrict__ scales,
                                                        float* __restrict__ rstd) {
  pdl_wait_and_trigger();
  const int lane = threadIdx.x & 31;
  const int nwarps = (gridDim.x * blockDim.x) >> 5;
  for (int t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; t < T; t += nwarps) {
    const uint16_t* hr = h + (size_t)t * d;
    float ss = 0.f;
    for (int k = lane * 4; k < d; k += 128) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(hr + k));
      const float a = __uint_as_float(v.x << 16), b = __uint_as_float(v.x & 0xFFFF0000u);
      const float c = __uint_as_float(v.y << 16), e = __uint_as_float(v.y & 0xFFFF0000u);
      ss = fmaf(a, a, ss);
      ss = fmaf(b, b, ss);
      ss = fmaf(c, c, ss);
      ss = fmaf(e, e, ss);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
    const float root = sqrtf(ss / (float)d + eps);
    if (lane == 0) rstd[t] = 1.f / root;
    for (int k0 = 0; k0 < d; k0 += 128) {
      const int k = k0 + lane * 4;
      const bool in = k < d;   // whole groups of 8 lanes: d is a multiple of 32
      const uint2 v = in ? __ldg(reinterpret_cast<const uint2*>(hr + k)) : make_uint2(0, 0);
      const float f0 = __uint_as_float(v.x << 16), f1 = __uint_as_float(v.x & 0xFFFF0000u);
      const float f2 = __uint_as_float(v.y << 16), f3 = __uint_as_float(v.y & 0xFFFF0000u);
      float amax = fmaxf(fmaxf(fabsf(f0), fabsf(f1)), fmaxf(fabsf(f2), fabsf(f3)));
#pragma unroll
      for (int off = 4; off > 0; off >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
      if (!in) continue;
      const int ex = mx_scale_exp<ACT_E4M3>(amax);
      const float inv = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
      *reinterpret_cast<uint32_t*>(q + (size_t)t * d + k) =
          f32x2_to_e4m3x2(f0 * inv, f1 * inv) | (f32x2_to_e4m3x2(f2 * inv, f3 * inv) << 16);
      if ((lane & 7) == 0)
        scales[(size_t)t * (d / 32) + k / 32] = static_cast<uint8_t>(ex + 127);
      if (x) {
        const float4 gv = __ldg(reinterpret_cast<const float4*>(g + k));
        *reinterpret_cast<uint2*>(x + (size_t)t * d + k) =
            make_uint2(pack_bf16((f0 / root) * gv.x, (f1 / root) * gv.y),
                       pack_bf16((f2 / root) * gv.z, (f3 / root) * gv.w));
      }
    }
  }
}

// One block per row in turn, each thread eight columns per chunk: the gain's
// gradient of those columns stays in registers over the block's rows.
template <bool Q8, int NC>
__global__ void __launch_bounds__(1024) norm_backward_kernel(
    const uint16_t* dx, const uint16_t* __restrict__ h, const uint8_t* __restrict__ q,
    const uint8_t* __restrict__ scales, const float* __restrict__ rstd,
    const float* __restrict__ g, const uint8_t* __restrict__ mask, int T, int d,
    const uint16_t* dh_in, uint16_t* dh, float* __restrict__ partial) {
  pdl_wait_and_trigger();
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int vec = d / 8;
  float dg[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[c][i] = 0.f;
  int buf = 0;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const bool live = mask == nullptr || mask[t] != 0;
    const float r = rstd[t];
    float n[NC][8], u[NC][8];
    float dot = 0.f;
    if (live) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int v = threadIdx.x + c * blockDim.x;
        if (v >= vec) continue;
        const uint4 dv = reinterpret_cast<const uint4*>(dx + (size_t)t * d)[v];
        const uint32_t dw[4] = {dv.x, dv.y, dv.z, dv.w};
        float hv[8];
        if (Q8) {
          const uint2 qv = __ldg(reinterpret_cast<const uint2*>(q + (size_t)t * d) + v);
          const float s = e8m0_to_f32(scales[(size_t)t * (d / 32) + v / 4]);
          const uint32_t qw[2] = {qv.x, qv.y};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = e4m3x2_to_f32x2((qw[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
            hv[2 * i] = f.x * s;
            hv[2 * i + 1] = f.y * s;
          }
        } else {
          const uint4 hw4 = __ldg(reinterpret_cast<const uint4*>(h + (size_t)t * d) + v);
          const uint32_t hw[4] = {hw4.x, hw4.y, hw4.z, hw4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            hv[2 * i] = __uint_as_float(hw[i] << 16);
            hv[2 * i + 1] = __uint_as_float(hw[i] & 0xFFFF0000u);
          }
        }
        const float4 g0 = __ldg(reinterpret_cast<const float4*>(g) + 2 * v);
        const float4 g1 = __ldg(reinterpret_cast<const float4*>(g) + 2 * v + 1);
        const float gv[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float dxv = __uint_as_float(i & 1 ? dw[i >> 1] & 0xFFFF0000u : dw[i >> 1] << 16);
          n[c][i] = hv[i] * r;
          u[c][i] = dxv * gv[i];
          dg[c][i] = fmaf(dxv, n[c][i], dg[c][i]);
          dot = fmaf(n[c][i], u[c][i], dot);
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, off);
    if (lane == 0) red[buf][warp] = dot;
    __syncthreads();
    float m = 0.f;
    for (int w = 0; w < warps; ++w) m += red[buf][w];
    m /= (float)d;
    buf ^= 1;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int v = threadIdx.x + c * blockDim.x;
      if (v >= vec) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = live ? r * (u[c][i] - n[c][i] * m) : 0.f;
      if (dh_in) {
        const uint4 dv = reinterpret_cast<const uint4*>(dh_in + (size_t)t * d)[v];
        const uint32_t dw[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[2 * i] += __uint_as_float(dw[i] << 16);
          o[2 * i + 1] += __uint_as_float(dw[i] & 0xFFFF0000u);
        }
      }
      reinterpret_cast<uint4*>(dh + (size_t)t * d)[v] =
          make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]),
                     pack_bf16(o[6], o[7]));
    }
  }
  float* pr = partial + (size_t)blockIdx.x * d;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int v = threadIdx.x + c * blockDim.x;
    if (v >= vec) continue;
    reinterpret_cast<float4*>(pr)[2 * v] = make_float4(dg[c][0], dg[c][1], dg[c][2], dg[c][3]);
    reinterpret_cast<float4*>(pr)[2 * v + 1] = make_float4(dg[c][4], dg[c][5], dg[c][6], dg[c][7]);
  }
}

// dg[i] (+)= sum over the blocks' rows, in block order within each of eight
// shares, the shares in order.
__global__ void __launch_bounds__(256) norm_dg_kernel(const float* __restrict__ partial, int rows,
                                                      int d, bool accumulate,
                                                      float* __restrict__ dg) {
  pdl_wait_and_trigger();
  __shared__ float sh[8][32];
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;   // d is a multiple of 32
  float s = 0.f;
  for (int r = share; r < rows; r += 8) s += __ldg(partial + (size_t)r * d + i);
  sh[share][lane] = s;
  __syncthreads();
  if (share == 0) {
#pragma unroll
    for (int w = 1; w < 8; ++w) s += sh[w][lane];
    dg[i] = accumulate ? dg[i] + s : s;
  }
}

constexpr int kNormBwdBlocks = 148 * 4;

struct NormBwdShape {
  int threads, chunks, blocks;
};

NormBwdShape norm_bwd_shape(int T, int d) {
  NormBwdShape s;
  const int vec = d / 8;                         // at most 2048
  s.chunks = vec > 1024 ? 2 : 1;
  s.threads = (vec / s.chunks + 31) / 32 * 32;
  while (s.threads * s.chunks < vec) s.threads += 32;
  s.blocks = T < kNormBwdBlocks ? (T > 0 ? T : 1) : kNormBwdBlocks;
  return s;
}

}  // namespace

cudaError_t launch_rms_norm_checkpoint(const uint16_t* h, const float* g, float eps, int T, int d,
                                       uint16_t* x, uint8_t* q, uint8_t* scales, float* rstd,
                                       cudaStream_t st) {
  const int64_t b = (static_cast<int64_t>(T) + 7) / 8;
  const int grid = static_cast<int>(b < 148 * 8 ? b : 148 * 8);
  return launch_kernel(norm_ckpt_kernel, dim3(grid), dim3(256), 0, st, h, g, eps, T, d, x, q,
                       scales, rstd);
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
  if (q)
    e = s.chunks == 1 ? go(norm_backward_kernel<true, 1>) : go(norm_backward_kernel<true, 2>);
  else
    e = s.chunks == 1 ? go(norm_backward_kernel<false, 1>) : go(norm_backward_kernel<false, 2>);
  if (e != cudaSuccess) return e;
  pdl_launches() = true;
  return launch_kernel(norm_dg_kernel, dim3(d / 32), dim3(256), 0, st, partial, s.blocks, d,
                       accumulate, dg);
}

}  // namespace moe
