// moe_router_grad.cu -- the router's training step: the load-balance and z
// loss with its gradient, the gradient through the selected-set softmax, and
// the gradients of the router product.
//
//   p[t] = softmax(s[t]) over all E experts, n live tokens, c_e pairs routed to
//   expert e:  f_e = c_e / (n k),  P_e = (1/n) sum_t p[t,e]
//   L = a E sum_e f_e P_e + b (1/n) sum_t lse(s[t])^2
//   dL/ds[t,e] = (1/n) p[t,e] (a E (f_e - sum_e' f_e' p[t,e']) + 2 b lse(s[t]))
//
//   out_t = sum_j p_j y_j over the selected set:  A_j = <dout_t, p_j y_j>,
//   dL/ds[t, idx_j] = p_j (dp_j - sum_l p_l dp_l) = A_j - p_j sum_l A_l
//                   = sum_l (p_l A_j - p_j A_l),  the p_l's sum being 1
//
//   s = x W^T + b:  dW = ds^T x,  db = sum_t ds,  dx = ds W
//
// ("llm-surgery-dark-arts-gpt-oss-40b-64a8-init", section 2, "Proof": s_i and
// p_i.) Sums over tokens are taken in a fixed order: results do not change
// from call to call.
#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include "moe_internal.h"
#include "moe_mx_convert.cuh"
#include "moe_ptx.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}
// Both sums at once: each half of the warp takes one of them (six shuffles, not ten).
__device__ __forceinline__ void warp_sum2(float& a, float& b, int lane) {
  const bool upper = lane & 16;
  float v = (upper ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, upper ? a : b, 16);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  const float w = __shfl_xor_sync(0xFFFFFFFFu, v, 16);
  a = upper ? w : v;
  b = upper ? v : w;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
  return v;
}

// -------------------------------------------------------- balance loss ----
// One warp per token; a block's sums are joined in shared memory and those of a
// cluster of four blocks over its shared memory, so that the finishing block has
// at most 32 rows of sums to add (in fp64): with a row per block it took longer
// than the pass over the logits. 32 clusters, because 36 do not fit the device at
// once (T = 16384, E = 128: 11 us against 16 in two waves). A batch that one cluster
// holds is finished in the same launch.

constexpr int kMaxE = 256;
constexpr int kBalCluster = 4, kBalClusters = 32, kBalWarps = 32;
constexpr int kBalOneCluster = 256;   // tokens: two per warp

// Warps of a block and clusters: one token per warp as long as the blocks last.
int balance_warps(int T) {
  const int blocks = T <= kBalOneCluster ? kBalCluster : kBalCluster * kBalClusters;
  const int w = T / blocks + (T % blocks != 0);
  return w < 4 ? 4 : w > kBalWarps ? kBalWarps : w;
}
int balance_clusters(int T) {
  if (T <= kBalOneCluster) return 1;
  const int per = balance_warps(T) * kBalCluster;
  const int c = T / per + (T % per != 0);
  return c > kBalClusters ? kBalClusters : c;
}

// Per cluster: sums over its tokens of p[e] and lse^2, the counts, live tokens.
struct BalanceScratch {
  float* p;        // [clusters][E]
  int32_t* counts; // [clusters][E]
  double* z;       // [clusters]
  int32_t* n;      // [clusters]
};

BalanceScratch balance_scratch(void* base, int E, int clusters) {
  BalanceScratch s;
  uint8_t* b = static_cast<uint8_t*>(base);
  s.z = reinterpret_cast<double*>(b);
  b += static_cast<size_t>(kBalClusters) * 8;
  s.n = reinterpret_cast<int32_t*>(b);
  b += static_cast<size_t>(kBalClusters) * 4;
  s.p = reinterpret_cast<float*>(b);
  b += static_cast<size_t>(clusters) * E * 4;
  s.counts = reinterpret_cast<int32_t*>(b);
  return s;
}

struct BalanceOut {
  float balance_coef, z_coef;
  float* stats;        // [4]
  int32_t* counts;     // [E]
  float* mean_probs;   // [E]
};

// A lane's NL (4 for at most 128 experts, else 8) of a row's experts: four
// neighbours at a time where rows are whole float4s (VEC), else lane, lane + 32, ...
template <bool VEC>
__device__ __forceinline__ int expert_of(int lane, int i) {
  return VEC ? 4 * lane + (i & 3) + 128 * (i >> 2) : lane + 32 * i;
}
template <bool VEC, int NL>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float (&v)[NL]) {
  if (VEC) {
#pragma unroll
    for (int h = 0; h < NL / 4; ++h) {
      const int e = 4 * lane + 128 * h;
      const float4 x = e < E ? __ldg(reinterpret_cast<const float4*>(row + e))
                             : make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F);
      v[4 * h] = x.x;
      v[4 * h + 1] = x.y;
      v[4 * h + 2] = x.z;
      v[4 * h + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i) v[i] = lane + 32 * i < E ? __ldg(row + lane + 32 * i) : -CUDART_INF_F;
  }
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}

// The loss from all sums: thread e < E has expert e's, z and n are the block's.
// Whole block (at least E threads, whole warps); red: 32 doubles of shared memory.
__device__ __forceinline__ void balance_results(double p, int c, double z, int n, int E, int k,
                                                const BalanceOut& o, double* red) {
  const int e = threadIdx.x;
  double term = 0.0;
  if (e < E) {
    const double mean = n > 0 ? p / n : 0.0;
    o.counts[e] = c;
    o.mean_probs[e] = static_cast<float>(mean);
    term = n > 0 ? mean * (static_cast<double>(c) / (static_cast<double>(n) * k)) : 0.0;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, off);
  if ((e & 31) == 0) red[e >> 5] = term;
  __syncthreads();
  if (e == 0) {
    double bal = 0.0;
    for (int w = 0; w < (E + 31) / 32; ++w) bal += red[w];
    bal *= E;
    const double zz = n > 0 ? z / n : 0.0;
    o.stats[0] = static_cast<float>(o.balance_coef * bal + o.z_coef * zz);
    o.stats[1] = static_cast<float>(bal);
    o.stats[2] = static_cast<float>(zz);
    o.stats[3] = static_cast<float>(n);
  }
}

// The next token's logits are loaded while this one's are summed. clusters == 1:
// the results too (at least E threads per block).
template <bool VEC, int NL>
__global__ void __launch_bounds__(kBalWarps * 32) balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const uint8_t* __restrict__ mask, int E, int k, int T, int clusters,
    float* __restrict__ lse_out, BalanceScratch sc, BalanceOut out) {
  pdl_wait_and_trigger();
  __shared__ float sp[kBalWarps][kMaxE];
  __shared__ float bp[kMaxE];              // the block's sums
  __shared__ int bc[kMaxE];
  __shared__ double sz[kBalWarps], bz, red[32];
  __shared__ int sn[kBalWarps], bn;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int e = threadIdx.x; e < E; e += blockDim.x) bc[e] = 0;
  __syncthreads();
  float acc[NL], next[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) acc[i] = 0.f;
  double z = 0.0;                          // a square of lse may pass fp32's range
  int n = 0, next_idx = -1;
  uint32_t next_live = 1;
  const int64_t step = static_cast<int64_t>(gridDim.x) * warps;
  auto load = [&](int64_t t) {
    if (t >= T) return;
    load_row<VEC, NL>(logits + t * E, E, lane, next);
    next_idx = lane < k ? __ldg(idx + t * k + lane) : -1;   // k is at most 32
    if (mask) next_live = __ldg(mask + t);
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * warps + warp;
  load(t);
  for (; t < T; t += step) {
    float v[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) v[i] = next[i];
    const int chosen = next_idx;
    const bool live = next_live != 0;
    load(t + step);
    if (!live) {
      if (lane == 0) lse_out[t] = 0.f;
      continue;
    }
    ++n;
    // the maximum leaves NaNs out; they reach the sum through their own term
    float m = v[0];
#pragma unroll
    for (int i = 1; i < NL; ++i) m = fmaxf(m, v[i]);
    m = warp_max(m);
    const float base = m == -CUDART_INF_F ? 0.f : m;   // places past E hold -inf: exp gives 0
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      v[i] = expf(v[i] - base);
      sum += v[i];
    }
    sum = warp_sum(sum);
    const bool none = sum == 0.f;                      // every logit is -inf
    const float l = none ? -CUDART_INF_F : base + logf(sum);
    const float inv = none ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < NL; ++i) acc[i] += v[i] * inv;
    if (lane == 0) {
      lse_out[t] = l;
      if (!none) z = fma(static_cast<double>(l), static_cast<double>(l), z);
    }
    if (static_cast<unsigned>(chosen) < static_cast<unsigned>(E)) atomicAdd(&bc[chosen], 1);
  }
#pragma unroll
  for (int i = 0; i < NL; ++i) sp[warp][expert_of<VEC>(lane, i)] = acc[i];
  if (lane == 0) {
    sz[warp] = z;
    sn[warp] = n;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float s = 0.f;
#pragma unroll 4
    for (int w = 0; w < warps; ++w) s += sp[w][e];
    bp[e] = s;
  }
  if (warp == 0) {
    double zz = lane < warps ? sz[lane] : 0.0;
    int nn = lane < warps ? sn[lane] : 0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      zz += __shfl_xor_sync(0xFFFFFFFFu, zz, off);
      nn += __shfl_xor_sync(0xFFFFFFFFu, nn, off);
    }
    if (lane == 0) {
      bz = zz;
      bn = nn;
    }
  }
  __syncthreads();
  cluster_sync();
  // over the cluster's blocks in order: every block a share of the experts, or
  // block 0 all of them where it goes on to the results
  const uint32_t rank = cluster_ctarank();
  const bool one = clusters == 1;
  const int cluster = blockIdx.x / kBalCluster;
  if (!one || rank == 0) {
    const int e = one ? threadIdx.x : threadIdx.x * kBalCluster + static_cast<int>(rank);
    float s[kBalCluster];
    int c[kBalCluster];
    double p = 0.0, zz = 0.0;
    int cnt = 0, nn = 0;
    if (e < E) {
#pragma unroll
      for (int r = 0; r < kBalCluster; ++r) {
        s[r] = ld_cluster_f32(mapa_shared(smem_u32(&bp[e]), r));
        c[r] = ld_cluster_s32(mapa_shared(smem_u32(&bc[e]), r));
      }
#pragma unroll
      for (int r = 0; r < kBalCluster; ++r) {
        p += s[r];
        cnt += c[r];
      }
    }
    if (one || threadIdx.x == 0)
#pragma unroll
      for (int r = 0; r < kBalCluster; ++r) {
        zz += ld_cluster_f64(mapa_shared(smem_u32(&bz), r));
        nn += ld_cluster_s32(mapa_shared(smem_u32(&bn), r));
      }
    if (one) {
      balance_results(p, cnt, zz, nn, E, k, out, red);
    } else {
      if (e < E) {
        sc.p[static_cast<size_t>(cluster) * E + e] = static_cast<float>(p);
        sc.counts[static_cast<size_t>(cluster) * E + e] = cnt;
      }
      if (rank == 0 && threadIdx.x == 0) {
        sc.z[cluster] = zz;
        sc.n[cluster] = nn;
      }
    }
  }
  cluster_sync();   // no block leaves while another reads its sums
}

// cols: E rounded up to a power of two; thread (share, e) adds every
// (1024 / cols)-th cluster's row, at most eight (32 clusters, four shares at least).
__global__ void __launch_bounds__(1024) balance_finish_kernel(BalanceScratch sc, int clusters, int E,
                                                              int cols, int k, BalanceOut out) {
  pdl_wait_and_trigger();
  __shared__ double sp[1024], red[32];
  __shared__ int scnt[1024];
  const int e = threadIdx.x & (cols - 1), share = threadIdx.x / cols, shares = 1024 / cols;
  double p = 0.0, z = 0.0;
  int c = 0, n = 0;
  if (e < E) {
    for (int b = share; b < clusters; b += shares) {
      p += __ldg(sc.p + static_cast<size_t>(b) * E + e);
      c += __ldg(sc.counts + static_cast<size_t>(b) * E + e);
    }
  }
  // every warp: z and n of all clusters
  const int lane = threadIdx.x & 31;
  for (int b = lane; b < clusters; b += 32) {
    z += __ldg(sc.z + b);
    n += __ldg(sc.n + b);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    z += __shfl_xor_sync(0xFFFFFFFFu, z, off);
    n += __shfl_xor_sync(0xFFFFFFFFu, n, off);
  }
  sp[threadIdx.x] = p;
  scnt[threadIdx.x] = c;
  __syncthreads();
  if (share == 0)
    for (int s = 1; s < shares; ++s) {
      p += sp[s * cols + e];
      c += scnt[s * cols + e];
    }
  balance_results(p, c, z, n, E, k, out, red);
}

template <bool VEC, int NL>
__global__ void __launch_bounds__(256) balance_backward_kernel(
    const float* __restrict__ logits, const float* __restrict__ lse,
    const int32_t* __restrict__ counts, const float* __restrict__ stats,
    const uint8_t* __restrict__ mask, int E, int k, int T, float balance_coef, float z_coef,
    const float* __restrict__ dloss, bool accumulate, float* dlogits) {
  pdl_wait_and_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  if (t >= T) return;
  // the first token's row and everything that does not depend on the token at once
  float v[NL], l = __ldg(lse + t), f[NL];
  uint32_t live_byte = mask ? __ldg(mask + t) : 1u;
  load_row<VEC, NL>(logits + t * E, E, lane, v);
  const float n = __ldg(stats + 3), up = dloss ? __ldg(dloss) : 1.f;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int e = expert_of<VEC>(lane, i);
    f[i] = e < E ? static_cast<float>(__ldg(counts + e)) : 0.f;
  }
  const float scale = n > 0.f ? up / n : 0.f, per = n > 0.f ? 1.f / (n * static_cast<float>(k)) : 0.f;
#pragma unroll
  for (int i = 0; i < NL; ++i) f[i] *= per;
  const float aE = balance_coef * static_cast<float>(E);
  for (; t < T; t += step) {
    const bool live = live_byte != 0 && l != -CUDART_INF_F;
    const float lt = l;
    // exp(s - lse) over its own sum: lse is fp32, off by up to 2^-24 |lse|, and every
    // exponential of the row by that much of itself (3e-4 at logits of 1e4)
    float p[NL], sum = 0.f, fp = 0.f;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      p[i] = live && expert_of<VEC>(lane, i) < E ? expf(v[i] - lt) : 0.f;
      sum += p[i];
      fp = fmaf(f[i], p[i], fp);
    }
    if (t + step < T) {
      l = __ldg(lse + t + step);
      if (mask) live_byte = __ldg(mask + t + step);
      load_row<VEC, NL>(logits + (t + step) * E, E, lane, v);
    }
    warp_sum2(fp, sum, lane);
    if (!live && accumulate) continue;   // left alone
    const float norm = 1.f / sum, to = scale * norm;
    fp *= norm;
    const float zt = 2.f * z_coef * lt;
#pragma unroll
    for (int i = 0; i < NL; ++i) p[i] = live ? to * p[i] * (aE * (f[i] - fp) + zt) : 0.f;
    float* row = dlogits + t * E;
    if (VEC) {
#pragma unroll
      for (int h = 0; h < NL / 4; ++h) {
        const int e = 4 * lane + 128 * h;
        if (e >= E) continue;
        float4 o = make_float4(p[4 * h], p[4 * h + 1], p[4 * h + 2], p[4 * h + 3]);
        if (accumulate) {
          const float4 b = *reinterpret_cast<const float4*>(row + e);
          o = make_float4(o.x + b.x, o.y + b.y, o.z + b.z, o.w + b.w);
        }
        *reinterpret_cast<float4*>(row + e) = o;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int e = lane + 32 * i;
        if (e < E) row[e] = accumulate ? row[e] + p[i] : p[i];
      }
    }
  }
}

// ------------------------------------------------------- gate gradient ----
// A token is read by `span` threads (whole warps), eight columns each, four
// slots at a time: the row of dout once, every row of yw once, all loads of four
// slots in flight together. A block holds several tokens where rows are short.
constexpr int kGateThreads = 512;
constexpr int kGateSlots = 4;

__global__ void __launch_bounds__(kGateThreads) gate_backward_kernel(
    const uint16_t* __restrict__ dout, const float* __restrict__ yw,
    const int32_t* __restrict__ idx, const float* __restrict__ w,
    const uint8_t* __restrict__ mask, int E, int k, int T, int d, int span, bool accumulate,
    float* dlogits) {
  pdl_wait_and_trigger();
  __shared__ float part[kGateThreads / 32][32];   // [warp][slot]
  __shared__ float grad[kGateThreads / 32][32];   // [token][slot]
  __shared__ int sidx[kGateThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tok = threadIdx.x / span, me = threadIdx.x % span, spans = blockDim.x / span;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * spans + tok;
  const bool in = t < T;
  const bool live = in && (!mask || mask[t] != 0);
  if (live) {
    const uint2* o = reinterpret_cast<const uint2*>(dout + t * d);
    for (int j0 = 0; j0 < k; j0 += kGateSlots) {
      float s[kGateSlots];
#pragma unroll
      for (int u = 0; u < kGateSlots; ++u) s[u] = 0.f;
      // four columns at v and four at v + span: whole 512-byte pieces per warp
      for (int v = me; v < d / 4; v += 2 * span) {
        const bool two = v + span < d / 4;
        float4 y[kGateSlots][2];
        uint2 ov[2];
#pragma unroll
        for (int u = 0; u < kGateSlots; ++u) {
          const float4* row = reinterpret_cast<const float4*>(yw + (t * k + min(j0 + u, k - 1)) * d) + v;
          y[u][0] = __ldcs(row);
          y[u][1] = two ? __ldcs(row + span) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        ov[0] = __ldg(o + v);
        ov[1] = two ? __ldg(o + v + span) : make_uint2(0, 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x0 = __uint_as_float(ov[h].x << 16), x1 = __uint_as_float(ov[h].x & 0xFFFF0000u);
          const float x2 = __uint_as_float(ov[h].y << 16), x3 = __uint_as_float(ov[h].y & 0xFFFF0000u);
#pragma unroll
          for (int u = 0; u < kGateSlots; ++u) {
            s[u] = fmaf(y[u][h].x, x0, s[u]);
            s[u] = fmaf(y[u][h].y, x1, s[u]);
            s[u] = fmaf(y[u][h].z, x2, s[u]);
            s[u] = fmaf(y[u][h].w, x3, s[u]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kGateSlots; ++u) {
        const float a = warp_sum(s[u]);
        if (lane == 0 && j0 + u < k) part[warp][j0 + u] = a;
      }
    }
  }
  __syncthreads();
  if (in && me < 32) {
    // A_j over the token's warps, then the sum over pairs of slots. With p_j near 1,
    // A_j - p_j sum A is a difference of near equals, and A_j (1 - sum p) with the
    // weights' roundings comes on top: at 1 - p_j = 1e-5 it was off by 1e-2 of itself.
    // A pair's two products are each rounded, so that a slot with itself gives zero.
    float a = 0.f, p = 0.f, g = 0.f;
    const int first = tok * (span / 32);
    if (live && lane < k)
      for (int x = 0; x < span / 32; ++x) a += part[first + x][lane];
    if (live && lane < k) p = __ldg(w + t * k + lane);
    for (int l = 0; l < k; ++l)
      g += __fmul_rn(__shfl_sync(0xFFFFFFFFu, p, l), a) - __fmul_rn(p, __shfl_sync(0xFFFFFFFFu, a, l));
    grad[tok][lane] = live && lane < k ? g : 0.f;
    sidx[tok][lane] = live && lane < k ? __ldg(idx + t * k + lane) : -1;
  }
  __syncthreads();
  if (!in) return;
  for (int e = me; e < E; e += span) {
    float v = 0.f;
    for (int j = 0; j < k; ++j)
      if (sidx[tok][j] == e) v += grad[tok][j];
    float* out = dlogits + t * E + e;
    if (!accumulate)
      *out = v;
    else if (live)
      *out += v;
  }
}

// ------------------------------------------- router gradient, few tokens ----
// One launch on the CUDA cores for batches whose three outputs take less time
// than the tensor-core path's three launches. Every block computes 8 rows by 128
// columns of a product out[r][i] = sum_k A[k][r] B[k][i]: dW (r experts, k
// tokens, B = x) or dx (r tokens, k experts, B = W). Its eight warps take every
// eighth k, eight of them with their loads in flight together (four groups with
// one load after another took 0.1 us a token), a lane four columns.

// Four columns of an input row: x, or q 2^(s - 127) r g.
struct RouterRows {
  const uint16_t* x;
  const uint8_t* q;
  const uint8_t* scales;
  const float* rstd;
  const float* g;
};
template <bool Q8>
__device__ __forceinline__ float4 router_row4(const RouterRows& r, int64_t t, int i, int d) {
  if (!Q8) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(r.x + t * d + i));
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
  }
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(r.q + t * d + i));
  const float n = __ldg(r.rstd + t), s = e8m0_of_row(__ldg(r.scales + t * (d / 32) + i / 32), n);
  const float2 a = e4m3x2_to_f32x2(w & 0xFFFFu), b = e4m3x2_to_f32x2(w >> 16);
  const float4 g = __ldg(reinterpret_cast<const float4*>(r.g + i));
  return make_float4(a.x * s * n * g.x, a.y * s * n * g.y, b.x * s * n * g.z, b.y * s * n * g.w);
}

struct SmallArgs {
  const float* dl;
  const float* W;
  RouterRows rows;
  const uint8_t* mask;
  int E, T, d, col_blocks, dw_blocks, dx_blocks;
  bool accumulate;
  const uint16_t* dx_in;
  float* dW;
  float* db;
  uint16_t* dx;
  int* status;
};

constexpr int kChunk = 64;    // k staged at a time, eight per warp

template <bool Q8>
__global__ void __launch_bounds__(256) router_small_kernel(const SmallArgs a) {
  pdl_wait_and_trigger();
  __shared__ float4 A[kChunk][2];          // eight rows of A
  __shared__ uint8_t keep[kChunk];
  __shared__ float4 part[4][8][32];        // sums of half of the warps
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int blk = blockIdx.x;
  if (blk == 0 && tid == 0) *a.status = 0;
  if (blk >= a.dw_blocks + a.dx_blocks) {
    // db: 32 experts, eight warps over the tokens
    __shared__ float sums[8][32];
    const int e = (blk - a.dw_blocks - a.dx_blocks) * 32 + lane;
    float s = 0.f;
    if (e < a.E) {
#pragma unroll 8
      for (int t = warp; t < a.T; t += 8)
        if (!a.mask || __ldg(a.mask + t) != 0) s += __ldg(a.dl + static_cast<int64_t>(t) * a.E + e);
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && e < a.E) {
      for (int k = 1; k < 8; ++k) s += sums[k][lane];
      a.db[e] = a.accumulate ? a.db[e] + s : s;
    }
    return;
  }
  const bool is_dw = blk < a.dw_blocks;
  if (!is_dw) blk -= a.dw_blocks;
  const int i = (blk % a.col_blocks) * 128 + lane * 4, r0 = blk / a.col_blocks * 8;
  const int K = is_dw ? a.T : a.E, R = is_dw ? a.E : a.T;
  float* Af = reinterpret_cast<float*>(A);
  float4 acc[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < K; k0 += kChunk) {
    const int n = K - k0 < kChunk ? K - k0 : kChunk;
    // this warp's rows of B, loaded whether or not their tokens are live
    float4 b[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int kk = warp + 8 * u;
      b[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (kk < n && i < a.d)
        b[u] = is_dw ? router_row4<Q8>(a.rows, k0 + kk, i, a.d)
                     : __ldg(reinterpret_cast<const float4*>(a.W + static_cast<int64_t>(k0 + kk) * a.d + i));
    }
    __syncthreads();
    for (int v = tid; v < kChunk * 8; v += 256) {
      const int kk = is_dw ? v >> 3 : v & (kChunk - 1), r = is_dw ? v & 7 : v / kChunk;
      const int64_t t = is_dw ? k0 + kk : r0 + r;
      const int e = is_dw ? r0 + r : k0 + kk;
      const bool live = t < a.T && (!a.mask || __ldg(a.mask + t) != 0);
      Af[kk * 8 + r] = live && e < a.E ? __ldg(a.dl + t * a.E + e) : 0.f;
      if (r == 0) keep[kk] = is_dw ? live : kk < n;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int kk = warp + 8 * u;
      if (!keep[kk]) continue;   // a padded token's row may hold anything
      const float4 lo = A[kk][0], hi = A[kk][1];
      const float w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        acc[r].x = fmaf(w[r], b[u].x, acc[r].x);
        acc[r].y = fmaf(w[r], b[u].y, acc[r].y);
        acc[r].z = fmaf(w[r], b[u].z, acc[r].z);
        acc[r].w = fmaf(w[r], b[u].w, acc[r].w);
      }
    }
  }
  // warps 4..7 hand their sums to 0..3, those to warp r (row r) in order
  auto add = [](float4 x, float4 y) { return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w); };
  if (warp >= 4)
#pragma unroll
    for (int r = 0; r < 8; ++r) part[warp - 4][r][lane] = acc[r];
  __syncthreads();
  if (warp < 4)
#pragma unroll
    for (int r = 0; r < 8; ++r) part[warp][r][lane] = add(acc[r], part[warp][r][lane]);
  __syncthreads();
  if (i >= a.d || r0 + warp >= R) return;
  float4 s = add(add(part[0][warp][lane], part[1][warp][lane]), add(part[2][warp][lane], part[3][warp][lane]));
  const int64_t at = static_cast<int64_t>(r0 + warp) * a.d + i;
  if (is_dw) {
    float4* o = reinterpret_cast<float4*>(a.dW + at);
    *o = a.accumulate ? add(s, *o) : s;
  } else {
    // a padded token's row stays dx_in's (its sum may be zero times an infinity)
    const bool live = !a.mask || __ldg(a.mask + r0 + warp) != 0;
    if (!live) s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.dx_in) {
      const uint2 v = *reinterpret_cast<const uint2*>(a.dx_in + at);
      if (!live) {
        *reinterpret_cast<uint2*>(a.dx + at) = v;
        return;
      }
      s = add(s, make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                             __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u)));
    }
    const __nv_bfloat162 p = __floats2bfloat162_rn(s.x, s.y), q = __floats2bfloat162_rn(s.z, s.w);
    *reinterpret_cast<uint2*>(a.dx + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&p),
                                                      *reinterpret_cast<const uint32_t*>(&q));
  }
}

// Which path. Measured, one launch against the tensor cores (bf16 rows, d = 2880
// unless said): E = 4, d = 512: T = 144 9.0 against 11.3 us, T = 192 10.6 against
// 10.3; E = 32: 9.8 against 12.1 and 11.4 against 12.0; E = 64: 13.7 against 15.2
// and 16.2 against 15.4; E = 128: T = 64 10.9 against 15.7, T = 96 17.0 against 16.3,
// T = 128 18.7 against 16.4; E = 248: T = 64 21.2 against 19.6, T = 96 29 against 20.
bool few_tokens(int E, int T, int d) { return T <= (static_cast<int64_t>(E) * d > 1 << 18 ? 96 : 144); }

}  // namespace

size_t balance_scratch_bytes(int E, int T) {
  // a row for every cluster there may be: one more token per warp can take fewer
  // clusters, and a workspace for more tokens serves fewer too
  const int rows = T <= kBalOneCluster ? 1 : kBalClusters;
  return static_cast<size_t>(kBalClusters) * 12 + static_cast<size_t>(rows) * E * 8;
}

cudaError_t launch_balance_loss(const float* logits, const int32_t* topk_idx, const uint8_t* mask,
                                int E, int k, int T, float balance_coef, float z_coef,
                                float* stats, int32_t* counts, float* mean_probs, float* lse,
                                void* scratch, cudaStream_t st) {
  const int clusters = balance_clusters(T);
  const BalanceScratch sc = balance_scratch(scratch, E, clusters);
  const BalanceOut out{balance_coef, z_coef, stats, counts, mean_probs};
  int warps = balance_warps(T);
  if (warps * 32 < E) warps = (E + 31) / 32;   // a thread per expert
  auto go = [&](auto kernel) {
    return launch_kernel_cluster(kernel, dim3(clusters * kBalCluster), dim3(warps * 32), 0, kBalCluster,
                                 st, logits, topk_idx, mask, E, k, T, clusters, lse, sc, out);
  };
  const cudaError_t e = E % 4 == 0
                            ? (E <= 128 ? go(balance_partial_kernel<true, 4>) : go(balance_partial_kernel<true, 8>))
                            : (E <= 128 ? go(balance_partial_kernel<false, 4>) : go(balance_partial_kernel<false, 8>));
  if (e != cudaSuccess || clusters == 1) return e;
  pdl_launches() = true;
  int cols = 32;
  while (cols < E) cols *= 2;
  return launch_kernel(balance_finish_kernel, dim3(1), dim3(1024), 0, st, sc, clusters, E, cols, k, out);
}

cudaError_t launch_balance_backward(const float* logits, const float* lse, const int32_t* counts,
                                    const float* stats, const uint8_t* mask, int E, int k, int T,
                                    float balance_coef, float z_coef, const float* dloss,
                                    bool accumulate, float* dlogits, cudaStream_t st) {
  const int64_t b = (static_cast<int64_t>(T) + 7) / 8;
  const dim3 grid(b < 148 * 8 ? static_cast<int>(b) : 148 * 8);
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, grid, dim3(256), 0, st, logits, lse, counts, stats, mask, E, k, T,
                         balance_coef, z_coef, dloss, accumulate, dlogits);
  };
  if (E % 4 == 0) return E <= 128 ? go(balance_backward_kernel<true, 4>) : go(balance_backward_kernel<true, 8>);
  return E <= 128 ? go(balance_backward_kernel<false, 4>) : go(balance_backward_kernel<false, 8>);
}

cudaError_t launch_gate_backward(const uint16_t* dout, const float* yw, const int32_t* topk_idx,
                                 const float* topk_w, const uint8_t* mask, int E, int k, int T,
                                 int d, bool accumulate, float* dlogits, cudaStream_t st) {
  // A warp per token once there are sixteen tokens per SM, more for fewer tokens, at
  // most a thread for eight columns. At d = 2880: T = 8192, k = 4: 76 us with one
  // warp, 78 with four, 113 with twelve; T = 64, k = 8: 19, 12 and 12 us.
  int64_t warps = (148 * 16 + static_cast<int64_t>(T) - 1) / T;
  const int most = (d / 8 + 31) / 32;
  if (warps > most) warps = most;
  if (warps > kGateThreads / 32) warps = kGateThreads / 32;
  const int span = static_cast<int>(warps) * 32;
  const int spans = span >= 256 ? 1 : 256 / span;
  const int64_t blocks = (static_cast<int64_t>(T) + spans - 1) / spans;
  return launch_kernel(gate_backward_kernel, dim3(static_cast<unsigned>(blocks)), dim3(span * spans), 0, st,
                       dout, yw, topk_idx, topk_w, mask, E, k, T, d, span, accumulate, dlogits);
}

size_t router_grad_scratch_bytes(int E, int T, int d) {
  return few_tokens(E, T, d) ? 16 : router_grad_tc_scratch_bytes(E, T, d);
}

cudaError_t launch_router_backward(const RouterGradProblem& p, cudaStream_t st) {
  if (!few_tokens(p.E, p.T, p.d)) return launch_router_backward_tc(p, st);
  SmallArgs a;
  a.dl = p.dlogits;
  a.W = p.W_r;
  a.rows = RouterRows{p.x, p.q, p.scales, p.rstd, p.g};
  a.mask = p.mask;
  a.E = p.E;
  a.T = p.T;
  a.d = p.d;
  a.col_blocks = (p.d + 127) / 128;
  a.dw_blocks = p.dW ? (p.E + 7) / 8 * a.col_blocks : 0;
  a.dx_blocks = p.dx ? (p.T + 7) / 8 * a.col_blocks : 0;
  a.accumulate = p.accumulate;
  a.dx_in = p.dx_in;
  a.dW = p.dW;
  a.db = p.db;
  a.dx = p.dx;
  a.status = p.status;
  const int blocks = a.dw_blocks + a.dx_blocks + (p.db ? (p.E + 31) / 32 : 0);
  if (blocks == 0) return cudaMemsetAsync(p.status, 0, sizeof(int), st);   // dx of no tokens
  return p.q ? launch_kernel(router_small_kernel<true>, dim3(blocks), dim3(256), 0, st, a)
             : launch_kernel(router_small_kernel<false>, dim3(blocks), dim3(256), 0, st, a);
}

}  // namespace moe
