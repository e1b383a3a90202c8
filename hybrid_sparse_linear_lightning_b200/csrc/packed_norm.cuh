// QK-RMSNorm (and RoPE) of packed tokens.
//
//   y = x / sqrt(mean_d(x^2) + eps) * w                    per (token, head) row
//   (y_i, y_{i+d/2}) turned by p_t theta_i,  theta_i = base^(-2i/d)   where positions are given
//
// (QK normalisation in every layer: MiniCPM-SALA paper, summary; RoPE in the
// linear layers only: acgfav.com "SALA 混合架构".)  The rectangular prefill
// calls do the same inside their kernels, from one start position; here every
// token brings its own position, so prompts of different lengths and single
// decode tokens share one launch.
//
// Bound by memory: each row is read once and written once as bf16 (4 bytes of
// traffic per bf16 value).  A row is held by d/16 threads as two 8-element
// halves (a rotation pair each), so a warp reads whole rows, four at a time for
// each thread; the cosines and sines of a token are formed once in shared
// memory and serve all its heads.
//
// 32768 tokens, 32 + 32 heads of 128, RoPE: 209 us, 5.1 TB/s (78 % of the copy
// rate).  Rows of a thread in flight: 1 281 us, 2 253, 4 209, 8 531 (spills);
// CTAs of 256 threads 227 us, of 64 207; 8 or 16 tokens per CTA the same.  fp32 q
// and k (6 bytes per value): 262 us, 6.2 TB/s.
#pragma once

#include "common.cuh"
#include "prologue.cuh"

namespace sala {

constexpr int kQkNormThreads = 128;
constexpr int kQkNormMaxTokens = 4;    // tokens per CTA
constexpr int kQkNormUnroll = 4;       // rows of a thread in flight

// 8 consecutive values as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* f) const { load8(reinterpret_cast<const __nv_bfloat16*>(&u), f); }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kQkNormThreads)
qk_norm_kernel(const T* q, const T* k, const float* __restrict__ wq,
               const float* __restrict__ wk, const int32_t* __restrict__ pos,
               __nv_bfloat16* qn, __nv_bfloat16* kn, int tokens,
               int tok_per_cta, int Hq, int Hk, const __grid_constant__ RopeFreq rf, float eps) {
  constexpr int TPR = D / 16;
  constexpr int kRows = kQkNormThreads / TPR;
  constexpr int U = kQkNormUnroll;
  __shared__ __align__(16) float cs[kQkNormMaxTokens * D / 2];
  __shared__ __align__(16) float sn[kQkNormMaxTokens * D / 2];
  const long long tok0 = (long long)blockIdx.x * tok_per_cta;
  const int ntok = (int)min((long long)tok_per_cta, tokens - tok0);
  const int c = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  const int H = Hq + Hk;
  const int rows = ntok * H;
  // Row r of the CTA is head r % H of token r / H, q's heads first.  Every thread
  // runs the same number of passes (the row sums shuffle between a row's threads);
  // rows past the end repeat the last one and are not stored.
  Raw8<T> lo[U], hi[U];
  auto offset = [&](int r, int* tt, bool* is_k) {
    r = min(r, rows - 1);
    *tt = r / H;
    const int h = r - *tt * H;
    *is_k = h >= Hq;
    return *is_k ? ((tok0 + *tt) * Hk + (h - Hq)) * (long long)D : ((tok0 + *tt) * Hq + h) * (long long)D;
  };
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int tt;
      bool is_k;
      const long long off = offset(base + u * kRows + rg, &tt, &is_k);
      const T* src = (is_k ? k : q) + off + 8 * c;
      lo[u].load(src);
      hi[u].load(src + D / 2);
    }
  };
  load(0);      // on their way while the angles are formed
  if (pos) {
    // the angle is formed and reduced modulo 2 pi in fp64 (|p| < 2^31), so far
    // positions lose nothing, and evaluated in fp32 on [-pi, pi]
    for (int e = threadIdx.x; e < ntok * (D / 2); e += kQkNormThreads) {
      const double a = (double)pos[tok0 + e / (D / 2)] * rf.inv[e % (D / 2)];
      constexpr double kTwoPi = 6.283185307179586476925286766559;
      sincosf((float)(a - rint(a * (1.0 / kTwoPi)) * kTwoPi), &sn[e], &cs[e]);
    }
    __syncthreads();
  }
  float wlo[2][8], whi[2][8];
  load8(wq + 8 * c, wlo[0]);
  load8(wq + D / 2 + 8 * c, whi[0]);
  load8(wk + 8 * c, wlo[1]);
  load8(wk + D / 2 + 8 * c, whi[1]);
  for (int base = 0; base < rows; base += U * kRows) {
    if (base > 0) load(base);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = base + u * kRows + rg;
      int tt;
      bool is_k;
      const long long off = offset(r, &tt, &is_k);
      float x[8], y[8];
      lo[u].get(x);
      hi[u].get(y);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, TPR);
      const float inv = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= inv * (is_k ? wlo[1][e] : wlo[0][e]);
        y[e] *= inv * (is_k ? whi[1][e] : whi[0][e]);
      }
      if (pos) rope_pair8(x, y, cs + tt * (D / 2) + 8 * c, sn + tt * (D / 2) + 8 * c);
      if (r < rows) {
        __nv_bfloat16* dst = (is_k ? kn : qn) + off + 8 * c;
        store8(dst, x);
        store8(dst + D / 2, y);
      }
    }
  }
}

}  // namespace sala
