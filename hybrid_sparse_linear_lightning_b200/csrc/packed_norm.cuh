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
// halves (a rotation pair each), so a warp reads whole 256-byte rows; the
// cosines and sines of a token are formed once in shared memory and serve all
// its heads.
#pragma once

#include "common.cuh"
#include "prologue.cuh"

namespace sala {

constexpr int kQkNormThreads = 256;
constexpr int kQkNormMaxTokens = 4;    // tokens per CTA

template <typename T, int D>
__global__ void __launch_bounds__(kQkNormThreads)
qk_norm_kernel(const T* __restrict__ q, const T* __restrict__ k, const float* __restrict__ wq,
               const float* __restrict__ wk, const int32_t* __restrict__ pos,
               __nv_bfloat16* __restrict__ qn, __nv_bfloat16* __restrict__ kn, int tokens,
               int tok_per_cta, int Hq, int Hk, const __grid_constant__ RopeFreq rf, float eps) {
  constexpr int TPR = D / 16;
  constexpr int kRows = kQkNormThreads / TPR;
  __shared__ __align__(16) float cs[kQkNormMaxTokens * D / 2];
  __shared__ __align__(16) float sn[kQkNormMaxTokens * D / 2];
  const long long tok0 = (long long)blockIdx.x * tok_per_cta;
  const int ntok = (int)min((long long)tok_per_cta, tokens - tok0);
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
  const int c = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  const int H = Hq + Hk;
  float wlo[2][8], whi[2][8];
  load8(wq + 8 * c, wlo[0]);
  load8(wq + D / 2 + 8 * c, whi[0]);
  load8(wk + 8 * c, wlo[1]);
  load8(wk + D / 2 + 8 * c, whi[1]);
  const int rows = ntok * H;
  // every thread runs the same number of passes (the row sums shuffle between
  // a row's threads); rows past the end repeat row 0 and are not stored
  for (int base = 0; base < rows; base += kRows) {
    const int r = base + rg;
    const bool active = r < rows;
    const int rc = active ? r : 0;
    const int tt = rc / H, h = rc % H;
    const bool is_k = h >= Hq;
    const long long off = is_k ? ((tok0 + tt) * Hk + (h - Hq)) * (long long)D
                               : ((tok0 + tt) * Hq + h) * (long long)D;
    const T* src = (is_k ? k : q) + off;
    float lo[8], hi[8];
    load8(src + 8 * c, lo);
    load8(src + D / 2 + 8 * c, hi);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(lo[e], lo[e], fmaf(hi[e], hi[e], ss));
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, TPR);
    const float inv = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] *= inv * (is_k ? wlo[1][e] : wlo[0][e]);
      hi[e] *= inv * (is_k ? whi[1][e] : whi[0][e]);
    }
    if (pos) rope_pair8(lo, hi, cs + tt * (D / 2) + 8 * c, sn + tt * (D / 2) + 8 * c);
    if (active) {
      __nv_bfloat16* dst = (is_k ? kn : qn) + off;
      store8(dst + 8 * c, lo);
      store8(dst + D / 2 + 8 * c, hi);
    }
  }
}

}  // namespace sala
