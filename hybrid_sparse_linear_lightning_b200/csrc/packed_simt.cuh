// Packed-batch attention on the CUDA cores: one warp per (row, q head), 32
// keys at a time with a running maximum and sum.
#pragma once

#include "common.cuh"
#include "packed_attn.cuh"
#include "packed_step.cuh"

namespace sala {

constexpr int kPkSimtWarps = 8;

// Running softmax state of one row: lane l holds columns [l D/32, (l+1) D/32).
template <int D>
struct RowSoftmax {
  static constexpr int E = D / 32;
  float m = -INFINITY, l = 0.f, o[E] = {};

  // keys / values of rows `n` (<= 32) starting at kp / vp, rows `stride` apart
  __device__ __forceinline__ void add(const float* qs, const __nv_bfloat16* kp,
                                      const __nv_bfloat16* vp, long long stride, int n, float sl2) {
    const int lane = threadIdx.x & 31;
    float x = -INFINITY;
    if (lane < n) {
      const __nv_bfloat16* kr = kp + lane * stride;
      float dot = 0.f;
      for (int c = 0; c < D; c += 8) {
        float f[8];
        load8(kr + c, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot = fmaf(qs[c + e], f[e], dot);
      }
      x = dot * sl2;
    }
    const float mn = fmaxf(m, warp_max(x));
    const float f = mn == -INFINITY ? 1.f : exp2f(m - mn);
    const float p = lane < n ? exp2f(x - mn) : 0.f;
    m = mn;
    l = l * f + warp_sum(p);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f;
    for (int j = 0; j < n; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(pj, to_f32(vp[j * stride + lane * E + e]), o[e]);
    }
  }
};

template <int D>
__global__ void __launch_bounds__(32 * kPkSimtWarps)
prefix_simt_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                   const __nv_bfloat16* __restrict__ v, const __nv_bfloat16* __restrict__ gate,
                   const __nv_bfloat16* __restrict__ pk, const __nv_bfloat16* __restrict__ pv,
                   __nv_bfloat16* __restrict__ kc, __nv_bfloat16* __restrict__ vc,
                   const int32_t* __restrict__ lens, const int32_t* __restrict__ slots,
                   __nv_bfloat16* __restrict__ out, int Hq, int Hkv, int prefix, long long cap,
                   int n_slots, float sl2) {
  __shared__ float qs[kPkSimtWarps][D];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y, h = blockIdx.x * kPkSimtWarps + w;
  const int slot = take_slot(slots, b, n_slots);
  if (slot < 0) return;
  const int len = lens[b];
  if (len < 0 || len >= cap) {
    if (threadIdx.x == 0) set_status(kStatusBounds);
    return;
  }
  if (h >= Hq) return;
  const int G = Hq / Hkv, g = h / G;
  const long long row = (long long)b * Hq + h;
  constexpr int E = D / 32;
  for (int e = 0; e < E; ++e) qs[w][lane * E + e] = to_f32(q[row * D + lane * E + e]);
  __syncwarp();
  RowSoftmax<D> a;
  const long long st = (long long)Hkv * D;
  for (int j = 0; j < prefix; j += 32)
    a.add(qs[w], pk + j * st + g * D, pv + j * st + g * D, st, min(32, prefix - j), sl2);
  const __nv_bfloat16 *ck = kc + slot * cap * st + g * D, *cv = vc + slot * cap * st + g * D;
  for (int j = 0; j < len; j += 32) a.add(qs[w], ck + j * st, cv + j * st, st, min(32, len - j), sl2);
  const long long nrow = ((long long)b * Hkv + g) * D;
  a.add(qs[w], k + nrow, v + nrow, st, 1, sl2);
  for (int e = 0; e < E; ++e) {
    const long long at = row * D + lane * E + e;
    out[at] = __float2bfloat16_rn(sigmoidf_(to_f32(gate[at])) * a.o[e] / a.l);
    if (h % G == 0) {
      kc[(slot * cap + len) * st + g * D + lane * E + e] = k[nrow + lane * E + e];
      vc[(slot * cap + len) * st + g * D + lane * E + e] = v[nrow + lane * E + e];
    }
  }
}

// The recurrence token by token: one CTA per (sequence, head, 32 value columns),
// the state in registers (thread: one column, D / 8 rows).
template <int D>
__global__ void __launch_bounds__(256)
linear_packed_simt_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                          const __nv_bfloat16* __restrict__ v,
                          const __nv_bfloat16* __restrict__ gate,
                          const float* __restrict__ lambda, const int32_t* __restrict__ cu,
                          const int32_t* __restrict__ slots, const float* __restrict__ state_in,
                          float* __restrict__ state_out, __nv_bfloat16* __restrict__ out,
                          int tokens, int H, int n_slots, float scale) {
  constexpr int R = D / 8;
  __shared__ float sq[D], sk[D], red[8][32];
  const int part = blockIdx.x % (D / 32), h = (blockIdx.x / (D / 32)) % H;
  const int i = blockIdx.x / (D / 32 * H);
  const int s0 = cu[i], s1 = cu[i + 1];
  if (!seq_ok(cu, i, tokens)) {
    if (threadIdx.x == 0) set_status(kStatusBounds);
    return;
  }
  const int slot = take_slot(slots, i, n_slots);
  const int c = threadIdx.x & 31, rg = threadIdx.x >> 5;
  const long long sbase = ((long long)slot * H + h) * D * D + part * 32 + c;
  float S[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    S[r] = state_in && slot >= 0 ? state_in[sbase + (long long)(rg * R + r) * D] : 0.f;
  const float lam = lambda[h];
  for (int t = s0; t < s1; ++t) {
    const long long row = ((long long)t * H + h) * D;
    __syncthreads();
    if (threadIdx.x < D) {
      sq[threadIdx.x] = to_f32(q[row + threadIdx.x]);
      sk[threadIdx.x] = to_f32(k[row + threadIdx.x]);
    }
    const float vv = to_f32(v[row + part * 32 + c]);
    __syncthreads();
    float o = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      S[r] = fmaf(lam, S[r], sk[rg * R + r] * vv);
      o = fmaf(sq[rg * R + r], S[r], o);
    }
    red[rg][c] = o;
    __syncthreads();
    if (rg == 0) {
      float sum = 0.f;
      for (int w = 0; w < 8; ++w) sum += red[w][c];
      const long long at = row + part * 32 + c;
      out[at] = __float2bfloat16_rn(sigmoidf_(to_f32(gate[at])) * scale * sum);
    }
  }
  if (state_out && slot >= 0)
#pragma unroll
    for (int r = 0; r < R; ++r) state_out[sbase + (long long)(rg * R + r) * D] = S[r];
}

}  // namespace sala
