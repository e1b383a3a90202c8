// Linear attention of packed prompts on the CUDA cores.
#pragma once

#include "common.cuh"
#include "packed_attn.cuh"
#include "packed_step.cuh"

namespace sala {

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
