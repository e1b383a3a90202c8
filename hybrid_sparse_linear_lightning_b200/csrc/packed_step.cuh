// Linear attention for one token of each request, states in a slot pool.
//
//   S <- lam_h S + k^T v  (fp32, in place),   out = sigmoid(gate) * scale * q S
//
// (Linear layers keep a constant-size state: MiniCPM-SALA paper, section 2.1.)
// Bound by memory: a state of d x d fp32 is read and written once per (row,
// head), 128 KB at d = 128, and everything else is a few KB.  A CTA holds COLS
// value columns of one state; its threads load their part of the state before
// anything else, so that all of it is in flight at once.  256 requests, 32 heads
// of 128: 168 us, 6.47 TB/s (99 % of the copy rate).  Where whole states would
// leave SMs idle, a CTA takes 32 columns (4 requests, 4 heads of 64: 1.9 us).
#pragma once

#include "common.cuh"

namespace sala {

constexpr int kStepThreads = 256;

// Row r of a batch may use its slot: inside [0, n_slots), and no earlier row
// names it too (the first one has it).  A negative slot marks a padded row.
// All threads of the CTA call this; a slot that is refused sets the bounds bit.
__device__ __forceinline__ int take_slot(const int32_t* slots, int r, int n_slots) {
  if (!slots) return r;
  const int s = slots[r];
  if (s < 0) return -1;
  if (s >= n_slots) {
    if (threadIdx.x == 0) set_status(kStatusBounds);
    return -1;
  }
  bool dup = false;
  for (int i = threadIdx.x; i < r; i += blockDim.x) dup |= slots[i] == s;
  if (__syncthreads_or(dup)) {
    if (threadIdx.x == 0) set_status(kStatusBounds);
    return -1;
  }
  return s;
}

template <typename T, int D, int COLS>
__global__ void __launch_bounds__(kStepThreads)
linear_step_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                   const T* __restrict__ v, const T* __restrict__ gate,
                   const float* __restrict__ lambda, const int32_t* __restrict__ slots,
                   float* __restrict__ state, T* __restrict__ out, int H, int n_slots,
                   float scale) {
  constexpr int LPR = COLS / 4;                  // lanes that share a state row
  constexpr int kRows = kStepThreads / LPR;      // rows of one pass
  constexpr int kPass = D / kRows;
  static_assert(kPass >= 1, "a pass covers at most the state's rows");
  __shared__ float sq[D], sk[D];
  __shared__ float4 red[kStepThreads / 32][LPR];
  constexpr int kSplit = D / COLS;
  const int part = blockIdx.x % kSplit;
  const int h = (blockIdx.x / kSplit) % H;
  const int r = blockIdx.x / (kSplit * H);
  const int slot = take_slot(slots, r, n_slots);
  if (slot < 0) return;
  const int tid = threadIdx.x, lc = tid % LPR, lr = tid / LPR;
  const long long row = ((long long)r * H + h) * D;
  float* S = state + ((long long)slot * H + h) * D * D + part * COLS + 4 * lc;
  float4 s[kPass];
#pragma unroll
  for (int i = 0; i < kPass; ++i)
    s[i] = *reinterpret_cast<const float4*>(S + (long long)(i * kRows + lr) * D);
  if (tid < D) {
    sq[tid] = to_f32(q[row + tid]);
    sk[tid] = to_f32(k[row + tid]);
  }
  const T* vp = v + row + part * COLS + 4 * lc;
  const float4 vv = make_float4(to_f32(vp[0]), to_f32(vp[1]), to_f32(vp[2]), to_f32(vp[3]));
  const float lam = lambda[h];
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    const int d = i * kRows + lr;
    const float kd = sk[d], qd = sq[d];
    s[i].x = fmaf(lam, s[i].x, kd * vv.x);
    s[i].y = fmaf(lam, s[i].y, kd * vv.y);
    s[i].z = fmaf(lam, s[i].z, kd * vv.z);
    s[i].w = fmaf(lam, s[i].w, kd * vv.w);
    o.x = fmaf(qd, s[i].x, o.x);
    o.y = fmaf(qd, s[i].y, o.y);
    o.z = fmaf(qd, s[i].z, o.z);
    o.w = fmaf(qd, s[i].w, o.w);
    *reinterpret_cast<float4*>(S + (long long)d * D) = s[i];
  }
  // sum over the rows: lanes that hold the same columns, then the warps, in a fixed order
#pragma unroll
  for (int m = 16; m >= LPR; m >>= 1) {
    o.x += __shfl_xor_sync(0xffffffffu, o.x, m);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, m);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, m);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, m);
  }
  if ((tid & 31) < LPR) red[tid >> 5][lc] = o;
  __syncthreads();
  if (tid < COLS) {
    const float* f = reinterpret_cast<const float*>(red);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kStepThreads / 32; ++w) sum += f[w * COLS + tid];
    const long long at = row + part * COLS + tid;
    out[at] = from_f32<T>(sigmoidf_(to_f32(gate[at])) * scale * sum);
  }
}

}  // namespace sala
