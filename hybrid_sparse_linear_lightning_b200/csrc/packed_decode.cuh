// One decode token of each request over a shared prefix and the request's own
// cache: softmax attention in two launches.
//
//   out = sigmoid(gate) softmax(scale q [K_prefix, K_own, k_new]^T) [V_prefix, V_own, v_new]
//
//   1. prefix_attn_kernel: the rows of all requests together against the
//      prefix on the tensor cores (packed_attn.cuh), its keys split so that the
//      units fill the card; leaves O, maximum and sum per row and split.
//   2. own_attn_kernel: a cluster per (request, kv head, 16 q heads) walks the
//      request's own keys (the new token's among them), joins the cluster's
//      parts through distributed shared memory with those of the prefix, gates,
//      and appends the token to the cache.
//
// A prefix that takes little to read once for every request (24 MB in all), and
// that gives no warp more than 18 steps of 16 keys, is walked by the second kernel
// with the own keys, and there is no first: 5 requests over 700 tokens 5.5 us against
// 9.0, 16 over 1000 (16 MB) 9.4 against 11.4, 8 over 4000 (33 MB) 14.8 against 14.7,
// 16 over 2000 of 8 kv heads (131 MB) 42 against 16.  Few requests have few clusters,
// whose warps take 0.7 us a step: one request of 2 kv heads over 8000 tokens (16
// steps) 17.7 us against 21.6, over 10000 (20) 20.4 against 17.9, over 20000 (39) 33
// against 24; one kv head over 32768 (64) 49 against 25.
//
// The second launch starts while the first runs out (programmatic dependent
// launch) and waits for it before it reads the prefix's parts.
//
// The own part is bound by memory: every key and value is used by one request
// alone, 4 d bytes each, against 16 padded rows on warp-level matrix
// instructions (m16n8k16).  A group of more than 16 q heads reads them once per 16:
// 12 requests with up to 16383 tokens of their own, 8 kv heads of 128, in 82 us for
// groups of 16, 118 of 17, 124 of 32, 210 of 64 and 376 of 128 (the rereads hit L2
// in part: 4.2 TB/s of keys asked for at 16, 7.2 at 128).  Each warp keeps kOwnStages steps of 16 keys in
// flight with asynchronous copies of its own, so warps never wait for one
// another before the final join.
//
// Measured, d = 128: 64 requests over a prefix of 32768 (32 q heads, 2 kv heads)
// 58 us, of which the prefix 35 (34 GFLOP); 12 requests with up to 16383 tokens of
// their own (8 kv heads) 75 us, 4.5 TB/s.  Clusters of 8 are the best size for the
// long ones (2: 115 us, 4: 78, 16: 119: sixteen CTAs seldom find places at once),
// and of 2 for caches of 1024 (8: 95 us); without the early start 62 and 82 us.
// Two or three steps in flight make no difference.
#pragma once

#include "common.cuh"
#include "packed_attn.cuh"
#include "packed_step.cuh"

namespace sala {

constexpr int kOwnWarps = 4;
constexpr int kOwnStages = 3;
constexpr int kOwnMaxSplits = 64;      // parts of the prefix
constexpr int kOwnMaxCluster = 8;
constexpr int kOwnMaxWalk = 18;        // steps of a warp over a walked prefix

template <int D>
struct OwnLayout {
  static constexpr int kStage = 2 * 16 * D * 2;                    // K, then V: 16 keys
  static constexpr int kWarp = kOwnStages * kStage;
  static constexpr int kRing = 0;                                  // reused for the warps' O, [warp][16][D] fp32
  static constexpr int kO = kOwnWarps * kWarp;                     // the CTA's O, [16][D] fp32
  static constexpr int kMl = kO + 16 * D * 4;                      // [16] (m, l) of the CTA
  static constexpr int kWarpMl = kMl + 16 * 8;                     // [warp][16] (m, l)
  static constexpr int kW = kWarpMl + kOwnWarps * 16 * 8;          // weights [16][cluster + splits]
  static constexpr int kBytes = kW + 16 * (kOwnMaxCluster + kOwnMaxSplits) * 4;
  static_assert(kWarp >= 16 * D * 4, "a warp's O fits into its ring");
};

__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c (16 x 8) += a (16 x 16, row) b (16 x 8, column)
__device__ __forceinline__ void mma16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Block: (split, pair of row tiles, kv head), heads fastest.
template <int D>
__global__ void __launch_bounds__(kPaThreads, 1)
prefix_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, float* __restrict__ part_o,
                   float2* __restrict__ part_ml, int batch, int Hq, int Hkv, int Tt, int pairs,
                   int prefix, int split_blocks, float sl2) {
  extern __shared__ __align__(1024) uint8_t smem_pp[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_pp) + 1023) & ~uintptr_t(1023));
  pdl_launch();
  pa_setup<D>(qmap, kmap, vmap, smem);
  __syncthreads();
  PaJob job;
  job.live = 1;
  job.g = blockIdx.x % Hkv;
  const int pair = (blockIdx.x / Hkv) % pairs;
  job.split = blockIdx.x / (Hkv * pairs);
  job.krow = job.split * split_blocks * kPaBlock;
  job.n_keys = min(prefix - job.krow, split_blocks * kPaBlock);
  const int nb = (job.n_keys + kPaBlock - 1) / kPaBlock;
  for (int t = 0; t < 2; ++t) {
    job.tok[t] = (2 * pair + t) * Tt;
    job.ntok[t] = max(0, min(Tt, batch - job.tok[t]));
    job.pos[t] = 0;
    job.nb[t] = job.ntok[t] > 0 ? nb : 0;
  }
  job.fix_from = nb;      // rows behind the prefix arrive as zeros
  pa_run<D, false>(qmap, kmap, vmap, smem, job, PaPrefix{part_o, part_ml}, batch, Hq, Hkv, Tt, sl2);
}

// Grid: cluster ranks fastest, then 16-row tiles of the group, kv heads, requests.
template <int D>
__global__ void __launch_bounds__(32 * kOwnWarps, 2)
own_attn_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                const __nv_bfloat16* __restrict__ v, const __nv_bfloat16* __restrict__ gate,
                const __nv_bfloat16* __restrict__ pk, const __nv_bfloat16* __restrict__ pv,
                __nv_bfloat16* __restrict__ kc, __nv_bfloat16* __restrict__ vc,
                const int32_t* __restrict__ lens, const int32_t* __restrict__ slots,
                const float* part_o, const float2* part_ml, __nv_bfloat16* __restrict__ out, int batch, int Hq, int Hkv, int mtiles, int prefix, int n_split,
                long long cap, int n_slots, float sl2) {
  using L = OwnLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem_ow[];
  const uint32_t cs = cluster_size(), rank = cluster_rank();
  const int unit = blockIdx.x / cs;
  const int mt = unit % mtiles, g = (unit / mtiles) % Hkv, b = unit / (mtiles * Hkv);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = Hq / Hkv;
  const int slot = take_slot(slots, b, n_slots);
  const int len = slot >= 0 ? lens[b] : -1;
  if (slot < 0 || len < 0 || len >= cap) {
    if (slot >= 0 && tid == 0) set_status(kStatusBounds);
    pdl_wait();
    return;
  }
  const int rows = min(16, G - 16 * mt);                       // q heads of this tile
  const long long row0 = (long long)b * Hq + g * G + 16 * mt;  // first (request, head) row
  const long long st = (long long)Hkv * D;
  __nv_bfloat16* ck = kc + slot * cap * st + g * D;
  __nv_bfloat16* cv = vc + slot * cap * st + g * D;
  const __nv_bfloat16* nk = k + ((long long)b * Hkv + g) * D;
  const __nv_bfloat16* nv = v + ((long long)b * Hkv + g) * D;

  // steps of 16 keys, dealt to the cluster's warps in turn: those of the prefix
  // (where it is not in parts), then the request's own with the new token's
  const int p_steps = (prefix + 15) / 16;
  const int n_steps = p_steps + len / 16 + 1;
  const int wstride = kOwnWarps * cs, first = rank * kOwnWarps + warp;
  const int mine = first < n_steps ? (n_steps - first + wstride - 1) / wstride : 0;
  uint8_t* ring = smem_ow + L::kRing + warp * L::kWarp;
  const uint32_t ring_a = tc::smem_u32(ring);
  constexpr int CH = D / 8;                 // 16-byte chunks of a row
  constexpr int RP = 32 / CH;               // rows of one pass of the warp
  auto load_step = [&](int i) {
    if (i < mine) {
      const int step = first + i * wstride;
      const bool own = step >= p_steps;
      const int key0 = (own ? step - p_steps : step) * 16;
      const int end = own ? len : prefix - 1;            // the last key there is
      const __nv_bfloat16 *kb = own ? ck : pk + g * D, *vb = own ? cv : pv + g * D;
      const uint32_t dst = ring_a + (i % kOwnStages) * L::kStage;
      const int c = lane % CH;
#pragma unroll
      for (int p = 0; p < 16 / RP; ++p) {
        const int r = p * RP + lane / CH, key = key0 + r;
        const bool is_new = own && key == len;
        const long long off = (long long)min(key, end) * st + 8 * c;
        const __nv_bfloat16* ks = is_new ? nk + 8 * c : kb + off;
        const __nv_bfloat16* vs = is_new ? nv + 8 * c : vb + off;
        const uint32_t at = dst + r * (D * 2) + ((c ^ (r & 7)) << 4);
        const int n = key <= end ? 16 : 0;   // rows past the end: zeros, nothing read
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(ks), "r"(n) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + 16 * D * 2), "l"(vs), "r"(n)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kOwnStages - 1; ++i) load_step(i);

  // Q fragments: rows lane / 4 and lane / 4 + 8, columns 16 kk + 2 (lane % 4) + {0, 1, 8, 9}
  uint32_t qf[D / 16][4];
  {
    const int r = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = r + 8 * (i & 1), cc = 16 * kk + c + 8 * (i >> 1);
        qf[kk][i] = rr < rows ? *reinterpret_cast<const uint32_t*>(q + (row0 + rr) * D + cc) : 0u;
      }
  }
  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
  float m[2] = {kPaLowest, kPaLowest}, l[2] = {0.f, 0.f};

  for (int i = 0; i < mine; ++i) {
    load_step(i + kOwnStages - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kOwnStages - 1) : "memory");
    __syncwarp();
    const uint32_t ks = ring_a + (i % kOwnStages) * L::kStage, vs = ks + 16 * D * 2;
    const int step = first + i * wstride;
    const bool own = step >= p_steps;
    const int left = (own ? len : prefix - 1) - (own ? step - p_steps : step) * 16;    // the last key's number here
    float s[2][4] = {};
    // matrices of one ldmatrix: keys 0-7 / 8-15 (bit 3 of the lane), column halves (bit 4)
    const int kr = (lane & 7) + (lane & 8), kh = lane >> 4;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t bf[4];
      ldsm4(bf, ks + kr * (D * 2) + (((2 * kk + kh) ^ (kr & 7)) << 4));
      mma16(s[0], qf[kk], bf[0], bf[2]);
      mma16(s[1], qf[kk], bf[1], bf[3]);
    }
    const int c0 = 2 * (lane & 3);
    float mx[2] = {kPaLowest, kPaLowest};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = c0 + 8 * n + (e & 1) <= left ? s[n][e] * sl2 : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
    }
    if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float mn = fmaxf(m[h], mx[h]);
        const float f = tc::ex2_approx(m[h] - mn);
        m[h] = mn;
        l[h] *= f;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[n][2 * h] *= f;
          o[n][2 * h + 1] *= f;
        }
      }
    }
    uint32_t pf[4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = tc::ex2_approx(s[n][e] - m[e >> 1]);
      l[0] += p[0] + p[1];
      l[1] += p[2] + p[3];
      __nv_bfloat162 a = __floats2bfloat162_rn(p[0], p[1]), c = __floats2bfloat162_rn(p[2], p[3]);
      pf[2 * n] = *reinterpret_cast<uint32_t*>(&a);
      pf[2 * n + 1] = *reinterpret_cast<uint32_t*>(&c);
    }
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t bf[4];
      ldsm4_t(bf, vs + kr * (D * 2) + (((2 * n + kh) ^ (kr & 7)) << 4));
      mma16(o[2 * n], pf, bf[0], bf[1]);
      mma16(o[2 * n + 1], pf, bf[2], bf[3]);
    }
    __syncwarp();
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  // ---- join the warps of the CTA
  __syncwarp();
  float* wo = reinterpret_cast<float*>(ring);                  // [16][D]
  float2* wml = reinterpret_cast<float2*>(smem_ow + L::kWarpMl);
  {
    const int r = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(wo + (r + 8 * h) * D + 8 * n + c) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
    if ((lane & 3) == 0) {
      wml[warp * 16 + r] = make_float2(m[0], l[0]);
      wml[warp * 16 + r + 8] = make_float2(m[1], l[1]);
    }
  }
  // the token enters the cache (nothing reads row `len` there: its key and
  // value above came from k and v)
  if (mt == 0 && rank == 0 && tid < 2 * CH) {
    const int c = tid % CH;
    const uint4 u = *reinterpret_cast<const uint4*>((tid < CH ? nk : nv) + 8 * c);
    *reinterpret_cast<uint4*>((tid < CH ? ck : cv) + (long long)len * st + 8 * c) = u;
  }
  __syncthreads();
  float2* cml = reinterpret_cast<float2*>(smem_ow + L::kMl);
  float* co = reinterpret_cast<float*>(smem_ow + L::kO);
  for (int e = tid; e < 16 * D / 4; e += 32 * kOwnWarps) {
    const int r = e / (D / 4);
    float M = kPaLowest;
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) M = fmaxf(M, wml[w * 16 + r].x);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) {
      const float2 x = wml[w * 16 + r];
      const float f = tc::ex2_approx(x.x - M);
      const float4 y = *reinterpret_cast<const float4*>(smem_ow + L::kRing + w * L::kWarp + e * 16);
      a.x = fmaf(f, y.x, a.x);
      a.y = fmaf(f, y.y, a.y);
      a.z = fmaf(f, y.z, a.z);
      a.w = fmaf(f, y.w, a.w);
      sum = fmaf(f, x.y, sum);
    }
    *reinterpret_cast<float4*>(co + 4 * e) = a;
    if (e % (D / 4) == 0) cml[r] = make_float2(M, sum);
  }
  cluster_sync();
  // ---- join the cluster's parts and the prefix's: weights per row, then a
  // slice of the 16 x D outputs per CTA
  pdl_wait();
  float* wts = reinterpret_cast<float*>(smem_ow + L::kW);      // [16][parts]
  const int parts = cs + n_split;
  const long long psz = (long long)batch * Hq;
  {
    const int r = tid >> 3, sub = tid & 7;
    const uint32_t ml_a = tc::smem_u32(cml);
    auto get = [&](int p) {
      if (p < (int)cs) return ld_cluster2(map_rank(ml_a + r * 8, p));
      return r < rows ? __ldcg(part_ml + (p - cs) * psz + row0 + r) : make_float2(kPaLowest, 0.f);
    };
    float M = kPaLowest;
    for (int p = sub; p < parts; p += 8) M = fmaxf(M, get(p).x);
#pragma unroll
    for (int x = 4; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x, 8));
    float sum = 0.f;
    for (int p = sub; p < parts; p += 8) {
      const float2 y = get(p);
      const float f = tc::ex2_approx(y.x - M);
      wts[r * parts + p] = f;
      sum = fmaf(f, y.y, sum);
    }
#pragma unroll
    for (int x = 4; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x, 8);
    const float inv = 1.f / sum;
    __syncwarp();
    for (int p = sub; p < parts; p += 8) wts[r * parts + p] *= inv;
  }
  __syncthreads();
  const int per = 16 * D / 4 / cs;
  const uint32_t co_a = tc::smem_u32(co);
  for (int e = rank * per + tid; e < (int)(rank + 1) * per; e += 32 * kOwnWarps) {
    const int r = e / (D / 4), c = 4 * (e % (D / 4));
    if (r >= rows) continue;
    const float* w = wts + r * parts;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float f, const float4& y) {
      a.x = fmaf(f, y.x, a.x);
      a.y = fmaf(f, y.y, a.y);
      a.z = fmaf(f, y.z, a.z);
      a.w = fmaf(f, y.w, a.w);
    };
    const float* po = part_o + (row0 + r) * D + c;
#pragma unroll 8
    for (int p = 0; p < n_split; ++p) add(w[cs + p], __ldcg(reinterpret_cast<const float4*>(po + p * psz * D)));
    for (uint32_t p = 0; p < cs; ++p) add(w[p], ld_cluster4(map_rank(co_a + 16 * e, p)));
    const long long at = (row0 + r) * D + c;
    const uint2 gr = *reinterpret_cast<const uint2*>(gate + at);
    const float2 g0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&gr.x));
    const float2 g1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&gr.y));
    __nv_bfloat162 r0 = __floats2bfloat162_rn(sigmoidf_(g0.x) * a.x, sigmoidf_(g0.y) * a.y);
    __nv_bfloat162 r1 = __floats2bfloat162_rn(sigmoidf_(g1.x) * a.z, sigmoidf_(g1.y) * a.w);
    *reinterpret_cast<uint2*>(out + at) =
        make_uint2(*reinterpret_cast<uint32_t*>(&r0), *reinterpret_cast<uint32_t*>(&r1));
  }
  cluster_sync();       // no CTA leaves while another reads its shared memory
}

}  // namespace sala
