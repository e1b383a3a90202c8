// Softmax attention of packed rows on the 5th-generation tensor cores: the
// dense form of the sparse layer over packed prompts, and the part of a shared
// prefix in a decode step.
//
//   out_r = sum_u p_ru v_u / sum_u p_ru,   p_ru = exp(scale q_r k_u - m_r)
//
// (Exact attention of the sparse layer: acgfav.com "SALA 混合架构"; output gate:
// MiniCPM-SALA paper, summary.)  A CTA holds 256 query rows of one kv head in
// two tiles of 128: row r of a tile is q head g G + r % G of token r / G, so
// all heads of a group share each K / V tile that is fetched, whatever the
// group size.  Keys come in blocks of 128:
//
//   S_t = Q_t K_j^T       (tcgen05, M = N = 128, fp32 in TMEM)
//   P_t = 2^(S_t sl2 - m) (one row per thread; bf16 pairs over S_t's columns)
//   O_t += P_t V_j        (tcgen05, A from TMEM)
//
// The two tiles take turns: while the softmax of one runs, the tensor core
// multiplies for the other.  The issue order per tile is S(0), PV(0), S(1),
// PV(1), ...: tcgen05.mma of one thread execute in order, so S(i+1) may
// overwrite P(i), and S(i+1) being complete says that PV(i) is too.  The
// running maximum is raised (O and l rescaled) only when a row's maximum grew
// by more than 2^8.  P is rounded to bf16 for its product, which is of the size
// of the output's own rounding; l sums the weights before that, in fp32.
//
// Isolation: a masked key has weight 0, but 0 x NaN and 0 x infinity are NaN
// on the tensor core.  In the blocks that hold masked keys (those on the
// diagonal and at a sequence's end), two warps go over the V tile first: rows
// past the end become 0, and so do non-finite values, which the epilogue then
// adds to the rows that do see them.
//
// Bound by the tensor core and, with it, the exponentials (128 x 128 of them
// per tile and block take as long as its two products).  One prompt of 32768
// tokens, 32 q heads over 2 kv heads, d = 128: 7.6 ms, 1160 TFLOP/s, 72 % of what
// this card's library product of 8192^3 reaches in a burst and 84 % of what it
// sustains.  Measured around it: P in one piece instead of two halves 7.8 ms;
// 1, 3 and 4 of 8 pairs of exponentials on the FMA pipe 7.67, 7.56 and 7.89 ms
// (none: 7.63); logits read from TMEM 32 at a time in rolled loops, without the 128
// registers, 8.2 to 8.4 ms.  Short prompts cost the set-up: 333 tokens in 6
// prompts take 9 us in one wave, 1.8 us until the first key block has landed and
// 1.3 us per block.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace sala {

constexpr int kPaThreads = 384;
constexpr int kPaBlock = 128;                // keys per block
constexpr int kPaRegsLow = 72, kPaRegsHigh = 216;
constexpr float kPaRescale = 8.0f;           // log2 units
constexpr float kPaLowest = -3.402823466e38f;

template <int D>
struct PaLayout {
  static constexpr int kAtoms = D / 64;
  static constexpr int kTile = 128 * D * 2;          // Q, K or V tile: atoms of 128 rows x 128 B
  static constexpr int kSlots = D == 128 ? 5 : 8;    // ring of K and V tiles
  static constexpr int kRing = 2 * kTile;
  static constexpr int kBar = kRing + kSlots * kTile;
  // q_full, ring_full[], ring_empty[], s_full[2], p_half[2], p_full[2], v_ready[3], fix_full[3], fin
  static constexpr int kNumBars = 1 + 2 * kSlots + 2 + 2 + 2 + 3 + 3 + 1;
  static constexpr int kMisc = kBar + 8 * kNumBars;  // TMEM address, flag
  static constexpr int kBytes = kMisc + 16 + 64;
  static constexpr int col_s(int t) { return 128 * t; }
  static constexpr int col_o(int t) { return 256 + D * t; }
};

// One CTA's work: two tiles of query rows against one run of keys.
struct PaJob {
  int live;        // 0: nothing to do
  int g;           // kv head
  int krow;        // first key's row in the K / V tensors
  int n_keys;      // keys behind krow that exist
  int tok[2];      // first token of each tile
  int ntok[2];     // tokens of each tile (0: tile unused)
  int pos[2];      // dense: key index of the tile's first token
  int nb[2];       // key blocks of each tile
  int fix_from;    // first block whose V tile is gone over
  int split;       // prefix: which part of the keys
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 16 bytes of shared memory by its 32-bit address.
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(a) : "memory");
  return u;
}
__device__ __forceinline__ void sts16(uint32_t a, const uint4& u) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w) : "memory");
}

// sigmoid(g) o for eight values: o / (1 + 2^(-g log2 e)), rounded to bf16.
__device__ __forceinline__ uint4 gate_pack(const uint4& g, const uint4& a, const uint4& b) {
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, ow[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    constexpr float kL = -1.4426950408889634f;
    const float2 z = __fmul2_rn(__bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&gw[e])), make_float2(kL, kL));
    const float2 d = __fadd2_rn(make_float2(tc::ex2_approx(z.x), tc::ex2_approx(z.y)), make_float2(1.f, 1.f));
    float2 q;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.y) : "f"(d.y));
    q = __fmul2_rn(q, make_float2(__uint_as_float(ow[2 * e]), __uint_as_float(ow[2 * e + 1])));
    const __nv_bfloat162 h2 = __floats2bfloat162_rn(q.x, q.y);
    r[e] = *reinterpret_cast<const uint32_t*>(&h2);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Non-finite bf16 values among the 8 of u: bit i set for value i.
__device__ __forceinline__ unsigned nonfinite8(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m |= ((w[i] & 0x7f80u) == 0x7f80u ? 1u : 0u) << (2 * i);
    m |= ((w[i] & 0x7f800000u) == 0x7f800000u ? 1u : 0u) << (2 * i + 1);
  }
  return m;
}

// The V tile of one block: rows from `valid` on become 0; non-finite values of
// the others become 0 and are reported.  Called by 64 threads (id 0..63).
template <int D>
__device__ __forceinline__ bool scrub_v(uint8_t* tile, int valid, int id) {
  bool found = false;
  for (int r = id; r < kPaBlock; r += 64) {
    uint4* row = reinterpret_cast<uint4*>(tile + r * 128);
#pragma unroll
    for (int a = 0; a < D / 64; ++a)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint4* p = row + a * 1024 + c;         // every chunk of the row: the swizzle only permutes them
        if (r >= valid) {
          *p = make_uint4(0, 0, 0, 0);
        } else {
          uint4 u = *p;
          const unsigned m = nonfinite8(u);
          if (m) {
            found = true;
            uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (m >> (2 * i) & 1) w[i] &= 0xffff0000u;
              if (m >> (2 * i + 1) & 1) w[i] &= 0xffffu;
            }
            *p = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
  }
  return found;
}

// What the epilogue does with a finished row.
//   dense:  out = sigmoid(gate) O / l, plus the non-finite values of V that the
//           row sees in blocks from fix_from on
//   prefix: O, m and l go to the workspace
struct PaDense {
  const __nv_bfloat16* v;
  const __nv_bfloat16* gate;
  __nv_bfloat16* out;
};
struct PaPrefix {
  float* part_o;       // [split, batch, Hq, D]
  float2* part_ml;     // [split, batch, Hq]: maximum (log2 units), sum
};

// What does not depend on the job, by warps 1 and 2, while warp 0 looks it up.
template <int D>
__device__ __forceinline__ void pa_setup(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                         uint8_t* smem) {
  using L = PaLayout<D>;
  if (threadIdx.x == 32) {
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
    for (int i = 0; i < L::kNumBars; ++i) {
      const int at = i - (1 + 2 * L::kSlots);       // p_half, p_full: the tile's four warps; v_ready: two warps
      tc::mbar_init(bars + i, at >= 2 && at < 6 ? 4 : at >= 6 && at < 9 ? 2 : 1);
    }
    tc::fence_barrier_init();
    tc::tma_prefetch(&qmap);
    tc::tma_prefetch(&kmap);
    tc::tma_prefetch(&vmap);
    *reinterpret_cast<volatile int*>(smem + L::kMisc + 4) = 0;
  }
  if (threadIdx.x >= 64 && threadIdx.x < 96) {
    tc::tmem_alloc(reinterpret_cast<uint32_t*>(smem + L::kMisc), 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
}

// Behind pa_setup and a barrier of the block.
template <int D, bool kDense, typename Epi>
__device__ __forceinline__ void pa_run(const CUtensorMap& qmap, const CUtensorMap& kmap,
                                       const CUtensorMap& vmap, uint8_t* smem, const PaJob& job,
                                       const Epi& epi, int batch, int Hq, int Hkv, int Tt, float sl2) {
  using L = PaLayout<D>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_full = bars;
  uint64_t* ring_full = bars + 1;
  uint64_t* ring_empty = ring_full + L::kSlots;
  uint64_t* s_full = ring_empty + L::kSlots;   // [2]
  // P is published in two halves of 64 keys: the first is multiplied while the
  // exponentials of the second are taken
  uint64_t* p_half = s_full + 2;               // [2]
  uint64_t* p_full = p_half + 2;               // [2]
  // block fix_from + k is published on v_ready[k]: two tiles hold at most 256
  // tokens, so their diagonal crosses at most three blocks
  uint64_t* v_ready = p_full + 2;
  // such a tile's load completes on fix_full[k] (and only counts a phase of its
  // ring barrier): those who go over it have not followed the ring's phases
  uint64_t* fix_full = v_ready + 3;
  uint64_t* fin = fix_full + 3;
  volatile int* found = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);

  // the same in all lanes, and known to be: branches on it are uniform
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = Hq / Hkv;
  const int nb = max(job.nb[0], job.nb[1]);
  tc::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<uint32_t*>(smem + L::kMisc);

  if (warp < 4) {
    tc::setmaxnreg_dec<kPaRegsLow>();
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      if (tc::elect_one()) {
        const uint32_t qb = (uint32_t)(G * Tt * 128 * L::kAtoms);
        tc::mbar_expect_tx(q_full, job.ntok[1] > 0 ? 2 * qb : qb);
        for (int t = 0; t < 2; ++t)
          if (job.ntok[t] > 0)
            for (int a = 0; a < L::kAtoms; ++a)
              tma_load_3d(smem + t * L::kTile + a * 16384, &qmap, q_full, 64 * a, job.g * G, job.tok[t]);
        int m = 0;
        for (; m < 2 * nb; ++m) {       // K(0) V(0) K(1) V(1) ...
          const int st = m % L::kSlots, use = m / L::kSlots;
          if (use > 0 && !tc::mbar_wait(ring_empty + st, (use - 1) & 1)) break;
          uint64_t* full = ring_full + st;
          if ((m & 1) && (m >> 1) >= job.fix_from) {
            tc::mbar_arrive(full);
            full = fix_full + ((m >> 1) - job.fix_from);
          }
          tc::mbar_expect_tx(full, L::kTile);
          uint8_t* dst = smem + L::kRing + st * L::kTile;
          const CUtensorMap* map = (m & 1) ? &vmap : &kmap;
          for (int a = 0; a < L::kAtoms; ++a)
            tc::tma_load_2d(dst + a * 16384, map, full, job.g * D + 64 * a, job.krow + (m >> 1) * kPaBlock);
        }
        // no copy is in flight when this warp ends, whatever became of the others
        for (int i = max(0, m - L::kSlots); i < m; ++i) {
          const int k = (i >> 1) - job.fix_from;
          if ((i & 1) && k >= 0) tc::mbar_wait(fix_full + k, 0);
          else tc::mbar_wait(ring_full + i % L::kSlots, (i / L::kSlots) & 1);
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (tc::elect_one()) {
        constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, D, false, true);
        const uint32_t q_addr = tc::smem_u32(smem), ring = q_addr + L::kRing;
        auto wait_tile = [&](int m) {
          return tc::mbar_wait(ring_full + m % L::kSlots, (m / L::kSlots) & 1);
        };
        // the last tile that reads block j's K (or V) lets its slot go
        auto release = [&](int t, int j, int m) {
          if (t == 1 || j >= job.nb[1]) tc::mma_commit(ring_empty + m % L::kSlots);
        };
        auto issue_s = [&](int t, int j) {
          const uint32_t k_addr = ring + ((2 * j) % L::kSlots) * L::kTile;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
            tc::mma_bf16_ss(tmem + L::col_s(t), tc::smem_desc_sw128(q_addr + t * L::kTile + off, 16, 1024),
                            tc::smem_desc_sw128(k_addr + off, 16, 1024), idesc_s, kk > 0);
          }
          tc::mma_commit(s_full + t);
          release(t, j, 2 * j);
        };
        auto issue_pv = [&](int t, int j, int half) {
          const uint32_t v_addr = ring + ((2 * j + 1) % L::kSlots) * L::kTile;
#pragma unroll
          for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
            tc::mma_bf16_ts(tmem + L::col_o(t), tmem + L::col_s(t) + kk * 8,
                            tc::smem_desc_sw128(v_addr + kk * 2048, 16384, 1024), idesc_o,
                            (j > 0 || kk > 0));
          if (half) release(t, j, 2 * j + 1);
        };
        bool ok = tc::mbar_wait(q_full, 0) && wait_tile(0);
        if (ok) {
          tc::tc_fence_after();
          for (int t = 0; t < 2; ++t)
            if (job.nb[t] > 0) issue_s(t, 0);
        }
        for (int j = 0; ok && j < nb; ++j) {
          if (!(ok = wait_tile(2 * j + 1))) break;
          if (j >= job.fix_from) {
            const int k = j - job.fix_from;
            if (!(ok = tc::mbar_wait(v_ready + k, 0))) break;
          }
          for (int t = 0; ok && t < 2; ++t) {
            if (j >= job.nb[t]) continue;
            if (!(ok = tc::mbar_wait(p_half + t, j & 1))) break;
            tc::tc_fence_after();
            issue_pv(t, j, 0);
            if (!(ok = tc::mbar_wait(p_full + t, j & 1))) break;
            tc::tc_fence_after();
            issue_pv(t, j, 1);
            if (j + 1 < job.nb[t]) {
              if (!(ok = wait_tile(2 * j + 2))) break;
              tc::tc_fence_after();
              issue_s(t, j + 1);
            }
          }
        }
        tc::mma_commit(fin);       // every product issued above is complete once this fires
        tc::mbar_wait(fin, 0);
      }
    } else {
      // ------------------------------------------------------------ V at masked keys
      bool bad = false;
      for (int j = job.fix_from; j < nb; ++j) {
        const int m = 2 * j + 1, k = j - job.fix_from;
        if (!__all_sync(0xffffffffu, tc::mbar_wait(fix_full + k, 0))) break;
        bad |= scrub_v<D>(smem + L::kRing + (m % L::kSlots) * L::kTile, job.n_keys - j * kPaBlock,
                          threadIdx.x - 64);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(v_ready + k);
      }
      if (bad) *found = 1;
      __threadfence_block();
      asm volatile("bar.arrive 1, 320;" ::: "memory");
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    tc::setmaxnreg_inc<kPaRegsHigh>();
    const int t = (warp - 4) >> 2;            // tile
    const int quad = warp & 3;                // TMEM lane quadrant
    const int r = quad * 32 + lane;           // row in the tile
    const int tt = r / G;                     // its token in the tile
    const bool valid = r < G * Tt && tt < job.ntok[t];
    const int nbt = job.nb[t];
    const int lim = !valid ? 0 : kDense ? job.pos[t] + tt + 1 : job.n_keys;   // keys it sees
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t o_addr = lane_base + L::col_o(t);
    const uint32_t s_addr = lane_base + L::col_s(t);
    const float2 sl2v = make_float2(sl2, sl2);
    float m = kPaLowest, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nbt; ++j) {
      ok = __all_sync(0xffffffffu, tc::mbar_wait(s_full + t, j & 1));
      if (!ok) break;
      tc::tc_fence_after();
      float x[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld32(s_addr + 32 * c, x + 32 * c);
      tc::tmem_wait_ld();
      const int vis = lim - j * kPaBlock;
      if (__any_sync(0xffffffffu, vis < kPaBlock)) {
#pragma unroll
        for (int c = 0; c < 128; ++c) x[c] = c < vis ? x[c] : -INFINITY;
      }
      // row maximum (NaN wins), scaled once (sl2 > 0)
      float mp[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) mp[k] = max_nan(x[k], x[8 + k]);
#pragma unroll
      for (int c = 16; c < 128; c += 16)
#pragma unroll
        for (int k = 0; k < 8; ++k) mp[k] = max3_nan(mp[k], x[c + k], x[c + 8 + k]);
      const float mx = max_nan(kPaLowest, sl2 * max3_nan(max3_nan(mp[0], mp[1], mp[2]), max3_nan(mp[3], mp[4], mp[5]),
                                                        max_nan(mp[6], mp[7])));
      if (j == 0) m = mx;
      if (j > 0 && __any_sync(0xffffffffu, mx > m + kPaRescale)) {
        const float mnew = fmaxf(m, mx);
        const float f = tc::ex2_approx(m - mnew);
        m = mnew;
        l *= f;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
          float o[16];
          tc::tmem_ld16(o_addr + c0, o);
          tc::tmem_wait_ld();
          uint32_t u[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) u[c] = __float_as_uint(o[c] * f);
          tc::tmem_st16_u(o_addr + c0, u);
        }
      }
      const float2 negm = make_float2(-m, -m);
      float2 acc4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
#pragma unroll
      for (int q0 = 0; q0 < 4; ++q0) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 z = __ffma2_rn(make_float2(x[32 * q0 + 2 * e], x[32 * q0 + 2 * e + 1]), sl2v, negm);
          const float2 pv = make_float2(tc::ex2_approx(z.x), tc::ex2_approx(z.y));
          acc4[e & 3] = __fadd2_rn(acc4[e & 3], pv);
          __nv_bfloat162 h2 = __floats2bfloat162_rn(pv.x, pv.y);
          pk[e] = *reinterpret_cast<uint32_t*>(&h2);
        }
        tc::tmem_st16_u(s_addr + 16 * q0, pk);
        if (q0 & 1) {
          tc::tmem_wait_st();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive((q0 == 1 ? p_half : p_full) + t);
        }
      }
      const float2 s01 = __fadd2_rn(__fadd2_rn(acc4[0], acc4[1]), __fadd2_rn(acc4[2], acc4[3]));
      // a NaN or infinite logit makes the row NaN: mx x 0 is NaN then, else 0
      l += s01.x + s01.y + mx * 0.f;
    }
    asm volatile("bar.sync 1, 320;" ::: "memory");
    // A thread holds a row; rows are D values apart or further.  64 columns at a
    // time go through the ring (8 KB for each warp, no tile is needed any more), so
    // that a row is read and written in pieces of 128 bytes or more.
    const long long head = job.g * G + (r - tt * G);
    const long long row = valid ? (long long)(job.tok[t] + tt) * Hq + head : -1;
    ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(fin, 0));
    if (ok && nbt > 0) {
      tc::tc_fence_after();
      const bool bad = kDense && *found;
      // logits that are all -infinity leave no weights: 0 / 0
      const float mul = !kDense ? 1.f : m == kPaLowest ? NAN : 1.f / l;
      const long long part = kDense ? 0 : (long long)job.split * batch * Hq;
      if constexpr (!kDense)
        if (valid) epi.part_ml[part + row] = make_float2(m, l);
      // 16-byte chunk x of a row of 64 fp32 lies at place (x >> 1 | (x & 1) << 3) ^ (row & 7)
      // of its 16: free of bank conflicts by rows and by pairs of chunks
      const uint32_t stg = tc::smem_u32(smem + L::kRing) + (warp - 4) * 8192;
      const uint32_t put_a = stg + lane * 256 + ((lane & 7) << 4);
      const int cr = lane >> 3, cq = lane & 7;          // row (+ 4 i) and 8-column chunk of a copy
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 64) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float o[32];
          tc::tmem_ld32(o_addr + c0 + 32 * h, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] *= mul;
          if constexpr (kDense) {
            if (bad && valid) {
              for (int u = job.fix_from * kPaBlock; u < lim; ++u) {
                const __nv_bfloat16* vr = epi.v + ((long long)(job.krow + u) * Hkv + job.g) * D + c0 + 32 * h;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  const float f = to_f32(vr[c]);
                  if (!isfinite(f)) o[c] += f;
                }
              }
            }
          }
#pragma unroll
          for (int x = 0; x < 8; ++x)
            sts16(put_a ^ (((8 * h + x) >> 1 | (x & 1) << 3) << 4),
                  make_uint4(__float_as_uint(o[4 * x]), __float_as_uint(o[4 * x + 1]), __float_as_uint(o[4 * x + 2]),
                             __float_as_uint(o[4 * x + 3])));
        }
        __syncwarp();
        long long at[8];
        uint4 g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          at[i] = __shfl_sync(0xffffffffu, row, cr + 4 * i);
          if constexpr (kDense)
            if (at[i] >= 0) g[i] = *reinterpret_cast<const uint4*>(epi.gate + at[i] * D + c0 + 8 * cq);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = cr + 4 * i;
          const uint32_t get_a = (stg + rr * 256 + ((rr & 7) << 4)) ^ (cq << 4);      // chunks 2 cq and 2 cq + 1
          const uint4 x = lds16(get_a), y = lds16(get_a ^ 128);
          if (at[i] >= 0) {
            if constexpr (kDense) {
              *reinterpret_cast<uint4*>(epi.out + at[i] * D + c0 + 8 * cq) = gate_pack(g[i], x, y);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(epi.part_o + (part + at[i]) * D + c0 + 8 * cq);
              dst[0] = x;
              dst[1] = y;
            }
          }
        }
        __syncwarp();
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Bounds of sequence i are usable by themselves.
__device__ __forceinline__ bool seq_ok(const int32_t* cu, int i, int tokens) {
  return cu[i] >= 0 && cu[i] <= cu[i + 1] && cu[i + 1] <= tokens;
}

// Lengths of sequences i0 .. i0 + 31, one per lane of a warp that asks for i0 = 0,
// 32, ... in turn; -1 where there is none or it is skipped.  Skipped is a sequence
// whose bounds are not usable, and one that begins below the end of an earlier
// usable one: those that are left are disjoint, and the grids and workspaces, sized
// from the number of tokens, hold their pieces.  Bounds that ascend need no more
// than a vote.  Overlap takes a descent somewhere, so the look at each pair of
// bounds, which sets the status, finds every call that holds a skipped sequence.
struct SeqLengths {
  int top = 0;       // highest end so far
  __device__ __forceinline__ int next(const int32_t* cu, int n_seqs, int tokens, int i0) {
    const int lane = threadIdx.x & 31, i = i0 + lane;
    const bool in = i < n_seqs;
    const int a = in ? cu[i] : 0, b = in ? cu[i + 1] : 0;
    bool ok = in && a >= 0 && a <= b && b <= tokens;
    int end = ok ? b : 0;
    if (__all_sync(0xffffffffu, !in || (ok && a >= top))) {
      end = __shfl_sync(0xffffffffu, end, min(31, n_seqs - 1 - i0));
    } else {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end = max(end, v);
      }
      const int before = __shfl_up_sync(0xffffffffu, end, 1);
      ok = ok && a >= (lane > 0 ? max(top, before) : top);
      end = __shfl_sync(0xffffffffu, end, 31);
    }
    top = max(top, end);
    return ok ? b - a : -1;
  }
};

// Work of different lengths, longest first: a launch's last blocks are then
// short ones, which keeps all SMs busy to its end.  Lengths are compared by
// their power of two (class k: 2^k to 2^(k+1) - 1 units); count(n, k) says how
// many pieces of class k a sequence of n tokens has.  Called by one warp: piece p
// of all, as a sequence, a class and a number among the sequence's pieces of that
// class.
struct PackedPiece {
  int seq, cls, idx;     // seq < 0: there are not so many
};

template <typename Count>
__device__ __forceinline__ PackedPiece find_piece(const int32_t* cu, int n_seqs, int tokens, int kmax, int p,
                                                  Count count) {
  const int lane = threadIdx.x & 31;
  int len = SeqLengths().next(cu, n_seqs, tokens, 0);
#pragma unroll 1
  for (int k = kmax; k >= 0; --k) {
    SeqLengths walk;
#pragma unroll 1
    for (int i0 = 0; i0 < n_seqs; i0 += 32) {
      if (n_seqs > 32) len = walk.next(cu, n_seqs, tokens, i0);
      const int n = len >= 0 ? count(len, k) : 0;
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, p < inc);
      if (hit) {
        const int w = __ffs(hit) - 1;
        return PackedPiece{i0 + w, k, p - __shfl_sync(0xffffffffu, inc - n, w)};
      }
      p -= __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  return PackedPiece{-1, 0, 0};
}

__device__ __forceinline__ int length_class(int n) { return 31 - __clz(max(n, 1)); }

template <int D>
__global__ void __launch_bounds__(kPaThreads, 1)
dense_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const int32_t* __restrict__ cu,
                  const __nv_bfloat16* __restrict__ v, const __nv_bfloat16* __restrict__ gate,
                  __nv_bfloat16* __restrict__ out, int tokens, int n_seqs, int Hq, int Hkv, int Tt,
                  int kmax, float sl2) {
  extern __shared__ __align__(1024) uint8_t smem_pa[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_pa) + 1023) & ~uintptr_t(1023));
  PaJob* slot = reinterpret_cast<PaJob*>(smem + PaLayout<D>::kMisc + 16);
  static_assert(sizeof(PaJob) <= 64, "the job's place in shared memory");
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < n_seqs; i += kPaThreads)
      if (!seq_ok(cu, i, tokens)) set_status(kStatusBounds);
  pa_setup<D>(qmap, kmap, vmap, smem);
  if (threadIdx.x < 32) {
    PaJob job = {};
    // pair j of a sequence's tiles sees the keys up to its last token: pairs of
    // class k or above begin where (2 j + 2) Tt exceeds 128 (2^k - 1) keys
    const uint32_t pair_tokens = 2 * Tt;
    const auto below = [&](int n, int k) {       // pairs of a sequence of n tokens below class k (k <= 24)
      const uint32_t keys = ((1u << k) - 1) * kPaBlock;
      return (int)((uint32_t)n <= keys ? (n + pair_tokens - 1) / pair_tokens : keys / pair_tokens);
    };
    const PackedPiece w = find_piece(cu, n_seqs, tokens, kmax, blockIdx.x / Hkv,
                                     [&](int n, int k) { return below(n, k + 1) - below(n, k); });
    if (w.seq >= 0) {
      const int s = w.seq, n = cu[s + 1] - cu[s];
      const int pair = below(n, w.cls + 1) - 1 - w.idx;
      job.live = 1;
      job.g = blockIdx.x % Hkv;
      job.krow = cu[s];
      job.n_keys = n;
      for (int t = 0; t < 2; ++t) {
        const int p0 = (2 * pair + t) * Tt;
        job.pos[t] = p0;
        job.tok[t] = cu[s] + p0;
        job.ntok[t] = max(0, min(Tt, n - p0));
        job.nb[t] = job.ntok[t] > 0 ? (p0 + job.ntok[t] + kPaBlock - 1) / kPaBlock : 0;
      }
      job.fix_from = (job.pos[0] + 1) / kPaBlock;   // the first token sees pos[0] + 1 keys
    }
    if (threadIdx.x == 0) *slot = job;
  }
  __syncthreads();
  const PaJob job = *slot;
  if (!job.live) {
    if (threadIdx.x >= 64 && threadIdx.x < 96) {
      tc::tc_fence_after();
      tc::tmem_dealloc(*reinterpret_cast<uint32_t*>(smem + PaLayout<D>::kMisc), 512);
    }
    return;
  }
  pa_run<D, true>(qmap, kmap, vmap, smem, job, PaDense{v, gate, out}, 0, Hq, Hkv, Tt, sl2);
}

}  // namespace sala
