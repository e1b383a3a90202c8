// Linear attention with a decay for each head over packed prompts, chunk-wise
// on the 5th-generation tensor cores.
//
//   S_t = lam S_{t-1} + k_t^T v_t,   out_t = sigmoid(gate_t) * scale * q_t S_t
//
// (Linear layers at O(N): acgfav.com "SALA 混合架构"; constant-size state:
// MiniCPM-SALA paper section 2.1.)  Per tile of L <= 128 tokens, from the state
// S that enters it:
//
//   P    = (Q K^T) . D,  D_ij = lam^(i-j) for j <= i, else 0
//   O_i  = lam^(i+1) (Q S)_i + (P V)_i
//   S   <- lam^L S + K^T V',  V'_j = lam^(L-1-j) v_j
//
// A sequence is cut into segments of whole tiles; a CTA walks one segment of
// one head (two heads where d = 64, side by side in 128 columns).  Sequences
// of several segments take three launches: the states that each segment but
// the last adds (kOut = false), a scan over them, and the outputs.
//
// Rounding.  States are fp32: V' is split into two bf16 parts (hi + lo, 2^-16),
// each tile's K^T V' is summed from zero on the tensor core and joined to S in
// registers, so the tensor core's own rounding never adds up over tiles.  P
// and the copy of S that Q multiplies are rounded to bf16; Q, K and V enter as
// they are.
//
// Isolation.  Rows past a sequence's end become 0 in K and V before anything is
// multiplied (0 x NaN is NaN).  So do non-finite values of V before P V, whose
// zeros above the diagonal would else hand them to earlier tokens; the epilogue
// adds them to the rows that do see them.
//
// Bound by memory: q, k, v, gate and out are 160 KB per tile and head (d = 128)
// against 2560 cycles of tensor core; at this card's copy rate a tile takes
// 7000 cycles of an SM.
#pragma once

#include "common.cuh"
#include "packed_attn.cuh"
#include "packed_step.cuh"
#include "tc_ptx.cuh"

namespace sala {

constexpr int kPlThreads = 512;
constexpr int kPlTile = 128;
// warpgroup 0: TMA, MMA, TMEM; 1: V; 2: P and outputs; 3: state.  The shares sum
// to the 4 x 128 registers that the block is launched with (warpgroup 2 keeps its own).
constexpr int kPlRegs0 = 48, kPlRegs1 = 152, kPlRegs2 = 128, kPlRegs3 = 184;
static_assert(kPlRegs0 + kPlRegs1 + kPlRegs2 + kPlRegs3 <= 4 * 128, "register split exceeds the launch");

struct PlLayout {
  static constexpr int kQ = 0, kK = 32768, kV = 65536;     // per stage, two 64-column atoms each
  static constexpr int kStage = 98304;
  static constexpr int kS = 2 * kStage;                    // S in bf16
  static constexpr int kPw = kS + 32768;                   // lam^m, m = 0..128, per head: [2][132]
  static constexpr int kBar = kPw + 2 * 132 * 4;
  // ld_full[2], ld_empty[2], kv_ok, qk_full, p_full, pv_done, o_full, o_empty, s_full, v_hi, v_lo,
  // hi_done, ds_full[2], fin
  static constexpr int kNumBars = 17;
  static constexpr int kMisc = kBar + 8 * kNumBars;        // TMEM address, unit, found[2][4]
  static constexpr int kBytes = kMisc + 96;
  static constexpr int kColQK = 0, kColO1 = 128, kColO2 = 256, kColDs = 384;
  static_assert(kBar % 8 == 0 && kMisc % 8 == 0, "alignment");
};

// How a call's sequences are cut: segments of seg_tokens.  What a CTA finds
// for its index p among the sequences' segments (all of them, or all but each
// sequence's last).
struct PlUnit {
  int seq, seg;      // sequence, segment in it; seq < 0: none
  int n_seg;         // segments of the sequence
  int ws;            // where the sequence's segment states begin
};

// Called by one warp.
__device__ __forceinline__ PlUnit find_segment(const int32_t* cu, int n_seqs, int tokens, int seg_tokens,
                                               bool all, int p) {
  const int lane = threadIdx.x & 31;
  int ws = 0;
  for (int i0 = 0; i0 < n_seqs; i0 += 32) {
    const int i = i0 + lane;
    int n = 0;
    if (i < n_seqs && seq_ok(cu, i, tokens)) n = max(1, (cu[i + 1] - cu[i] + seg_tokens - 1) / seg_tokens);
    const int e = max(n - 1, 0), own = all ? n : e;
    int inc = own, ince = e;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, inc, o), b = __shfl_up_sync(0xffffffffu, ince, o);
      if (lane >= o) {
        inc += a;
        ince += b;
      }
    }
    const unsigned hit = __ballot_sync(0xffffffffu, p < inc);
    if (hit) {
      const int w = __ffs(hit) - 1;
      PlUnit u;
      u.seq = i0 + w;
      u.n_seg = __shfl_sync(0xffffffffu, n, w);
      u.seg = p - __shfl_sync(0xffffffffu, inc - own, w);
      u.ws = ws + __shfl_sync(0xffffffffu, ince - e, w);
      return u;
    }
    p -= __shfl_sync(0xffffffffu, inc, 31);
    ws += __shfl_sync(0xffffffffu, ince, 31);
  }
  return PlUnit{-1, 0, 0, 0};
}

// bf16 pair (w) times (f, f): high and low bf16 parts.
__device__ __forceinline__ void split_pair(uint32_t w, float f, uint32_t* hi, uint32_t* lo) {
  const float2 x = __fmul2_rn(__bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w)), make_float2(f, f));
  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
  const float2 hf = __bfloat1622float2(h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(x.x - hf.x, x.y - hf.y);
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = *reinterpret_cast<const uint32_t*>(&l);
}

template <int D, bool kOut>
__global__ void __launch_bounds__(kPlThreads, 1)
linear_packed_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __nv_bfloat16* __restrict__ v,
                     const __nv_bfloat16* __restrict__ gate, const float* __restrict__ lambda,
                     const int32_t* __restrict__ cu, const int32_t* __restrict__ slots,
                     const float* state_in, float* state_out, float* __restrict__ ws,
                     __nv_bfloat16* __restrict__ out, int tokens, int n_seqs, int n_slots, int H,
                     int seg_tokens, float scale) {
  using L = PlLayout;
  constexpr int NH = 128 / D;               // heads side by side
  extern __shared__ __align__(1024) uint8_t smem_pl[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_pl) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  // Every barrier's phase is waited for by all who wait on it before the next
  // one can complete.  Where kOut is false, tiles of even and odd number use
  // kv_ok / v_hi (V' written) and o_empty / s_full (sum read) in turn for that.
  uint64_t* ld_full = bars;            // [2] Q, K, V of a tile have landed
  uint64_t* ld_empty = bars + 2;       // [2]
  uint64_t* kv_ok = bars + 4;          // rows past the end and non-finite values are 0
  uint64_t* qk_full = bars + 5;
  uint64_t* p_full = bars + 6;
  uint64_t* pv_done = bars + 7;        // V may be overwritten by V'
  uint64_t* o_full = bars + 8;
  uint64_t* o_empty = bars + 9;
  uint64_t* s_full = bars + 10;        // the bf16 copy of S
  uint64_t* v_hi = bars + 11;
  uint64_t* v_lo = bars + 12;
  uint64_t* hi_done = bars + 13;
  uint64_t* ds_full = bars + 14;       // [2]
  uint64_t* fin = bars + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  PlUnit* unit = reinterpret_cast<PlUnit*>(smem + L::kMisc + 8);
  volatile int* found = reinterpret_cast<volatile int*>(smem + L::kMisc + 32);   // [2][4]
  float* pw = reinterpret_cast<float*>(smem + L::kPw);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_hg = (H + NH - 1) / NH;
  const int hg = blockIdx.x % n_hg;
  if (kOut && blockIdx.x == 0)
    for (int i = threadIdx.x; i < n_seqs; i += kPlThreads)
      if (!seq_ok(cu, i, tokens)) set_status(kStatusBounds);
  if (warp == 0) {
    const PlUnit u = find_segment(cu, n_seqs, tokens, seg_tokens, kOut, blockIdx.x / n_hg);
    if (lane == 0) *unit = u;
  }
  __syncthreads();
  const PlUnit u = *unit;
  if (u.seq < 0) return;
  const int slot = kOut ? take_slot(slots, u.seq, n_slots) : 0;
  const int s0 = cu[u.seq] + u.seg * seg_tokens;
  const int n_tok = min(cu[u.seq + 1] - s0, seg_tokens);
  const int nt = (n_tok + kPlTile - 1) / kPlTile;
  const bool last = u.seg + 1 == u.n_seg;
  // where this thread's state row lives: row r of the 128 is key dim r % D of head r / D
  const int r_own = threadIdx.x & 127;
  const int hsub = r_own / D, h_own = hg * NH + hsub;
  const long long srow = (((long long)slot * H + h_own) * D + r_own % D) * D;
  const float* s_src = nullptr;
  if (h_own < H && kOut) {
    if (u.seg > 0) s_src = ws + (((long long)(u.ws + u.seg - 1) * H + h_own) * D + r_own % D) * D;
    else if (state_in && slot >= 0) s_src = state_in + srow;
  }
  float* s_dst = nullptr;
  if (h_own < H) {
    if (!kOut) s_dst = ws + (((long long)(u.ws + u.seg) * H + h_own) * D + r_own % D) * D;
    else if (last && state_out && slot >= 0) s_dst = state_out + srow;
  }
  if (nt == 0) {        // an empty sequence hands its state on
    if (threadIdx.x < 128 && s_dst)
      for (int c = 0; c < D; c += 4)
        *reinterpret_cast<float4*>(s_dst + c) =
            s_src ? *reinterpret_cast<const float4*>(s_src + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  // tiles whose K^T V' is wanted
  const bool keep = !kOut || (last && state_out && slot >= 0);
  const int nds = keep ? nt : nt - 1;
  auto tile_len = [&](int c) { return min(kPlTile, n_tok - c * kPlTile); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(ld_full + i, 1);
      tc::mbar_init(ld_empty + i, 1);
      tc::mbar_init(ds_full + i, 1);
    }
    tc::mbar_init(kv_ok, 4);
    tc::mbar_init(qk_full, 1);
    tc::mbar_init(p_full, 4);
    tc::mbar_init(pv_done, 1);
    tc::mbar_init(o_full, 1);
    tc::mbar_init(o_empty, 4);
    tc::mbar_init(s_full, 4);
    tc::mbar_init(v_hi, 4);
    tc::mbar_init(v_lo, 4);
    tc::mbar_init(hi_done, 1);
    tc::mbar_init(fin, 1);
    tc::fence_barrier_init();
  }
  for (int e = threadIdx.x; e < NH * 129; e += kPlThreads) {
    const int hh = e / 129, x = e % 129;
    const double lam = hg * NH + hh < H ? (double)lambda[hg * NH + hh] : 0.0;
    pw[hh * 132 + x] = (float)pow(lam, (double)x);
  }
  if (warp == 2) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    tc::setmaxnreg_dec<kPlRegs0>();
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      if (tc::elect_one()) {
        int c = 0;
        for (; c < nt; ++c) {
          const int st = c & 1, use = c >> 1;
          if (use > 0 && !tc::mbar_wait(ld_empty + st, (use - 1) & 1)) break;
          uint8_t* stage = smem + st * L::kStage;
          tc::mbar_expect_tx(ld_full + st, kOut ? 98304 : 65536);
          for (int a = 0; a < 2; ++a) {
            const int x = hg * 128 + 64 * a, y = s0 + c * kPlTile;
            tc::tma_load_2d(stage + L::kK + a * 16384, &kmap, ld_full + st, x, y);
            if (kOut) tc::tma_load_2d(stage + L::kQ + a * 16384, &qmap, ld_full + st, x, y);
            tc::tma_load_2d(stage + L::kV + a * 16384, &vmap, ld_full + st, x, y);
          }
        }
        // no copy is in flight when this warp ends, whatever became of the others
        for (int i = max(0, c - 2); i < c; ++i) tc::mbar_wait(ld_full + (i & 1), (i >> 1) & 1);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (tc::elect_one()) {
        constexpr uint32_t id_kk = tc::idesc_bf16_f32(128, 128, false, false);   // A, B K-major
        constexpr uint32_t id_pv = tc::idesc_bf16_f32(128, D, false, true);      // B MN-major
        constexpr uint32_t id_nn = tc::idesc_bf16_f32(128, 128, true, true);     // A, B MN-major
        const uint32_t base = tc::smem_u32(smem);
        const uint32_t sb = base + L::kS;
        auto part = [&](int c, int which) { return base + (c & 1) * L::kStage + which; };
        auto issue_qk = [&](int c, int hs) {
          const uint32_t q = part(c, L::kQ), k = part(c, L::kK);
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const int kk = hs * (D / 16) + x;
            const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
            tc::mma_bf16_ss(tmem + L::kColQK, tc::smem_desc_sw128(q + off, 16, 1024),
                            tc::smem_desc_sw128(k + off, 16, 1024), id_kk, x > 0);
          }
          tc::mma_commit(qk_full);
        };
        auto issue_ds = [&](int c, int which, uint32_t col, bool acc) {
          const uint32_t k = part(c, L::kK), w = part(c, which);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc::mma_bf16_ss(tmem + col, tc::smem_desc_sw128(k + kk * 2048, 16384, 1024),
                            tc::smem_desc_sw128(w + kk * 2048, 16384, 1024), id_nn, acc || kk > 0);
        };
        auto loaded = [&](int c) {
          return tc::mbar_wait(ld_full + (c & 1), (c >> 1) & 1) && tc::mbar_wait(kv_ok, c & 1);
        };
        bool ok = true;
        if constexpr (kOut) {
          ok = loaded(0);
          if (ok) {
            tc::tc_fence_after();
            issue_qk(0, 0);
          }
          for (int c = 0; ok && c < nt; ++c) {
            // O2 = P V, head by head
            if (c > 0 && !(ok = tc::mbar_wait(o_empty, (c - 1) & 1))) break;
#pragma unroll
            for (int hs = 0; hs < NH; ++hs) {
              if (!(ok = tc::mbar_wait(p_full, (c * NH + hs) & 1))) break;
              tc::tc_fence_after();
              const uint32_t vv = part(c, L::kV) + hs * 16384;
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc::mma_bf16_ts(tmem + L::kColO2 + hs * D, tmem + L::kColQK + kk * 8,
                                tc::smem_desc_sw128(vv + kk * 2048, 16384, 1024), id_pv, kk > 0);
              if (hs + 1 < NH) issue_qk(c, hs + 1);
            }
            if (!ok) break;
            tc::mma_commit(pv_done);
            // O1 = Q S
            if (!(ok = tc::mbar_wait(s_full, c & 1))) break;
            tc::tc_fence_after();
            const uint32_t q = part(c, L::kQ);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {     // key dims 16 kk .. 16 kk + 15, of head hs
              const int hs = kk * 16 / D;
              const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
              tc::mma_bf16_ss(tmem + L::kColO1 + hs * D, tc::smem_desc_sw128(q + off, 16, 1024),
                              tc::smem_desc_sw128(sb + hs * 16384 + kk * 2048, 16384, 1024), id_pv,
                              kk * 16 % D > 0);
            }
            tc::mma_commit(o_full);
            // K^T V', high parts, then (while the low parts are written) the next
            // tile's Q K^T, then the low parts
            if (c < nds) {
              if (!(ok = tc::mbar_wait(v_hi, c & 1))) break;
              tc::tc_fence_after();
              issue_ds(c, L::kV, L::kColDs, false);
              tc::mma_commit(hi_done);
            }
            if (c + 1 < nt) {
              if (!(ok = loaded(c + 1))) break;
              tc::tc_fence_after();
              issue_qk(c + 1, 0);
            }
            if (c < nds) {
              if (!(ok = tc::mbar_wait(v_lo, c & 1))) break;
              tc::tc_fence_after();
              issue_ds(c, L::kV, L::kColDs, true);
              tc::mma_commit(ds_full);
              tc::mma_commit(ld_empty + (c & 1));
            }
          }
        } else {
          // high parts lie in V's place, low parts in Q's
          for (int c = 0; ok && c < nt; ++c) {
            const int x = c & 1, use = c >> 1;
            if (!(ok = tc::mbar_wait(ld_full + x, use & 1) && tc::mbar_wait(x ? v_hi : kv_ok, use & 1))) break;
            // the buffer's last sum has been read
            if (use > 0 && !(ok = tc::mbar_wait(x ? s_full : o_empty, (use - 1) & 1))) break;
            tc::tc_fence_after();
            issue_ds(c, L::kV, L::kColDs - 128 * (c & 1), false);
            issue_ds(c, L::kQ, L::kColDs - 128 * (c & 1), true);
            tc::mma_commit(ds_full + (c & 1));
            tc::mma_commit(ld_empty + (c & 1));
          }
        }
        tc::mma_commit(fin);
        tc::mbar_wait(fin, 0);
      }
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- V
    tc::setmaxnreg_inc<kPlRegs1>();
    const int r = r_own;                      // token row of the tile
    auto chunk = [&](uint8_t* tile, int i) {  // 16-byte chunk i (of 16) of this row
      return reinterpret_cast<uint4*>(tile + (i >> 3) * 16384 + r * 128 + (((i & 7) ^ (r & 7)) << 4));
    };
    uint4 raw[16];
    // reads the row into registers and makes the tile safe to multiply
    auto enter = [&](int c) {
      if (!__all_sync(0xffffffffu, tc::mbar_wait(ld_full + (c & 1), (c >> 1) & 1))) return false;
      uint8_t* stage = smem + (c & 1) * L::kStage;
      if (r < tile_len(c)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) raw[i] = *chunk(stage + L::kV, i);
      } else {
        const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          raw[i] = z;
          *chunk(stage + L::kV, i) = z;
          *chunk(stage + L::kK, i) = z;
        }
      }
      return true;
    };
    bool ok = enter(0);
    if constexpr (kOut) {
      uint4 lo[16];
      // before P V: non-finite values become 0 in the tile
      auto make_safe = [&](int c) {
        uint32_t acc = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          acc |= (raw[i].x & 0x7f807f80u) + 0x00800080u;
          acc |= (raw[i].y & 0x7f807f80u) + 0x00800080u;
          acc |= (raw[i].z & 0x7f807f80u) + 0x00800080u;
          acc |= (raw[i].w & 0x7f807f80u) + 0x00800080u;
        }
        const bool bad = (acc & 0x80008000u) != 0;
        if (bad) {
#pragma unroll 1
          for (int i = 0; i < 16; ++i) {
            uint4* p = chunk(smem + (c & 1) * L::kStage + L::kV, i);
            const uint4 x = *p;
            const unsigned m = nonfinite8(x);
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (m >> (2 * e) & 1) w[e] &= 0xffff0000u;
              if (m >> (2 * e + 1) & 1) w[e] &= 0xffffu;
            }
            *p = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        const bool any = __any_sync(0xffffffffu, bad);
        if (lane == 0) found[(c & 1) * 4 + (warp & 3)] = any;
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(kv_ok);
      };
      if (ok) make_safe(0);
      for (int c = 0; ok && c < nt; ++c) {
        const bool want = c < nds;
        if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(pv_done, c & 1)))) break;
        if (want) {
          const int Lt = tile_len(c);
          uint8_t* tile = smem + (c & 1) * L::kStage + L::kV;
          const float f0 = r < Lt ? pw[Lt - 1 - r] : 0.f;
          const float f1 = NH == 1 ? f0 : (r < Lt ? pw[132 + Lt - 1 - r] : 0.f);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint4 hi;
            const float f = i < 8 ? f0 : f1;
            split_pair(raw[i].x, f, &hi.x, &lo[i].x);
            split_pair(raw[i].y, f, &hi.y, &lo[i].y);
            split_pair(raw[i].z, f, &hi.z, &lo[i].z);
            split_pair(raw[i].w, f, &hi.w, &lo[i].w);
            *chunk(tile, i) = hi;
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(v_hi);
        }
        if (c + 1 < nt) {
          if (!(ok = enter(c + 1))) break;
          make_safe(c + 1);
        }
        if (want) {
          if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(hi_done, c & 1)))) break;
          uint8_t* tile = smem + (c & 1) * L::kStage + L::kV;
#pragma unroll
          for (int i = 0; i < 16; ++i) *chunk(tile, i) = lo[i];
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(v_lo);
        }
      }
    } else {
      for (int c = 0; ok && c < nt; ++c) {
        const int Lt = tile_len(c);
        uint8_t* stage = smem + (c & 1) * L::kStage;
        const float f0 = r < Lt ? pw[Lt - 1 - r] : 0.f;
        const float f1 = NH == 1 ? f0 : (r < Lt ? pw[132 + Lt - 1 - r] : 0.f);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint4 hi, lo;
          const float f = i < 8 ? f0 : f1;
          split_pair(raw[i].x, f, &hi.x, &lo.x);
          split_pair(raw[i].y, f, &hi.y, &lo.y);
          split_pair(raw[i].z, f, &hi.z, &lo.z);
          split_pair(raw[i].w, f, &hi.w, &lo.w);
          *chunk(stage + L::kV, i) = hi;
          *chunk(stage + L::kQ, i) = lo;
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(c & 1 ? v_hi : kv_ok);
        if (c + 1 < nt) ok = enter(c + 1);
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------- P and gated outputs
    if constexpr (kOut) {
      const int quad = warp & 3, r = r_own;      // token row
      const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
      const int cols = min(128, H * D - hg * 128);      // columns of heads that exist
      for (int c = 0; c < nt; ++c) {
        if (!__all_sync(0xffffffffu, tc::mbar_wait(kv_ok, c & 1))) break;
        const volatile int* fc = found + (c & 1) * 4;
        const bool bad = fc[0] | fc[1] | fc[2] | fc[3];
        bool ok = true;
#pragma unroll 1
        for (int hs = 0; hs < NH; ++hs) {
          if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(qk_full, (c * NH + hs) & 1)))) break;
          tc::tc_fence_after();
          const float* pwh = pw + hs * 132;
          // 32-column chunk u of P (bf16 pairs) lands on columns [16 u, 16 u + 16),
          // read with chunk u / 2 <= u: each is written back as it is built
#pragma unroll
          for (int q0 = 0; q0 < 4; ++q0) {
            uint32_t pk[16];
            if (q0 <= quad) {
              float xv[32];
              tc::tmem_ld32(lane_base + L::kColQK + 32 * q0, xv);
              tc::tmem_wait_ld();
              if (q0 == quad) {
#pragma unroll
                for (int e = 0; e < 32; ++e) xv[e] = e <= lane ? xv[e] * pwh[lane - e] : 0.f;
              } else {
                const int a = r - 32 * q0;            // element e decays by lam^(a - e)
                float2 dcy = make_float2(pwh[a - 30], pwh[a - 31]);
                const float2 l2 = make_float2(pwh[2], pwh[2]);
#pragma unroll
                for (int e = 30; e >= 0; e -= 2) {
                  const float2 y = __fmul2_rn(make_float2(xv[e], xv[e + 1]), dcy);
                  xv[e] = y.x;
                  xv[e + 1] = y.y;
                  dcy = __fmul2_rn(dcy, l2);
                }
              }
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                __nv_bfloat162 h2 = __floats2bfloat162_rn(xv[2 * e], xv[2 * e + 1]);
                pk[e] = *reinterpret_cast<uint32_t*>(&h2);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = 0u;
            }
            tc::tmem_st16_u(lane_base + L::kColQK + 16 * q0, pk);
          }
          tc::tmem_wait_st();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(p_full);
        }
        if (!ok) break;
        // ---- out = sigmoid(gate) scale (lam^(r+1) O1 + O2)
        const bool valid = r < tile_len(c);
        const long long row = ((long long)(s0 + c * kPlTile + r) * H) * D + hg * 128;
        uint4 g[16];
        if (valid) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (8 * i < cols) g[i] = *reinterpret_cast<const uint4*>(gate + row + 8 * i);
        }
        if (!__all_sync(0xffffffffu, tc::mbar_wait(o_full, c & 1))) break;
        tc::tc_fence_after();
#pragma unroll
        for (int j = 0; j < 8; ++j) {                   // 16 columns at a time
          float o1[16], o2[16];
          tc::tmem_ld16(lane_base + L::kColO1 + 16 * j, o1);
          tc::tmem_ld16(lane_base + L::kColO2 + 16 * j, o2);
          tc::tmem_wait_ld();
          if (j == 7) {
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(o_empty);
          }
          const float f = pw[(16 * j / D) * 132 + r + 1];
#pragma unroll
          for (int e = 0; e < 16; ++e) o1[e] = fmaf(f, o1[e], o2[e]);
          if (bad && valid && 16 * j < cols) {
            for (int t = 0; t <= r; ++t) {
              const __nv_bfloat16* vr = v + (long long)(s0 + c * kPlTile + t) * H * D + hg * 128 + 16 * j;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float x = to_f32(vr[e]);
                if (!isfinite(x)) o1[e] += x;
              }
            }
          }
          if (valid && 16 * j < cols) {
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
              float gv[8];
              load8(reinterpret_cast<const __nv_bfloat16*>(&g[2 * j + e / 8]), gv);
#pragma unroll
              for (int x = 0; x < 8; ++x) gv[x] = sigmoidf_(gv[x]) * (scale * o1[e + x]);
              store8(out + row + 16 * j + e, gv);
            }
          }
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- state
    tc::setmaxnreg_inc<kPlRegs3>();
    const int quad = warp & 3, r = r_own;      // key row of S (of head hsub)
    const uint32_t ds_addr = tmem + ((uint32_t)(quad * 32) << 16) + L::kColDs + hsub * D % 128;
    const float* pwh = pw + hsub * 132;
    float S[D];
#pragma unroll
    for (int e = 0; e < D; e += 4) {
      const float4 x = s_src ? __ldcg(reinterpret_cast<const float4*>(s_src + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
      S[e] = x.x;
      S[e + 1] = x.y;
      S[e + 2] = x.z;
      S[e + 3] = x.w;
    }
    auto publish = [&]() {
#pragma unroll
      for (int j = 0; j < D / 32; ++j) sw128_store_row32(smem + L::kS, r, hsub * (D / 32) + j, S + 32 * j);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(s_full);
    };
    if (kOut) publish();
    bool ok = true;
    for (int c = 0; ok && c < nds; ++c) {
      // ds_full of tile c says that Q S of tile c has read the copy of S as well
      uint64_t* full = kOut ? ds_full : ds_full + (c & 1);
      if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(full, kOut ? c & 1 : (c >> 1) & 1)))) break;
      tc::tc_fence_after();
      const float f = pwh[tile_len(c)];
      const uint32_t src = ds_addr - (kOut ? 0 : 128 * (c & 1));
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        float x[16];
        tc::tmem_ld16(src + 16 * j, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) S[16 * j + e] = fmaf(f, S[16 * j + e], x[e]);
      }
      tc::tc_fence_before();
      if constexpr (kOut) {
        if (c + 1 < nt) publish();
      } else {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(c & 1 ? s_full : o_empty);
      }
    }
    if (ok && s_dst) {
#pragma unroll
      for (int e = 0; e < D; e += 4)
        *reinterpret_cast<float4*>(s_dst + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Between the two: the k-th sequence of several segments turns what each of
// its segments but the last adds into the state that enters the next one.
// Four state values per thread.
constexpr int kPlScanThreads = 256;

template <int D>
__global__ void __launch_bounds__(kPlScanThreads)
linear_packed_scan_kernel(const float* __restrict__ lambda, const int32_t* __restrict__ cu,
                          const int32_t* __restrict__ slots, const float* __restrict__ state_in, float* ws,
                          int tokens, int n_seqs, int n_slots, int H, int seg_tokens) {
  __shared__ PlUnit unit;
  if (threadIdx.x < 32) {
    // the k-th sequence that has more than one segment
    int k = blockIdx.y, base = 0;
    PlUnit u = {-1, 0, 0, 0};
    const int lane = threadIdx.x;
    for (int i0 = 0; i0 < n_seqs; i0 += 32) {
      const int i = i0 + lane;
      int e = 0;
      if (i < n_seqs && seq_ok(cu, i, tokens)) e = max(0, (cu[i + 1] - cu[i] + seg_tokens - 1) / seg_tokens - 1);
      const unsigned multi = __ballot_sync(0xffffffffu, e > 0);
      if (k < __popc(multi)) {
        const int w = __fns(multi, 0, k + 1);
        u.seq = i0 + w;
        u.n_seg = __shfl_sync(0xffffffffu, e, w) + 1;
        int before = lane < w ? e : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
        u.ws = base + before;
        break;
      }
      k -= __popc(multi);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
      base += e;
    }
    if (lane == 0) unit = u;
  }
  __syncthreads();
  const PlUnit u = unit;
  if (u.seq < 0) return;
  const int slot = take_slot(slots, u.seq, n_slots);
  const long long e = 4 * ((long long)blockIdx.x * kPlScanThreads + threadIdx.x);
  const long long per = (long long)H * D * D;
  if (e >= per) return;
  const float f = (float)pow((double)lambda[e / (D * D)], (double)seg_tokens);
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (state_in && slot >= 0) S = *reinterpret_cast<const float4*>(state_in + slot * per + e);
  float* p = ws + u.ws * per + e;
  const int n = u.n_seg - 1;
  for (int s0 = 0; s0 < n; s0 += 8) {          // eight sums in flight
    float4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s0 + i < n) x[i] = *reinterpret_cast<const float4*>(p + (s0 + i) * per);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s0 + i < n) {
        S.x = fmaf(f, S.x, x[i].x);
        S.y = fmaf(f, S.y, x[i].y);
        S.z = fmaf(f, S.z, x[i].z);
        S.w = fmaf(f, S.w, x[i].w);
        *reinterpret_cast<float4*>(p + (s0 + i) * per) = S;
      }
  }
}

}  // namespace sala
