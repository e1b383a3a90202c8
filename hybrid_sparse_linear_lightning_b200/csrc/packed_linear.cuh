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
// of several segments take three launches: what each segment adds to the state
// (kOut = false), a scan over them, which also gives the leaving state, and the
// outputs.
//
// Rounding.  States are fp32: V' is split into three bf16 parts (24 bits; two,
// 16 bits, where the state does not leave), each tile's K^T V' is summed from
// zero on the tensor core and joined to S in registers, so the tensor core's own
// rounding never adds up over tiles.  P
// and the copy of S that Q multiplies are rounded to bf16; Q, K and V enter as
// they are.
//
// The gate's sigmoid is an exponential and a reciprocal, as in the other calls: a
// closed gate's output keeps its relative accuracy.  1/2 + tanh(g / 2) / 2 on the
// hardware's tanh takes half the special-function operations (64K prompt 912 us),
// but its error of 2^-12 is absolute: 10 % of the output at g = -6.  Every other
// exponential on the FMA pipe, or one reciprocal for two values, gain nothing (980
// and 1075 us).
//
// Isolation.  Rows past a sequence's end become 0 in K and V before anything is
// multiplied (0 x NaN is NaN).  So do non-finite values of V before P V, whose
// zeros above the diagonal would else hand them to earlier tokens; the epilogue
// makes the rows that do see them NaN, which is what q S gives for a column of
// infinities of both signs.
//
// q, k, v, gate and out are 160 KB per tile and head (d = 128), 7000 cycles of
// an SM at this card's copy rate, against 2560 cycles of tensor core.  What binds
// is the chain of a tile through the warps that build P, split V and carry S, and
// shared memory, which the products, the tiles and the staged outputs share (670
// KB per tile, 5250 cycles): 9000 cycles per tile.  One prompt of 65536 tokens, 32
// heads: 980 us, 2.74 TB/s; 13 prompts of 9001 tokens: 190 us.  What it took: the
// roles as functions of their own (their registers in memory cost 3000 cycles per
// tile), loops rolled to fit the instruction caches, V and S shared by two
// warpgroups, outputs in 128-byte pieces, states by TMA (12 us less per CTA than
// row by row).  A third part of V' costs 15 %.
#pragma once

#include "common.cuh"
#include "packed_attn.cuh"
#include "packed_step.cuh"
#include "tc_ptx.cuh"

namespace sala {

constexpr int kPlThreads = 512;
constexpr int kPlTile = 128;
// warpgroup 0: TMA, MMA, TMEM; 1 and 3: P, V and the state, half the columns
// each; 2: outputs.  The shares sum to the 4 x 128 registers that the block is
// launched with.
constexpr int kPlRegs0 = 56, kPlRegsV = 176, kPlRegs2 = 104;
static_assert(kPlRegs0 + 2 * kPlRegsV + kPlRegs2 <= 4 * 128, "register split exceeds the launch");

struct PlLayout {
  static constexpr int kQ = 0, kK = 32768, kV = 65536;     // per stage, two 64-column atoms each
  static constexpr int kStage = 98304;
  static constexpr int kS = 2 * kStage;                    // S in bf16
  static constexpr int kPw = kS + 32768;                   // lam^m, m = 0..128, per head: [2][132]
  static constexpr int kBar = kPw + 2 * 132 * 4;
  // ld_full[2], ld_empty[2], kv_ok, qk_full, p_full, pv_done, o_full, o_empty, s_full, v_hi, v_lo,
  // hi_done, ds_full[2], fin, s_ld, e_sync, v_sync
  static constexpr int kNumBars = 26;
  // Barriers by their byte offset.  Every barrier's phase is waited for by all who
  // wait on it before the next one can complete.  Where kOut is false, tiles of
  // even and odd number use kv_ok and v_hi (V' written) in turn for that.
  enum : uint32_t {
    ld_full = 0,         // [2] K and V of a tile have landed
    ld_empty = 16,       // [2] K^T V' is done
    kv_ok = 32,          // rows past the end and non-finite values are 0
    qk_full = 40,
    p_full = 48,
    pv_done = 56,        // V may be overwritten by V'
    o_full = 64,
    o_empty = 72,
    s_full = 80,         // the bf16 copy of S
    v_hi = 88,
    v_lo = 96,
    hi_done = 104,
    ds_full = 112,       // [2]
    fin = 128,
    s_ld = 136,          // the entering state has landed
    e_sync = 144,        // among the warps that write outputs
    v_sync = 152,        // the leaving state lies in shared memory
    q_full = 160,        // [2] Q has landed
    q_empty = 176,       // [2] outputs are written
    v_low = 192,         // the third part of V'
    lo_done = 200,
  };
  static constexpr int kMisc = kBar + 8 * kNumBars;        // TMEM address, unit, found[2][8]
  static constexpr int kShared = kMisc + 96;               // PlShared
  static constexpr int kBytes = kShared + 64;
  static constexpr int kColQK = 0, kColO1 = 128, kColO2 = 256, kColDs = 384;
  static_assert(kBar % 8 == 0 && kMisc % 8 == 0, "alignment");
};

// lam^n by squaring in fp64 (n >= 0): no call of a library function, across
// which the kernel's values would have to be kept in memory.
__device__ __forceinline__ float decay_pow(float lam, int n) {
  double p = 1.0, b = lam;
  for (; n > 0; n >>= 1) {
    if (n & 1) p *= b;
    b *= b;
  }
  return (float)p;
}

// Read by the roles where they need it.
struct PlShared {
  const __nv_bfloat16 *v, *gate;
  __nv_bfloat16* out;
  const CUtensorMap* dst_map;      // of the leaving state
  int dst_row;                     // its first row, -1 for nowhere
  int s0, H, hg;
  float scale;
};
static_assert(sizeof(PlShared) <= 64, "its place in shared memory");

// How a call's sequences are cut: segments of seg_tokens.  What a CTA finds
// for its index p among the sequences' segments (all of them, or all but each
// sequence's last).
struct PlUnit {
  int seq, seg;      // sequence, segment in it; seq < 0: none
  int n_seg;         // segments of the sequence
  int ws;            // where its n_seg + 1 states in the workspace begin (none where n_seg is 1)
};

__device__ __forceinline__ int segments_of(int n, int seg_tokens) {
  return max(1, (n + seg_tokens - 1) / seg_tokens);
}

// Called by one warp: index p among all segments (longest first), or among
// those of the sequences that have several.
__device__ __forceinline__ PlUnit find_segment(const int32_t* cu, int n_seqs, int tokens, int seg_tokens,
                                               bool all, int p) {
  const int kseg = length_class(seg_tokens / kPlTile);
  const PackedPiece w = find_piece(cu, n_seqs, tokens, all ? kseg : 0, p, [&](int n, int k) {
    const int n_seg = segments_of(n, seg_tokens);
    if (!all) return n_seg > 1 ? n_seg : 0;
    const int whole = n / seg_tokens, rest = n - whole * seg_tokens;
    const bool has_rest = rest > 0 || n == 0;
    return (k == kseg ? whole : 0) + (has_rest && k == length_class((rest + kPlTile - 1) / kPlTile));
  });
  PlUnit u = {w.seq, 0, 0, 0};
  if (w.seq < 0) return u;
  const int n = cu[w.seq + 1] - cu[w.seq];
  u.n_seg = segments_of(n, seg_tokens);
  // the rest of a sequence comes behind its whole segments, alone in its class
  // where that is another one
  u.seg = !all || w.cls == kseg ? w.idx : u.n_seg - 1;
  if (u.n_seg > 1) {
    int before = 0;
    SeqLengths walk;
    for (int i0 = 0; i0 < w.seq; i0 += 32) {
      const int len = walk.next(cu, n_seqs, tokens, i0);
      const int e = segments_of(len, seg_tokens);
      if (e > 1 && i0 + (int)(threadIdx.x & 31) < w.seq) before += e + 1;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    u.ws = before;
  }
  return u;
}

// A load that stays where it is written: the compiler would else move it to
// its first use, behind the wait that is to cover its latency.  Gates and outputs
// pass the L1 cache by: what shared memory leaves of it keeps spilled registers.
__device__ __forceinline__ uint4 ld_now(const __nv_bfloat16* p) {
  uint4 u;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  return u;
}

__device__ __forceinline__ void st_out(__nv_bfloat16* p, const uint4& u) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w)
               : "memory");
}

// 2D tiled store of one box.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}

// bf16 pair (w) times (f, f) in three bf16 parts.
__device__ __forceinline__ void split_pair(uint32_t w, float f, uint32_t* hi, uint32_t* lo, uint32_t* low) {
  const float2 x = __fmul2_rn(__bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w)), make_float2(f, f));
  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
  const float2 hf = __bfloat1622float2(h);
  const float2 d = __fadd2_rn(x, make_float2(-hf.x, -hf.y));
  const __nv_bfloat162 l = __floats2bfloat162_rn(d.x, d.y);
  const float2 lf = __bfloat1622float2(l);
  const float2 e = __fadd2_rn(d, make_float2(-lf.x, -lf.y));
  const __nv_bfloat162 m = __floats2bfloat162_rn(e.x, e.y);
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = *reinterpret_cast<const uint32_t*>(&l);
  *low = *reinterpret_cast<const uint32_t*>(&m);
}

// The warps that build P, split V and carry the state.  A function of its own,
// not inlined: its registers are then allocated apart from the other roles'
// (inlined, the compiler keeps 30 of them in memory inside the loop over tiles).
// What it needs rarely is in shared memory (PlShared), not among its arguments,
// which the compiler would keep in memory too.
template <int D, bool kOut, bool kThree>
__device__ __noinline__ void linear_state_role(uint32_t o_smem, uint32_t tmem, int n_tok, int nds, int flags) {
  using L = PlLayout;
  constexpr int NH = 128 / D;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const bool has_src = flags & 1;
  const int nt = (n_tok + kPlTile - 1) / kPlTile, heads = flags >> 1;
  // --------------------------------------------- V and the state (half the columns each)
  tc::setmaxnreg_inc<kPlRegsV>();
  auto o_len = [&](int c) { return min(kPlTile, n_tok - c * kPlTile); };
  const uint32_t bar = o_smem + L::kBar;
  const float* pw = reinterpret_cast<const float*>(__cvta_shared_to_generic(o_smem + L::kPw));
  volatile int* found = reinterpret_cast<volatile int*>(__cvta_shared_to_generic(o_smem + L::kMisc + 32));
  const volatile PlShared* sh = reinterpret_cast<const volatile PlShared*>(__cvta_shared_to_generic(o_smem + L::kShared));
  const int r_own = threadIdx.x & 127, hsub = r_own / D;
  const int quad = warp & 3, half = warp >= 12;
  const int r = r_own;                      // token row of V, key row of S (of head hsub)
  // 16-byte chunk i (of 8) of this half row of the tile at offset `part` of stage c & 1
  const uint32_t row_a = o_smem + half * 16384 + r * 128 + ((r & 7) << 4);
  auto chunk = [&](int c, int part, int i) { return (row_a + (c & 1) * L::kStage + part) ^ (i << 4); };
  // makes the tile safe to multiply; says whether this part of V held values
  // that are not finite (they are 0 now).  False where a wait ran out.
  auto enter = [&](int c, bool* bad) {
    if (!__all_sync(0xffffffffu, tc::mbar_wait(bar + L::ld_full + 8 * (c & 1), (c >> 1) & 1))) return false;
    *bad = false;
    if (r >= o_len(c)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sts16(chunk(c, L::kV, i), make_uint4(0, 0, 0, 0));
        sts16(chunk(c, L::kK, i), make_uint4(0, 0, 0, 0));
      }
    } else if (kOut) {
      __nv_bfloat162 top = __float2bfloat162_rn(0.f);       // largest magnitudes, NaN above all
#pragma unroll
      for (int i0 = 0; i0 < 8; i0 += 4) {
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = lds16(chunk(c, L::kV, i0 + i));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[e])));
        }
      }
      const uint32_t tw = *reinterpret_cast<const uint32_t*>(&top);
      *bad = (tw & 0x7f80u) == 0x7f80u || (tw & 0x7f800000u) == 0x7f800000u;
      if (*bad) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const uint4 x = lds16(chunk(c, L::kV, i));
          const unsigned m = nonfinite8(x);
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (m >> (2 * e) & 1) w[e] &= 0xffff0000u;
            if (m >> (2 * e + 1) & 1) w[e] &= 0xffffu;
          }
          sts16(chunk(c, L::kV, i), make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
    }
    if (kOut) {
      const bool any = __any_sync(0xffffffffu, *bad);
      if (lane == 0) found[(c & 1) * 8 + half * 4 + quad] = any;
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar + L::kv_ok);
    }
    return true;
  };
  const float* pwv = pw + (NH == 1 ? 0 : half) * 132;     // decays of the half's head
  // the state: columns [64 half, 64 half + 64) of row r; where two heads lie
  // side by side only the half of the row's own head
  const bool mine = NH == 1 || half == hsub;
  const uint32_t ds_addr = tmem + ((uint32_t)(quad * 32) << 16) + L::kColDs + 64 * half;
  // where the row's 64 columns lie while the state is loaded or stored: boxes of
  // 32 columns, swizzled like the tiles
  const uint32_t box_a = o_smem + L::kK + (hsub * (D / 32) + (NH == 1 ? 2 * half : 0)) * (D * 128) + (r % D) * 128 +
                         ((r & 7) << 4);
  float S[64];
#pragma unroll
  for (int e = 0; e < 64; ++e) S[e] = 0.f;
  bool ok = true;
  if (has_src) {
    ok = __all_sync(0xffffffffu, tc::mbar_wait(bar + L::s_ld, 0));
    if (ok && mine && hsub < heads) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint4 x = lds16((box_a + L::kStage + (i >> 3) * (D * 128)) ^ ((i & 7) << 4));
        S[4 * i] = __uint_as_float(x.x);
        S[4 * i + 1] = __uint_as_float(x.y);
        S[4 * i + 2] = __uint_as_float(x.z);
        S[4 * i + 3] = __uint_as_float(x.w);
      }
    }
  }
  auto publish = [&]() {
    if (mine) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 h2 = __floats2bfloat162_rn(S[8 * i + 2 * e], S[8 * i + 2 * e + 1]);
          w[e] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        sts16(chunk(0, L::kS, i), make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar + L::s_full);
  };
  // S <- lam^L S + K^T V' of tile c
  auto join = [&](int c, uint32_t full, int parity, uint32_t src) {
    if (!__all_sync(0xffffffffu, tc::mbar_wait(full, parity))) return false;
    tc::tc_fence_after();
    const float f = pw[hsub * 132 + o_len(c)];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[16];
      tc::tmem_ld16(src + 16 * j, x);
      tc::tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) S[16 * j + e] = fmaf(f, S[16 * j + e], x[e]);
    }
    tc::tc_fence_before();
    return true;
  };
  // P of one head: (Q K^T)_rj lam^(r-j) for j <= r, this half's 64 columns.
  // Its bf16 pairs take the first 32 of the columns that it read.
  auto make_p = [&](int c, int hs) {
    if (!__all_sync(0xffffffffu, tc::mbar_wait(bar + L::qk_full, (c * NH + hs) & 1))) return false;
    tc::tc_fence_after();
    const float* pwh = pw + hs * 132;
    const uint32_t qk = tmem + ((uint32_t)(quad * 32) << 16) + L::kColQK + 64 * half;
#pragma unroll 1
    for (int x0 = 0; x0 < 2; ++x0) {
      const int q0 = 2 * half + x0;         // 32-column chunk
      uint32_t pk[16];
      if (q0 <= quad) {
        float xv[32];
        tc::tmem_ld32(qk + 32 * x0, xv);
        tc::tmem_wait_ld();
        if (q0 == quad) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float d = pwh[max(lane - e, 0)];
            xv[e] = e <= lane ? xv[e] * d : 0.f;
          }
        } else {
          // element e decays by lam^(a - e): four pairs with powers of their own,
          // lam^8 from one to the next, from the largest power down
          const int a = r - 32 * q0;
          float2 dcy[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) dcy[x] = make_float2(pwh[a - 24 - 2 * x], pwh[a - 25 - 2 * x]);
          const float2 l8 = make_float2(pwh[8], pwh[8]);
#pragma unroll
          for (int e0 = 24; e0 >= 0; e0 -= 8)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int e = e0 + 2 * x;
              const float2 y = __fmul2_rn(make_float2(xv[e], xv[e + 1]), dcy[x]);
              xv[e] = y.x;
              xv[e + 1] = y.y;
              dcy[x] = __fmul2_rn(dcy[x], l8);
            }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const __nv_bfloat162 h2 = __floats2bfloat162_rn(xv[2 * e], xv[2 * e + 1]);
          pk[e] = *reinterpret_cast<const uint32_t*>(&h2);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) pk[e] = 0u;
      }
      tc::tmem_st16_u(qk + 16 * x0, pk);
    }
    tc::tmem_wait_st();
    tc::tc_fence_before();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar + L::p_full);
    return true;
  };
  bool bad = false, bad_next = false;
  if (kOut && ok) publish();
  // kOut: round c finishes tile c and begins tile c + 1
  if (!kOut) ok = ok && enter(0, &bad);
#pragma unroll 1
  for (int c = kOut ? -1 : 0; ok && c < nt; ++c) {
    const int Lt = o_len(c);
    if constexpr (kOut) {
      const bool want = c >= 0 && c < nds;
      if (c >= 0 && !(ok = __all_sync(0xffffffffu, tc::mbar_wait(bar + L::pv_done, c & 1)))) break;
      uint4 lo[8] = {}, low[8] = {};
      if (want) {
        const float f = r < Lt ? pwv[Lt - 1 - r] : 0.f;
        if (bad) {         // the state takes the row as it came
          const __nv_bfloat16* vr = sh->v + (long long)(sh->s0 + c * kPlTile + r) * sh->H * D + sh->hg * 128 + 64 * half;
#pragma unroll 1
          for (int i = 0; i < 8; ++i) sts16(chunk(c, L::kV, i), *reinterpret_cast<const uint4*>(vr + 8 * i));
        }
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += 4) {
          uint4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = lds16(chunk(c, L::kV, i0 + i));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 hi;
            split_pair(x[i].x, f, &hi.x, &lo[i0 + i].x, &low[i0 + i].x);
            split_pair(x[i].y, f, &hi.y, &lo[i0 + i].y, &low[i0 + i].y);
            split_pair(x[i].z, f, &hi.z, &lo[i0 + i].z, &low[i0 + i].z);
            split_pair(x[i].w, f, &hi.w, &lo[i0 + i].w, &low[i0 + i].w);
            sts16(chunk(c, L::kV, i0 + i), hi);
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar + L::v_hi);
      }
      if (c + 1 < nt && !(ok = enter(c + 1, &bad_next))) break;
      if (want) {
        if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(bar + L::hi_done, c & 1)))) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) sts16(chunk(c, L::kV, i), lo[i]);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar + L::v_lo);
      }
      if (kThree && want) {
        if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(bar + L::lo_done, c & 1)))) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) sts16(chunk(c, L::kV, i), low[i]);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar + L::v_low);
      }
      if (c + 1 < nt) {
#pragma unroll 1
        for (int hs = 0; ok && hs < NH; ++hs) ok = make_p(c + 1, hs);
      }
      if (!ok) break;
      if (want) {
        // the products being done says that Q S of this tile has read the copy of S too
        if (!(ok = join(c, bar + L::ds_full, c & 1, ds_addr))) break;
        if (c + 1 < nt) publish();
      }
      bad = bad_next;
    } else {
      const float f = r < Lt ? pwv[Lt - 1 - r] : 0.f;
      uint4 low[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 x = lds16(chunk(c, L::kV, i));
        uint4 hi, lo;
        split_pair(x.x, f, &hi.x, &lo.x, &low[i].x);
        split_pair(x.y, f, &hi.y, &lo.y, &low[i].y);
        split_pair(x.z, f, &hi.z, &lo.z, &low[i].z);
        split_pair(x.w, f, &hi.w, &lo.w, &low[i].w);
        sts16(chunk(c, L::kV, i), hi);
        sts16(chunk(c, L::kQ, i), lo);
      }
      // the third part's place is free once its products for the last tile are done
      if (c > 0 && !(ok = __all_sync(0xffffffffu, tc::mbar_wait(bar + L::lo_done, (c - 1) & 1)))) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) sts16(chunk(0, L::kS, i), low[i]);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar + (c & 1 ? L::v_hi : L::kv_ok));
      // the next tile's parts are written while this one is multiplied
      if (c > 0 && !(ok = join(c - 1, bar + L::ds_full + 8 * ((c - 1) & 1), ((c - 1) >> 1) & 1, ds_addr - 128 * ((c - 1) & 1)))) break;
      if (c + 1 < nt) ok = enter(c + 1, &bad_next);
    }
  }
  if (!kOut && ok)
    ok = join(nt - 1, bar + L::ds_full + 8 * ((nt - 1) & 1), ((nt - 1) >> 1) & 1, ds_addr - 128 * ((nt - 1) & 1));
  // every product and every load is done: the state leaves through stage 0
  const int dst_row = sh->dst_row;
  if (dst_row >= 0) {
    if (ok) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (mine)
          sts16((box_a + (i >> 3) * (D * 128)) ^ ((i & 7) << 4),
                make_uint4(__float_as_uint(S[4 * i]), __float_as_uint(S[4 * i + 1]), __float_as_uint(S[4 * i + 2]),
                           __float_as_uint(S[4 * i + 3])));
    }
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (ok && lane == 0) tc::mbar_arrive(bar + L::v_sync);
    if (warp == 4 && lane == 0 && ok && tc::mbar_wait(bar + L::v_sync, 0)) {
      for (int i = 0; i < heads * (D / 32); ++i)
        tma_store_2d(sh->dst_map, o_smem + L::kK + i * (D * 128), 32 * (i % (D / 32)),
                     dst_row + i / (D / 32) * D);
      asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncwarp();
  }
}

// The warps that write the outputs, a function of its own like the last.
//
// out = sigmoid(gate) scale (lam^(r+1) O1 + O2).  A thread holds a token's row,
// whose neighbours lie H d values apart: 64 columns at a time go through the
// tile's Q, which no product needs any more, so that gate and out are read and
// written 128 bytes a row.
template <int D>
__device__ __noinline__ void linear_output_role(uint32_t o_smem, uint32_t tmem, int n_tok) {
  using L = PlLayout;
  tc::setmaxnreg_dec<kPlRegs2>();
  const float* pw = reinterpret_cast<const float*>(__cvta_shared_to_generic(o_smem + L::kPw));
  const volatile int* found =
      reinterpret_cast<const volatile int*>(__cvta_shared_to_generic(o_smem + L::kMisc + 32));
  const volatile PlShared* sh = reinterpret_cast<const volatile PlShared*>(__cvta_shared_to_generic(o_smem + L::kShared));
  const int s0 = sh->s0, H = sh->H, hg = sh->hg;
  const float scale = sh->scale;
  const __nv_bfloat16* gate = sh->gate;
  __nv_bfloat16* out = sh->out;
  const uint32_t bar = o_smem + L::kBar;
  const int quad = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, r = threadIdx.x & 127;          // token row
  const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
  const int cols = min(128, H * D - hg * 128);           // columns of heads that exist
  const int cr = quad * 4 + (lane >> 3), cq = lane & 7;      // row (+ 16 i) and 8-column chunk of a copy
  const long long rs = (long long)H * D;                   // from token to token
  uint32_t phase = 0;
  auto sync = [&]() {              // the four warps, with a bound
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar + L::e_sync);
    const bool ok = __all_sync(0xffffffffu, tc::mbar_wait(bar + L::e_sync, phase & 1));
    ++phase;
    return ok;
  };
#pragma unroll 1
  for (int c = 0; kPlTile * c < n_tok; ++c) {
    const int Lt = min(kPlTile, n_tok - c * kPlTile);
    const long long t0 = s0 + c * kPlTile;
    const long long at = (t0 + cr) * rs + hg * 128 + 8 * cq;
    uint4 g[8];
    auto load_gate = [&](int h) {
      const __nv_bfloat16* p = gate + at + 64 * h;
#pragma unroll
      for (int i = 0; i < 8; ++i, p += 16 * rs)
        if (cr + 16 * i < Lt && 64 * h < cols) g[i] = ld_now(p);
    };
    load_gate(0);
    if (!__all_sync(0xffffffffu, tc::mbar_wait(bar + L::o_full, c & 1))) break;
    tc::tc_fence_after();
    const volatile int* fc = found + (c & 1) * 8;
    const bool bad = fc[0] | fc[1] | fc[2] | fc[3] | fc[4] | fc[5] | fc[6] | fc[7];
    // 16-byte chunk x of a row of 64 fp32 lies at place (x >> 1 | (x & 1) << 3) ^ (row & 7)
    // of its 16: free of bank conflicts by rows and by pairs of chunks
    const uint32_t stg = o_smem + (c & 1) * L::kStage + L::kQ;
    const uint32_t put_a = stg + r * 256 + ((r & 7) << 4);
    const uint32_t get_a = (stg + cr * 256 + ((cr & 7) << 4)) ^ (cq << 4);     // chunks 2 cq and 2 cq + 1
    // 16 columns of the row into chunks x0 .. x0 + 3
    auto combine = [&](int col, int x0, bool end) {
      float o[16], o2[16];
      tc::tmem_ld16(lane_base + L::kColO1 + col, o);
      tc::tmem_ld16(lane_base + L::kColO2 + col, o2);
      tc::tmem_wait_ld();
      if (end) {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar + L::o_empty);
      }
      const float f = scale * pw[(col / D) * 132 + r + 1];
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float2 y = __ffma2_rn(make_float2(f, f), make_float2(o[e], o[e + 1]),
                                    __fmul2_rn(make_float2(scale, scale), make_float2(o2[e], o2[e + 1])));
        o[e] = y.x;
        o[e + 1] = y.y;
      }
      if (bad && r < Lt && col < cols) {       // the values of V that P V left out
        for (int t = 0; t <= r; ++t) {
          const __nv_bfloat16* vr = sh->v + (t0 + t) * rs + hg * 128 + col;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float x = to_f32(vr[e]);
            if (!isfinite(x)) o[e] = NAN;
          }
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        sts16(put_a ^ (x0 << 3) ^ ((x >> 1 | (x & 1) << 3) << 4), make_uint4(__float_as_uint(o[4 * x]), __float_as_uint(o[4 * x + 1]),
                                              __float_as_uint(o[4 * x + 2]), __float_as_uint(o[4 * x + 3])));
    };
    // the staged half: gated and written
    auto store = [&](int h) {
      constexpr int kB = 8;            // rows of a thread at a time
      __nv_bfloat16* p = out + at + 64 * h;
#pragma unroll
      for (int i0 = 0; i0 < 8; i0 += kB) {
        uint4 a[kB], b[kB];
#pragma unroll
        for (int i = 0; i < kB; ++i) {
          a[i] = lds16(get_a + (i0 + i) * 4096);
          b[i] = lds16((get_a ^ 128) + (i0 + i) * 4096);
        }
#pragma unroll
        for (int i = 0; i < kB; ++i) a[i] = gate_pack(g[i0 + i], a[i], b[i]);
#pragma unroll
        for (int i = 0; i < kB; ++i, p += 16 * rs)
          if (cr + 16 * (i0 + i) < Lt && 64 * h < cols) st_out(p, a[i]);
      }
    };
    // rolled: every role's straight-line code together would not fit the
    // instruction caches
    bool ok = true;
#pragma unroll 1
    for (int h = 0; ok && h < 2; ++h) {
#pragma unroll 1
      for (int j = 0; j < 4; ++j) combine(64 * h + 16 * j, 4 * j, h == 1 && j == 3);
      if (!(ok = sync())) break;
      store(h);
      if (h == 0) load_gate(1);
      else tc::fence_proxy_async_smem();      // the next load writes there
      ok = sync();
    }
    if (!ok) break;
    if (threadIdx.x == 256) tc::mbar_arrive(bar + L::q_empty + 8 * (c & 1));
  }
}

template <int D, bool kOut>
__global__ void __launch_bounds__(kPlThreads, 1)
linear_packed_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap gmap,
                     const __grid_constant__ CUtensorMap simap, const __grid_constant__ CUtensorMap somap,
                     const __grid_constant__ CUtensorMap wsmap, const __nv_bfloat16* __restrict__ v,
                     const __nv_bfloat16* __restrict__ gate,
                     const float* __restrict__ lambda,
                     const int32_t* __restrict__ cu, const int32_t* __restrict__ slots,
                     const float* state_in, float* state_out, __nv_bfloat16* __restrict__ out, int tokens, int n_seqs, int n_slots, int H,
                     int seg_tokens, float scale) {
  using L = PlLayout;
  constexpr int NH = 128 / D;               // heads side by side
  extern __shared__ __align__(1024) uint8_t smem_pl[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_pl) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  PlUnit* unit = reinterpret_cast<PlUnit*>(smem + L::kMisc + 8);
  float* pw = reinterpret_cast<float*>(smem + L::kPw);

  // the same in all lanes, and known to be: branches on it are uniform
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
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
  // the entering and the leaving state: rows of D values from `row` on, key dims
  // of the heads one after the other
  const bool has_src = kOut && (u.n_seg > 1 || (state_in && slot >= 0));
  const bool has_dst = !kOut || (u.n_seg == 1 && state_out && slot >= 0);
  const int heads = min(NH, H - hg * NH);              // heads that exist
  const int own_row = (slot * H + hg * NH) * D;        // in the caller's pools
  if (nt == 0) {        // an empty sequence hands its state on
    if (has_dst)
      for (int e = threadIdx.x; e < heads * D * D / 4; e += kPlThreads) {
        const long long at = (long long)own_row * D + 4 * e;
        *reinterpret_cast<float4*>(state_out + at) =
            has_src ? *reinterpret_cast<const float4*>(state_in + at) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    return;
  }
  // tiles whose K^T V' is wanted
  const int nds = has_dst ? nt : nt - 1;
  // A state that leaves keeps fp32's accuracy with V' in three parts; one that only
  // Q multiplies, after a rounding to bf16, has two.
  const bool three = has_dst;
  auto tile_len = [&](int c) { return min(kPlTile, n_tok - c * kPlTile); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bars + L::ld_full / 8 + i, 1);
      tc::mbar_init(bars + L::ld_empty / 8 + i, 1);
      tc::mbar_init(bars + L::q_full / 8 + i, 1);
      tc::mbar_init(bars + L::q_empty / 8 + i, 1);
      tc::mbar_init(bars + L::ds_full / 8 + i, 1);
    }
    PlShared* sh = reinterpret_cast<PlShared*>(smem + L::kShared);
    *sh = PlShared{v, gate, out, kOut ? &somap : &wsmap,
                   !has_dst ? -1 : kOut ? own_row : ((u.ws + u.seg + 1) * H + hg * NH) * D, s0, H, hg, scale};
    tc::mbar_init(bars + L::kv_ok / 8, 8);
    tc::mbar_init(bars + L::qk_full / 8, 1);
    tc::mbar_init(bars + L::p_full / 8, 8);
    tc::mbar_init(bars + L::pv_done / 8, 1);
    tc::mbar_init(bars + L::o_full / 8, 1);
    tc::mbar_init(bars + L::o_empty / 8, 4);
    tc::mbar_init(bars + L::s_full / 8, 8);
    tc::mbar_init(bars + L::v_hi / 8, 8);
    tc::mbar_init(bars + L::v_lo / 8, 8);
    tc::mbar_init(bars + L::hi_done / 8, 1);
    tc::mbar_init(bars + L::v_low / 8, 8);
    tc::mbar_init(bars + L::lo_done / 8, 1);
    tc::mbar_init(bars + L::fin / 8, 1);
    tc::mbar_init(bars + L::s_ld / 8, 1);
    tc::mbar_init(bars + L::e_sync / 8, 4);
    tc::mbar_init(bars + L::v_sync / 8, 8);
    tc::fence_barrier_init();
  }
  for (int e = threadIdx.x; e < NH * 129; e += kPlThreads) {
    const int hh = e / 129, x = e % 129;
    pw[hh * 132 + x] = hg * NH + hh < H ? decay_pow(lambda[hg * NH + hh], x) : 0.f;
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
    const uint32_t o_smem = tc::smem_u32(smem), bar = o_smem + L::kBar;
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      if (tc::elect_one()) {
        int c = 0, q_tiles = 0;
        for (; c < nt; ++c) {
          const int st = c & 1, use = c >> 1;
          if (use > 0 && !tc::mbar_wait(bar + L::ld_empty + 8 * st, (use - 1) & 1)) break;
          // stage 1 holds the entering state until its copy has been published
          // (the next one cannot be before tile 1 is here)
          if (c == 1 && has_src && !tc::mbar_wait(bar + L::s_full, 0)) break;
          const uint32_t stage = o_smem + st * L::kStage;
          tc::mbar_expect_tx(bar + L::ld_full + 8 * st, 65536);
          for (int a = 0; a < 2; ++a) {
            const int x = hg * 128 + 64 * a, y = s0 + c * kPlTile;
            tc::tma_load_2d(stage + L::kK + a * 16384, &kmap, bar + L::ld_full + 8 * st, x, y);
            tc::tma_load_2d(stage + L::kV + a * 16384, &vmap, bar + L::ld_full + 8 * st, x, y);
            if (kOut) tc::tma_prefetch_l2_2d(&gmap, x, y);     // its loads come a tile later
          }
          if (kOut) {            // Q's place is the outputs' until they are written
            if (use > 0 && !tc::mbar_wait(bar + L::q_empty + 8 * st, (use - 1) & 1)) {
              ++c;
              break;
            }
            tc::mbar_expect_tx(bar + L::q_full + 8 * st, 32768);
            for (int a = 0; a < 2; ++a)
              tc::tma_load_2d(stage + L::kQ + a * 16384, &qmap, bar + L::q_full + 8 * st, hg * 128 + 64 * a,
                              s0 + c * kPlTile);
            q_tiles = c + 1;
          }
          if (c == 0 && has_src) {
            const int row = u.n_seg > 1 ? ((u.ws + u.seg) * H + hg * NH) * D : own_row;
            tc::mbar_expect_tx(bar + L::s_ld, heads * D * D * 4);
            for (int i = 0; i < heads * (D / 32); ++i)
              tc::tma_load_2d(o_smem + L::kStage + L::kK + i * (D * 128), u.n_seg > 1 ? &wsmap : &simap, bar + L::s_ld,
                              32 * (i % (D / 32)), row + i / (D / 32) * D);
          }
        }
        if (has_src) tc::mbar_wait(bar + L::s_ld, 0);
        // no copy is in flight when this warp ends, whatever became of the others
        for (int i = max(0, c - 2); i < c; ++i) tc::mbar_wait(bar + L::ld_full + 8 * (i & 1), (i >> 1) & 1);
        for (int i = max(0, q_tiles - 2); i < q_tiles; ++i) tc::mbar_wait(bar + L::q_full + 8 * (i & 1), (i >> 1) & 1);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (tc::elect_one()) {
        constexpr uint32_t id_kk = tc::idesc_bf16_f32(128, 128, false, false);   // A, B K-major
        constexpr uint32_t id_pv = tc::idesc_bf16_f32(128, D, false, true);      // B MN-major
        constexpr uint32_t id_nn = tc::idesc_bf16_f32(128, 128, true, true);     // A, B MN-major
        const uint32_t base = o_smem;
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
          tc::mma_commit(bar + L::qk_full);
        };
        auto issue_ds = [&](int c, int which, uint32_t col, bool acc) {
          const uint32_t k = part(c, L::kK), w = which == L::kS ? sb : part(c, which);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc::mma_bf16_ss(tmem + col, tc::smem_desc_sw128(k + kk * 2048, 16384, 1024),
                            tc::smem_desc_sw128(w + kk * 2048, 16384, 1024), id_nn, acc || kk > 0);
        };
        auto loaded = [&](int c) {
          return tc::mbar_wait(bar + L::ld_full + 8 * (c & 1), (c >> 1) & 1) && tc::mbar_wait(bar + L::kv_ok, c & 1) &&
                 tc::mbar_wait(bar + L::q_full + 8 * (c & 1), (c >> 1) & 1);
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
            if (c > 0 && !(ok = tc::mbar_wait(bar + L::o_empty, (c - 1) & 1))) break;
#pragma unroll
            for (int hs = 0; hs < NH; ++hs) {
              if (!(ok = tc::mbar_wait(bar + L::p_full, (c * NH + hs) & 1))) break;
              tc::tc_fence_after();
              const uint32_t vv = part(c, L::kV) + hs * 16384;
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc::mma_bf16_ts(tmem + L::kColO2 + hs * D, tmem + L::kColQK + (kk >> 2) * 64 + (kk & 3) * 8,
                                tc::smem_desc_sw128(vv + kk * 2048, 16384, 1024), id_pv, kk > 0);
              if (hs + 1 < NH) issue_qk(c, hs + 1);
            }
            if (!ok) break;
            tc::mma_commit(bar + L::pv_done);
            // O1 = Q S
            if (!(ok = tc::mbar_wait(bar + L::s_full, c & 1))) break;
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
            tc::mma_commit(bar + L::o_full);
            // K^T V', high parts, then (while the low parts are written) the next
            // tile's Q K^T, then the low parts
            if (c < nds) {
              if (!(ok = tc::mbar_wait(bar + L::v_hi, c & 1))) break;
              tc::tc_fence_after();
              issue_ds(c, L::kV, L::kColDs, false);
              tc::mma_commit(bar + L::hi_done);
            }
            if (c + 1 < nt) {
              if (!(ok = loaded(c + 1))) break;
              tc::tc_fence_after();
              issue_qk(c + 1, 0);
            }
            if (c < nds) {
              if (!(ok = tc::mbar_wait(bar + L::v_lo, c & 1))) break;
              tc::tc_fence_after();
              issue_ds(c, L::kV, L::kColDs, true);
              if (three) {       // written once the second part has been read
                tc::mma_commit(bar + L::lo_done);
                if (!(ok = tc::mbar_wait(bar + L::v_low, c & 1))) break;
                tc::tc_fence_after();
                issue_ds(c, L::kV, L::kColDs, true);
              }
              tc::mma_commit(bar + L::ds_full);
              tc::mma_commit(bar + L::ld_empty + 8 * (c & 1));
            }
          }
        } else {
          // the parts lie in V's place, in Q's, and in that of the copy of S
          for (int c = 0; ok && c < nt; ++c) {
            const int x = c & 1, use = c >> 1;
            if (!(ok = tc::mbar_wait(bar + L::ld_full + 8 * x, use & 1) && tc::mbar_wait(bar + (x ? L::v_hi : L::kv_ok), use & 1))) break;
            // (who wrote V' of this tile has read the sum of tile c - 2 before)
            tc::tc_fence_after();
            issue_ds(c, L::kS, L::kColDs - 128 * (c & 1), false);     // its place is free first
            tc::mma_commit(bar + L::lo_done);
            issue_ds(c, L::kQ, L::kColDs - 128 * (c & 1), true);
            issue_ds(c, L::kV, L::kColDs - 128 * (c & 1), true);
            tc::mma_commit(bar + L::ds_full + 8 * (c & 1));
            tc::mma_commit(bar + L::ld_empty + 8 * (c & 1));
          }
        }
        tc::mma_commit(bar + L::fin);
        tc::mbar_wait(bar + L::fin, 0);
      }
    }
  } else if (warp >= 8 && warp < 12) {
    if constexpr (kOut) linear_output_role<D>(tc::smem_u32(smem), tmem, n_tok);
    else tc::setmaxnreg_dec<kPlRegs2>();
  } else {
    const int flags = has_src | heads << 1;
    if (!kOut || three) linear_state_role<D, kOut, true>(tc::smem_u32(smem), tmem, n_tok, nds, flags);
    else linear_state_role<D, kOut, false>(tc::smem_u32(smem), tmem, n_tok, nds, flags);
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Between the two: the k-th sequence of several segments turns what each of
// its segments adds (entry s + 1 for segment s) into the state that enters
// segment s (entry s), and hands on the last.
// Four state values per thread.
constexpr int kPlScanThreads = 256;

template <int D>
__global__ void __launch_bounds__(kPlScanThreads)
linear_packed_scan_kernel(const float* __restrict__ lambda, const int32_t* __restrict__ cu,
                          const int32_t* __restrict__ slots, const float* state_in, float* state_out, float* ws,
                          int tokens, int n_seqs, int n_slots, int H, int seg_tokens, int entries) {
  __shared__ PlUnit unit;
  if (threadIdx.x < 32) {
    // the k-th sequence that has more than one segment
    int k = blockIdx.y, base = 0;
    PlUnit u = {-1, 0, 0, 0};
    const int lane = threadIdx.x;
    SeqLengths walk;
    for (int i0 = 0; i0 < n_seqs; i0 += 32) {
      int e = segments_of(walk.next(cu, n_seqs, tokens, i0), seg_tokens);
      e = e < 2 ? 0 : e + 1;
      const unsigned multi = __ballot_sync(0xffffffffu, e > 0);
      if (k < __popc(multi)) {
        const int w = __fns(multi, 0, k + 1);
        u.seq = i0 + w;
        u.n_seg = __shfl_sync(0xffffffffu, e, w) - 1;
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
  // the plan has room for all sequences that are not skipped; bounds that another
  // stream changes while the call runs may still ask for more
  if (u.ws + u.n_seg + 1 > entries) {
    if (threadIdx.x == 0) set_status(kStatusBounds);
    return;
  }
  const int slot = take_slot(slots, u.seq, n_slots);
  const long long e = 4 * ((long long)blockIdx.x * kPlScanThreads + threadIdx.x);
  const long long per = (long long)H * D * D;
  if (e >= per) return;
  const float lam = lambda[e / (D * D)];
  const float whole = decay_pow(lam, seg_tokens);
  const int n = u.n_seg;
  const float rest = decay_pow(lam, cu[u.seq + 1] - cu[u.seq] - (n - 1) * seg_tokens);
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (state_in && slot >= 0) S = *reinterpret_cast<const float4*>(state_in + slot * per + e);
  float* p = ws + u.ws * per + e;
  *reinterpret_cast<float4*>(p) = S;           // state_out may be state_in: the outputs read it from here
  p += per;
  for (int s0 = 0; s0 < n; s0 += 8) {          // eight sums in flight
    float4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s0 + i < n) x[i] = *reinterpret_cast<const float4*>(p + (s0 + i) * per);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s0 + i < n) {
        const bool end = s0 + i + 1 == n;
        const float f = end ? rest : whole;
        S.x = fmaf(f, S.x, x[i].x);
        S.y = fmaf(f, S.y, x[i].y);
        S.z = fmaf(f, S.z, x[i].z);
        S.w = fmaf(f, S.w, x[i].w);
        if (!end) *reinterpret_cast<float4*>(p + (s0 + i) * per) = S;
      }
  }
  if (state_out && slot >= 0) *reinterpret_cast<float4*>(state_out + slot * per + e) = S;
}

}  // namespace sala
