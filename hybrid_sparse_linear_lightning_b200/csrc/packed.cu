// Entry points for packed batches: prompts of different lengths in one call,
// one token for each of many requests.
#include <algorithm>
#include <type_traits>

#include "host.cuh"
#include "packed_attn.cuh"
#include "packed_decode.cuh"
#include "packed_norm.cuh"
#include "packed_linear.cuh"
#include "packed_step.cuh"

using namespace sala;

namespace sala {
// Reads and clears this translation unit's status word.
cudaError_t packed_take_status(unsigned* bits) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *bits = v;
  return e;
}
}  // namespace sala

namespace {

using bf16 = __nv_bfloat16;

inline bool dtype_ok(sala_dtype t) { return t == SALA_F32 || t == SALA_BF16; }
inline bool dim_ok(int d) { return d == 64 || d == 128; }

sala_status check_qk_norm(const sala_qk_norm_desc* d) {
  if (!d || d->tokens < 1 || d->q_heads < 1 || d->k_heads < 1 || !dtype_ok(d->dtype))
    return SALA_ERR_INVALID_ARG;
  if (!(d->rms_eps >= 0.f) || !(d->rope_base > 0.f)) return SALA_ERR_INVALID_ARG;
  if (!dim_ok(d->head_dim)) return SALA_ERR_UNSUPPORTED;
  if ((int64_t)d->q_heads + d->k_heads > 8192) return SALA_ERR_UNSUPPORTED;
  return SALA_OK;
}

// Head counts of grouped attention: a group's heads share the 128 rows of a
// tensor-core tile.
sala_status check_heads(int q_heads, int kv_heads, int head_dim) {
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0) return SALA_ERR_INVALID_ARG;
  if (!dim_ok(head_dim) || q_heads / kv_heads > 128 || q_heads > 8192) return SALA_ERR_UNSUPPORTED;
  return SALA_OK;
}

sala_status check_dense(const sala_dense_desc* d) {
  if (!d || d->tokens < 1 || d->n_seqs < 1 || !dtype_ok(d->dtype) || !isfinite(d->scale))
    return SALA_ERR_INVALID_ARG;
  const sala_status s = check_heads(d->q_heads, d->kv_heads, d->head_dim);
  if (s != SALA_OK) return s;
  return d->dtype == SALA_BF16 ? SALA_OK : SALA_ERR_UNSUPPORTED;
}

sala_status check_packed_linear(const sala_packed_linear_desc* d) {
  if (!d || d->tokens < 1 || d->n_seqs < 1 || d->n_slots < 1 || d->heads < 1 ||
      !dtype_ok(d->dtype) || !isfinite(d->scale))
    return SALA_ERR_INVALID_ARG;
  if (!dim_ok(d->head_dim) || d->heads > 8192) return SALA_ERR_UNSUPPORTED;
  return SALA_OK;
}

sala_status check_prefix(const sala_prefix_desc* d) {
  if (!d || d->batch < 1 || d->prefix_len < 0 || d->n_slots < 1 || d->cache_capacity < 1 ||
      !dtype_ok(d->dtype) || !isfinite(d->scale))
    return SALA_ERR_INVALID_ARG;
  const sala_status s = check_heads(d->q_heads, d->kv_heads, d->head_dim);
  if (s != SALA_OK) return s;
  // more cache rows than any card holds; keys are counted in 32 bits
  if (d->cache_capacity > 0x7fffffffll / d->n_slots) return SALA_ERR_UNSUPPORTED;
  return d->dtype == SALA_BF16 ? SALA_OK : SALA_ERR_UNSUPPORTED;
}

inline float softmax_scale(float scale, int head_dim) {
  return scale > 0.f ? scale : 1.0f / sqrtf((float)head_dim);
}

template <typename T, int D>
sala_status run_qk_norm(const sala_qk_norm_desc* d, const void* q, const void* k, const float* wq,
                        const float* wk, const int32_t* pos, void* qn, void* kn, cudaStream_t st) {
  // several tokens per CTA only where there are CTAs enough to fill the card (32 + 32
  // heads of 128: 8 tokens 3.4 us against 8.0 with four, 1024 tokens 8.4 against 9.7,
  // 2048 14.1 and 14.5, 16384 110 against 103)
  const int tpc = d->tokens >= 2048 ? kQkNormMaxTokens : 1;
  // the last frequency table stays: forming one takes longer than a small launch
  static thread_local float base = 0.f;
  static thread_local RopeFreq freq;
  if (pos && base != d->rope_base) {
    freq = rope_freq(D, d->rope_base);
    base = d->rope_base;
  }
  qk_norm_kernel<T, D><<<(d->tokens + tpc - 1) / tpc, kQkNormThreads, 0, st>>>(
      static_cast<const T*>(q), static_cast<const T*>(k), wq, wk, pos, static_cast<bf16*>(qn),
      static_cast<bf16*>(kn), d->tokens, tpc, d->q_heads, d->k_heads, freq, d->rms_eps);
  return launch_status();
}

template <typename T, int D>
sala_status run_step(const sala_packed_linear_desc* d, const void* q, const void* k, const void* v,
                     const void* gate, const float* lambda, const int32_t* slots, float* state,
                     void* out, cudaStream_t st) {
  const long long units = (long long)d->n_seqs * d->heads;
  auto launch = [&](auto kern, int split) {
    kern<<<(unsigned)(units * split), kStepThreads, 0, st>>>(
        static_cast<const bf16*>(q), static_cast<const bf16*>(k), static_cast<const T*>(v),
        static_cast<const T*>(gate), lambda, slots, state, static_cast<T*>(out), d->heads,
        d->n_slots, d->scale);
    return launch_status();
  };
  // 32 columns a CTA where whole states would leave a third of the SMs idle (d = 128:
  // 4 states 2.1 us against 2.8 whole, 96 states 3.1 against 3.2, 128 states 3.5
  // against 3.2, 4096 states 87 against 81)
  if (3 * units < 2 * std::max(device_sms(), 1)) return launch(linear_step_kernel<T, D, 32>, D / 32);
  return launch(linear_step_kernel<T, D, D>, 1);
}

template <int D>
sala_status run_dense(const sala_dense_desc* d, const void* q, const void* k, const void* v,
                      const void* gate, const int32_t* cu, void* out, float sl2, cudaStream_t st) {
  const int G = d->q_heads / d->kv_heads, Tt = 128 / G;
  CUtensorMap qm, km, vm;
  const uint64_t kv_cols = (uint64_t)d->kv_heads * D;
  if (!make_tmap_rows(&qm, q, D, d->q_heads, d->tokens, G, Tt) ||
      !make_tmap_bf16(&km, k, kv_cols, d->tokens, 64, kPaBlock) ||
      !make_tmap_bf16(&vm, v, kv_cols, d->tokens, 64, kPaBlock))
    return SALA_ERR_CUDA;
  auto kern = dense_attn_kernel<D>;
  const size_t smem = PaLayout<D>::kBytes + 1024;
  static std::atomic<uint64_t> allowed{0};
  if (allow_smem_once(kern, smem, &allowed) != cudaSuccess) return SALA_ERR_CUDA;
  // every sequence ends in a pair of tiles that may be part empty
  const int64_t pairs = (int64_t)d->tokens / (2 * Tt) + d->n_seqs;
  if (pairs * d->kv_heads > 0x7fffffffll) return SALA_ERR_UNSUPPORTED;
  int kmax = 0;      // class of the longest sequence there can be, in key blocks
  while ((int64_t)kPaBlock << (kmax + 1) <= (int64_t)d->tokens + kPaBlock - 1) ++kmax;
  kern<<<(unsigned)(pairs * d->kv_heads), kPaThreads, smem, st>>>(
      qm, km, vm, cu, static_cast<const bf16*>(v), static_cast<const bf16*>(gate),
      static_cast<bf16*>(out), d->tokens, d->n_seqs, d->q_heads, d->kv_heads, Tt, kmax, sl2);
  return launch_status();
}

// How packed prompts are cut for linear attention.
struct LinearPlan {
  int seg_tokens;
  int64_t extra;        // most segments behind a sequence's first
  int64_t multi;        // most sequences of several segments
  int64_t entries;      // states of theirs: before and behind each segment
  size_t total;         // workspace: the states that enter them
};

LinearPlan linear_plan(const sala_packed_linear_desc* d) {
  constexpr int64_t kSms = 148;
  LinearPlan p;
  const int64_t groups = (d->heads + 128 / d->head_dim - 1) / (128 / d->head_dim);
  const int64_t tiles = ((int64_t)d->tokens + kPlTile - 1) / kPlTile * groups;
  // Tiles per segment: whole waves of CTAs over the card, taking the tokens for
  // one sequence and three tiles' time for what a segment costs besides.  With
  // sequences enough to fill the card twice, only what one SM would take more than
  // twice the whole card's time for is cut: the sums of the segments read keys and
  // values once more (13 prompts of up to 23 tiles at 32 heads: 190 us whole, 197
  // cut at 17).
  const int64_t per_head = ((int64_t)d->tokens + kPlTile - 1) / kPlTile;
  int64_t seg = per_head;
  if (d->n_seqs * groups < 2 * kSms) {
    int64_t best = INT64_MAX;
    for (int64_t n = 1; n <= 64; ++n) {
      const int64_t len = (per_head + n - 1) / n;
      const int64_t cost = (n * groups + kSms - 1) / kSms * (len + 3);
      if (cost < best) {
        best = cost;
        seg = len;
      }
    }
  } else {
    seg = tiles / 64;
  }
  // Down to two tiles, where there are 8 in all and a sequence has one on average:
  // prompts of 1024, 3000 and 8192 tokens at 4 heads of 64 37 us, 38 and 39 against
  // 72, 84 and 84 with 8 tiles, at 32 heads of 128 37, 70 and 158 against 63, 81 and
  // 158.  Shorter calls are left whole, as the two launches more take longer (600
  // tokens in 4 prompts, 32 heads of 128: 30 us, 45 cut at two), and so are many
  // short prompts (20 of 1500 tokens, 8 heads of 128: 37 against 46).
  const bool whole = per_head < 8 || d->tokens < (int64_t)kPlTile * d->n_seqs;
  seg = std::min<int64_t>(std::max<int64_t>(seg, whole ? 8 : 2), 1 << 20);
  p.seg_tokens = (int)(seg * kPlTile);
  p.extra = d->tokens / p.seg_tokens;
  p.multi = std::min<int64_t>(p.extra, d->n_seqs);
  p.entries = p.extra + 2 * p.multi;
  p.total = align_up((size_t)p.entries * d->heads * d->head_dim * d->head_dim * sizeof(float));
  return p;
}

template <int D>
sala_status run_linear(const sala_packed_linear_desc* d, const void* q, const void* k, const void* v,
                       const void* gate, const float* lambda, const int32_t* cu, const int32_t* slots,
                       const float* state_in, float* state_out, void* out, float* ws, cudaStream_t st) {
  const LinearPlan p = linear_plan(d);
  const int64_t groups = (d->heads + 128 / D - 1) / (128 / D);
  CUtensorMap qm, km, vm, gm;
  const uint64_t cols = (uint64_t)d->heads * D;
  if (!make_tmap_bf16(&qm, q, cols, d->tokens, 64, kPlTile) ||
      !make_tmap_bf16(&km, k, cols, d->tokens, 64, kPlTile) ||
      !make_tmap_bf16(&vm, v, cols, d->tokens, 64, kPlTile) ||
      !make_tmap_bf16(&gm, gate, cols, d->tokens, 64, kPlTile))
    return SALA_ERR_CUDA;
  // states as rows of D fp32, read and written in boxes of 32 columns x one head
  CUtensorMap sim = {}, som = {}, wsm = {};
  const uint64_t rows = (uint64_t)d->n_slots * d->heads * D, ws_rows = (uint64_t)p.entries * d->heads * D;
  if (rows > 0x7fffffffull || ws_rows > 0x7fffffffull) return SALA_ERR_UNSUPPORTED;
  if ((state_in && !make_tmap_f32(&sim, state_in, D, rows, 32, D)) ||
      (state_out && !make_tmap_f32(&som, state_out, D, rows, 32, D)) ||
      (p.extra > 0 && !make_tmap_f32(&wsm, ws, D, ws_rows, 32, D)))
    return SALA_ERR_CUDA;
  const size_t smem = PlLayout::kBytes + 1024;
  const int64_t units = (p.extra + d->n_seqs) * groups;
  if (units > 0x7fffffffll) return SALA_ERR_UNSUPPORTED;
  static std::atomic<uint64_t> allowed[2];
  auto launch = [&](auto kern, int64_t grid, std::atomic<uint64_t>* done) {
    if (allow_smem_once(kern, smem, done) != cudaSuccess) return SALA_ERR_CUDA;
    kern<<<(unsigned)grid, kPlThreads, smem, st>>>(
        qm, km, vm, gm, sim, som, wsm, static_cast<const bf16*>(v), static_cast<const bf16*>(gate), lambda, cu,
        slots, state_in, state_out, static_cast<bf16*>(out), d->tokens, d->n_seqs, d->n_slots, d->heads, p.seg_tokens,
        d->scale);
    return launch_status();
  };
  if (p.extra > 0) {
    sala_status s = launch(linear_packed_kernel<D, false>, (p.extra + p.multi) * groups, &allowed[0]);
    if (s != SALA_OK) return s;
    const int64_t per = (int64_t)d->heads * D * D / 4;
    const dim3 grid((unsigned)((per + kPlScanThreads - 1) / kPlScanThreads),
                    (unsigned)p.multi);
    if (grid.y > 65535) return SALA_ERR_UNSUPPORTED;
    linear_packed_scan_kernel<D><<<grid, kPlScanThreads, 0, st>>>(
        lambda, cu, slots, state_in, state_out, ws, d->tokens, d->n_seqs, d->n_slots, d->heads, p.seg_tokens,
        (int)p.entries);
    s = launch_status();
    if (s != SALA_OK) return s;
  }
  return launch(linear_packed_kernel<D, true>, units, &allowed[1]);
}

// How a decode step over a shared prefix is cut up.
struct PrefixPlan {
  int Tt, pairs;                 // requests per row tile, pairs of row tiles
  int mtiles;                    // 16-row tiles of a group
  bool walked;                   // the prefix is read with each request's own keys
  int cluster;                   // CTAs that share a request's keys
  int split_blocks, n_split;     // else: key blocks per part of the prefix, parts
  size_t o, ml, total;           // workspace: parts of O, of (maximum, sum)
};

// CTAs per cluster for `units` of up to `keys` keys each: clusters grow until
// their CTAs fill the card twice over (two CTAs live on an SM), as long as every
// warp has eight steps, and over SMs that would stay idle down to two steps.
int own_cluster(int64_t units, int64_t keys) {
  int cs = 1;
  while (cs < kOwnMaxCluster && units * cs < 4 * 148 && keys > (int64_t)cs * kOwnWarps * 16 * 8) cs *= 2;
  while (cs < kOwnMaxCluster && units * cs * 2 <= 148 && keys > (int64_t)cs * kOwnWarps * 16 * 2) cs *= 2;
  return cs;
}

PrefixPlan prefix_plan(const sala_prefix_desc* d) {
  constexpr int kSms = 148;
  PrefixPlan p = {};
  p.Tt = 128 / (d->q_heads / d->kv_heads);
  const int64_t tiles = ((int64_t)d->batch + p.Tt - 1) / p.Tt;
  p.pairs = (int)((tiles + 1) / 2);
  const int64_t blocks = ((int64_t)d->prefix_len + kPaBlock - 1) / kPaBlock;
  p.mtiles = (d->q_heads / d->kv_heads + 15) / 16;
  // walked where that reads little and is short for each warp: packed_decode.cuh
  // has both sides
  const int64_t own_units = (int64_t)d->batch * d->kv_heads * p.mtiles;
  p.cluster = own_cluster(own_units, d->cache_capacity + d->prefix_len);
  p.walked = (double)own_units * d->prefix_len * d->head_dim * 4 <= 24e6 &&
             d->prefix_len <= p.cluster * kOwnWarps * 16 * kOwnMaxWalk;
  if (!p.walked) p.cluster = own_cluster(own_units, d->cache_capacity);
  if (blocks > 0 && !p.walked) {
    // the number of parts whose waves of units take the fewest block times; a
    // unit costs two blocks' time to start and to hand over its part
    const int64_t units = d->kv_heads * (int64_t)p.pairs;
    int64_t best = INT64_MAX;
    for (int64_t n = 1; n <= std::min<int64_t>(blocks, kOwnMaxSplits); ++n) {
      const int64_t per = (blocks + n - 1) / n;
      const int64_t cost = ((units * n + kSms - 1) / kSms) * (per + 2);
      if (cost < best) {
        best = cost;
        p.split_blocks = (int)per;
      }
    }
    p.n_split = (int)((blocks + p.split_blocks - 1) / p.split_blocks);
  }
  const size_t rows = (size_t)p.n_split * d->batch * d->q_heads;
  p.o = 0;
  p.ml = align_up(rows * d->head_dim * sizeof(float));
  p.total = rows ? p.ml + align_up(rows * sizeof(float2)) : 0;
  return p;
}

template <int D>
sala_status run_prefix(const sala_prefix_desc* d, const void* q, const void* k, const void* v,
                       const void* gate, const void* pk, const void* pv, void* kc, void* vc,
                       const int32_t* lens, const int32_t* slots, void* out, uint8_t* ws,
                       cudaStream_t st) {
  const PrefixPlan p = prefix_plan(d);
  const float sl2 = softmax_scale(d->scale, D) * 1.4426950408889634f;
  float* part_o = reinterpret_cast<float*>(ws + p.o);
  float2* part_ml = reinterpret_cast<float2*>(ws + p.ml);
  const int G = d->q_heads / d->kv_heads;
  if (p.n_split > 0) {
    CUtensorMap qm, km, vm;
    const uint64_t kv_cols = (uint64_t)d->kv_heads * D;
    if (!make_tmap_rows(&qm, q, D, d->q_heads, d->batch, G, p.Tt) ||
        !make_tmap_bf16(&km, pk, kv_cols, d->prefix_len, 64, kPaBlock) ||
        !make_tmap_bf16(&vm, pv, kv_cols, d->prefix_len, 64, kPaBlock))
      return SALA_ERR_CUDA;
    const size_t smem = PaLayout<D>::kBytes + 1024;
    static std::atomic<uint64_t> allowed{0};
    if (allow_smem_once(prefix_attn_kernel<D>, smem, &allowed) != cudaSuccess) return SALA_ERR_CUDA;
    const int64_t units = (int64_t)p.n_split * p.pairs * d->kv_heads;
    prefix_attn_kernel<D><<<(unsigned)units, kPaThreads, smem, st>>>(
        qm, km, vm, part_o, part_ml, d->batch, d->q_heads, d->kv_heads, p.Tt, p.pairs, d->prefix_len,
        p.split_blocks, sl2);
    const sala_status s = launch_status();
    if (s != SALA_OK) return s;
  }
  const int mtiles = p.mtiles, walked = p.walked ? d->prefix_len : 0, cs = p.cluster;
  const int64_t units = (int64_t)d->batch * d->kv_heads * mtiles;
  if (units * cs > 0x7fffffffll) return SALA_ERR_UNSUPPORTED;
  auto kern = own_attn_kernel<D>;
  const size_t smem = OwnLayout<D>::kBytes;
  static std::atomic<uint64_t> allowed{0};
  if (allow_smem_once(kern, smem, &allowed) != cudaSuccess) return SALA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cs));
  cfg.blockDim = dim3(32 * kOwnWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.n_split > 0 ? 2 : 1;    // alone, the kernel starts after what came before it
  cudaLaunchKernelEx(&cfg, kern, static_cast<const bf16*>(q), static_cast<const bf16*>(k),
                     static_cast<const bf16*>(v), static_cast<const bf16*>(gate), static_cast<const bf16*>(pk),
                     static_cast<const bf16*>(pv), static_cast<bf16*>(kc), static_cast<bf16*>(vc), lens, slots, static_cast<const float*>(part_o),
                     static_cast<const float2*>(part_ml), static_cast<bf16*>(out), d->batch, d->q_heads,
                     d->kv_heads, mtiles, walked, p.n_split, (long long)d->cache_capacity, d->n_slots, sl2);
  return launch_status();
}

}  // namespace

extern "C" {

sala_status sala_qk_norm(const sala_qk_norm_desc* d, const void* q, const void* k, const float* wq,
                         const float* wk, const int32_t* positions, void* q_norm, void* k_norm,
                         void* stream) {
  const sala_status s = check_qk_norm(d);
  if (s != SALA_OK) return s;
  if (!aligned16(q) || !aligned16(k) || !aligned16(wq) || !aligned16(wk) || !aligned16(q_norm) ||
      !aligned16(k_norm) || !aligned4_or_null(positions))
    return SALA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->dtype == SALA_BF16) {
    if (d->head_dim == 128) return run_qk_norm<bf16, 128>(d, q, k, wq, wk, positions, q_norm, k_norm, st);
    return run_qk_norm<bf16, 64>(d, q, k, wq, wk, positions, q_norm, k_norm, st);
  }
  if (d->head_dim == 128) return run_qk_norm<float, 128>(d, q, k, wq, wk, positions, q_norm, k_norm, st);
  return run_qk_norm<float, 64>(d, q, k, wq, wk, positions, q_norm, k_norm, st);
}

size_t sala_dense_workspace_size(const sala_dense_desc* d) {
  if (check_dense(d) != SALA_OK) return 0;
  return 0;
}

sala_status sala_dense_prefill(const sala_dense_desc* d, const void* q_norm, const void* k_norm,
                               const void* v, const void* gate, const int32_t* cu_seqlens,
                               void* out, void* workspace, size_t ws_bytes, void* stream) {
  const sala_status s = check_dense(d);
  if (s != SALA_OK) return s;
  if (!aligned16(q_norm) || !aligned16(k_norm) || !aligned16(v) || !aligned16(gate) ||
      !aligned4(cu_seqlens) || !aligned16(out))
    return SALA_ERR_INVALID_ARG;
  (void)workspace;
  (void)ws_bytes;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const float sl2 = softmax_scale(d->scale, d->head_dim) * 1.4426950408889634f;
  if (d->head_dim == 128) return run_dense<128>(d, q_norm, k_norm, v, gate, cu_seqlens, out, sl2, st);
  return run_dense<64>(d, q_norm, k_norm, v, gate, cu_seqlens, out, sl2, st);
}

size_t sala_linear_packed_workspace_size(const sala_packed_linear_desc* d) {
  if (check_packed_linear(d) != SALA_OK || d->dtype != SALA_BF16) return 0;
  return linear_plan(d).total;
}

sala_status sala_linear_packed_prefill(const sala_packed_linear_desc* d, const void* q_norm,
                                       const void* k_norm, const void* v, const void* gate,
                                       const float* lambda, const int32_t* cu_seqlens,
                                       const int32_t* slots, const float* state_in,
                                       float* state_out, void* out, void* workspace,
                                       size_t ws_bytes, void* stream) {
  const sala_status s = check_packed_linear(d);
  if (s != SALA_OK) return s;
  if (d->dtype != SALA_BF16) return SALA_ERR_UNSUPPORTED;
  if (!aligned16(q_norm) || !aligned16(k_norm) || !aligned16(v) || !aligned16(gate) ||
      !aligned4(lambda) || !aligned4(cu_seqlens) || !aligned4_or_null(slots) ||
      !aligned16_or_null(state_in) || !aligned16_or_null(state_out) || !aligned16(out))
    return SALA_ERR_INVALID_ARG;
  if (!slots && d->n_slots < d->n_seqs) return SALA_ERR_INVALID_ARG;
  const size_t need = linear_plan(d).total;
  if (need > 0 && (!workspace || ws_bytes < need)) return SALA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return SALA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* ws = static_cast<float*>(workspace);
  if (d->head_dim == 128)
    return run_linear<128>(d, q_norm, k_norm, v, gate, lambda, cu_seqlens, slots, state_in, state_out, out, ws, st);
  return run_linear<64>(d, q_norm, k_norm, v, gate, lambda, cu_seqlens, slots, state_in, state_out, out, ws, st);
}

sala_status sala_linear_packed_step(const sala_packed_linear_desc* d, const void* q_norm,
                                    const void* k_norm, const void* v, const void* gate,
                                    const float* lambda, const int32_t* slots, float* state,
                                    void* out, void* stream) {
  const sala_status s = check_packed_linear(d);
  if (s != SALA_OK) return s;
  if (d->tokens != d->n_seqs) return SALA_ERR_INVALID_ARG;
  if (!aligned16(q_norm) || !aligned16(k_norm) || !aligned16(v) || !aligned16(gate) ||
      !aligned4(lambda) || !aligned4_or_null(slots) || !aligned16(state) || !aligned16(out))
    return SALA_ERR_INVALID_ARG;
  if (!slots && d->n_slots < d->n_seqs) return SALA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->dtype == SALA_BF16) {
    if (d->head_dim == 128) return run_step<bf16, 128>(d, q_norm, k_norm, v, gate, lambda, slots, state, out, st);
    return run_step<bf16, 64>(d, q_norm, k_norm, v, gate, lambda, slots, state, out, st);
  }
  if (d->head_dim == 128) return run_step<float, 128>(d, q_norm, k_norm, v, gate, lambda, slots, state, out, st);
  return run_step<float, 64>(d, q_norm, k_norm, v, gate, lambda, slots, state, out, st);
}

size_t sala_prefix_workspace_size(const sala_prefix_desc* d) {
  if (check_prefix(d) != SALA_OK) return 0;
  return prefix_plan(d).total;
}

sala_status sala_prefix_decode(const sala_prefix_desc* d, const void* q_norm, const void* k_norm,
                               const void* v, const void* gate, const void* prefix_k,
                               const void* prefix_v, void* k_cache, void* v_cache,
                               const int32_t* lens, const int32_t* slots, void* out,
                               void* workspace, size_t ws_bytes, void* stream) {
  const sala_status s = check_prefix(d);
  if (s != SALA_OK) return s;
  if (!aligned16(q_norm) || !aligned16(k_norm) || !aligned16(v) || !aligned16(gate) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned4(lens) || !aligned4_or_null(slots) ||
      !aligned16(out))
    return SALA_ERR_INVALID_ARG;
  if (d->prefix_len > 0 && (!aligned16(prefix_k) || !aligned16(prefix_v))) return SALA_ERR_INVALID_ARG;
  if (!slots && d->n_slots < d->batch) return SALA_ERR_INVALID_ARG;
  const size_t need = prefix_plan(d).total;
  if (need > 0 && (!workspace || ws_bytes < need)) return SALA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return SALA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (d->head_dim == 128)
    return run_prefix<128>(d, q_norm, k_norm, v, gate, prefix_k, prefix_v, k_cache, v_cache, lens, slots, out, ws, st);
  return run_prefix<64>(d, q_norm, k_norm, v, gate, prefix_k, prefix_v, k_cache, v_cache, lens, slots, out, ws, st);
}

}  // extern "C"
