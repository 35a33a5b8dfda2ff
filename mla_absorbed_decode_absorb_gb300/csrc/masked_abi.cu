// The C entry points of decoding with drafted tokens and with a limited view of the
// cache: argument validation, split planning and the launches.
#include <limits.h>

#include "internal.cuh"
#include "view.cuh"

namespace {

using namespace mla;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

mla_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

bool view_ok(int window, int sinks) { return window >= 0 && sinks >= 0 && (window > 0 || sinks == 0); }

// From this many query tokens on the finish takes the kernel with a head's weights resident (for at most two splits).
constexpr int kManyTokens = 33;  // 64 tokens: 10.2 us against 12.5 for the other, 1024: 68 against 175; 32: 9.7 against 6.4

// The split of a query's view over pairs of CTAs.  Automatic choice: the split count of least time, in ns: waves of as
// many units as pairs fit on the GPU at once, each of a split's tiles (two pages) and of what a unit costs besides
// (query load, pipeline fill, epilogue: six tiles); and the partials, which are written and read in float32 (384
// tokens of 47 tiles over the FP8 cache: 371 us with one split, 429 with two; 8 tokens of four tiles: 21.8 us with one
// split, 18.3 with four).  Where the units alone fill more than a wave, splits have to gain a sixth: the plan knows the
// longest sequence only, and the units of a ragged batch, longest first, fill the last wave by themselves (8 x 13
// tokens of 1000 to 5000: 92 us with one split, 105 with two; all of 5000: 143 and 130).
constexpr int kFixedTiles = 6, kTileNs = 1450;
// What the merge of splits adds to the finish: by its bytes in the kernel for many tokens; in the other one a split's
// turn, and 7 us for every further wave of its CTAs, which hold 64 rows each (8 tokens of 8 splits 8.4 us, of 9 16.9).
// Waves are counted over the SMs that pairs of CTAs fill, 148 of the 152 here; over all of them a few plans of very long
// contexts had one split more and took 1 to 2% longer (16 x 5 tokens of 32000: 544 us for 534).
inline int64_t merge_ns(int64_t queries, int splits, int64_t slots) {
  if (splits == 1) return 0;
  if (splits <= 2 && queries >= kManyTokens) return 30 * queries * splits;
  const int64_t tile = splits > 2 ? 64 / splits : 32, ctas = kHeads * ((queries + tile - 1) / tile);
  return 100 * splits + 7000 * ((ctas - 1) / (2 * slots));
}

mla_status masked_plan(int B, int n_q, int max_kv_len, int window, int sinks, int split_pages, SplitPlan* plan) {
  if (B < 0 || n_q < 1 || n_q > MLA_MAX_TREE || max_kv_len < n_q || split_pages < 0 || !view_ok(window, sinks))
    return MLA_ERR_INVALID_ARG;
  const int64_t queries = static_cast<int64_t>(B) * n_q;
  if (queries * kHeads > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  plan->short_path = false;
  plan->max_pages = max_view_pages(n_q, max_kv_len, window, sinks);
  if (split_pages == 0) {
    const int64_t slots = masked_cluster_slots(), units = queries > 0 ? queries : 1;
    const int max_tiles = (plan->max_pages + 1) / 2;
    int64_t best = -1;
    for (int s = 1; s <= max_tiles && s <= 64; ++s) {
      const int tiles = (max_tiles + s - 1) / s;
      const int64_t waves = (units * ((max_tiles + tiles - 1) / tiles) + slots - 1) / slots;
      int64_t cost = waves * (tiles + kFixedTiles) * kTileNs + merge_ns(units, (max_tiles + tiles - 1) / tiles, slots);
      if (tiles < max_tiles && units > slots) cost += cost / 6;
      if (best < 0 || cost < best) {
        best = cost;
        split_pages = 2 * tiles;
      }
    }
  }
  plan->split_pages = split_pages < plan->max_pages ? split_pages : plan->max_pages;
  plan->num_splits = (plan->max_pages + plan->split_pages - 1) / plan->split_pages;
  if (2 * queries * plan->num_splits > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  if (plan->num_splits > kMaxMaskedSplits) {  // the merge takes no more: longer splits
    plan->split_pages = (plan->max_pages + kMaxMaskedSplits - 1) / kMaxMaskedSplits;
    plan->num_splits = (plan->max_pages + plan->split_pages - 1) / plan->split_pages;
  }
  const size_t rows = static_cast<size_t>(queries) * plan->num_splits * kHeads;
  plan->o_part_bytes = (rows * kLatent * sizeof(float) + 255) / 256 * 256;
  plan->lse_part_bytes = (rows * sizeof(float) + 255) / 256 * 256;
  plan->workspace_bytes = plan->num_splits > 1 ? plan->o_part_bytes + plan->lse_part_bytes : 0;
  return MLA_OK;
}

bool workspace_ok(const SplitPlan& plan, const void* workspace, size_t bytes) {
  return plan.workspace_bytes == 0 || (workspace != nullptr && bytes >= plan.workspace_bytes && aligned(workspace, 16));
}

// The checks and the launch of both cache formats.
mla_status masked_partial(MaskedArgs a, int split_pages, void* workspace, size_t workspace_bytes, float* o_latent,
                          float* lse, cudaStream_t stream) {
  SplitPlan plan;
  const mla_status s = masked_plan(a.B, a.n_q, a.max_kv_len, a.window, a.sinks, split_pages, &plan);
  if (s != MLA_OK) return s;
  if (a.B == 0) return MLA_OK;
  if (!a.q_abs || !a.page_table || !a.kv_lens || !o_latent || a.num_pages < 1 || a.pt_stride < 1)
    return MLA_ERR_INVALID_ARG;
  if (!aligned(a.q_abs, 16) || !aligned(o_latent, 16) || !aligned(a.words, 8)) return MLA_ERR_INVALID_ARG;
  if (a.num_pages > INT32_MAX / kPage) return MLA_ERR_UNSUPPORTED;
  if (!workspace_ok(plan, workspace, workspace_bytes)) return MLA_ERR_WORKSPACE;
  int* st = device_status_word();
  if (st == nullptr) return MLA_ERR_CUDA;
  float* o_out = o_latent;
  float* lse_out = lse;
  if (plan.num_splits > 1) {
    o_out = static_cast<float*>(workspace);
    lse_out = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.o_part_bytes);
  }
  return from_cuda(launch_decode_masked(a, plan, o_out, lse_out, st, stream));
}

mla_status append_tree(const mla_bf16* c_kv_new, const mla_bf16* k_pe_new, const mla_bf16* q_nope,
                       const mla_bf16* q_rope, const int32_t* seq_lens_before, const int32_t* depths,
                       const int32_t* page_table, int pt_stride, const mla_bf16* w_uk, const float* rope_table,
                       int rope_max_pos, mla_bf16* cache, uint8_t* c8, float* scale, uint16_t* kr, int64_t num_pages,
                       mla_bf16* q_abs, int B, int n_q, cudaStream_t stream) {
  if (B < 0 || n_q < 1 || n_q > MLA_MAX_TREE) return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(B) * n_q * kHeads > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  if (B == 0) return MLA_OK;
  if (!c_kv_new || !k_pe_new || !q_nope || !q_rope || !seq_lens_before || !depths || !page_table || !w_uk ||
      !rope_table || !q_abs)
    return MLA_ERR_INVALID_ARG;
  if (pt_stride < 1 || rope_max_pos < 1 || num_pages < 1) return MLA_ERR_INVALID_ARG;
  if (!aligned(c_kv_new, 16) || !aligned(cache, 16) || !aligned(c8, 16) || !aligned(q_nope, 16) ||
      !aligned(q_rope, 16) || !aligned(w_uk, 16) || !aligned(q_abs, 16))
    return MLA_ERR_INVALID_ARG;
  int* st = device_status_word();
  if (st == nullptr) return MLA_ERR_CUDA;
  return from_cuda(launch_append_absorb_q_tree(c_kv_new, k_pe_new, q_nope, q_rope, seq_lens_before, depths, page_table,
                                               pt_stride, w_uk, rope_table, rope_max_pos, cache, c8, scale, kr,
                                               num_pages, q_abs, B, n_q, st, stream));
}

mla_status accept(mla_bf16* cache, uint8_t* c8, float* scale, uint16_t* kr, int64_t num_pages,
                  const int32_t* page_table, int pt_stride, const int32_t* seq_lens_before, const int32_t* path,
                  const int32_t* counts, int B, int n_q, cudaStream_t stream) {
  if (B < 0 || n_q < 1 || n_q > MLA_MAX_TREE) return MLA_ERR_INVALID_ARG;
  if (B == 0) return MLA_OK;
  if (!page_table || !seq_lens_before || !path || !counts || num_pages < 1 || pt_stride < 1) return MLA_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || !aligned(c8, 16) || !aligned(scale, 4) || !aligned(kr, 16)) return MLA_ERR_INVALID_ARG;
  int* st = device_status_word();
  if (st == nullptr) return MLA_ERR_CUDA;
  return from_cuda(launch_accept_tokens(cache, c8, scale, kr, num_pages, page_table, pt_stride, seq_lens_before, path,
                                        counts, B, n_q, st, stream));
}

}  // namespace

extern "C" {

mla_status mla_tree_prepare(const int32_t* parents, const int32_t* seq_lens_before, int window, int sinks,
                            int32_t* depths, uint64_t* tree_mask, int B, int n_q, cudaStream_t stream) {
  if (B < 0 || n_q < 1 || n_q > MLA_MAX_TREE || !view_ok(window, sinks)) return MLA_ERR_INVALID_ARG;
  if (B == 0) return MLA_OK;
  if (!parents || !seq_lens_before || !depths || !tree_mask || !aligned(tree_mask, 8)) return MLA_ERR_INVALID_ARG;
  int* st = device_status_word();
  if (st == nullptr) return MLA_ERR_CUDA;
  return from_cuda(launch_tree_prepare(parents, seq_lens_before, window, sinks, depths, tree_mask, B, n_q, st, stream));
}

mla_status mla_append_absorb_q_tree(const mla_bf16* c_kv_new, const mla_bf16* k_pe_new, const mla_bf16* q_nope,
                                    const mla_bf16* q_rope, const int32_t* seq_lens_before, const int32_t* depths,
                                    const int32_t* page_table, int pt_stride, const mla_bf16* w_uk,
                                    const float* rope_table, int rope_max_pos, mla_bf16* cache, int64_t num_pages,
                                    mla_bf16* q_abs, int B, int n_q, cudaStream_t stream) {
  if (B > 0 && !cache) return MLA_ERR_INVALID_ARG;
  return append_tree(c_kv_new, k_pe_new, q_nope, q_rope, seq_lens_before, depths, page_table, pt_stride, w_uk,
                     rope_table, rope_max_pos, cache, nullptr, nullptr, nullptr, num_pages, q_abs, B, n_q, stream);
}

mla_status mla_append_absorb_q_tree_fp8(const mla_bf16* c_kv_new, const mla_bf16* k_pe_new, const mla_bf16* q_nope,
                                        const mla_bf16* q_rope, const int32_t* seq_lens_before, const int32_t* depths,
                                        const int32_t* page_table, int pt_stride, const mla_bf16* w_uk,
                                        const float* rope_table, int rope_max_pos, uint8_t* cache_c8,
                                        float* cache_scale, uint16_t* cache_kr, int64_t num_pages, mla_bf16* q_abs,
                                        int B, int n_q, cudaStream_t stream) {
  if (B > 0 && (!cache_c8 || !cache_scale || !cache_kr)) return MLA_ERR_INVALID_ARG;
  return append_tree(c_kv_new, k_pe_new, q_nope, q_rope, seq_lens_before, depths, page_table, pt_stride, w_uk,
                     rope_table, rope_max_pos, nullptr, cache_c8, cache_scale, cache_kr, num_pages, q_abs, B, n_q,
                     stream);
}

mla_status mla_masked_workspace_size(int B, int n_q, int max_kv_len, int window, int sinks, int split_pages,
                                     size_t* bytes) {
  SplitPlan plan;
  if (bytes == nullptr) return MLA_ERR_INVALID_ARG;
  const mla_status s = masked_plan(B, n_q, max_kv_len, window, sinks, split_pages, &plan);
  if (s == MLA_OK) *bytes = plan.workspace_bytes;
  return s;
}

mla_status mla_masked_num_splits(int B, int n_q, int max_kv_len, int window, int sinks, int split_pages,
                                 int* num_splits) {
  SplitPlan plan;
  if (num_splits == nullptr) return MLA_ERR_INVALID_ARG;
  const mla_status s = masked_plan(B, n_q, max_kv_len, window, sinks, split_pages, &plan);
  if (s == MLA_OK) *num_splits = plan.num_splits;
  return s;
}

mla_status mla_decode_attn_masked_partial(const mla_bf16* q_abs, const mla_bf16* cache, int64_t num_pages,
                                          const int32_t* page_table, int pt_stride, const int32_t* kv_lens,
                                          const uint64_t* tree_mask, const int32_t* depths, int window, int sinks,
                                          int B, int n_q, int max_kv_len, int split_pages, void* workspace,
                                          size_t workspace_bytes, float* o_latent, float* lse, cudaStream_t stream) {
  if (B > 0 && (!cache || !aligned(cache, 16))) return MLA_ERR_INVALID_ARG;
  const MaskedArgs a{q_abs,   cache,     nullptr,   nullptr, nullptr, num_pages, page_table, pt_stride,
                     kv_lens, tree_mask, depths,    window,  sinks,   B,         n_q,        max_kv_len};
  return masked_partial(a, split_pages, workspace, workspace_bytes, o_latent, lse, stream);
}

mla_status mla_decode_attn_masked_fp8_partial(const mla_bf16* q_abs, const uint8_t* cache_c8, const float* cache_scale,
                                              const uint16_t* cache_kr, int64_t num_pages, const int32_t* page_table,
                                              int pt_stride, const int32_t* kv_lens, const uint64_t* tree_mask,
                                              const int32_t* depths, int window, int sinks, int B, int n_q,
                                              int max_kv_len, int split_pages, void* workspace, size_t workspace_bytes,
                                              float* o_latent, float* lse, cudaStream_t stream) {
  if (B > 0 && (!cache_c8 || !cache_scale || !cache_kr || !aligned(cache_c8, 16) || !aligned(cache_scale, 16) ||
                !aligned(cache_kr, 16)))
    return MLA_ERR_INVALID_ARG;
  const MaskedArgs a{q_abs,   nullptr,   cache_c8, cache_scale, cache_kr, num_pages, page_table, pt_stride,
                     kv_lens, tree_mask, depths,   window,      sinks,    B,         n_q,        max_kv_len};
  return masked_partial(a, split_pages, workspace, workspace_bytes, o_latent, lse, stream);
}

mla_status mla_masked_combine_out_absorb(int B, int n_q, int max_kv_len, int window, int sinks, int split_pages,
                                         const void* workspace, size_t workspace_bytes, const float* o_latent,
                                         const mla_bf16* w_uv, mla_bf16* out, float* lse, cudaStream_t stream) {
  SplitPlan plan;
  const mla_status s = masked_plan(B, n_q, max_kv_len, window, sinks, split_pages, &plan);
  if (s != MLA_OK) return s;
  if (B == 0) return MLA_OK;
  if (!w_uv || !out || (plan.num_splits == 1 && !o_latent)) return MLA_ERR_INVALID_ARG;
  void* od = nullptr;
  if (!output_address(out, static_cast<size_t>(B) * n_q * kHeads * kNope * 2, &od)) return MLA_ERR_INVALID_ARG;
  if (!aligned(o_latent, 16) || !aligned(w_uv, 16) || !aligned(od, 16)) return MLA_ERR_INVALID_ARG;
  if (!workspace_ok(plan, workspace, workspace_bytes)) return MLA_ERR_WORKSPACE;
  int* st = device_status_word();
  if (st == nullptr) return MLA_ERR_CUDA;
  const bool one = plan.num_splits == 1;
  const float* src = one ? o_latent : static_cast<const float*>(workspace);
  const float* lse_part =
      one ? nullptr : reinterpret_cast<const float*>(static_cast<const char*>(workspace) + plan.o_part_bytes);
  const auto finish = plan.num_splits <= 2 && B * n_q >= kManyTokens ? launch_out_absorb_many : launch_out_absorb_exact;
  return from_cuda(finish(src, lse_part, plan.num_splits, w_uv, static_cast<uint16_t*>(od), lse, B * n_q, st, stream));
}

mla_status mla_accept_tokens(mla_bf16* cache, int64_t num_pages, const int32_t* page_table, int pt_stride,
                             const int32_t* seq_lens_before, const int32_t* path, const int32_t* counts, int B,
                             int n_q, cudaStream_t stream) {
  if (B > 0 && !cache) return MLA_ERR_INVALID_ARG;
  return accept(cache, nullptr, nullptr, nullptr, num_pages, page_table, pt_stride, seq_lens_before, path, counts, B,
                n_q, stream);
}

mla_status mla_accept_tokens_fp8(uint8_t* cache_c8, float* cache_scale, uint16_t* cache_kr, int64_t num_pages,
                                 const int32_t* page_table, int pt_stride, const int32_t* seq_lens_before,
                                 const int32_t* path, const int32_t* counts, int B, int n_q, cudaStream_t stream) {
  if (B > 0 && (!cache_c8 || !cache_scale || !cache_kr)) return MLA_ERR_INVALID_ARG;
  return accept(nullptr, cache_c8, cache_scale, cache_kr, num_pages, page_table, pt_stride, seq_lens_before, path,
                counts, B, n_q, stream);
}

mla_status mla_decompress_kv_window(const mla_bf16* cache, int64_t num_pages, const int32_t* page_table, int pt_stride,
                                    const int32_t* kv_lens, int B, int n_q, int max_kv_len, int window, int sinks,
                                    const mla_bf16* w_uk, const mla_bf16* w_uv, mla_bf16* k_nope, mla_bf16* v,
                                    cudaStream_t stream) {
  if (!view_ok(window, sinks) || n_q < 0 || max_kv_len < n_q) return MLA_ERR_INVALID_ARG;
  if (window == 0)
    return mla_decompress_kv(cache, num_pages, page_table, pt_stride, kv_lens, B, max_kv_len, w_uk, w_uv, k_nope, v,
                             stream);
  if (B < 0 || num_pages < 0 || pt_stride < 0) return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(B) * kHeads * (static_cast<int64_t>(max_kv_len) + kPage) > INT32_MAX)
    return MLA_ERR_UNSUPPORTED;
  if (B == 0 || n_q == 0) return MLA_OK;
  if (!cache || !page_table || !kv_lens || !w_uk || !w_uv || !k_nope || !v) return MLA_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || !aligned(w_uk, 16) || !aligned(w_uv, 16) || !aligned(k_nope, 16) || !aligned(v, 16))
    return MLA_ERR_INVALID_ARG;
  if (pt_stride < (max_kv_len + kPage - 1) / kPage) return MLA_ERR_INVALID_ARG;
  int* st = device_status_word();
  if (st == nullptr) return MLA_ERR_CUDA;
  return from_cuda(launch_decompress_kv_window(cache, num_pages, page_table, pt_stride, kv_lens, B, n_q, max_kv_len,
                                               window, sinks, w_uk, w_uv, k_nope, v, st, stream));
}

mla_status mla_prefill_attn_window(const mla_bf16* q_nope, const mla_bf16* q_rope, const int32_t* seq_lens_before,
                                   const float* rope_table, int rope_max_pos, const mla_bf16* k_nope,
                                   const mla_bf16* v, int max_kv_len, const mla_bf16* cache, int64_t num_pages,
                                   const int32_t* page_table, int pt_stride, const int32_t* kv_lens, int B, int n_q,
                                   int window, int sinks, mla_bf16* out, float* lse, cudaStream_t stream) {
  if (!view_ok(window, sinks)) return MLA_ERR_INVALID_ARG;
  if (window == 0)
    return mla_prefill_attn(q_nope, q_rope, seq_lens_before, rope_table, rope_max_pos, k_nope, v, max_kv_len, cache,
                            num_pages, page_table, pt_stride, kv_lens, B, n_q, out, lse, stream);
  if (B < 0 || n_q < 0 || max_kv_len < n_q || num_pages < 0 || pt_stride < 0 || rope_max_pos < 0)
    return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(B) * kHeads * (static_cast<int64_t>(max_kv_len) + 128) > INT32_MAX)
    return MLA_ERR_UNSUPPORTED;
  if (B == 0 || n_q == 0) return MLA_OK;
  if (!q_nope || !q_rope || !seq_lens_before || !rope_table || !k_nope || !v || !cache || !page_table || !kv_lens ||
      !out)
    return MLA_ERR_INVALID_ARG;
  if (!aligned(q_nope, 16) || !aligned(q_rope, 16) || !aligned(rope_table, 16) || !aligned(k_nope, 16) ||
      !aligned(v, 16) || !aligned(cache, 16) || !aligned(out, 16))
    return MLA_ERR_INVALID_ARG;
  if (pt_stride < (max_kv_len + kPage - 1) / kPage) return MLA_ERR_INVALID_ARG;
  int* st = device_status_word();
  if (st == nullptr) return MLA_ERR_CUDA;
  return from_cuda(launch_prefill_attn_window(q_nope, q_rope, seq_lens_before, rope_table, rope_max_pos, k_nope, v,
                                              max_kv_len, cache, num_pages, page_table, pt_stride, kv_lens, B, n_q,
                                              window, sinks, out, lse, st, stream));
}

}  // extern "C"
