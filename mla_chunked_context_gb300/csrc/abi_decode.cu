// C-ABI entry points of the decode calls: argument checks and the choice of
// kernel.  Everything runs on the caller's stream, in one or two launches,
// with no host-side state, so the calls can be captured into graphs.
#include <cmath>

#include "abi_util.h"

namespace mla {

// kernels (append.cu, latent.cu, tree.cu, verify.cu)
int launch_append(const mla_dims_t &d, const void *kv_a, int64_t kv_a_ld, const void *norm_weight,
                  float eps, int T, int R, const int32_t *qsl, const int32_t *seq_lens,
                  const int32_t *positions, const float *rope, int max_pos, int interleaved,
                  void *kv_cache, int num_blocks, const int32_t *block_table, int bt_stride,
                  void *new_latent, const void *q, void *q_pe, int64_t q_pe_ld, int32_t *status,
                  cudaStream_t s);
int launch_absorb_simt(const mla_dims_t &d, const void *q, int T, const void *w, int rope_columns,
                       void *q_latent, cudaStream_t s);
int launch_expand_simt(const mla_dims_t &d, const void *o_latent, int T, const void *w, void *out,
                       cudaStream_t s);
bool latent_simt_ok(const mla_dims_t &d);
int launch_latent_attn_simt(const mla_dims_t &d, int causal, const TreeMask &tree, int R,
                            const int32_t *qsl, const int32_t *seq_lens, int T, const void *q,
                            const void *cache,
                            int num_blocks, const int32_t *block_table, int bt_stride, void *o,
                            float *lse, int32_t *status, cudaStream_t s);
// sm103_heads.cu, sm103_latent.cu
int launch_absorb_tc(const mla_dims_t &d, const void *q, int T, const void *w, int rope_columns,
                     void *q_latent, cudaStream_t s);
int launch_expand_tc(const mla_dims_t &d, const void *o_latent, int T, const void *w, void *out,
                     cudaStream_t s);
int launch_latent_attn_tc(const mla_dims_t &d, int causal, const TreeMask &tree, int R,
                          const int32_t *qsl, const int32_t *seq_lens, int T, const void *q,
                          const void *cache, int num_blocks, const int32_t *block_table,
                          int bt_stride, float *part_o, float *part_lse, void *desc, int max_ctas,
                          void *o, float *lse, int32_t *status, cudaStream_t s);
int launch_tree_layout(const int32_t *parents, const int32_t *qsl, const int32_t *seq_lens, int T,
                       int R, int words, uint64_t *mask, int32_t *positions, int32_t *status,
                       cudaStream_t s);
int launch_commit(const mla_dims_t &d, const int32_t *path, int path_ld, const int32_t *kept, int T,
                  int R, const int32_t *qsl, const int32_t *seq_lens, void *const *caches,
                  int layers, int num_blocks, const int32_t *block_table, int bt_stride,
                  int32_t *new_lens, int32_t *status, cudaStream_t s);
int launch_verify(const void *p, int64_t p_ld, const void *q, int64_t q_ld, int dtype, int V,
                  const int32_t *tokens, const int32_t *parents, int T, int R, const int32_t *qsl,
                  const float *u, const float *u_next, int32_t *path, int path_ld, int32_t *kept,
                  int32_t *next, int32_t *status, cudaStream_t s);

namespace {

// Tokens x heads a call may have: grids (65535 tiles of 64 tokens) and row
// indices (31 bits) hold them.
int check_rows(const mla_dims_t &d, int T) {
  if (T < 0) return MLA_ERR_INVALID;
  if (d.num_heads > 65535 || T > 65535 * 64 || int64_t(T) * d.num_heads > (int64_t(1) << 30))
    return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

// Workspace of mla_latent_attn for the tensor-core shape: partial results of
// key ranges.  A CTA has at most two (the unit it starts in the middle of and
// the one it leaves unfinished), each 64 rows of 512 float32 and a log-sum.
constexpr int kMaxCtas = 160;
struct LatentWorkspace {
  float *part_o = nullptr, *part_lse = nullptr;
  void *desc = nullptr;  // two int4 a cluster: its unfinished unit
};
size_t latent_workspace(const mla_dims_t &d, void *base, LatentWorkspace &w) {
  if (!tc_shape(d)) return 0;
  // 16-byte aligned bases are enough: every part is a multiple of 256 bytes
  Carve cv(base);
  w.part_o = static_cast<float *>(cv.take(size_t(2) * kMaxCtas * 64 * 512 * sizeof(float)));
  w.part_lse = static_cast<float *>(cv.take(size_t(2) * kMaxCtas * 64 * sizeof(float)));
  w.desc = cv.take(size_t(kMaxCtas) * 8 * sizeof(int32_t));
  return cv.off;
}

bool aligned_to(const void *p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & uintptr_t(bytes - 1)) == 0;
}

// Do two of n caches of `bytes` share memory?  (As a rule a list rises or falls.)
bool share_memory(void *const *caches, int n, int64_t bytes) {
  auto apart = [&](int i, int j) {
    const int64_t d = int64_t(reinterpret_cast<uintptr_t>(caches[j])) -
                      int64_t(reinterpret_cast<uintptr_t>(caches[i]));
    return d >= bytes ? 1 : -d >= bytes ? -1 : 0;
  };
  int way = 0;
  for (int i = 0; i + 1 < n; ++i) way += apart(i, i + 1);
  if (way == n - 1 || way == 1 - n) return false;
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if (!apart(i, j)) return true;
  return false;
}

// Do n and m 32-bit integers share memory?
bool overlap(const int32_t *a, int64_t n, const int32_t *b, int64_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + uintptr_t(m) * 4 && y < x + uintptr_t(n) * 4;
}

// mla_latent_attn, and with a mask mla_tree_attn
int attend(const mla_dims_t *d, int causal, const TreeMask &tree, int num_seqs,
           const int32_t *query_start_loc, const int32_t *seq_lens, int num_tokens,
           const void *q_latent, const void *kv_cache, int num_blocks, const int32_t *block_table,
           int block_table_stride, void *workspace, size_t workspace_bytes, void *o_latent,
           float *lse, int32_t *dev_status, mla_stream_t stream) {
  if (!query_start_loc || !seq_lens || !q_latent || !kv_cache || !block_table || !o_latent)
    return MLA_ERR_INVALID;
  const int es = elem_bytes(d->dtype);
  if (!aligned_to(q_latent, es) || !aligned_to(o_latent, es) || !aligned4(lse) ||
      !aligned16(kv_cache))
    return MLA_ERR_INVALID;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tc_shape(*d)) {
    LatentWorkspace w;
    const size_t need = latent_workspace(*d, workspace, w);
    if (!workspace || !aligned16(workspace)) return MLA_ERR_INVALID;
    if (workspace_bytes < need) return MLA_ERR_TOO_SMALL;
    if (!aligned16(q_latent) || !aligned16(o_latent) || !tc_available())
      return MLA_ERR_UNSUPPORTED;
    return launch_latent_attn_tc(*d, causal, tree, num_seqs, query_start_loc, seq_lens, num_tokens,
                                 q_latent, kv_cache, num_blocks, block_table, block_table_stride,
                                 w.part_o, w.part_lse, w.desc, kMaxCtas, o_latent, lse, dev_status,
                                 s);
  }
  if (!latent_simt_ok(*d)) return MLA_ERR_UNSUPPORTED;
  return launch_latent_attn_simt(*d, causal, tree, num_seqs, query_start_loc, seq_lens, num_tokens,
                                 q_latent, kv_cache, num_blocks, block_table, block_table_stride,
                                 o_latent, lse, dev_status, s);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_append_latent(const mla_dims_t *d, const void *kv_a, int64_t kv_a_ld,
                                 const void *norm_weight, float norm_eps, int32_t num_tokens,
                                 int32_t num_seqs, const int32_t *query_start_loc,
                                 const int32_t *seq_lens, const int32_t *positions,
                                 const float *rope_table, int32_t max_positions,
                                 int32_t interleaved, void *kv_cache, int32_t num_blocks,
                                 const int32_t *block_table, int32_t block_table_stride,
                                 void *new_latent, const void *q, void *q_pe_out, int64_t q_pe_ld,
                                 int32_t *dev_status, mla_stream_t stream) {
  int rc = check_dims(d);
  if (rc) return rc;
  rc = check_rows(*d, num_tokens);
  if (rc) return rc;
  if (num_seqs < 0 || num_blocks < 0 || block_table_stride < 1 || max_positions < 0 ||
      kv_a_ld < d->kv_lora_rank + d->qk_rope_dim || (interleaved != 0 && interleaved != 1))
    return MLA_ERR_INVALID;
  if (norm_weight && !(norm_eps >= 0.f && std::isfinite(norm_eps))) return MLA_ERR_INVALID;
  if (num_tokens == 0 || num_seqs == 0) return MLA_OK;
  if (!kv_a || !query_start_loc || !seq_lens || !kv_cache || !block_table ||
      (q == nullptr) != (q_pe_out == nullptr))
    return MLA_ERR_INVALID;
  if (q && q_pe_ld < d->qk_rope_dim) return MLA_ERR_INVALID;
  const int es = elem_bytes(d->dtype);
  if (!aligned16(kv_cache) || !aligned16(new_latent) || !aligned_to(kv_a, es) ||
      !aligned_to(norm_weight, es) || !aligned_to(q, es) || !aligned_to(q_pe_out, es) ||
      !aligned4(rope_table))
    return MLA_ERR_INVALID;
  if (rope_table && d->qk_rope_dim % 2 != 0) return MLA_ERR_UNSUPPORTED;
  if (d->qk_rope_dim == 0) q = q_pe_out = nullptr;
  return launch_append(*d, kv_a, kv_a_ld, norm_weight, norm_eps, num_tokens, num_seqs,
                       query_start_loc, seq_lens, positions, rope_table, max_positions,
                       interleaved, kv_cache, num_blocks, block_table, block_table_stride,
                       new_latent, q, q_pe_out, q_pe_ld, dev_status,
                       static_cast<cudaStream_t>(stream));
}

extern "C" int mla_absorb_query(const mla_dims_t *d, const void *q, int32_t num_tokens,
                                const void *w_kv_b, int32_t rope_columns, void *q_latent,
                                mla_stream_t stream) {
  int rc = check_dims(d);
  if (rc) return rc;
  rc = check_rows(*d, num_tokens);
  if (rc) return rc;
  if (rope_columns != 0 && rope_columns != 1) return MLA_ERR_INVALID;
  if (num_tokens == 0) return MLA_OK;
  const int es = elem_bytes(d->dtype);
  if (!q || !w_kv_b || !q_latent || !aligned_to(q, es) || !aligned_to(w_kv_b, es) ||
      !aligned_to(q_latent, es))
    return MLA_ERR_INVALID;
  if (tc_shape(*d)) {
    if (!aligned16(q) || !aligned16(w_kv_b) || !aligned16(q_latent) || !tc_available())
      return MLA_ERR_UNSUPPORTED;
    return launch_absorb_tc(*d, q, num_tokens, w_kv_b, rope_columns, q_latent,
                            static_cast<cudaStream_t>(stream));
  }
  return launch_absorb_simt(*d, q, num_tokens, w_kv_b, rope_columns, q_latent,
                            static_cast<cudaStream_t>(stream));
}

extern "C" int mla_expand_output(const mla_dims_t *d, const void *o_latent, int32_t num_tokens,
                                 const void *w_kv_b, void *out, mla_stream_t stream) {
  int rc = check_dims(d);
  if (rc) return rc;
  rc = check_rows(*d, num_tokens);
  if (rc) return rc;
  if (num_tokens == 0) return MLA_OK;
  const int es = elem_bytes(d->dtype);
  if (!o_latent || !w_kv_b || !out || !aligned_to(o_latent, es) || !aligned_to(w_kv_b, es) ||
      !aligned_to(out, es))
    return MLA_ERR_INVALID;
  if (tc_shape(*d)) {
    if (!aligned16(o_latent) || !aligned16(w_kv_b) || !aligned16(out) || !tc_available())
      return MLA_ERR_UNSUPPORTED;
    return launch_expand_tc(*d, o_latent, num_tokens, w_kv_b, out,
                            static_cast<cudaStream_t>(stream));
  }
  return launch_expand_simt(*d, o_latent, num_tokens, w_kv_b, out,
                            static_cast<cudaStream_t>(stream));
}

extern "C" int mla_latent_attn_workspace_bytes(const mla_dims_t *d, int32_t num_tokens,
                                               int32_t num_seqs, size_t *bytes) {
  int rc = check_dims(d);
  if (rc) return rc;
  rc = check_rows(*d, num_tokens);
  if (rc) return rc;
  if (num_seqs < 0 || !bytes) return MLA_ERR_INVALID;
  LatentWorkspace w;
  *bytes = latent_workspace(*d, nullptr, w);
  return MLA_OK;
}

extern "C" int mla_latent_attn(const mla_dims_t *d, int32_t causal, int32_t num_seqs,
                               const int32_t *query_start_loc, const int32_t *seq_lens,
                               int32_t num_tokens, const void *q_latent, const void *kv_cache,
                               int32_t num_blocks, const int32_t *block_table,
                               int32_t block_table_stride, void *workspace,
                               size_t workspace_bytes, void *o_latent, float *lse,
                               int32_t *dev_status, mla_stream_t stream) {
  int rc = check_dims(d);
  if (rc) return rc;
  rc = check_rows(*d, num_tokens);
  if (rc) return rc;
  if ((causal != 0 && causal != 1) || num_seqs < 0 || num_blocks < 0 || block_table_stride < 1)
    return MLA_ERR_INVALID;
  if (num_tokens == 0 || num_seqs == 0) return MLA_OK;
  return attend(d, causal, TreeMask(), num_seqs, query_start_loc, seq_lens, num_tokens, q_latent,
                kv_cache, num_blocks, block_table, block_table_stride, workspace, workspace_bytes,
                o_latent, lse, dev_status, stream);
}

extern "C" int mla_tree_layout(int32_t num_tokens, int32_t num_seqs,
                               const int32_t *query_start_loc, const int32_t *seq_lens,
                               const int32_t *parents, int32_t mask_words, uint64_t *tree_mask,
                               int32_t *positions, int32_t *dev_status, mla_stream_t stream) {
  if (num_tokens < 0 || num_seqs < 0 || mask_words < 1) return MLA_ERR_INVALID;
  if (num_tokens == 0 || num_seqs == 0) return MLA_OK;
  if (!query_start_loc || !parents || !tree_mask || (positions && !seq_lens) ||
      !aligned_to(tree_mask, 8) || !aligned4(parents) || !aligned4(positions))
    return MLA_ERR_INVALID;
  return launch_tree_layout(parents, query_start_loc, positions ? seq_lens : nullptr, num_tokens,
                            num_seqs, mask_words, tree_mask, positions, dev_status,
                            static_cast<cudaStream_t>(stream));
}

extern "C" int mla_tree_attn(const mla_dims_t *d, int32_t num_seqs, const int32_t *query_start_loc,
                             const int32_t *seq_lens, const uint64_t *tree_mask,
                             int32_t mask_words, int32_t num_tokens, const void *q_latent,
                             const void *kv_cache, int32_t num_blocks, const int32_t *block_table,
                             int32_t block_table_stride, void *workspace, size_t workspace_bytes,
                             void *o_latent, float *lse, int32_t *dev_status,
                             mla_stream_t stream) {
  int rc = check_dims(d);
  if (rc) return rc;
  rc = check_rows(*d, num_tokens);
  if (rc) return rc;
  if (num_seqs < 0 || num_blocks < 0 || block_table_stride < 1 || mask_words < 1)
    return MLA_ERR_INVALID;
  if (num_tokens == 0 || num_seqs == 0) return MLA_OK;
  if (!tree_mask || !aligned_to(tree_mask, 8)) return MLA_ERR_INVALID;
  return attend(d, 0, TreeMask{tree_mask, mask_words}, num_seqs, query_start_loc, seq_lens,
                num_tokens, q_latent, kv_cache, num_blocks, block_table, block_table_stride,
                workspace, workspace_bytes, o_latent, lse, dev_status, stream);
}

extern "C" int mla_verify_tree(int32_t dtype, int32_t num_tokens, int32_t num_seqs, int32_t vocab,
                               const void *target, int64_t target_ld, const void *draft,
                               int64_t draft_ld, const int32_t *tokens, const int32_t *parents,
                               const int32_t *query_start_loc, const float *uniform,
                               const float *uniform_next, int32_t *path, int32_t path_ld,
                               int32_t *num_kept, int32_t *next_tokens, int32_t *dev_status,
                               mla_stream_t stream) {
  if (!valid_dtype(dtype) || num_tokens < 0 || num_seqs < 0 || vocab < 1 || path_ld < 1 ||
      target_ld < vocab || (draft && draft_ld < vocab))
    return MLA_ERR_INVALID;
  constexpr int kMost = 1 << 24;
  if (vocab > kMost || num_tokens > kMost || num_seqs > kMost) return MLA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return MLA_OK;
  const int es = elem_bytes(dtype);
  if (!query_start_loc || !path || !num_kept || !next_tokens || !aligned4(path) ||
      !aligned4(num_kept) || !aligned4(next_tokens) || !aligned4(query_start_loc))
    return MLA_ERR_INVALID;
  if (num_tokens > 0 && (!target || !tokens || !parents ||
                         (uniform == nullptr) != (uniform_next == nullptr) ||
                         !aligned_to(target, es) ||
                         !aligned_to(draft, es) || !aligned4(tokens) || !aligned4(parents) ||
                         !aligned4(uniform) || !aligned4(uniform_next)))
    return MLA_ERR_INVALID;
  return launch_verify(target, target_ld, uniform ? draft : nullptr, draft_ld, dtype, vocab, tokens,
                       parents, num_tokens, num_seqs, query_start_loc, uniform, uniform_next, path,
                       path_ld, num_kept, next_tokens, dev_status,
                       static_cast<cudaStream_t>(stream));
}

extern "C" int mla_commit_tree(const mla_dims_t *d, int32_t num_seqs, int32_t num_tokens,
                               const int32_t *path, int32_t path_ld, const int32_t *num_kept,
                               const int32_t *query_start_loc, const int32_t *seq_lens,
                               void *const *kv_caches, int32_t num_layers, int32_t num_blocks,
                               const int32_t *block_table, int32_t block_table_stride,
                               int32_t *new_seq_lens, int32_t *dev_status, mla_stream_t stream) {
  int rc = check_dims(d);
  if (rc) return rc;
  if (num_seqs < 0 || num_tokens < 0 || path_ld < 1 || num_layers < 0 || num_blocks < 0 ||
      block_table_stride < 1)
    return MLA_ERR_INVALID;
  if (num_seqs == 0) return MLA_OK;
  if (!path || !num_kept || !query_start_loc || !seq_lens || !block_table ||
      (num_layers > 0 && !kv_caches) ||
      (new_seq_lens && overlap(new_seq_lens, num_seqs, seq_lens, num_seqs)))
    return MLA_ERR_INVALID;
  for (int32_t l = 0; l < num_layers; ++l)
    if (!kv_caches[l] || !aligned16(kv_caches[l])) return MLA_ERR_INVALID;
  const int64_t row = int64_t(d->kv_lora_rank + d->qk_rope_dim) * elem_bytes(d->dtype);
  if (num_blocks > 0 && share_memory(kv_caches, num_layers, row * d->block_size * num_blocks))
    return MLA_ERR_INVALID;
  // blocks of other layers still read these when a sequence's new length is written
  const int64_t R = num_seqs;
  if (new_seq_lens &&
      (overlap(new_seq_lens, R, num_kept, R) || overlap(new_seq_lens, R, query_start_loc, R + 1) ||
       overlap(new_seq_lens, R, path, R * path_ld) ||
       overlap(new_seq_lens, R, block_table, R * block_table_stride)))
    return MLA_ERR_UNSUPPORTED;
  return launch_commit(*d, path, path_ld, num_kept, num_tokens, num_seqs, query_start_loc, seq_lens,
                       kv_caches, num_layers, num_blocks, block_table, block_table_stride,
                       new_seq_lens, dev_status, static_cast<cudaStream_t>(stream));
}
