// Host-side launchers of the drafted-token kernels (internal to the library).
#pragma once

#include "mb_kernels.h"

namespace mb {

// bf16 tensor of any rank up to 5, 128-byte swizzle (strides[i]: of dimension i + 1)
cudaError_t encode_tmap(CUtensorMap *map, const void *base, int rank, const uint64_t *dims,
                        const uint64_t *strides_bytes, const uint32_t *box);
// The KV pool's map: one (page, K/V, head) block of 16 x hd per copy, blocks = pages * 2 * Hkv
cudaError_t encode_kv_tmap(CUtensorMap *map, const void *base, uint64_t blocks, int hd);

// rope_append_run for a step with drafted trees: tok_slot [T] is the place of
// each token in its request's cache (tok_pos the position of its rotation).
cudaError_t rope_append_tree_run(const RopeArgs &a, const int32_t *tok_slot, cudaStream_t st);

constexpr int kMaxTreeNodes = 128;        // nodes of one request's tree
constexpr int kMaxPoolsPerLaunch = 128;   // pools of one page-operation launch (their bases are kernel arguments)

struct TreeArgs {
  const void *q;            // [T][Hq][hd] bf16 (rotated)
  const void *pool;         // [P][2][Hkv][16][hd]
  void *o;                  // [T][Hq hd] bf16
  const int32_t *qo_indptr, *kv_len, *bt_indptr, *bt, *parent;   // device
  int n_reqs, T, Hq, Hkv, hd, num_pages;
  void *workspace;          // tree_workspace_bytes()
  int *err;
  const int32_t *is_tree = nullptr;   // [n_reqs], or null: requests to leave alone hold 0
};
size_t tree_workspace_bytes();
cudaError_t tree_attention_run(const TreeArgs &a, cudaStream_t st);

struct VerifyArgs {
  const void *logits;       // [T][vocab] bf16
  const int32_t *tokens;    // [T]
  const float *probs;       // [T][vocab] or null
  const int32_t *qo_indptr, *parent;
  const float *temperature, *u_accept, *u_final;
  int32_t *n_accepted, *path, *next_token;
  int n_reqs, T, vocab, max_path;
  int *err;
};
cudaError_t verify_tree_run(const VerifyArgs &a, cudaStream_t st);

struct CompactArgs {
  void *const *pools;       // host array of device pointers
  int n_pools, num_pages, Hkv, hd, n_reqs, max_path;
  const int32_t *qo_indptr, *kv_len, *bt_indptr, *bt, *count, *path;
  int32_t *new_kv_len;
  int *err;
};
cudaError_t kv_compact_run(const CompactArgs &a, cudaStream_t st);
// src and dst: host page ids (checked by the caller)
cudaError_t kv_copy_pages_run(void *const *pools, int n_pools, int Hkv, int hd, const int32_t *src, const int32_t *dst,
                              int n_pairs, cudaStream_t st);

}  // namespace mb
