// Host-side launchers of the latent-cache kernels and of the descriptors built
// on the GPU (internal to the library).
#pragma once

#include "mb_kernels.h"

namespace mb {

constexpr int kLatentRope = 64;          // dimensions of the rotated key that all heads share
constexpr int kLatentMaxReqs = 1 << 20;  // requests of an attention call (a thread's range of them is counted in 32 bits)
constexpr int kTablesMaxReqs = 8192;     // requests of one descriptor (their sums sit in shared memory)
constexpr int kTablesMaxSlots = 65536;   // rows of the tables (a bit each, twice, in shared memory)
constexpr int kTablesMaxPages = 1 << 20; // pages of one request: 2^24 tokens

struct TablesArgs {
  const int32_t *slots, *cached, *new_tokens;   // [n]
  int n, T, bt_cap, max_slots, max_pages, num_pages;
  int32_t *tables;                              // [max_slots][max_pages]
  int32_t *owned;                               // [max_slots]
  int32_t *ring;                                // [num_pages]
  int32_t *state;                               // {head, count, 0, 0}
  int32_t *qo_indptr, *kv_len, *bt_indptr, *bt, *tok_req, *tok_pos, *tok_slot;
  int *err;
};
cudaError_t batch_tables_run(const TablesArgs &a, cudaStream_t st);
cudaError_t tables_release_run(const TablesArgs &a, cudaStream_t st);

struct LatentAppendArgs {
  const void *ckv;          // [T] rows of ld elements: rank, then 64
  const void *q;            // [T][H][hd + 64]
  const void *gain;         // [rank]
  void *pool;               // [P][16][rank + 64]
  void *q_rope;             // [T][H][64]
  const int32_t *tok_pos, *tok_slot;
  int64_t ld;
  int T, num_pages, H, hd, rank;
  float eps, theta;
  int *err;
};
cudaError_t latent_append_run(const LatentAppendArgs &a, cudaStream_t st);

struct LatentArgs {
  const void *q;            // [T][H][hd + 64]
  const void *q_rope;       // [T][H][64]
  const void *w_kv;         // [H][2 hd][rank]: each head's key rows, then its value rows
  const void *pool;         // [P][16][rank + 64]
  void *o;                  // [T][H hd]
  const int32_t *qo_indptr, *kv_len, *bt_indptr, *bt;   // device
  int n_reqs, T, H, hd, rank, num_pages;
  float scale;
  void *workspace;
  int *err;
  int kv_tokens;            // expanded form: room for the batch's keys
};
size_t latent_attention_workspace_bytes(int64_t T, int64_t H, int64_t rank);
cudaError_t latent_attention_run(const LatentArgs &a, cudaStream_t st);
size_t latent_prefill_workspace_bytes(int64_t kv_tokens, int64_t n_reqs, int64_t H, int64_t hd);   // (of any rank)
cudaError_t latent_prefill_run(const LatentArgs &a, cudaStream_t st);

}  // namespace mb
