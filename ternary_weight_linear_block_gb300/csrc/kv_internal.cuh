// Launchers of the paged-cache and tree-attention kernels; they assume
// validated arguments.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/tern.h"

namespace tern {

int kv_sm_count();
cudaError_t launch_kv_plan(const int32_t* ctx_len, const int32_t* new_len, int64_t B,
                           int64_t page_size, int32_t* table, int64_t table_stride,
                           int64_t table_width, const int32_t* held, const int32_t* free_pages,
                           int64_t n_free, const int32_t* free_head, int32_t* row_start,
                           int64_t capacity, int64_t* slots, int32_t* positions, int32_t* request,
                           int32_t* held_out, int32_t* info, cudaStream_t st);
cudaError_t launch_kv_write(const tern_kv_cache& c, const void* k, const void* v, int64_t k_token,
                            int64_t k_head, int64_t v_token, int64_t v_head, const int64_t* slots,
                            int64_t T, cudaStream_t st);
cudaError_t launch_kv_commit(const tern_kv_cache* caches, int64_t layers, const int32_t* table,
                             int64_t table_stride, int64_t table_width, const int32_t* ctx_len,
                             const int32_t* path, int64_t path_width, const int32_t* path_len,
                             int32_t* ctx_out, int64_t B, cudaStream_t st);

cudaError_t launch_kv_rotate_write(const tern_kv_cache* c, const tern_kv_cache8* c8,
                                   const tern_kv_rows& r, cudaStream_t st);
cudaError_t launch_kv8_read(const tern_kv_cache8& c, const int64_t* slots, int64_t T, void* k, void* v,
                            int dtype, cudaStream_t st);
cudaError_t launch_kv8_commit(const tern_kv_cache8* caches, int64_t layers, const int32_t* table,
                              int64_t table_stride, int64_t table_width, const int32_t* ctx_len,
                              const int32_t* path, int64_t path_width, const int32_t* path_len,
                              int32_t* ctx_out, int64_t B, cudaStream_t st);

cudaError_t launch_sample(const void* logits, int64_t row_stride, int64_t rows, int64_t vocab,
                          int dtype, const float* u, const float* temperature,
                          const int32_t* top_k, const float* top_p, const float* min_p,
                          int32_t* token, cudaStream_t st);
cudaError_t launch_tree_accept(const int32_t* tokens, const int32_t* target, const int32_t* parent,
                               const int32_t* row_start, int64_t B, int64_t T, int64_t path_width,
                               int32_t* path, int32_t* path_len, int32_t* next, cudaStream_t st);

// One tree-attention call.
struct TreeAttnCall {
  const void* q;
  int64_t q_token_stride, q_head_stride;
  tern_kv_cache cache;
  const int32_t* table;
  int64_t table_stride, table_width;
  const int32_t* ctx_len;
  const int32_t* row_start;
  const uint64_t* mask;
  int64_t mask_words, B, T, Hq, max_new;
  float scale;
  void* out;
  float* lse;
  void* ws;
};
size_t tree_attention_workspace_bytes(int64_t max_new, int64_t Hq, int64_t H, int64_t D);
cudaError_t launch_tree_attention(const TreeAttnCall& call, cudaStream_t st);
cudaError_t attn_read_clear_error(unsigned int* err);

// One tree-attention call over an 8-bit cache.
struct TreeAttn8Call {
  const void* q;
  int64_t q_token_stride, q_head_stride;
  int dtype;
  tern_kv_cache8 cache;
  const int32_t* table;
  int64_t table_stride, table_width;
  const int32_t* ctx_len;
  const int32_t* row_start;
  const uint64_t* mask;
  int64_t mask_words, B, T, Hq, max_new;
  float scale;
  void* out;
  float* lse;
  void* ws;
};
size_t tree_attention8_workspace_bytes(int64_t max_new, int64_t Hq, int64_t H, int64_t D);
cudaError_t launch_tree_attention8(const TreeAttn8Call& call, cudaStream_t st);
cudaError_t attn8_read_clear_error(unsigned int* err);

}  // namespace tern
