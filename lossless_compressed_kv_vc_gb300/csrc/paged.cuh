// Drafted trees over a cache of pages: declarations shared by the C-ABI layer (paged_api.cu) and the kernels behind it.
#pragma once

#include "vc_internal.cuh"

namespace vc {

struct PagedDev {
  bf16 *k, *v;
  int32_t *refs, *free_pages, *n_free, *table, *len, *held, *next;
  int32_t n_pages, shift, n_seq, max_pages;  // a page has 1 << shift rows

  __device__ __forceinline__ int rows() const { return 1 << shift; }
  // Pages and rows of context of a sequence, within what its table can hold whatever the state says.
  __device__ __forceinline__ int held_of(int seq) const { return min(max(held[seq], 0), max_pages); }
  __device__ __forceinline__ bool has_page(int p) const { return (uint32_t)p < (uint32_t)n_pages; }
  __device__ __forceinline__ int32_t* pages_of(int seq) const { return table + (int64_t)seq * max_pages; }
};

struct ReserveParams {
  PagedDev kv;
  vc_reserve_req req[VC_MAX_BATCH];
  int4* copies;  // [B] old page, new page, rows
  int32_t B, Hkv;
  int32_t* dev_status;
};
struct ForkParams {
  PagedDev kv;
  vc_fork_req req[VC_MAX_BATCH];
  int32_t* dev_status;
};
struct TrimParams {
  PagedDev kv;
  vc_trim_req req[VC_MAX_BATCH];
  int32_t B;
  int32_t* dev_status;
};
struct CompactParams {
  PagedDev kv;
  int32_t Hkv;
  int32_t* head;  // [4] pages to move, pages in use
  int32_t *hole, *from, *back;  // [n_pages / 2 + 1] twice, [n_pages]
  int32_t* dev_status;
};
struct CommitParams {
  PagedDev kv;
  vc_commit_req req[VC_MAX_BATCH];
  int32_t Hkv;
  int32_t* dev_status;
};
cudaError_t launch_pages_init(const PagedDev& kv, cudaStream_t s);
cudaError_t launch_reserve(const ReserveParams& p, int d, cudaStream_t s);
cudaError_t launch_fork(const ForkParams& p, int B, cudaStream_t s);
cudaError_t launch_trim(const TrimParams& p, cudaStream_t s);
cudaError_t launch_compact(const CompactParams& p, int d, cudaStream_t s);
cudaError_t launch_commit(const CommitParams& p, int B, int d, cudaStream_t s);

struct RopePageReqDev {
  const bf16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t* off;
  int64_t off_stride;
  bf16* q_out;
  int32_t seq;
};
struct RopePageParams {
  PagedDev kv;
  int32_t tok_begin[VC_MAX_BATCH];  // first token of each request in the call's token sequence, INT32_MAX behind the last
  RopePageReqDev req[VC_MAX_BATCH];
  double turns[VC_ROPE_MAX_PAIRS];  // turns a position: theta / 2 pi
  uint64_t axis[2];                 // two bits a pair: each thread's own byte of the parameters would be read one by one
  int32_t Hq, Hkv, rot, inter, n_tok;
  float amp;
  int32_t* dev_status;
};
cudaError_t launch_rope_pages(const RopePageParams& p, int d, cudaStream_t s);

struct TreeMaskArgs {
  const int32_t *parent, *n_nodes;
  uint32_t* mask;
  int32_t* depth;
  int32_t B, N_max;
};
struct TreeAcceptArgs {
  const float* logits;
  const int32_t *token, *parent, *n_nodes;
  int32_t *out_tokens, *path, *n_acc;
  int32_t B, N_max, V;
};
cudaError_t launch_tree_mask(const TreeMaskArgs& a, cudaStream_t s);
cudaError_t launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t s);

struct TreeReqDev {
  const bf16* q;
  bf16* o;
  const uint32_t* mask;
  int32_t mask_words, seq, n_rows;
  int32_t tok_begin;  // first query token of the request in the call's token sequence
};
struct TreeArgs {
  PagedDev kv;
  TreeReqDev req[VC_MAX_BATCH];  // those with tokens
  int32_t B, Hq, Hkv, d, n_tok;
  void* ws;
  size_t ws_bytes;
  int32_t* dev_status;
};
size_t tree_workspace_size(const vc_shape* s, int32_t max_rows);
// VC_ERR_WORKSPACE, VC_ERR_UNSUPPORTED or VC_ERR_CUDA in *st: nothing launched
cudaError_t launch_tree_attn(const TreeArgs& a, cudaStream_t s, vc_status* st);

}  // namespace vc
