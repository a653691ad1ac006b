// Greedy accept: "VeriCache: Turning Lossy KV Cache into Lossless LLM Inference", "Core
// algorithm" step 3 — accept drafts up to the first mismatch with the full-cache prediction, plus
// one bonus token when all of them match.
//
// Two launches: one CTA per logits row finds the row's argmax (first maximal index) with 16-byte
// loads and writes it into the request's output slot; then one warp per request finds the first
// mismatch with a ballot, pads the output with -1 and writes the accepted count. Slots i <= n
// already hold the right token: a_i == draft_i for i < n, and a_n is the correction or the bonus.
//
// Trees of drafts: ancestor masks and depths, and acceptance along the tree, further down.
#include "paged.cuh"

#include <limits.h>
#include <math.h>

namespace vc {

__device__ __forceinline__ void better(float& bv, int& bi, float v, int i) {
  if (v > bv || (v == bv && i < bi)) {
    bv = v;
    bi = i;
  }
}

// L[b] from the device, held to [0, L_max] so that no row or draft outside request b's is read.
__device__ __forceinline__ int clamp_L(int Lb, int L_max) { return Lb < 0 ? 0 : (Lb > L_max ? L_max : Lb); }

constexpr int kAcceptThreads = 512;

// The first maximal index of x[0 .. V-1], known to thread 0 of the block (INT_MAX where all are NaN).
__device__ __forceinline__ int row_argmax(const float* x, int V) {
  float bv = -INFINITY;
  int bi = INT_MAX;
  // scalar head up to 16-byte alignment, vector body, scalar tail
  int pre = (int)(((16 - ((uintptr_t)x & 15)) & 15) >> 2);
  if (pre > V) pre = V;
  if ((int)threadIdx.x < pre) better(bv, bi, __ldg(x + threadIdx.x), threadIdx.x);
  const int nv = (V - pre) >> 2;
  const float4* xv = reinterpret_cast<const float4*>(x + pre);
  int j = threadIdx.x;
#pragma unroll 1
  for (; j + 3 * kAcceptThreads < nv; j += 4 * kAcceptThreads) {
    float4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = __ldg(xv + j + u * kAcceptThreads);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int base = pre + 4 * (j + u * kAcceptThreads);
      better(bv, bi, v[u].x, base);
      better(bv, bi, v[u].y, base + 1);
      better(bv, bi, v[u].z, base + 2);
      better(bv, bi, v[u].w, base + 3);
    }
  }
  for (; j < nv; j += kAcceptThreads) {
    const float4 v = __ldg(xv + j);
    const int base = pre + 4 * j;
    better(bv, bi, v.x, base);
    better(bv, bi, v.y, base + 1);
    better(bv, bi, v.z, base + 2);
    better(bv, bi, v.w, base + 3);
  }
  const int tail0 = pre + 4 * nv;
  if (tail0 + (int)threadIdx.x < V) better(bv, bi, __ldg(x + tail0 + threadIdx.x), tail0 + threadIdx.x);
  // warp then block reduction
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float ov = __shfl_xor_sync(0xffffffffu, bv, off);
    const int oi = __shfl_xor_sync(0xffffffffu, bi, off);
    better(bv, bi, ov, oi);
  }
  __shared__ float sv[kAcceptThreads / 32];
  __shared__ int si[kAcceptThreads / 32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    sv[w] = bv;
    si[w] = bi;
  }
  __syncthreads();
  if (w == 0) {
    bv = lane < kAcceptThreads / 32 ? sv[lane] : -INFINITY;
    bi = lane < kAcceptThreads / 32 ? si[lane] : INT_MAX;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, bv, off);
      const int oi = __shfl_xor_sync(0xffffffffu, bi, off);
      better(bv, bi, ov, oi);
    }
  }
  return bi;
}

__global__ void __launch_bounds__(kAcceptThreads) accept_argmax_kernel(AcceptArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x;
  const int rows = a.L_max + 1;
  const int b = row / rows, i = row % rows;
  if (i > clamp_L(__ldg(a.L + b), a.L_max)) return;
  const int bi = row_argmax(a.logits + (size_t)row * a.V, a.V);
  if (threadIdx.x == 0) a.out_tokens[(size_t)b * rows + i] = bi;
}

__global__ void accept_finalize_kernel(AcceptArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (b >= a.B) return;
  const int rows = a.L_max + 1;
  const int Lb = clamp_L(__ldg(a.L + b), a.L_max);
  int32_t* out = a.out_tokens + (size_t)b * rows;
  const int32_t* x = a.draft + (size_t)b * a.L_max;
  int n = Lb;
  for (int i0 = 0; i0 < Lb; i0 += 32) {
    const int i = i0 + lane;
    const bool mis = i < Lb && out[i] != x[i];
    const unsigned ball = __ballot_sync(0xffffffffu, mis);
    if (ball) {
      n = i0 + __ffs(ball) - 1;
      break;
    }
  }
  __syncwarp();
  for (int i = lane; i < rows; i += 32)
    if (i > n) out[i] = -1;
  if (lane == 0) a.n_acc[b] = n + 1;
}

cudaError_t launch_accept(const AcceptArgs& a, cudaStream_t s) {
  cudaError_t e = launch_pdl(accept_argmax_kernel, dim3(a.B * (a.L_max + 1)), dim3(kAcceptThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(accept_finalize_kernel, dim3((a.B + 3) / 4), dim3(128), 0, s, a);
}

// ---- trees of drafts -----------------------------------------------------------------------------------
// Masks: a thread per node walks to the root in shared memory; ancestors come in descending order, so each
// word of the node's bits is written once, full. Bound by the walk, about 30 clocks an ancestor (16 trees of 32:
// 4 us, which is a launch and one round trip).
__global__ void __launch_bounds__(256) tree_mask_kernel(TreeMaskArgs a) {
  __shared__ int16_t up[VC_TREE_MAX_NODES];
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x, N = a.N_max, words = (N + 31) / 32;
  const int nodes = a.n_nodes[b], n = min(max(nodes, 0), N);
  const int32_t* parent = a.parent + (size_t)b * N;
  for (int i = threadIdx.x; i < N; i += blockDim.x) {  // those behind the last node too: not one after the other's load
    const int p = parent[i];
    up[i] = (int16_t)(p >= 0 && p < i ? p : -1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < N; i += blockDim.x) {
    uint32_t* row = a.mask + ((size_t)b * N + i) * words;
    int w = words - 1, depth = -1;
    uint32_t bits = 0;
    for (int j = i < n ? i : -1; j >= 0; j = up[j], ++depth) {
      for (; w > (j >> 5); --w, bits = 0) row[w] = bits;
      bits |= 1u << (j & 31);
    }
    for (; w >= 0; --w, bits = 0) row[w] = bits;
    if (a.depth) a.depth[(size_t)b * N + i] = max(depth, 0);
  }
}

// Acceptance: the argmax of each node's row, then a block per request: every node that carries its parent's
// token offers itself as its parent's next one (the lowest wins), and one thread follows them from node 0. Bound by
// reading the logits once (16 trees of up to 32 with 128256 tokens, 222 MB: 36 us, 0.92 of the copy rate).
__global__ void __launch_bounds__(kAcceptThreads) tree_argmax_kernel(TreeAcceptArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x, b = row / a.N_max;
  if (row - b * a.N_max >= min(a.n_nodes[b], a.N_max)) return;
  const int bi = row_argmax(a.logits + (size_t)row * a.V, a.V);
  if (threadIdx.x == 0) a.out_tokens[row] = bi == INT_MAX ? 0 : bi;
}

__global__ void __launch_bounds__(256) tree_walk_kernel(TreeAcceptArgs a) {
  __shared__ int32_t pick[VC_TREE_MAX_NODES], next[VC_TREE_MAX_NODES];
  __shared__ int16_t path[VC_TREE_MAX_NODES];
  __shared__ int s_len;
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x, N = a.N_max;
  const int n = min(max(a.n_nodes[b], 0), N);
  const size_t at = (size_t)b * N;
  // a node a thread, up to four: one round trip for all three arrays (a node behind the last one is read and not used)
  int up[VC_TREE_MAX_NODES / 256], tok[VC_TREE_MAX_NODES / 256];
#pragma unroll
  for (int u = 0; u < VC_TREE_MAX_NODES / 256; ++u) {
    const int i = threadIdx.x + u * blockDim.x;
    if (i < N) {
      up[u] = a.parent[at + i];
      tok[u] = a.token[at + i];
      pick[i] = a.out_tokens[at + i];
      next[i] = INT_MAX;
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < VC_TREE_MAX_NODES / 256; ++u) {
    const int i = threadIdx.x + u * blockDim.x;
    if (i < n && up[u] >= 0 && up[u] < i && tok[u] == pick[up[u]]) atomicMin(&next[up[u]], i);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int len = 0;
    for (int cur = n > 0 ? 0 : INT_MAX; cur < n; cur = next[cur]) path[len++] = (int16_t)cur;
    s_len = len;
    a.n_acc[b] = len;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < N; i += blockDim.x) {
    const int node = i < s_len ? path[i] : -1;
    a.path[at + i] = node;
    a.out_tokens[at + i] = node >= 0 ? pick[node] : -1;
  }
}

cudaError_t launch_tree_mask(const TreeMaskArgs& a, cudaStream_t s) {
  const int threads = a.N_max >= 256 ? 256 : (a.N_max + 31) / 32 * 32;
  return launch_pdl(tree_mask_kernel, dim3(a.B), dim3(threads), 0, s, a);
}

cudaError_t launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t s) {
  cudaError_t e = launch_pdl(tree_argmax_kernel, dim3(a.B * a.N_max), dim3(kAcceptThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  const int threads = a.N_max >= 256 ? 256 : (a.N_max + 31) / 32 * 32;
  return launch_pdl(tree_walk_kernel, dim3(a.B), dim3(threads), 0, s, a);
}

}  // namespace vc
