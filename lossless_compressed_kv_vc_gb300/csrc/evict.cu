// Eviction from live caches by accumulated attention weight, in place.
//
// Select: of a KV head's n rows the `keep` of largest rank stay, the rank being the order-preserving
// 32-bit image of the score (guarded rows above everything, NaN below everything) and, among equals,
// the lower row. A 4-pass MSB radix select gives the rank T of the keep-th row and how many rows of
// rank T stay; one ordered pass then numbers the rows: a row below `keep` that goes is hole
// i - kept(i), a row behind it that stays is move kept(i) - (keep - moves), with kept(i) the kept rows
// before row i. There are as many holes as moves, and move j goes into hole j.
// Move: only the rows behind the budget that stay are read and written (K, V, score, position).
#include "vc_internal.cuh"

namespace vc {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;

__device__ __forceinline__ uint32_t evict_rank(float s, int pos, int sink, int recent_from) {
  if (pos < sink || pos >= recent_from) return 0xffffffffu;
  uint32_t u = __float_as_uint(s);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;  // NaN
  if (u == 0x80000000u) u = 0u;                    // -0 == +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const EvictReqDev& r = p.req[blockIdx.y];
  const int n = r.n, keep = r.keep;
  const float* score = r.score + (size_t)h * r.cap;
  const int32_t* pos = r.pos + (size_t)h * r.cap;
  int32_t* plan = r.plan + (size_t)h * r.plan_stride;
  auto rank = [&](int i) { return evict_rank(score[i], pos[i], r.sink, r.recent_from); };
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_prefix, s_rem;
  __shared__ int s_cnt[2][kEvWarps];
  if (tid == 0) {
    s_prefix = 0;
    s_rem = (uint32_t)keep;
  }
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < 256; i += kEvThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix, mask = pass ? 0xffffffffu << (shift + 8) : 0u;
    for (int i = tid; i < n; i += kEvThreads) {
      const uint32_t u = rank(i);
      if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t rem = s_rem, cum = 0;
      int dg = 255;
      for (; dg > 0 && cum + hist[dg] < rem; --dg) cum += hist[dg];
      s_rem = rem - cum;
      s_prefix = prefix | ((uint32_t)dg << shift);
    }
    __syncthreads();
  }
  const uint32_t T = s_prefix;
  const int need_eq = (int)s_rem;
  // ordered pass: warps own consecutive segments
  const int seg = ((n + 31) / 32 + kEvWarps - 1) / kEvWarps * 32;
  const int w0 = min(n, warp * seg), w1 = min(n, w0 + seg);
  int gt = 0, eq = 0;
  for (int base = w0; base < w1; base += 32) {
    const int i = base + lane;
    const uint32_t u = i < w1 ? rank(i) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, i < w1 && u > T));
    eq += __popc(__ballot_sync(0xffffffffu, i < w1 && u == T));
  }
  if (lane == 0) {
    s_cnt[0][warp] = gt;
    s_cnt[1][warp] = eq;
  }
  __syncthreads();
  int gt_run = 0, eq_run = 0;
  for (int w = 0; w < warp; ++w) {
    gt_run += s_cnt[0][w];
    eq_run += s_cnt[1][w];
  }
  const unsigned lt = (1u << lane) - 1u;
  for (int base = w0; base < w1; base += 32) {
    const int i = base + lane;
    const uint32_t u = i < w1 ? rank(i) : 0u;
    const unsigned mg = __ballot_sync(0xffffffffu, i < w1 && u > T), me = __ballot_sync(0xffffffffu, i < w1 && u == T);
    if (i < w1) {
      const int eq_before = eq_run + __popc(me & lt);
      const int kept = gt_run + __popc(mg & lt) + min(eq_before, need_eq);  // kept rows before row i
      const bool stays = u > T || (u == T && eq_before < need_eq);
      if (i < keep) {
        if (!stays && i - kept < r.room) plan[4 + i - kept] = i;
        if (i == keep - 1) plan[0] = keep - kept - (stays ? 1 : 0);
      } else if (stays && keep - 1 - kept < r.room) {
        plan[4 + r.room + keep - 1 - kept] = i;  // from the last move backwards
      }
    }
    gt_run += __popc(mg);
    eq_run += __popc(me);
  }
}

template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int LANES = D / 8;  // 16-byte pieces of a K or V row
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.y;
  const EvictReqDev& r = p.req[blockIdx.z];
  const int32_t* plan = r.plan + (size_t)h * r.plan_stride;
  const int m = plan[0];
  if (m < 0 || m > r.room) {
    if (threadIdx.x == 0) set_status(p.dev_status, VC_DEV_INTERNAL);
    return;
  }
  const int part = threadIdx.x % (2 * LANES);  // K pieces, then V pieces
  const int step = gridDim.x * (256 / (2 * LANES));
  const size_t head = (size_t)h * r.cap;
  uint4* rows = reinterpret_cast<uint4*>((part < LANES ? r.k : r.v) + head * D) + part % LANES;
  for (int j = blockIdx.x * (256 / (2 * LANES)) + threadIdx.x / (2 * LANES); j < m; j += step) {
    const int dst = plan[4 + j], src = plan[4 + r.room + m - 1 - j];
    if (dst < 0 || dst >= r.keep || src < r.keep || src >= r.n) {
      set_status(p.dev_status, VC_DEV_INTERNAL);
      continue;
    }
    rows[(size_t)dst * LANES] = rows[(size_t)src * LANES];
    if (part == 0) r.score[head + dst] = r.score[head + src];
    if (part == 1) r.pos[head + dst] = r.pos[head + src];
  }
}

cudaError_t launch_evict(const EvictParams& p, int d, cudaStream_t s) {
  cudaError_t e = launch_pdl(evict_select_kernel, dim3(p.Hkv, p.B), dim3(kEvThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  int room = 1;
  for (int b = 0; b < p.B; ++b) room = p.req[b].room > room ? p.req[b].room : room;
  const int rows = 256 / (d / 4);  // moves a CTA makes at a time
  const int64_t want = ((int64_t)room + rows - 1) / rows, wave = (152 * 8 + p.Hkv * p.B - 1) / (p.Hkv * p.B);
  const dim3 grid((unsigned)(want < wave ? want : wave), p.Hkv, p.B);
  return d == 128 ? launch_pdl(evict_move_kernel<128>, grid, dim3(256), 0, s, p)
                  : launch_pdl(evict_move_kernel<64>, grid, dim3(256), 0, s, p);
}

}  // namespace vc
