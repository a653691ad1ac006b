// Eviction from live caches by accumulated attention weight, in place.
//
// Select: of a KV head's n rows the `keep` of largest rank stay, the rank being the order-preserving
// 32-bit image of the score (guarded rows above everything, NaN below everything) and, among equals,
// the lower row. A radix select, most significant digit first (11, 11 and 10 bits), gives the rank T of
// the keep-th row and how many rows of rank T stay; one ordered pass then numbers the rows: a row below
// `keep` that goes is hole i - kept(i), a row behind it that stays is move kept(i) - (keep - moves),
// with kept(i) the kept rows before row i. There are as many holes as moves, and move j goes into hole j.
// Scores and positions are read once: each thread keeps its rows' ranks in registers.
//
// Move: only the rows behind the budget that stay are read and written (K, V, score, position). A warp
// takes consecutive moves: their plan, scores and positions lane by lane (neighbours in memory), then
// their K and V rows, several in flight.
#include "vc_internal.cuh"

namespace vc {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvKeys = 16;  // ranks a thread holds
constexpr int kEvSlice = kEvThreads * kEvKeys;
constexpr int kEvCluster = 8;
constexpr int kEvBins = 2048;

__device__ __forceinline__ uint32_t evict_rank(float s, int pos, int sink, int recent_from) {
  if (pos < sink || pos >= recent_from) return 0xffffffffu;
  uint32_t u = __float_as_uint(s);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;  // NaN
  if (u == 0x80000000u) u = 0u;                    // -0 == +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ev_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of every CTA of the cluster arrives; writes before it are visible to reads after it.
__device__ __forceinline__ void ev_cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of CTA `rank`'s shared memory at the address of `p` in this CTA's.
__device__ __forceinline__ uint32_t ev_ld_cluster(const void* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// CL CTAs (a cluster) per (KV head, request), each with a consecutive slice of the rows, each warp with a
// consecutive segment of the slice. HELD: a warp's segment is at most 32 kEvKeys rows and its ranks stay
// in registers; otherwise they are taken from memory again in every pass.
template <int CL, bool HELD>
__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ uint32_t hist[2][kEvBins];  // this CTA's histogram, double-buffered by pass
  __shared__ uint32_t s_warp[kEvWarps];
  __shared__ uint32_t s_prefix, s_rem;
  __shared__ int s_cnt[2][kEvWarps];
  __shared__ int s_cta[2];  // this CTA's rows above T and equal to T
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = CL > 1 ? ev_cluster_rank() : 0u;
  const int h = blockIdx.x / CL;
  const EvictReqDev& r = p.req[blockIdx.y];
  const int n = r.n, keep = r.keep;
  const float* score = r.score + (size_t)h * r.cap;
  const int32_t* pos = r.pos + (size_t)h * r.cap;
  int32_t* plan = r.plan + (size_t)h * r.plan_stride;
  const int per = (n + CL - 1) / CL;                               // rows of a slice
  const int s0 = min((int64_t)n, (int64_t)rank * per), s1 = min((int64_t)n, (int64_t)s0 + per);
  const int seg = ((s1 - s0 + 31) / 32 + kEvWarps - 1) / kEvWarps * 32;  // rows of a warp
  const int w0 = min(s1, s0 + warp * seg), w1 = min(s1, w0 + seg);
  auto load = [&](int i) { return i < w1 ? evict_rank(__ldg(score + i), __ldg(pos + i), r.sink, r.recent_from) : 0u; };
  uint32_t key[kEvKeys];
  if (HELD) {
#pragma unroll
    for (int k = 0; k < kEvKeys; ++k) key[k] = load(w0 + 32 * k + lane);
  }
  // f(row, rank) for the warp's rows, 32 at a time (the last may be beyond w1)
  auto each = [&](auto f) {
    if (HELD) {
#pragma unroll
      for (int k = 0; k < kEvKeys; ++k)
        if (w0 + 32 * k < w1) f(w0 + 32 * k + lane, key[k]);
    } else {
      for (int base = w0; base < w1; base += 32) f(base + lane, load(base + lane));
    }
  };
  if (tid == 0) {
    s_prefix = 0;
    s_rem = (uint32_t)keep;
  }
  uint32_t mask = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 1023u : 2047u;
    uint32_t* hs = hist[pass & 1];  // last read by the cluster before the previous cluster barrier
    for (int i = tid; i < kEvBins; i += kEvThreads) hs[i] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    each([&](int i, uint32_t u) {
      // rows of the warp's commonest case, one digit for most lanes (guarded rows, rows without any
      // weight, one exponent), are added up before they reach the histogram
      const bool in = i < w1 && (u & mask) == prefix;
      const uint32_t dg = (u >> shift) & digit;
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (!act) return;
      const int lead = __ffs(act) - 1;
      const uint32_t lead_dg = __shfl_sync(0xffffffffu, dg, lead);
      const unsigned same = __ballot_sync(0xffffffffu, in && dg == lead_dg);
      if (lane == lead)
        atomicAdd(&hs[dg], (uint32_t)__popc(same));
      else if (in && !((same >> lane) & 1u))
        atomicAdd(&hs[dg], 1u);
    });
    if (CL > 1)
      ev_cluster_sync();
    else
      __syncthreads();
    // thread t owns the bins 2t', 2t'+1 from the top: counts of larger digits come from the threads before
    const int b1 = kEvBins - 1 - 2 * tid, b0 = b1 - 1;
    uint32_t c1 = 0, c0 = 0;
    if (CL > 1) {
#pragma unroll
      for (int q = 0; q < CL; ++q) {
        c1 += ev_ld_cluster(&hs[b1], q);
        c0 += ev_ld_cluster(&hs[b0], q);
      }
    } else {
      c1 = hs[b1];
      c0 = hs[b0];
    }
    uint32_t sum = c1 + c0;  // inclusive prefix over the warp's threads
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += o;
    }
    if (lane == 31) s_warp[warp] = sum;
    const uint32_t rem = s_rem;
    __syncthreads();
    uint32_t before = lane < warp ? s_warp[lane] : 0u;  // warps before this one
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
    const uint32_t cum1 = before + sum - c1 - c0, cum0 = cum1 + c1;  // larger digits than b1, than b0
    if (cum1 < rem && cum1 + c1 >= rem) {  // exactly one digit satisfies this
      s_rem = rem - cum1;
      s_prefix = prefix | ((uint32_t)b1 << shift);
    }
    if (cum0 < rem && cum0 + c0 >= rem) {
      s_rem = rem - cum0;
      s_prefix = prefix | ((uint32_t)b0 << shift);
    }
    mask |= digit << shift;
    __syncthreads();
  }
  const uint32_t T = s_prefix;
  const int need_eq = (int)s_rem;
  int gt = 0, eq = 0;
  each([&](int i, uint32_t u) {
    gt += __popc(__ballot_sync(0xffffffffu, i < w1 && u > T));
    eq += __popc(__ballot_sync(0xffffffffu, i < w1 && u == T));
  });
  if (lane == 0) {
    s_cnt[0][warp] = gt;
    s_cnt[1][warp] = eq;
  }
  __syncthreads();
  // rows above and equal to T in the warps (and, through the cluster, the CTAs) before this one
  int gt_run = lane < kEvWarps ? s_cnt[0][lane] : 0, eq_run = lane < kEvWarps ? s_cnt[1][lane] : 0;
  int gt_all = gt_run, eq_all = eq_run;
  gt_run = lane < warp ? gt_run : 0;
  eq_run = lane < warp ? eq_run : 0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    gt_run += __shfl_xor_sync(0xffffffffu, gt_run, off);
    eq_run += __shfl_xor_sync(0xffffffffu, eq_run, off);
    gt_all += __shfl_xor_sync(0xffffffffu, gt_all, off);
    eq_all += __shfl_xor_sync(0xffffffffu, eq_all, off);
  }
  if constexpr (CL > 1) {
    if (tid == 0) {
      s_cta[0] = gt_all;
      s_cta[1] = eq_all;
    }
    ev_cluster_sync();
    for (uint32_t q = 0; q < rank; ++q) {
      gt_run += (int)ev_ld_cluster(&s_cta[0], q);
      eq_run += (int)ev_ld_cluster(&s_cta[1], q);
    }
  }
  const unsigned lt = (1u << lane) - 1u;
  each([&](int i, uint32_t u) {
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
  });
  if (CL > 1) ev_cluster_sync();  // no CTA leaves while another may still read its shared memory
}

// grid (x, Hkv, B): warps take per_warp consecutive moves (at most 32) at a time.
template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictParams p, int per_warp) {
  constexpr int LANES = D / 4;       // 16-byte pieces of a row of K and of V
  constexpr int RW = 32 / LANES;     // rows a warp copies at a time
  constexpr int U = 4;               // of those, in flight
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.y, lane = threadIdx.x & 31;
  const EvictReqDev& r = p.req[blockIdx.z];
  const int32_t* plan = r.plan + (size_t)h * r.plan_stride;
  const int m = plan[0];
  if (m < 0 || m > r.room) {
    if (threadIdx.x == 0) set_status(p.dev_status, VC_DEV_INTERNAL);
    return;
  }
  const size_t head = (size_t)h * r.cap;
  const int part = lane % LANES;  // K pieces, then V pieces
  uint4* rows = reinterpret_cast<uint4*>((part < LANES / 2 ? r.k : r.v) + head * D) + part % (LANES / 2);
  const int64_t step = (int64_t)gridDim.x * 8 * per_warp;
  for (int64_t j0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * per_warp; j0 < m; j0 += step) {
    const int cnt = (int)min((int64_t)per_warp, m - j0);
    int dst = -1, src = 0;
    if (lane < cnt) {
      dst = plan[4 + j0 + lane];
      src = plan[4 + r.room + m - 1 - j0 - lane];
      if (dst < 0 || dst >= r.keep || src < r.keep || src >= r.n) {
        set_status(p.dev_status, VC_DEV_INTERNAL);
        dst = -1;
      } else {
        r.score[head + dst] = r.score[head + src];
        r.pos[head + dst] = r.pos[head + src];
      }
    }
    for (int c0 = 0; c0 < cnt; c0 += RW * U) {
      uint4 v[U];
      int to[U];
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int c = c0 + e * RW + lane / LANES;  // rows beyond cnt have dst -1, those beyond 31 wrap to one
        to[e] = __shfl_sync(0xffffffffu, dst, c & 31);
        const int from = __shfl_sync(0xffffffffu, src, c & 31);
        if (c >= cnt) to[e] = -1;
        if (to[e] >= 0) v[e] = rows[(size_t)from * (LANES / 2)];
      }
#pragma unroll
      for (int e = 0; e < U; ++e)
        if (to[e] >= 0) rows[(size_t)to[e] * (LANES / 2)] = v[e];
    }
  }
}

template <int CL, bool HELD>
static cudaError_t launch_select(const EvictParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.Hkv * CL, p.B);
  cfg.blockDim = dim3(kEvThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<CL, HELD>, p);
}

cudaError_t launch_evict(const EvictParams& p, int d, cudaStream_t s) {
  int n = 0;
  int64_t room = 0;
  for (int b = 0; b < p.B; ++b) {
    n = p.req[b].n > n ? p.req[b].n : n;
    room = p.req[b].room > room ? p.req[b].room : room;
  }
  cudaError_t e = n <= kEvSlice                ? launch_select<1, true>(p, s)
                  : n <= kEvSlice * kEvCluster ? launch_select<kEvCluster, true>(p, s)
                                               : launch_select<kEvCluster, false>(p, s);
  if (e != cudaSuccess) return e;
  // enough warps to fill the GPU before each takes more moves at a time, up to a lane each
  const int64_t heads = (int64_t)p.Hkv * p.B, warps = 152 * 64;
  int64_t per = (room * heads + warps - 1) / warps;
  per = per < 4 ? 4 : per > 32 ? 32 : per;
  const int64_t want = (room + 8 * per - 1) / (8 * per), wave = (warps / 8 + heads - 1) / heads;
  const dim3 grid((unsigned)(want < wave ? want : wave), p.Hkv, p.B);
  return d == 128 ? launch_pdl(evict_move_kernel<128>, grid, dim3(256), 0, s, p, (int)per)
                  : launch_pdl(evict_move_kernel<64>, grid, dim3(256), 0, s, p, (int)per);
}

}  // namespace vc
