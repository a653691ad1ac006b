// Eviction from live caches by accumulated attention weight, in place.
//
// Select: of a KV head's n rows the `keep` of largest rank stay, the rank being the order-preserving
// 32-bit image of the score (guarded rows above everything, NaN below everything) and, among equals,
// the lower row. A radix select, most significant digit first (11, 11 and 10 bits), gives the rank T of
// the keep-th row and how many rows of rank T stay; one ordered pass then numbers the rows: a row below
// `keep` that goes is hole i - kept(i), a row behind it that stays is move kept(i) - (keep - moves),
// with kept(i) the kept rows before row i. There are as many holes as moves, and move j goes into hole j.
// Scores and positions are read once: the ranks are held in shared memory.
//
// Move: only the rows behind the budget that stay are read and written (K, V, score, position). A warp
// takes consecutive moves: their plan, scores and positions lane by lane (neighbours in memory), then
// their K and V rows, several in flight.
//
// What bounds it. 32 heads of 131072 rows shrunk to 32768: select 30 us (34 MB; the shared atomics of the first
// pass, then barriers), move 131 us (804 MB in rows of 256 bytes, 0.91 of the copy rate). 64 heads, 32 rows over
// 8192: 12 us, three passes over the held ranks with their barriers, and two launches.
#include "vc_internal.cuh"

namespace vc {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvHeld = 40 * 1024;  // ranks a CTA holds at most (160 KB)
constexpr int kEvBins = 2048;
constexpr int kEvCoarse = kEvBins / 32;  // sums of 32 consecutive bins

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
// consecutive segment of the slice. HELD: the slice's ranks stay in shared memory; otherwise (more than
// kEvHeld rows a CTA) they are taken from memory again in every pass.
template <int CL, bool HELD>
__global__ void __launch_bounds__(kEvThreads, 2) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t held[];  // [seg * kEvWarps] ranks
  __shared__ uint32_t count[kEvBins];
  __shared__ uint32_t fine[2][kEvBins], coarse[2][kEvCoarse];  // by pass: the cluster may still read the last one's
  __shared__ uint32_t s_prefix, s_rem;
  __shared__ int s_cnt[2][kEvWarps];
  __shared__ int s_cta[2];  // this CTA's rows above T and equal to T
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kEvBins; i += kEvThreads) count[i] = 0;
  if (tid == 0) s_prefix = 0;
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t rank = CL > 1 ? ev_cluster_rank() : 0u;
  const int h = blockIdx.x / CL;
  const EvictReqDev& r = p.req[blockIdx.y];
  const int n = r.n, keep = r.keep, sink = r.sink, recent_from = r.recent_from, room = r.room;
  const float* score = r.score + (size_t)h * r.cap;
  const int32_t* pos = r.pos + (size_t)h * r.cap;
  int32_t* plan = r.plan + (size_t)h * r.plan_stride;
  const int per = (n + CL - 1) / CL;                               // rows of a slice
  const int s0 = min((int64_t)n, (int64_t)rank * per), s1 = min((int64_t)n, (int64_t)s0 + per);
  const int seg = ((s1 - s0 + 31) / 32 + kEvWarps - 1) / kEvWarps * 32;  // rows of a warp
  const int w0 = min(s1, s0 + warp * seg), w1 = min(s1, w0 + seg);
  uint32_t* mine = held + warp * seg;
  auto load = [&](int i) { return i < w1 ? evict_rank(__ldcg(score + i), __ldcg(pos + i), sink, recent_from) : 0u; };
  auto rank_of = [&](int i) { return HELD ? mine[i - w0] : load(i); };
  // A shared atomic a row, whatever the digits: 32 heads of 131072 rows take 28.8 us with one digit for all rows
  // and 27.9 with evenly spread scores; adding up a warp's equal digits first, or a thread's, cost more than it
  // saved (by 3 to 20 us).
  auto tally = [&](bool in, uint32_t dg) {
    if (in) atomicAdd(&count[dg], 1u);
  };
  if (tid == 0) s_rem = (uint32_t)keep;
  __syncthreads();
  uint32_t mask = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 1023u : 2047u;
    const uint32_t prefix = s_prefix;
    if (pass == 0) {
#pragma unroll 1
      for (int base = w0; base < w1; base += 32 * 4) {  // four groups of 32 rows: eight loads in flight
        float sc[4];
        int ps[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = base + 32 * k + lane;
          sc[k] = i < w1 ? __ldcg(score + i) : 0.f;
          ps[k] = i < w1 ? __ldcg(pos + i) : 0;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = base + 32 * k + lane;
          const uint32_t u = evict_rank(sc[k], ps[k], sink, recent_from);
          if (HELD && i < w1) mine[i - w0] = u;
          tally(i < w1, u >> shift);
        }
      }
    } else {
#pragma unroll 1
      for (int base = w0; base < w1; base += 32 * 2) {
        uint32_t u[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) u[k] = base + 32 * k + lane < w1 ? rank_of(base + 32 * k + lane) : 0u;
#pragma unroll
        for (int k = 0; k < 2; ++k) tally(base + 32 * k + lane < w1 && (u[k] & mask) == prefix, (u[k] >> shift) & digit);
      }
    }
    __syncthreads();
    // the sums of 32 bins each: only these, and then the 32 bins of one of them, are
    // added up over the cluster (reading all bins of all CTAs kept the cluster's network busy for longer
    // than everything else)
    for (int c = warp; c < kEvCoarse; c += kEvWarps) {
      uint32_t v = count[32 * c + lane];
      count[32 * c + lane] = 0;  // for the next pass
      fine[pass & 1][32 * c + lane] = v;
      v = __reduce_add_sync(0xffffffffu, v);
      if (lane == 0) coarse[pass & 1][c] = v;
    }
    if (CL > 1)
      ev_cluster_sync();
    else
      __syncthreads();
    if (warp == 0) {
      auto total = [&](const uint32_t* word) {
        if constexpr (CL == 1) return *word;
        uint32_t v = 0;
#pragma unroll
        for (int q = 0; q < CL; ++q) v += ev_ld_cluster(word, q);
        return v;
      };
      // of a row of counts (lane 0 the largest digit) the lane in which the rem-th row stands, -1: behind
      // them; rem becomes its number among that lane's
      auto find = [&](uint32_t cnt, uint32_t& rem) -> int {
        uint32_t sum = cnt;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint32_t o = __shfl_up_sync(0xffffffffu, sum, off);
          if (lane >= off) sum += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, sum >= rem);
        if (!hit) {
          rem -= __shfl_sync(0xffffffffu, sum, 31);
          return -1;
        }
        const int at = __ffs(hit) - 1;
        rem -= __shfl_sync(0xffffffffu, sum - cnt, at);
        return at;
      };
      uint32_t rem = s_rem;
      const uint32_t hi = total(&coarse[pass & 1][kEvCoarse - 1 - lane]), lo = total(&coarse[pass & 1][31 - lane]);
      int c = find(hi, rem);
      c = c >= 0 ? kEvCoarse - 1 - c : 31 - max(0, find(lo, rem));
      const int at = max(0, find(total(&fine[pass & 1][32 * c + 31 - lane]), rem));
      if (lane == 0) {
        s_rem = rem;
        s_prefix = prefix | ((uint32_t)(32 * c + 31 - at) << shift);
      }
    }
    mask |= digit << shift;
    __syncthreads();
  }
  const uint32_t T = s_prefix;
  const int need_eq = (int)s_rem;
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t u = rank_of(i);
    gt += u > T;
    eq += u == T;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    s_cnt[0][warp] = gt;
    s_cnt[1][warp] = eq;
  }
  __syncthreads();
  // rows above and equal to T in the warps (and, through the cluster, the CTAs) before this one
  const int gw = s_cnt[0][lane], ew = s_cnt[1][lane];
  int gt_run = __reduce_add_sync(0xffffffffu, lane < warp ? gw : 0), eq_run = __reduce_add_sync(0xffffffffu, lane < warp ? ew : 0);
  if constexpr (CL > 1) {
    const int gt_all = __reduce_add_sync(0xffffffffu, gw), eq_all = __reduce_add_sync(0xffffffffu, ew);
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
#pragma unroll 2
  for (int base = w0; base < w1; base += 32) {
    const int i = base + lane;
    const uint32_t u = i < w1 ? rank_of(i) : 0u;
    const unsigned mg = __ballot_sync(0xffffffffu, i < w1 && u > T), me = __ballot_sync(0xffffffffu, i < w1 && u == T);
    if (i < w1) {
      const int eq_before = eq_run + __popc(me & lt);
      const int kept = gt_run + __popc(mg & lt) + min(eq_before, need_eq);  // kept rows before row i
      const bool stays = u > T || (u == T && eq_before < need_eq);
      if (i < keep) {
        if (!stays && i - kept < room) plan[4 + i - kept] = i;
        if (i == keep - 1) plan[0] = keep - kept - (stays ? 1 : 0);
      } else if (stays && keep - 1 - kept < room) {
        plan[4 + room + keep - 1 - kept] = i;  // from the last move backwards
      }
    }
    gt_run += __popc(mg);
    eq_run += __popc(me);
  }
  if (CL > 1) ev_cluster_sync();  // no CTA leaves while another may still read its shared memory
}

// grid (x, Hkv, B): warps take per_warp consecutive moves (at most 32) at a time.
template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictParams p, int per_warp) {
  constexpr int LANES = D / 4;       // 16-byte pieces of a row of K and of V
  constexpr int RW = 32 / LANES;     // rows a warp copies at a time
  constexpr int U = 8;               // of those, in flight
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
        src = 0;
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
        v[e] = rows[(size_t)from * (LANES / 2)];  // some row where there is none to move: no branch between the loads
      }
#pragma unroll
      for (int e = 0; e < U; ++e)
        if (to[e] >= 0) rows[(size_t)to[e] * (LANES / 2)] = v[e];
    }
  }
}

template <int CL, bool HELD>
static cudaError_t launch_select(const EvictParams& p, int n, cudaStream_t s) {
  const int per = (n + CL - 1) / CL;  // the largest slice; a warp's part is a multiple of 32 rows
  const int smem = HELD ? ((per + 31) / 32 + kEvWarps - 1) / kEvWarps * 32 * kEvWarps * 4 : 0;
  static std::atomic<uint64_t> attr_set{0};
  if (HELD) {
    const cudaError_t e = raise_smem_limit(evict_select_kernel<CL, HELD>, kEvHeld * 4, attr_set);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.Hkv * CL, p.B);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
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
  // CTAs per head: enough to hold the ranks; one an SM where the heads leave SMs free and there are 16384 rows to
  // cut (8 heads: 1 and 8 CTAs a head take 15.4 and 12.0 us at 16384 rows, 11.1 and 11.7 at 8192: the passes'
  // fixed part, and the cluster's); and rather four than two with more heads than that, which even out over the SMs
  // (96 heads, 65536 rows: 52.2 us with 2, 42.6 with 4, 56.7 with 8; 64 heads: 28.0, 32.3, 40.5).
  const int64_t all = (int64_t)p.Hkv * p.B;
  int cl = 1;
  while (cl < 8 && (n > cl * kEvHeld || (n >= 16384 && all * cl * 2 <= 152) || (cl == 2 && all > 76))) cl *= 2;
  cudaError_t e = n > 8 * kEvHeld ? launch_select<8, false>(p, n, s)
                  : cl == 8       ? launch_select<8, true>(p, n, s)
                  : cl == 4       ? launch_select<4, true>(p, n, s)
                  : cl == 2       ? launch_select<2, true>(p, n, s)
                                  : launch_select<1, true>(p, n, s);
  if (e != cudaSuccess) return e;
  // enough warps to fill the GPU before each takes more moves at a time, up to a lane each
  const int64_t heads = all, warps = 152 * 64;
  int64_t per = (room * heads + warps - 1) / warps;
  per = per < 4 ? 4 : per > 32 ? 32 : per;
  const int64_t want = (room + 8 * per - 1) / (8 * per), wave = (warps / 8 + heads - 1) / heads;
  const dim3 grid((unsigned)(want < wave ? want : wave), p.Hkv, p.B);
  return d == 128 ? launch_pdl(evict_move_kernel<128>, grid, dim3(256), 0, s, p, (int)per)
                  : launch_pdl(evict_move_kernel<64>, grid, dim3(256), 0, s, p, (int)per);
}

}  // namespace vc
