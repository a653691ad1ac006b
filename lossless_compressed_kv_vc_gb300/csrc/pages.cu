// A pool of pages: room for new rows, forks, pages given back, the pages in use moved together, and the rows of
// an accepted path joined to the context.
//
// The state is whole numbers in device memory, up to a few hundred a turn: one CTA moves it on (a launch and some
// dependent loads, 3 to 10 us; long sequences reserved or given back at once take more, see there), and whatever
// must not depend on the order of threads is settled by position in the call: pages are taken from and put on the
// stack at places given by a prefix sum. What is copied, K and V, is left to grids that fill the GPU.
#include "paged.cuh"

namespace vc {

constexpr int kPageThreads = 1024;
constexpr int kPageWarps = kPageThreads / 32;

// The last i in [0, VC_MAX_BATCH) with begin[i] <= x (begin of requests that take nothing equals the next one's).
__device__ __forceinline__ int page_req_of(const int32_t* begin, int x) {
  int lo = 0;
#pragma unroll
  for (int s = VC_MAX_BATCH / 2; s > 0; s >>= 1)
    if (begin[lo + s] <= x) lo += s;
  return lo;
}

__device__ __forceinline__ int warp_scan(int v, int lane) {  // sum over lanes 0 .. lane
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += o;
  }
  return v;
}

// Rows of context, within the pages held whatever the state says; `ok` falls where it does not add up.
__device__ __forceinline__ int context_rows(const PagedDev& kv, int seq, int held, bool& ok) {
  const int n = kv.len[seq], cap = held << kv.shift;
  if (n < 0 || n > cap || held != kv.held[seq]) ok = false;
  return min(max(n, 0), cap);
}

__global__ void __launch_bounds__(256) pages_init_kernel(PagedDev kv) {
  pdl_wait();
  const int step = gridDim.x * blockDim.x;
  for (int64_t i = blockIdx.x * blockDim.x + threadIdx.x; i < kv.n_pages; i += step) {
    kv.refs[i] = 0;
    kv.free_pages[i] = kv.n_pages - 1 - (int)i;
  }
  for (int64_t i = blockIdx.x * blockDim.x + threadIdx.x; i < kv.n_seq; i += step) kv.len[i] = kv.held[i] = kv.next[i] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *kv.n_free = kv.n_pages;
}

// ---- reserve ------------------------------------------------------------------------------------------
// One warp takes the requests, a lane each: what they need follows from the state alone unless the stack runs
// short. The block then hands out the pages (8192 of one sequence 9 us, 32 x 1000 23 us).
__device__ __forceinline__ void reserve_plan(const ReserveParams& p) {
  __shared__ int32_t begin[VC_MAX_BATCH], s_held[VC_MAX_BATCH], s_tail[VC_MAX_BATCH], s_old[VC_MAX_BATCH], s_rows[VC_MAX_BATCH];
  __shared__ int s_total, s_free;
  const PagedDev& kv = p.kv;
  if (threadIdx.x < 32) {
    const int r = threadIdx.x, page = kv.rows();
    const bool here = r < p.B;
    const vc_reserve_req q = p.req[here ? r : 0];
    int held = 0, n = 0, old = -1, refs = 0, more = 0;
    bool ok = here, shared = false;
    const int avail = min(max(*kv.n_free, 0), kv.n_pages);
    if (here) {
      held = kv.held_of(q.seq);
      n = context_rows(kv, q.seq, held, ok);
      const int64_t want = ((int64_t)n + q.rows + page - 1) >> kv.shift;
      more = (int)min(max(want - held, (int64_t)0), (int64_t)avail);
      if (want > kv.max_pages || want - held > avail) ok = false;
      if (ok && q.rows > 0 && (n & (page - 1)) != 0) {  // n <= held * page: the table has this page
        old = kv.pages_of(q.seq)[n >> kv.shift];
        if (kv.has_page(old))
          refs = kv.refs[old];
        else
          ok = false;
      }
    }
    // of the requests that go on in one page, each that takes a copy leaves it to one sequence less
    const unsigned same = __match_any_sync(0xffffffffu, ok && old >= 0 ? old : -1 - r), lt = (1u << r) - 1u;
    shared = ok && old >= 0 && refs - __popc(same & lt) > 1;
    int take = ok ? more + shared : 0;
    // 32 requests' sum takes more than 32 bits
    const int64_t all = ((int64_t)__reduce_add_sync(0xffffffffu, take >> 16) << 16) + __reduce_add_sync(0xffffffffu, take & 0xffff);
    if (all > avail) {  // one after the other, as long as pages last
      int left = avail;
      unsigned copied = 0;
      for (int i = 0; i < p.B; ++i) {
        const bool sh = ok && old >= 0 && refs - __popc(same & copied & lt) > 1;
        const bool served = ok && more + sh <= left;
        if (r == i) {
          shared = sh;
          take = served ? more + sh : 0;
          ok = served;
        }
        copied |= (unsigned)__shfl_sync(0xffffffffu, (int)(served && sh), i) << i;
        left -= __shfl_sync(0xffffffffu, take, i);
      }
    }
    if (here && !ok) set_status(p.dev_status, VC_DEV_PAGES);
    shared = shared && ok;
    const int end = warp_scan(take, r);
    begin[r] = end - take;
    s_held[r] = held;
    s_tail[r] = n >> kv.shift;
    s_old[r] = shared ? old : -1;
    s_rows[r] = n & (page - 1);
    if (here) {
      if (shared) atomicSub(&kv.refs[old], 1);
      if (take > shared) kv.held[q.seq] = held + take - shared;
      if (!shared) p.copies[r] = make_int4(0, 0, 0, 0);
    }
    if (r == 31) {
      s_total = end;
      s_free = avail;
      if (end > 0) *kv.n_free = avail - end;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < s_total; i += kPageThreads) {
    const int r = page_req_of(begin, i), copy = s_old[r] >= 0, j = i - begin[r];
    const int page = kv.free_pages[s_free - 1 - i];
    const bool good = kv.has_page(page);
    kv.pages_of(p.req[r].seq)[j < copy ? s_tail[r] : s_held[r] + j - copy] = page;
    if (good)
      kv.refs[page] = 1;
    else
      set_status(p.dev_status, VC_DEV_PAGES);
    if (j < copy) p.copies[r] = good ? make_int4(s_old[r], page, s_rows[r], 0) : make_int4(0, 0, 0, 0);
  }
}

__global__ void __launch_bounds__(kPageThreads) reserve_plan_kernel(const __grid_constant__ ReserveParams p) {
  pdl_launch_dependents();
  pdl_wait();
  reserve_plan(p);
}

// Plan and copies in one launch, by a cluster whose first CTA plans: most calls have no page to copy, and pay for one
// launch instead of two. Call after call without a copy 4.1 us (the host's time), with two launches 5.9; alone 8, and
// 9.5. With a page to copy for every request, 32 KB each: one 10.8 us, two launches 12.2; eight (512 KB in all) 12.3,
// 13.2; 31 (2 MB) 16.4, 14.8.
constexpr int kReserveCtas = 8;
__global__ void __cluster_dims__(kReserveCtas, 1, 1) __launch_bounds__(kPageThreads)
reserve_kernel(const __grid_constant__ ReserveParams p, int d) {
  __shared__ int4 s_copies[VC_MAX_BATCH];
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0) reserve_plan(p);
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if ((int)threadIdx.x < p.B) s_copies[threadIdx.x] = __ldcg(&p.copies[threadIdx.x]);
  __syncthreads();
  // a warp takes 256 pieces of 16 bytes of a head's K or V in one of the pages, all on their way at once
  constexpr int U = 8;
  const int row = d / 8, page = p.kv.rows() * row, parts = (page + 32 * U - 1) / (32 * U);
  for (int w = blockIdx.x * kPageWarps + threadIdx.x / 32; w < p.B * 2 * p.Hkv * parts; w += kReserveCtas * kPageWarps) {
    const int r = w / (2 * p.Hkv * parts), head = (w / parts) % p.Hkv, v0 = (w / (p.Hkv * parts)) & 1;
    const int4 c = s_copies[r];
    const int n = c.z * row, i0 = (w % parts) * 32 * U + (threadIdx.x & 31);
    uint4* pool = reinterpret_cast<uint4*>(v0 ? p.kv.v : p.kv.k);
    const uint4* src = pool + ((int64_t)c.x * p.Hkv + head) * page;
    uint4* dst = pool + ((int64_t)c.y * p.Hkv + head) * page;
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + 32 * u < n) x[u] = src[i0 + 32 * u];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + 32 * u < n) dst[i0 + 32 * u] = x[u];
  }
}

// grid (KV head, request, K or V): a head's rows of a page lie together.
__global__ void __launch_bounds__(256) reserve_copy_kernel(const __grid_constant__ ReserveParams p, int d) {
  pdl_launch_dependents();
  pdl_wait();
  const int4 c = p.copies[blockIdx.y];
  const int n = c.z * (d / 8), pieces = p.kv.rows() * (d / 8);
  uint4* pool = reinterpret_cast<uint4*>(blockIdx.z ? p.kv.v : p.kv.k);
  const uint4* src = pool + ((int64_t)c.x * p.Hkv + blockIdx.x) * pieces;
  uint4* dst = pool + ((int64_t)c.y * p.Hkv + blockIdx.x) * pieces;
  for (int i0 = threadIdx.x; i0 < n; i0 += 4 * 256) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * 256 < n) v[u] = src[i0 + u * 256];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * 256 < n) dst[i0 + u * 256] = v[u];
  }
}

// ---- fork ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) fork_kernel(const __grid_constant__ ForkParams p) {
  const PagedDev& kv = p.kv;
  pdl_launch_dependents();
  pdl_wait();
  const vc_fork_req q = p.req[blockIdx.x];
  bool ok = kv.held[q.dst] == 0;
  const int n = context_rows(kv, q.src, kv.held_of(q.src), ok), pages = (n + kv.rows() - 1) >> kv.shift;
  __syncthreads();  // all have looked at dst
  if (!ok) {
    if (threadIdx.x == 0) set_status(p.dev_status, VC_DEV_PAGES);
    return;
  }
  const int32_t* from = kv.pages_of(q.src);
  int32_t* to = kv.pages_of(q.dst);
  for (int i = threadIdx.x; i < pages; i += blockDim.x) {
    const int page = from[i];
    to[i] = page;
    if (kv.has_page(page))
      atomicAdd(&kv.refs[page], 1);
    else
      set_status(p.dev_status, VC_DEV_PAGES);
  }
  if (threadIdx.x == 0) {
    kv.held[q.dst] = pages;
    kv.len[q.dst] = n;
    kv.next[q.dst] = kv.next[q.src];
  }
}

// ---- trim ---------------------------------------------------------------------------------------------
// All pages given back by the call in one list, by request and from a sequence's last page to its first. A page
// that several of them held leaves with the last: counts fall first; then the pages that nobody holds take the
// largest place in the list of those that named them, as a negative count; and that one puts it on the stack.
// Bound by latency: three passes of one CTA, each round of 1024 pages a table load and an access to its count that
// depends on it (100 pages 5 us, 32 x 100 13 us, 8192 of one sequence 23 us, 32 x 1000 81 us, 32 x 8192 655 us).
__global__ void __launch_bounds__(kPageThreads) trim_kernel(const __grid_constant__ TrimParams p) {
  __shared__ int32_t begin[VC_MAX_BATCH], s_last[VC_MAX_BATCH];
  __shared__ int32_t sums[kPageWarps];
  __shared__ int s_total, s_free;
  const PagedDev& kv = p.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x < 32) {
    const int r = threadIdx.x;
    int cnt = 0, held = 0;
    if (r < p.B) {
      const vc_trim_req q = p.req[r];
      bool ok = true;
      held = kv.held_of(q.seq);
      int n = context_rows(kv, q.seq, held, ok);
      if (!ok) set_status(p.dev_status, VC_DEV_PAGES);
      if (q.rows < n) {
        n = q.rows;
        kv.next[q.seq] = q.next;
      }
      const int keep = (int)(((int64_t)n + kv.rows() - 1) >> kv.shift);
      cnt = held - keep;
      kv.len[q.seq] = n;
      kv.held[q.seq] = keep;
    }
    const int end = warp_scan(cnt, r);
    begin[r] = end - cnt;
    s_last[r] = held - 1;
    if (r == 31) s_total = end;
    if (r == 0) s_free = min(max(*kv.n_free, 0), kv.n_pages);
  }
  __syncthreads();
  const int total = s_total;
  auto page_at = [&](int i) {
    const int r = page_req_of(begin, i);
    return kv.pages_of(p.req[r].seq)[s_last[r] - (i - begin[r])];
  };
  for (int i = threadIdx.x; i < total; i += kPageThreads) {
    const int page = page_at(i);
    if (!kv.has_page(page) || atomicSub(&kv.refs[page], 1) <= 0) set_status(p.dev_status, VC_DEV_PAGES);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += kPageThreads) {
    const int page = page_at(i);
    if (kv.has_page(page) && __ldcg(&kv.refs[page]) <= 0) atomicMin(&kv.refs[page], -1 - i);
  }
  __syncthreads();
  int top = s_free;
  for (int i0 = 0; i0 < total; i0 += kPageThreads) {
    const int i = i0 + threadIdx.x, page = i < total ? page_at(i) : -1;
    const bool gone = kv.has_page(page) && __ldcg(&kv.refs[page]) == -1 - i;
    const unsigned all = __ballot_sync(0xffffffffu, gone);
    if (lane == 0) sums[warp] = __popc(all);
    __syncthreads();
    const int before = warp_scan(sums[lane], lane);  // every warp adds up all of them
    const int at = top + __shfl_sync(0xffffffffu, before, warp) - __popc(all >> lane);
    if (gone) {
      kv.refs[page] = 0;
      if (at >= 0 && at < kv.n_pages)
        kv.free_pages[at] = page;
      else
        set_status(p.dev_status, VC_DEV_PAGES);
    }
    top += __shfl_sync(0xffffffffu, before, 31);
    __syncthreads();
  }
  if (threadIdx.x == 0 && top != s_free) *kv.n_free = min(max(top, 0), kv.n_pages);
}

// ---- compact ------------------------------------------------------------------------------------------
// Plan: with U pages in use, page i < U that is free is hole i - used(i), page i >= U in use is the
// U - 1 - used(i)-th to move, counted from the last, where used(i) counts the pages in use before page i.
// Warps take consecutive segments: a pass that counts, and one that numbers.
__global__ void __launch_bounds__(kPageThreads) compact_plan_kernel(const __grid_constant__ CompactParams p) {
  __shared__ int32_t sums[kPageWarps];
  const PagedDev& kv = p.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seg = ((kv.n_pages + 31) / 32 + kPageWarps - 1) / kPageWarps * 32;
  const int w0 = (int)min((int64_t)kv.n_pages, (int64_t)warp * seg), w1 = (int)min((int64_t)kv.n_pages, (int64_t)w0 + seg);
  pdl_launch_dependents();
  pdl_wait();
  int cnt = 0;
#pragma unroll 8
  for (int i = w0 + lane; i < w1; i += 32) cnt += kv.refs[i] > 0;
  cnt = __reduce_add_sync(0xffffffffu, cnt);
  if (lane == 0) sums[warp] = cnt;
  __syncthreads();
  const int upto = warp_scan(sums[lane], lane);
  const int U = __shfl_sync(0xffffffffu, upto, 31), room = kv.n_pages / 2 + 1;
  int run = __shfl_sync(0xffffffffu, upto, warp) - cnt;
#pragma unroll 4
  for (int base = w0; base < w1; base += 32) {
    const int i = base + lane;
    const bool used = i < w1 && kv.refs[i] > 0;
    const unsigned all = __ballot_sync(0xffffffffu, used);
    const int before = run + __popc(all & ((1u << lane) - 1u));
    if (i < w1) {
      if (i < U) {
        if (!used && i - before < room) p.hole[i - before] = i;
        if (i == U - 1) p.head[0] = U - before - used;
      } else if (used) {
        const int back = U - 1 - before;
        p.back[i] = back;
        if (back < room) p.from[back] = i;
      }
    }
    run += __popc(all);
  }
  if (threadIdx.x == 0) {
    p.head[1] = U;
    if (U == 0) p.head[0] = 0;
  }
}

// Pages' K and V in units of 16 KB, then the whole numbers. Bound by DRAM: 4017 pages of 64 KB (K and V) moved, 527 MB
// in 77 to 80 us, the copy rate; the plan before it takes 8 us for 16384 pages.
constexpr int kMoveUnit = 1024;  // 16-byte pieces
__global__ void __launch_bounds__(256) compact_move_kernel(const __grid_constant__ CompactParams p, int d) {
  const PagedDev& kv = p.kv;
  pdl_launch_dependents();
  pdl_wait();
  const int M = p.head[0], U = p.head[1];
  const int64_t pieces = ((int64_t)p.Hkv << kv.shift) * (d / 8), units = (pieces + kMoveUnit - 1) / kMoveUnit;
  for (int64_t w = blockIdx.x; w < 2 * M * units; w += gridDim.x) {
    const int64_t m = w / (2 * units), part = w - m * 2 * units, at = (part >> 1) * kMoveUnit;
    uint4* pool = reinterpret_cast<uint4*>(part & 1 ? kv.v : kv.k);
    const uint4* src = pool + p.from[M - 1 - m] * pieces;
    uint4* dst = pool + p.hole[m] * pieces;
    uint4 v[kMoveUnit / 256];
#pragma unroll
    for (int u = 0; u < kMoveUnit / 256; ++u)
      if (at + u * 256 + threadIdx.x < pieces) v[u] = src[at + u * 256 + threadIdx.x];
#pragma unroll
    for (int u = 0; u < kMoveUnit / 256; ++u)
      if (at + u * 256 + threadIdx.x < pieces) dst[at + u * 256 + threadIdx.x] = v[u];
  }
  const int64_t step = (int64_t)gridDim.x * 256, first = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int64_t i = first; i < M; i += step) {
    const int src = p.from[M - 1 - i];
    kv.refs[p.hole[i]] = kv.refs[src];
    kv.refs[src] = 0;
  }
  for (int64_t i = first; i < (int64_t)kv.n_seq * kv.max_pages; i += step) {
    const int seq = (int)(i / kv.max_pages);
    if (i - (int64_t)seq * kv.max_pages >= kv.held[seq]) continue;
    const int page = kv.table[i];
    if (page < U && page >= 0) continue;
    const int back = kv.has_page(page) ? p.back[page] : -1;
    if (back >= 0 && back < M && p.from[back] == page)
      kv.table[i] = p.hole[M - 1 - back];
    else
      set_status(p.dev_status, VC_DEV_PAGES);
  }
  for (int64_t i = first; i < kv.n_pages - U; i += step) kv.free_pages[i] = kv.n_pages - 1 - (int)i;
  if (first == 0) *kv.n_free = kv.n_pages - U;
}

// ---- commit -------------------------------------------------------------------------------------------
// A block per request, a thread per 16-byte column of the heads' K and V rows, which it moves from the first
// row to the last: row i takes row path[i] >= i, so that no row is written that a later one still needs.
// vc_rope_pages has written the turn's rows if all of them lie in pages that the sequence holds alone, which is so
// where vc_pages_reserve served it. Otherwise nothing becomes context, and the turn can be made again. Bound by
// latency (one token of 32 sequences 4.0 us, a prompt of 2048 4.2; 5 drafts along a path 5.9, and 5.0 if the pages were
// not looked at).
constexpr int kCommitRows = 256;  // rows of the path looked up at a time
template <int D>
__global__ void __launch_bounds__(256) commit_kernel(const __grid_constant__ CommitParams p) {
  __shared__ int64_t s_src[kCommitRows], s_dst[kCommitRows];  // first piece of the row in head 0; dst < 0: stays
  __shared__ int s_m;
  const PagedDev& kv = p.kv;
  pdl_launch_dependents();
  pdl_wait();
  const vc_commit_req q = p.req[blockIdx.x];
  const int held = kv.held_of(q.seq), page = kv.rows();
  const int32_t* pages = kv.pages_of(q.seq);
  bool ok = true;
  const int n = context_rows(kv, q.seq, held, ok);
  const int early = q.path && (int)threadIdx.x < q.n_rows ? q.path[threadIdx.x] : 0;  // beside the other state, not behind it
  const int m = q.n_acc ? min(max(*q.n_acc, 0), q.n_rows) : q.n_rows;
  const int end = (int)(((int64_t)n + q.n_rows + page - 1) >> kv.shift);
  if (end > held)
    ok = false;
  else
#pragma unroll 4
    for (int j = (n >> kv.shift) + threadIdx.x; j < end; j += blockDim.x) {
      const int own = pages[j];
      if (!kv.has_page(own) || kv.refs[own] != 1) ok = false;
    }
  if (threadIdx.x == 0) s_m = m;
  if (!__syncthreads_and(ok)) {
    if (threadIdx.x == 0) set_status(p.dev_status, VC_DEV_PAGES);
    return;
  }
  const int head = page * (D / 8), cols = p.Hkv * (D / 8);  // pieces of a head's page; 16-byte columns of K
  auto piece = [&](int row) { return ((int64_t)pages[row >> kv.shift] * p.Hkv * page + (row & (page - 1))) * (D / 8); };
  if (q.path)
    for (int i0 = 0; i0 < m; i0 += kCommitRows) {
      __syncthreads();
      for (int i = i0 + threadIdx.x; i < min(m, i0 + kCommitRows); i += blockDim.x) {
        const int from = i < (int)blockDim.x ? early : q.path[i];
        const bool good = from >= i && from < q.n_rows;
        int64_t src = 0, dst = -1;
        if (good && from != i) {  // both among the turn's rows
          src = piece(n + from);
          dst = piece(n + i);
        }
        if (!good) {
          atomicMin(&s_m, i);
          set_status(p.dev_status, VC_DEV_PAGES);
        }
        s_src[i - i0] = src;
        s_dst[i - i0] = dst;
      }
      __syncthreads();
      const int end = min(s_m, i0 + kCommitRows) - i0;
      for (int c = threadIdx.x; c < 2 * cols; c += blockDim.x) {
        const int col = c < cols ? c : c - cols;
        uint4* pool = reinterpret_cast<uint4*>(c < cols ? kv.k : kv.v) + (int64_t)(col / (D / 8)) * head + col % (D / 8);
        constexpr int U = 16;  // rows in flight
        for (int i = 0; i < end; i += U) {
          uint4 v[U];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (i + u < end && s_dst[i + u] >= 0) v[u] = pool[s_src[i + u]];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (i + u < end && s_dst[i + u] >= 0) pool[s_dst[i + u]] = v[u];
        }
      }
      if (s_m < i0 + kCommitRows) break;
    }
  __syncthreads();
  if (threadIdx.x == 0) {
    kv.len[q.seq] = n + s_m;
    kv.next[q.seq] += q.advance < 0 ? s_m : q.advance;
  }
}

// ------------------------------------------------------------------------------------------------
cudaError_t launch_pages_init(const PagedDev& kv, cudaStream_t s) {
  const int n = kv.n_pages > kv.n_seq ? kv.n_pages : kv.n_seq, blocks = (n - 1) / 256 + 1;
  return launch_pdl(pages_init_kernel, dim3(blocks < 608 ? blocks : 608), dim3(256), 0, s, kv);
}

cudaError_t launch_reserve(const ReserveParams& p, int d, cudaStream_t s) {
  // up to 2 MB of copies if every request had one: beyond that a cluster is slow for them
  if (((int64_t)p.B * p.Hkv << p.kv.shift) * d * 4 <= 2 << 20) return launch_pdl(reserve_kernel, dim3(kReserveCtas), dim3(kPageThreads), 0, s, p, d);
  const cudaError_t e = launch_pdl(reserve_plan_kernel, dim3(1), dim3(kPageThreads), 0, s, p);
  return e != cudaSuccess ? e : launch_pdl(reserve_copy_kernel, dim3(p.Hkv, p.B, 2), dim3(256), 0, s, p, d);
}

cudaError_t launch_fork(const ForkParams& p, int B, cudaStream_t s) {
  return launch_pdl(fork_kernel, dim3(B), dim3(256), 0, s, p);
}

cudaError_t launch_trim(const TrimParams& p, cudaStream_t s) {
  return launch_pdl(trim_kernel, dim3(1), dim3(kPageThreads), 0, s, p);
}

cudaError_t launch_compact(const CompactParams& p, int d, cudaStream_t s) {
  const cudaError_t e = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPageThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  // no more blocks than units that half the pages could need, or numbers to rewrite
  const int64_t units = ((((int64_t)p.Hkv << p.kv.shift) * (d / 8) + kMoveUnit - 1) / kMoveUnit) * p.kv.n_pages;
  const int64_t words = ((int64_t)p.kv.n_seq * p.kv.max_pages + 255) / 256;
  const int64_t want = units > words ? units : words;
  return launch_pdl(compact_move_kernel, dim3((unsigned)(want < 152 * 8 ? want : 152 * 8)), dim3(256), 0, s, p, d);
}

cudaError_t launch_commit(const CommitParams& p, int B, int d, cudaStream_t s) {
  return d == 128 ? launch_pdl(commit_kernel<128>, dim3(B), dim3(256), 0, s, p)
                  : launch_pdl(commit_kernel<64>, dim3(B), dim3(256), 0, s, p);
}

}  // namespace vc
