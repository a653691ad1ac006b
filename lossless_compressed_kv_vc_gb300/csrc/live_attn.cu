// Attention of new rows over live caches and an optional shared prefix, on tcgen05 tensor cores; with
// the weights that eviction ranks by.
//
// Row i of a request's n_rows rows sees every prefix row and own rows t <= n - n_rows + i:
//   s_t = q . k_t / sqrt(d),  o = sum_t 2^(s_t - lse) v_t  (log2 domain),  score[t] += sum_rows 2^(s_t - lse).
//
// Work decomposition. A group is a key sequence with the query rows that read it: the prefix with the
// rows of all requests, or one request's own cache with its rows. The rows of one KV head (tokens x
// G = Hq / Hkv heads) are cut into units of up to 256, the keys into tiles of 128. The prefix's tiles, [unit]
// [head][tile], and the own caches', [request][unit][head][tile], form a sequence each; CTAs (one per SM: 8
// softmax warps, 4 MMA issuers, 1 loader) are shared out between the two by cost, and each takes an equal
// range of its sequence. A CTA's part of a unit of a head (a piece) leaves (o, lse) partials; a second kernel
// merges a row's partials over both its groups. So the prefix is read once for up to 256 rows, whatever
// requests they come from, and a request's own rows cost what they are. With several units of prefix rows the
// CTAs are dealt out so that every unit's ranges are cut at the same tiles: they read a tile at about the same
// time, and it comes from DRAM once.
//
// Within a CTA two chains run side by side, each an issuer thread and a warpgroup of softmax threads (a
// thread per query row): S = Q K^T into TMEM, softmax in registers, P (bf16) over S in TMEM, O += P V with P
// read from TMEM. The chains meet only in the ring of K and V tiles, so one's softmax runs while the
// tensor cores work for the other. A unit of more than 128 rows gives each chain 128 rows and every tile
// (a tile serves 256 rows and costs 2); one of up to 128 rows gives both chains the same rows and a half of
// every tile (which costs 1), and each leaves its own partial. So both chains walk through every tile.
//
// What bounds it. One token a request: K and V from DRAM (8 caches of 8200 rows, 8 heads of 128: 49 us with the
// merge, 236 MB, 0.71 of the copy rate; 4 of 131072: 385 us, 0.83), the rest start-up and, where scores are
// kept, the second kernel's pass over them. Drafts over a prefix (2000 rows of a KV head, 65536 keys): 394 us back
// to back on two sets of inputs, 414 to 418 with others in each call, 1.15 to 1.22 PFLOP/s, 0.61 to 0.64 of the bf16
// peak: shared memory's bandwidth, since a pair of chains moves 320 KB a tile (Q
// twice 64, as S steps of 64 keys read it twice, K and V twice 32 each, and 64 in from L2), 2560 clocks at 128
// bytes each of about 3000; leaving out all exponentials changes nothing. Many short caches (a few tiles a
// piece): the pieces' fixed part, about 6 us each, of which instruction fetch is the largest.
#include "tc05.cuh"

#include <cudaTypedefs.h>
#include <math.h>
#include <string.h>

namespace vc {

constexpr int LM = 128;         // query rows of a chain
constexpr int LN = 128;         // keys per tile
constexpr int LS = 64;          // keys per step: S and P of half a tile, double-buffered
constexpr int LU = 2 * LM;      // query rows of a unit
// warps 0-3, 4-7 softmax of chains 0 and 1; 8, 9 issue their S; 10, 11 their P V; 12 TMA; 13-15 idle (they
// make a warpgroup with it: registers are handed over by warpgroup)
constexpr int LTHREADS = 512;
// Registers a thread: launched with 128 (65536 / 512), then 144 in the softmax warpgroups and 80 in the others
constexpr int LREG_SOFTMAX = 144, LREG_ISSUE = 80;
static_assert(256 * (LREG_SOFTMAX + LREG_ISSUE) <= 65536, "no more than the block was launched with");
constexpr int SCORE_KEYS = 1024;  // keys of a score block at most: 256 a pass
static_assert(SCORE_KEYS % 256 == 0 && LN % 4 == 0, "whole vectors of scores");
static_assert(VC_SCORED_MAX_ROWS <= LU, "a head's scored rows are one unit");

struct LiveGroup {
  int32_t n;          // keys
  int32_t rows;       // query rows of one KV head
  int32_t tok_begin;  // first query token (of the call)
  int32_t causal;     // 1: row of token i sees keys <= n - n_rows + i; 0: every row sees every key
  int32_t n_rows;     // query tokens
  int32_t units;      // ceil(rows / LU) of a head; all but the last have LU rows
  int32_t tiles;      // ceil(n / LN)
  int32_t unit_begin; // first (unit, head) among those of its kind (prefix or own)
  float* score;
  int64_t cap;        // row stride of score
  float* s;           // scored: q . k of every row and key, [Hkv][tiles * LN / 4][rows][4 keys], -inf where not seen
};

// K and V of each group: read by the attention kernel alone.
struct LiveMaps {
  CUtensorMap tm[VC_MAX_BATCH + 1][2];
};

struct LiveParams {
  // what is searched lies together: a scan over the groups' own fields took the constant cache 8 us to
  // bring in at 33 groups
  int32_t cost_begin[VC_MAX_BATCH + 2];   // first cost of each group in its kind's sequence [units][Hkv][tiles]
  int32_t chunk_begin[VC_MAX_BATCH + 2];  // scored: first score block of each group, [Hkv][ceil(n / 2^score_shift)]
  int32_t tok_begin[VC_MAX_BATCH + 1];    // first query token of each request
  int32_t own_of[VC_MAX_BATCH];           // group of the request's own cache, -1: empty
  LiveGroup grp[VC_MAX_BATCH + 1];        // the prefix first where there is one
  const bf16* q[VC_MAX_BATCH];
  bf16* o[VC_MAX_BATCH];
  int32_t B, Hq, Hkv, G, n_tok;
  int32_t n_grp, has_prefix;
  // by kind: its CTAs, the cost of each one's range and how many (the first) have one more
  int32_t n_cta[2], cta_cost[2], cta_more[2];
  int32_t keep_ws;                      // tiles read once leave L2 (evict first) to the workspace
  int32_t merge_blocks, merge_warps;    // blocks of the merge, warps a row (1, 2, 4 or 8; 0: several rows a warp)
  int32_t score_blocks, score_shift;    // blocks of 2^score_shift keys: 256, 512 or 1024
  int32_t slot_rows[2];                 // partial rows of a slot: prefix, own
  float* ws_o[2];                       // [slots][slot_rows][d]; slot = CTA of the kind + (unit, head)
  float* ws_lse[2];                     // [slots][slot_rows], log2 domain, -inf: saw nothing
  float scale_log2;
  int32_t* dev_status;
};

// The last i in [0, n) with begin[i] <= x.
__device__ __forceinline__ int last_begin(const int32_t* begin, int n, int x) {
  int lo = 0;
#pragma unroll
  for (int s = 32; s > 0; s >>= 1)
    if (lo + s < n && begin[lo + s] <= x) lo += s;
  return lo;
}

// CTA c of a kind has the costs from cta_begin(c) on; x lies in those of cta_of(x).
__device__ __forceinline__ int cta_begin(const LiveParams& p, int kind, int c) {
  return c * p.cta_cost[kind] + min(c, p.cta_more[kind]);
}
__device__ __forceinline__ int cta_of(const LiveParams& p, int kind, int x) {
  const int each = p.cta_cost[kind], more = p.cta_more[kind], e = more * (each + 1);
  return x < e ? x / (each + 1) : more + (x - e) / each;
}

// Steps of tile j of n keys: its second half only where it holds keys.
__device__ __forceinline__ int live_steps(int n, int j) { return n - j * LN > LS ? 2 : 1; }

// A CTA's part of a unit of a head: tiles [j0, j1). Every role of the CTA walks through the same pieces.
struct LPiece {
  int g, hk, u, j0, j1;  // group, KV head, unit of its rows, tiles
  int rows, tiles;       // the unit's query rows, the group's tiles
  int at, end;           // cost at which the head's tiles start, end of the CTA's range
  bool split;            // both chains hold the same rows, chain w takes half w of every tile

  __device__ __forceinline__ bool valid() const { return at < end; }
  __device__ __forceinline__ int cost() const { return split ? 1 : 2; }
  // chain w's steps of tile j of a group of n keys are its halves [h0, h1)
  __device__ __forceinline__ int h0(int w) const { return split ? w : 0; }
  __device__ __forceinline__ int h1(int w, int n, int j) const { return min(live_steps(n, j), split ? w + 1 : 2); }
  // it has none in the whole piece: chain 1 of a split unit's last, short tile
  __device__ __forceinline__ bool idle(int w, int n) const { return split && w == 1 && j1 - j0 == 1 && live_steps(n, j0) == 1; }
  __device__ __forceinline__ void fit(const LiveParams& p) {
    const LiveGroup& R = p.grp[g];
    rows = min(LU, R.rows - u * LU);
    tiles = R.tiles;
    split = rows <= LM;
  }
  __device__ __forceinline__ void cut() { j1 = min(tiles, (end - at + cost() - 1) / cost()); }
  __device__ __forceinline__ void next(const LiveParams& p) {
    at += cost() * tiles;
    if (!valid()) return;
    if (++hk == p.Hkv) {
      hk = 0;
      if (++u == p.grp[g].units) {
        u = 0;
        ++g;
      }
      fit(p);
    }
    j0 = 0;
    cut();
  }
};

template <int D>
struct LCfg {
  static constexpr int KB = D / 64;            // 64-channel (128-byte) blocks
  static constexpr int T_BYTES = KB * LN * 128;  // a K, V or Q tile
  static constexpr int NST = D == 128 ? 5 : 10;  // K and V tiles in flight or in use
  static constexpr int OFF_T = 2 * T_BYTES;    // behind a Q tile per chain
  static constexpr int OFF_BAR = OFF_T + NST * T_BYTES;
  static constexpr int SMEM = OFF_BAR + 448;
  static_assert(SMEM <= 227 * 1024, "one CTA's shared memory");
  static_assert((2 * NST + 20) * 8 + 32 + sizeof(LPiece) <= 448, "barriers fit");
  static constexpr int OCOL = 4 * LS;          // TMEM: S (and P) of chain w at (2 w + step % 2) LS, O at OCOL + w D
  static constexpr uint32_t TCOLS = 512;
  static_assert(OCOL + 2 * D <= (int)TCOLS, "TMEM");
};

__device__ __forceinline__ LPiece live_first(const LiveParams& p) {
  LPiece q;
  const int kind = (int)blockIdx.x < p.n_cta[0] ? 0 : 1, c = blockIdx.x - (kind ? p.n_cta[0] : 0);
  const int beg = cta_begin(p, kind, c);
  q.end = cta_begin(p, kind, c + 1);
  q.g = kind ? p.has_prefix + last_begin(p.cost_begin + p.has_prefix, p.n_grp - p.has_prefix, beg) : 0;
  const LiveGroup& R = p.grp[q.g];
  int rem = beg - p.cost_begin[q.g];
  const int unit = 2 * R.tiles * p.Hkv;  // of a unit of more than LM rows
  q.u = min(rem / unit, R.units - 1);
  rem -= q.u * unit;
  q.fit(p);
  q.hk = rem / (q.cost() * q.tiles);
  rem -= q.hk * q.cost() * q.tiles;
  q.at = beg - rem;
  q.j0 = (rem + q.cost() - 1) / q.cost();
  q.cut();
  if (q.j0 >= q.j1) q.next(p);  // the range starts in a head's last tile, which is the CTA's before
  return q;
}

__device__ __forceinline__ int live_req_of(const LiveParams& p, int tok) { return last_begin(p.tok_begin, p.B, tok); }

__device__ __forceinline__ void prefetch_tmap(const void* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// Bounded mbarrier wait that also gives up when another role of the CTA has aborted.
__device__ __forceinline__ bool lwait(uint64_t* bar, uint32_t parity, int32_t* st, volatile int* abort) {
  for (uint32_t it = 0; it < kSpinLimit; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 31u && *abort) return false;
  }
  set_status(st, VC_DEV_TIMEOUT);
  *abort = 1;
  return false;
}

// The same by a whole warp, which goes on or gives up together: its collective instructions need every lane.
__device__ __forceinline__ bool lwait_warp(uint64_t* bar, uint32_t parity, int32_t* st, volatile int* abort) {
  bool done = false;
  for (uint32_t it = 0; it < kSpinLimit && !done; ++it) {
    done = mbar_try_wait(bar, parity);
    if ((it & 31u) == 31u && *abort) break;
  }
  if (__all_sync(0xffffffffu, done)) return true;
  if (!*abort) set_status(st, VC_DEV_TIMEOUT);
  *abort = 1;
  return false;
}

// Arrives where `on`, without a branch.
__device__ __forceinline__ void mbar_arrive_if(uint64_t* bar, bool on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"((uint32_t)on)
      : "memory");
}

__device__ __forceinline__ bool nonfinite_bf16x2(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <int D, bool SCORED>
__global__ void __launch_bounds__(LTHREADS, 1) live_attn_kernel(const __grid_constant__ LiveParams p, const __grid_constant__ LiveMaps maps) {
  using C = LCfg<D>;
  constexpr int NST = C::NST;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem) & 1023u) {  // the swizzled layouts need 1024-byte aligned tiles
    pdl_wait();
    if (tid == 0) set_status(p.dev_status, VC_DEV_INTERNAL);
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [NST] tile landed
  uint64_t* empty = full + NST;   // [NST] both chains' MMAs are done with it
  uint64_t* sfull = empty + NST;  // [2][2] S of the chain's step in TMEM buffer step & 1
  uint64_t* pfull = sfull + 4;    // [2][2] the step's P in the same place (4 warps)
  uint64_t* ofull = pfull + 4;    // [2][2] its P V done: the buffer may take the S of two steps on
  uint64_t* qfull = ofull + 4;    // [2] the piece's Q tile in shared memory (4 warps)
  uint64_t* vbar = qfull + 2;     // [2] the chain's warps have looked through a V tile (4 warps)
  uint64_t* xbar = vbar + 2;      // [4] drain of an issuer's MMAs
  uint32_t* tslot = reinterpret_cast<uint32_t*>(xbar + 4);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tslot + 1);
  // [2][2] by S buffer, as the barriers are: 1 + the chain's last step in it whose P V the softmax warps took. A
  // warp may be a step ahead of the others, and so ahead of the P V issuer, which reads a step's word once all
  // four have left the step; the word's next step needs the issuer's commit behind that.
  volatile uint32_t* s_odd = tslot + 2;
  volatile uint32_t* s_issued = tslot + 6;  // loads issued so far
  LPiece* s_first = reinterpret_cast<LPiece*>(tslot + 8);  // the CTA's first piece

  if (warp == 12) tc05::alloc(tslot, C::TCOLS);
  if (tid == 13 * 32) *s_first = live_first(p);  // once: its code and parameters are cold in every cache
  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);
    }
    for (int w = 0; w < 2; ++w) {
      for (int i = 2 * w; i < 2 * w + 2; ++i) {
        mbar_init(&sfull[i], 1);
        mbar_init(&pfull[i], 4);
        mbar_init(&ofull[i], 1);
        s_odd[i] = 0;
      }
      mbar_init(&qfull[w], 4);
      mbar_init(&vbar[w], 4);
      mbar_init(&xbar[w], 1);
      mbar_init(&xbar[2 + w], 1);
    }
    fence_mbar_init();
    *s_abort = 0;
    *s_issued = 0;
  }
  tc05::fence_before();
  __syncthreads();
  tc05::fence_after();
  const uint32_t tmem = *tslot;
  const int kind = (int)blockIdx.x < p.n_cta[0] ? 0 : 1;
  pdl_wait();
  pdl_launch_dependents();

  // Load `it` has landed; `seen` is the caller's count of loads it knows to be issued. A role does not see
  // every phase of a stage's barrier (the S issuers wait for K tiles only, the P V issuers for V tiles), so the
  // parity alone could be that of two phases before: once the load is issued, the phase before it is over, and
  // its own cannot pass until this role releases the stage.
  // The chains' barriers are kept per S buffer: step s + 2 cannot complete a phase of one before step s's
  // has been waited for, while with one barrier for both, steps s and s + 1 could both pass unseen.
  auto landed = [&](uint32_t it, uint32_t& seen) -> bool {
    for (uint32_t i = 0; seen <= it; ++i) {
      seen = *s_issued;
      if (i >= kSpinLimit || ((i & 31u) == 31u && *s_abort)) {
        if (!*s_abort) set_status(p.dev_status, VC_DEV_TIMEOUT);
        *s_abort = 1;
        return false;
      }
    }
    return lwait(&full[it % NST], (it / NST) & 1, p.dev_status, s_abort);
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LREG_ISSUE));
    if (warp == 12) {
      // ---- TMA: tiles in order, K then V of each ---------------------------------------------------
      if (lane == 0) {
        LPiece q = *s_first;
        prefetch_tmap(&maps.tm[q.g][1]);
        const uint64_t pol = l2_evict_first_policy();
        uint32_t it = 0;
        bool ok = true;
        for (; q.valid() && ok; q.next(p)) {
          if (q.end - q.at > q.cost() * q.tiles && q.g + 1 < p.n_grp) {  // the range goes on: maybe to the next group
            prefetch_tmap(&maps.tm[q.g + 1][0]);
            prefetch_tmap(&maps.tm[q.g + 1][1]);
          }
          const bool once = p.keep_ws && p.grp[q.g].units == 1;  // tiles that one CTA reads once
          for (int j = q.j0; j < q.j1 && ok; ++j)
            for (int kv = 0; kv < 2; ++kv) {
              const uint32_t st = it % NST;
              if (it >= (uint32_t)NST && !lwait(&empty[st], (it / NST - 1) & 1, p.dev_status, s_abort)) {
                ok = false;
                break;
              }
              uint8_t* dst = smem + C::OFF_T + st * C::T_BYTES;
              mbar_arrive_expect_tx(&full[st], C::T_BYTES);
              if (once) {
#pragma unroll
                for (int kb = 0; kb < C::KB; ++kb)
                  tc05::tma_load_3d_hint(dst + kb * (LN * 128), &maps.tm[q.g][kv], kb * 64, j * LN, q.hk, &full[st], pol);
              } else {
#pragma unroll
                for (int kb = 0; kb < C::KB; ++kb)
                  tc05::tma_load_3d(dst + kb * (LN * 128), &maps.tm[q.g][kv], kb * 64, j * LN, q.hk, &full[st]);
              }
              __threadfence_block();
              *s_issued = ++it;
            }
        }
        if (*s_abort)  // drain (bounded): a ring's worth of loads may still be landing
          for (uint32_t i = it > (uint32_t)NST ? it - NST : 0; i < it; ++i)
            mbar_wait_bounded(&full[i % NST], (i / NST) & 1, p.dev_status);
      }
    } else if (warp == 10 || warp == 11) {
      // ---- P V issue of chain w: as soon as a step's P is there ---------------------------------------
      if (lane == 0) {
        const int w = warp - 10;
        constexpr uint32_t IDESC_O = tc05::idesc_bf16(LM, D, true);
        const uint32_t aT = smem_u32(smem + C::OFF_T), tS = tmem + 2 * w * LS, tO = tmem + C::OCOL + w * D;
        LPiece q = *s_first;
        uint32_t g = 0, t = 0, seen = 0;  // tiles of the CTA, steps of the chain
        bool ok = true;
        for (; q.valid() && ok; q.next(p)) {
          const int n = p.grp[q.g].n;
          bool acc = false;
          for (int j = q.j0; j < q.j1 && ok; ++j, ++g) {
            const uint32_t iv = 2 * g + 1, sv = iv % NST, vaddr = aT + sv * C::T_BYTES;
            ok = landed(iv, seen);
            const int h1 = q.h1(w, n, j);
            for (int h = q.h0(w); h < h1 && ok; ++h, ++t) {
              if (!lwait(&pfull[2 * w + (t & 1)], (t >> 1) & 1, p.dev_status, s_abort)) {
                ok = false;
                break;
              }
              tc05::fence_after();
              if (s_odd[2 * w + (t & 1)] != t + 1) {
                const uint32_t tP = tS + (t & 1) * LS, va = vaddr + h * (LS / 16) * 2048;
#pragma unroll
                for (int kk = 0; kk < LS / 16; ++kk)
                  tc05::mma_ts(tO, tP + kk * 8, tc05::sdesc_sw128(va + kk * 2048, LN * 128, 1024), IDESC_O,
                               (acc || kk > 0) ? 1u : 0u);
              }
              tc05::commit(&ofull[2 * w + (t & 1)]);
              acc = true;
            }
            if (ok) tc05::commit(&empty[sv]);
          }
        }
        // every MMA issued so far has completed before TMEM is released (bounded, even after an abort)
        tc05::commit(&xbar[2 + w]);
        mbar_wait_bounded(&xbar[2 + w], 0, p.dev_status);
      }
    } else if (warp < 10) {
      // ---- S issue of chain w: a step ahead of its softmax --------------------------------------------
      if (lane == 0) {
        const int w = warp - 8;
        constexpr uint32_t IDESC_S = tc05::idesc_bf16(LM, LS, false);
        const uint32_t aQ = smem_u32(smem) + w * C::T_BYTES, aT = smem_u32(smem + C::OFF_T);
        const uint32_t tS = tmem + 2 * w * LS;
        LPiece q = *s_first;
        uint32_t g = 0, t = 0, u = 0, seen = 0;  // tiles of the CTA, steps and pieces of the chain
        bool ok = true;
        for (; q.valid() && ok; q.next(p)) {
          const int n = p.grp[q.g].n;
          if (!q.idle(w, n)) {
            ok = lwait(&qfull[w], u & 1, p.dev_status, s_abort);
            ++u;
          }
          for (int j = q.j0; j < q.j1 && ok; ++j, ++g) {
            const uint32_t ik = 2 * g, sk = ik % NST, kaddr = aT + sk * C::T_BYTES;
            ok = landed(ik, seen);
            const int h1 = q.h1(w, n, j);
            for (int h = q.h0(w); h < h1 && ok; ++h, ++t) {
              // the P V that read its P from this S buffer is done
              if (t > 1 && !lwait(&ofull[2 * w + (t & 1)], ((t - 2) >> 1) & 1, p.dev_status, s_abort)) {
                ok = false;
                break;
              }
              tc05::fence_after();
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * (LN * 128) + (kk & 3) * 32;
                tc05::mma_bf16(tS + (t & 1) * LS, tc05::sdesc_sw128(aQ + off, 16, 1024),
                               tc05::sdesc_sw128(kaddr + h * LS * 128 + off, 16, 1024), IDESC_S, kk > 0);
              }
              tc05::commit(&sfull[2 * w + (t & 1)]);
            }
            if (ok) tc05::commit(&empty[sk]);
          }
        }
        tc05::commit(&xbar[w]);
        mbar_wait_bounded(&xbar[w], 0, p.dev_status);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(LREG_SOFTMAX));
    // ---- softmax of chain w: thread rt owns TMEM lane rt = row rt of the chain ----------------------
    const int w = warp >> 2, rt = tid & (LM - 1);
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + 2 * w * LS, tO = tmem + lane_off + C::OCOL + w * D;
    uint8_t* sQ = smem + w * C::T_BYTES;
    LPiece q = *s_first;
    uint32_t g = 0, t = 0, looked = 0, seen = 0;
    // P V of step s done (and with it those before): asked for steps whose S has been read, so the phase
    // before on that buffer is over
    auto pv_done = [&](uint32_t s) { return lwait_warp(&ofull[2 * w + (s & 1)], (s >> 1) & 1, p.dev_status, s_abort); };
    bool ok = true;
    auto slot_of = [&](const LiveGroup& R) {
      return (size_t)(blockIdx.x - (kind ? p.n_cta[0] : 0)) + R.unit_begin + q.u * p.Hkv + q.hk;
    };
    // Q of the next piece with steps for this chain, into its Q tile (the chain's S on the last one are all
    // done: their softmax is); pieces without any leave an empty partial
    auto fetch = [&]() {
      for (; q.valid(); g += q.j1 - q.j0, q.next(p)) {
        const LiveGroup& R = p.grp[q.g];
        const int ru = q.split ? rt : w * LM + rt, row = q.u * LU + ru;  // row of the unit, of the head
        const bool row_ok = ru < q.rows;
        if (q.idle(w, R.n)) {
          const size_t slot = slot_of(R);
          if (row_ok) p.ws_lse[kind][slot * p.slot_rows[kind] + w * q.rows + ru] = -INFINITY;
          continue;
        }
        const bf16* src = nullptr;  // this thread's row
        if (row_ok) {
          const int tok = R.tok_begin + row / p.G, b = live_req_of(p, tok);
          src = p.q[b] + ((size_t)(tok - p.tok_begin[b]) * p.Hq + q.hk * p.G + row % p.G) * D;
        }
        // the warp's 32 rows, a row's 16-byte pieces in neighbouring lanes (a lane per row would touch 32 lines a load)
        constexpr int PR = D / 8, RW = 32 / PR;  // pieces of a row, rows a load
#pragma unroll
        for (int i = 0; i < 32 / RW; ++i) {
          const int r = i * RW + lane / PR, c = lane % PR, rr = (warp & 3) * 32 + r;
          const bf16* from = reinterpret_cast<const bf16*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), r));
          const uint4 v = from ? __ldcg(reinterpret_cast<const uint4*>(from) + c) : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(sQ + (c >> 3) * (LM * 128) + rr * 128 + (((c ^ rr) & 7) << 4)) = v;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&qfull[w]);
        return;
      }
    };
    // the chain's partial of the piece before: written once the next one's S are under way
    size_t part = 0;
    float m_run = 0.f, l_run = 0.f;
    bool row_ok = false, have = false;
    while (ok) {
      fetch();
      if (have) {
        // after its last P V
        if (!pv_done(t - 1)) break;
        tc05::fence_after();
        const float inv = l_run != 0.f ? 1.f / l_run : 0.f;
        // rows in the order of an MMA's accumulator: four lanes hold 8 neighbouring channels (whole 32-byte
        // sectors), where a lane per row would write 32 lines at a time
        float* o_row0 = p.ws_o[kind] + (part - (rt & 31)) * D + 2 * (lane & 3);  // of the warp's first row
        const unsigned rows_ok = __ballot_sync(0xffffffffu, row_ok);
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh) {
          if (!((rows_ok >> (16 * hh)) & 0xffffu)) continue;
          const int r0 = hh * 16 + (lane >> 2), r1 = r0 + 8;
          const float i0 = __shfl_sync(0xffffffffu, inv, r0), i1 = __shfl_sync(0xffffffffu, inv, r1);
          const bool ok0 = (rows_ok >> r0) & 1u, ok1 = (rows_ok >> r1) & 1u;
#pragma unroll 1
          for (int cb = 0; cb < D / 32; ++cb) {
            uint32_t r[16];
            tc05::ld16x256_x4(tO + ((uint32_t)(hh * 16) << 16) + cb * 32, r);  // warp-collective: every lane loads
            tc05::wait_ld();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (ok0)
                *reinterpret_cast<float2*>(o_row0 + (size_t)r0 * D + cb * 32 + 8 * k) =
                    make_float2(__uint_as_float(r[4 * k]) * i0, __uint_as_float(r[4 * k + 1]) * i0);
              if (ok1)
                *reinterpret_cast<float2*>(o_row0 + (size_t)r1 * D + cb * 32 + 8 * k) =
                    make_float2(__uint_as_float(r[4 * k + 2]) * i1, __uint_as_float(r[4 * k + 3]) * i1);
            }
          }
        }
        if (row_ok) p.ws_lse[kind][part] = l_run != 0.f ? m_run + log2f(l_run) : -INFINITY;
        tc05::fence_before();
      }
      if (!q.valid()) break;
      have = true;
      const LiveGroup& R = p.grp[q.g];
      const int ru = q.split ? rt : w * LM + rt;
      row_ok = ru < q.rows;
      const int row = q.u * LU + ru, tl = row / p.G;
      part = slot_of(R) * p.slot_rows[kind] + (q.split ? w * q.rows : 0) + ru;
      // last key the row sees, and the first one that some row of the chain does not
      const int n = R.n;
      const int last_key = R.causal ? n - R.n_rows + tl : n - 1;
      const int blind = R.causal ? n - R.n_rows + (q.u * LU + (q.split ? 0 : w * LM)) / p.G + 1 : n;
      const int s_rows = R.rows;
      float4* s_row = SCORED ? reinterpret_cast<float4*>(R.s) + (size_t)q.hk * R.tiles * (LN / 4) * s_rows + row : nullptr;
      m_run = -INFINITY, l_run = 0.f;
      bool fresh = true;  // the piece's first step
      for (int j = q.j0; j < q.j1 && ok; ++j, ++g) {
        const int h1 = q.h1(w, n, j);
        for (int h = q.h0(w); h < h1; ++h, ++t, fresh = false) {
          const int k0 = j * LN + h * LS;  // the step's first key
          const uint32_t tP = tS + (t & 1) * LS;
          if (!lwait_warp(&sfull[2 * w + (t & 1)], (t >> 1) & 1, p.dev_status, s_abort)) {
            ok = false;
            break;
          }
          tc05::fence_after();
          float x[LS];
#pragma unroll
          for (int cb = 0; cb < LS / 32; ++cb) {
            uint32_t r[32];
            tc05::ld32(tP + cb * 32, r);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[cb * 32 + e] = __uint_as_float(r[e]);
          }
          tc05::wait_ld();
          const int last = last_key - k0;
          if (last < LS - 1) {
            // as bits, several of which become predicates at a time: half the instructions of 64 comparisons
            const uint32_t lo = last >= 31 ? 0xffffffffu : last < 0 ? 0u : (2u << last) - 1u;  // keys that are seen
            const uint32_t hi = last < 32 ? 0u : (2u << (last - 32)) - 1u;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (!((lo >> e) & 1u)) x[e] = -INFINITY;
              if (!((hi >> e) & 1u)) x[32 + e] = -INFINITY;
            }
          }
          if constexpr (SCORED) {
            if (row_ok) {  // four keys of neighbouring rows in neighbouring lanes: whole lines
              float4* d = s_row + (size_t)(k0 / 4) * s_rows;
#pragma unroll
              for (int e = 0; e < LS / 4; ++e, d += s_rows) *d = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            }
          }
          // P = 2^(x scale - m), bf16, over S: the MMA wants both operands in one 16-bit type, and V is bf16 (its range
          // is not fp16's). A weight is off by 2^-8 of itself at most; with the output's own rounding the outputs are
          // 0.0020 to 0.0023 from 64 bits (relative L2), where fp32 weights leave 0.0017. A second product with what
          // P lacks would double P V's share of the tensor cores and of shared memory. Sums and lse take the weights
          // unrounded.
          // The running maximum is taken as it is: the row's new one is found alongside, and only when it is larger by
          // more than 2^8 (or this is the piece's first step) is m moved, O rescaled after the P V before, and P
          // computed again. TMEM loads and stores are warp-collective: the warp does it together.
          uint32_t r[LS / 2];
          float u0, u1, mx = -INFINITY, my = -INFINITY, mz = -INFINITY, mw = -INFINITY;
#pragma unroll 1
          for (int again = 0; again < 2; ++again) {
            const float mu = m_run == -INFINITY ? 0.f : m_run;
            const uint64_t sc = f2_pack(p.scale_log2, p.scale_log2), nm = f2_pack(-mu, -mu);
            uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int e = 0; e < LS / 2; ++e) {
              float a0, a1;
              f2_unpack(f2_fma(f2_pack(x[2 * e], x[2 * e + 1]), sc, nm), a0, a1);
              const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
              acc[e & 3] = f2_add(acc[e & 3], f2_pack(p0, p1));
              r[e] = pack_bf16x2(p0, p1);
              float& m = (e & 3) == 0 ? mx : (e & 3) == 1 ? my : (e & 3) == 2 ? mz : mw;
              m = max3f(m, x[2 * e], x[2 * e + 1]);
            }
            f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), u0, u1);
            if (again) break;
            const float m_new = fmaxf(m_run, fmaxf(fmaxf(mx, my), fmaxf(mz, mw)) * p.scale_log2);
            const bool need = m_new > m_run + 8.f;  // from -infinity, any finite score
            if (!__any_sync(0xffffffffu, need)) break;
            if (fresh) {
              m_run = m_new;
              continue;
            }
            if (!pv_done(t - 1)) {
              ok = false;
              break;
            }
            tc05::fence_after();
            float f = 1.f;
            if (need) {
              f = ex2_approx(m_run - m_new);
              l_run *= f;
              m_run = m_new;
            }
#pragma unroll 1
            for (int cb = 0; cb < D / 32; ++cb) {
              uint32_t o[32];
              tc05::ld32(tO + cb * 32, o);
              tc05::wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tc05::st32(tO + cb * 32, o);
            }
          }
          if (!ok) break;
          tc05::st32(tP, r);
          l_run += u0 + u1;
          tc05::wait_st();
          // A step with keys that some rows see and others do not: a weight of 0 would carry an infinite or
          // NaN value row to the latter, so if V holds any, the threads add up the seen keys themselves.
          if (blind < min(n, k0 + LS)) {
            const uint32_t iv = 2 * g + 1;
            if (!__all_sync(0xffffffffu, landed(iv, seen))) {
              ok = false;
              break;
            }
            const uint8_t* sV = smem + C::OFF_T + (iv % NST) * C::T_BYTES;
            bool bad = false;
            const int kv = h * LS + (rt & (LS - 1));  // two threads look through each of the step's rows
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const int c = (rt / LS) * (D / 16) + i;
              const uint4 v = *reinterpret_cast<const uint4*>(sV + (c >> 3) * (LN * 128) + kv * 128 + (((c ^ kv) & 7) << 4));
              bad |= nonfinite_bf16x2(v.x) || nonfinite_bf16x2(v.y) || nonfinite_bf16x2(v.z) || nonfinite_bf16x2(v.w);
            }
            if (bad) s_odd[2 * w + (t & 1)] = t + 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&vbar[w]);
            if (!lwait_warp(&vbar[w], looked & 1, p.dev_status, s_abort)) {
              ok = false;
              break;
            }
            ++looked;
            if (s_odd[2 * w + (t & 1)] == t + 1) {
              if (!fresh && !pv_done(t - 1)) {
                ok = false;
                break;
              }
              tc05::fence_after();
#pragma unroll 1
              for (int cb = 0; cb < D / 32; ++cb) {
                uint32_t r[32];
                if (!fresh) {
                  tc05::ld32(tO + cb * 32, r);
                  tc05::wait_ld();
                } else {
#pragma unroll
                  for (int e = 0; e < 32; ++e) r[e] = 0u;
                }
#pragma unroll 1
                for (int kp = 0; kp < LS / 2; ++kp) {  // two keys a column; rare, so kept small
                  const uint32_t pw = tc05::ld1(tP + kp);
                  tc05::wait_ld();
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const int k = 2 * kp + e, kt = h * LS + k;
                    const float pk = __uint_as_float(e ? pw & 0xffff0000u : pw << 16);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                      const int ch = cb * 4 + c;
                      const uint4 v = *reinterpret_cast<const uint4*>(sV + (ch >> 3) * (LN * 128) + kt * 128 + (((ch ^ kt) & 7) << 4));
                      const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                      for (int i = 0; i < 8; ++i) {
                        const float val = __uint_as_float(i & 1 ? vw[i >> 1] & 0xffff0000u : vw[i >> 1] << 16);
                        const float a = __uint_as_float(r[c * 8 + i]);
                        r[c * 8 + i] = __float_as_uint(k <= last ? fmaf(pk, val, a) : a);
                      }
                    }
                  }
                }
                tc05::st32(tO + cb * 32, r);
              }
              tc05::wait_st();
            }
          }
          tc05::fence_before();
          __syncwarp();
          mbar_arrive_if(&pfull[2 * w + (t & 1)], lane == 0);
        }
      }
      if (!ok) break;
      q.next(p);
    }
  }

  tc05::fence_before();
  __syncthreads();
  tc05::fence_after();
  if (warp == 12) tc05::dealloc(tmem, C::TCOLS);
}

// Where a row of a group (KV head hk, row r of the head) left its partials: `count` of them, number i at
// index at(i) of the kind's partial rows. A split unit has two a slot.
struct LParts {
  size_t base;
  int count, stride, second;  // stride: a slot's rows; second: rows to the slot's second partial, 0: none
  __device__ __forceinline__ size_t at(int i) const {
    return second ? base + (size_t)(i >> 1) * stride + (i & 1) * second : base + (size_t)i * stride;
  }
};

__device__ __forceinline__ LParts live_parts(const LiveParams& p, int kind, int g, int hk, int r) {
  LParts q;
  const LiveGroup& R = p.grp[g];
  const int u = r / LU, rows = min(LU, R.rows - u * LU), cost = rows <= LM ? 1 : 2;
  const int at = p.cost_begin[g] + (u * 2 * p.Hkv + hk * cost) * R.tiles;
  const int c0 = cta_of(p, kind, at), c1 = cta_of(p, kind, at + cost * (R.tiles - 1));  // of its first and last tile
  q.second = rows <= LM ? rows : 0;
  q.count = (c1 - c0 + 1) * (q.second ? 2 : 1);
  q.stride = p.slot_rows[kind];
  q.base = (size_t)(c0 + R.unit_begin + u * p.Hkv + hk) * q.stride + (r - u * LU);
  return q;
}

// Weight of a partial beside the largest lse M: 0 where it saw nothing; M stays -inf only beside a NaN.
__device__ __forceinline__ float merge_weight(float l, float M) { return l == -INFINITY ? 0.f : M == -INFINITY ? NAN : exp2f(l - M); }

// Merge: one to eight warps per (token, query head), o = sum_k 2^(lse_k - M) o_k / sum_k 2^(lse_k - M) over the
// partials of the prefix and of the own cache: a lane per partial takes the weights, then the warp adds
// up the partials' channels, four loads in flight. Scores: a block per 256 to 1024 keys of a (request, KV head)
// merges the head's rows' lse, four rows a warp at a time, then sums 2^(s scale - lse) over the rows for each key.
template <int D, bool SCORED>
__global__ void __launch_bounds__(256, SCORED ? 3 : 4) live_finish_kernel(const __grid_constant__ LiveParams p) {
  constexpr int E = D / 32;  // channels a lane
  constexpr int PF = 4;      // partials in flight
  constexpr int SP = SCORE_KEYS / 256;
  __shared__ float s_lse[VC_SCORED_MAX_ROWS];
  __shared__ float s_acc[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto warp_max = [](float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
  };
  auto warp_sum = [](float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  };
  if (!SCORED || (int)blockIdx.x >= p.score_blocks) {  // the longer score blocks go first
    const int wpr = p.merge_warps, part = warp % wpr;  // warps of a row, this one among them
    const int64_t id = (int64_t)(blockIdx.x - p.score_blocks) * (8 / wpr) + warp / wpr;
    const bool live = id < (int64_t)p.n_tok * p.Hq;
    LParts a{0, 0, 0, 0}, o{0, 0, 0, 0};  // of the prefix, of the own cache
    bf16* dst = nullptr;
    if (live) {
      const int tok = (int)(id / p.Hq), hq = (int)(id - (int64_t)tok * p.Hq), hk = hq / p.G, gq = hq - hk * p.G;
      const int b = live_req_of(p, tok), i = tok - p.tok_begin[b], own = p.own_of[b];
      if (p.has_prefix) a = live_parts(p, 0, 0, hk, tok * p.G + gq);
      if (own >= 0) o = live_parts(p, 1, own, hk, i * p.G + gq);
      dst = p.o[b] + ((size_t)i * p.Hq + hq) * D + lane * E;
    }
    pdl_wait();  // what needs the parameters alone is done
    pdl_launch_dependents();
    const int total = a.count + o.count;
    auto lse_of = [&](int k, int end) {
      return k >= end ? -INFINITY : k < a.count ? p.ws_lse[0][a.at(k)] : p.ws_lse[1][o.at(k - a.count)];
    };
    float M = -INFINITY;
    for (int k0 = 0; k0 < total; k0 += 32) M = fmaxf(M, lse_of(k0 + lane, total));
    M = warp_max(M);
    float L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    const int beg = total * part / wpr, end = total * (part + 1) / wpr;
    for (int k0 = beg; k0 < end; k0 += 32) {
      const float l = lse_of(k0 + lane, end), f = merge_weight(l, M);
      const unsigned wrote = __ballot_sync(0xffffffffu, l != -INFINITY);
      L += f;
      const int cnt = min(32, end - k0);
      for (int c0 = 0; c0 < cnt; c0 += PF) {
        float v[PF][E], fc[PF];
#pragma unroll
        for (int c = 0; c < PF; ++c) {
          fc[c] = __shfl_sync(0xffffffffu, f, c0 + c);  // c0 + c < 32; nothing was written beyond cnt
#pragma unroll
          for (int e = 0; e < E; ++e) v[c][e] = 0.f;
          if ((wrote >> (c0 + c)) & 1u) {  // a partial that saw nothing was not written
            const int k = k0 + c0 + c;
            const float* src = (k < a.count ? p.ws_o[0] + a.at(k) * D : p.ws_o[1] + o.at(k - a.count) * D) + lane * E;
            if constexpr (E == 4)
              *reinterpret_cast<float4*>(v[c]) = __ldcg(reinterpret_cast<const float4*>(src));
            else
              *reinterpret_cast<float2*>(v[c]) = __ldcg(reinterpret_cast<const float2*>(src));
          }
        }
#pragma unroll
        for (int c = 0; c < PF; ++c)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(fc[c], v[c][e], acc[e]);
      }
    }
    L = warp_sum(L);
    if (wpr > 1) {  // the row's warps meet
#pragma unroll
      for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
      if (lane == 0) s_lse[warp] = L;
      __syncthreads();
      if (part != 0) return;
      for (int u = 1; u < wpr; ++u) {
        L += s_lse[warp + u];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += s_acc[warp + u][lane * E + e];
      }
    }
    if (!live) return;
    const float inv = L != 0.f ? 1.f / L : 0.f;
    uint32_t out[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) out[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = out[0];
    return;
  }
  if constexpr (SCORED) {
    const int id = blockIdx.x;
    const int g = last_begin(p.chunk_begin, p.n_grp, id);
    const LiveGroup& R = p.grp[g];
    const int chunks = (R.n + (1 << p.score_shift) - 1) >> p.score_shift;
    const int hk = (id - p.chunk_begin[g]) / chunks, k0 = (id - p.chunk_begin[g] - hk * chunks) << p.score_shift;
    const int rows = R.rows, gl = threadIdx.x & 3;  // four lanes share a group of four keys, rows gl, gl + 4, ...
    const float4* s = reinterpret_cast<const float4*>(R.s) + ((size_t)hk * R.tiles * (LN / 4) + k0 / 4 + threadIdx.x / 4) * rows;
    float* score = R.score + (size_t)hk * R.cap + k0 + threadIdx.x;  // its key in a pass of 256
    const int keys = min(R.n - k0, 1 << p.score_shift);  // of this block
    const int left = keys - (int)threadIdx.x, quads = (keys + 3) / 4 - (int)threadIdx.x / 4;
    LParts part{0, 0, 0, 0};  // of row 0; row r's are r further on
    if (warp < rows) part = live_parts(p, 1, g, hk, 0);
    pdl_wait();
    pdl_launch_dependents();
    float4 v[SP][2];
    auto load2 = [&](int r0) {
#pragma unroll
      for (int c = 0; c < SP; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (r0 + 4 * e < rows && 64 * c < quads) v[c][e] = __ldcg(s + (size_t)(64 * c) * rows + r0 + 4 * e);
    };
    load2(gl);  // in flight while the rows' lse are merged
    float w[SP];
#pragma unroll
    for (int c = 0; c < SP; ++c) w[c] = 256 * c < left ? score[256 * c] : 0.f;
    constexpr int LR = 4;  // rows a warp merges at a time
    for (int r0 = warp; r0 < rows; r0 += 8 * LR) {
      float M[LR], L[LR];
#pragma unroll
      for (int e = 0; e < LR; ++e) M[e] = -INFINITY, L[e] = 0.f;
      for (int k = lane; k < part.count; k += 32) {
        const float* l = p.ws_lse[1] + part.at(k) + r0;
#pragma unroll
        for (int e = 0; e < LR; ++e)
          if (r0 + 8 * e < rows) M[e] = fmaxf(M[e], l[8 * e]);
      }
#pragma unroll
      for (int e = 0; e < LR; ++e)
        if (r0 + 8 * e < rows) M[e] = warp_max(M[e]);
      for (int k = lane; k < part.count; k += 32) {
        const float* l = p.ws_lse[1] + part.at(k) + r0;
#pragma unroll
        for (int e = 0; e < LR; ++e)
          if (r0 + 8 * e < rows) L[e] += merge_weight(l[8 * e], M[e]);
      }
#pragma unroll
      for (int e = 0; e < LR; ++e)
        if (r0 + 8 * e < rows) {
          const float l = warp_sum(L[e]);
          if (lane == 0) s_lse[r0 + 8 * e] = l != 0.f ? M[e] + log2f(l) : INFINITY;  // a row that sees nothing has weights 2^-inf
        }
    }
    __syncthreads();
    float4 sum[SP];
#pragma unroll
    for (int c = 0; c < SP; ++c) sum[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int r0 = gl; r0 < rows; r0 += 8) {
      if (r0 != gl) load2(r0);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (r0 + 4 * e < rows) {
          const float lse = s_lse[r0 + 4 * e];
          if (lse != lse) {  // the row's weights are NaN: those of the keys it sees, not of the ones behind them
            const int seen = R.n - R.n_rows + (r0 + 4 * e) / p.G - (k0 + (threadIdx.x & ~3));  // last one, from the group's first
#pragma unroll
            for (int c = 0; c < SP; ++c) {
              if (256 * c <= seen) sum[c].x = lse;
              if (256 * c + 1 <= seen) sum[c].y = lse;
              if (256 * c + 2 <= seen) sum[c].z = lse;
              if (256 * c + 3 <= seen) sum[c].w = lse;
            }
            continue;
          }
#pragma unroll
          for (int c = 0; c < SP; ++c) {
            sum[c].x += ex2_approx(fmaf(v[c][e].x, p.scale_log2, -lse));
            sum[c].y += ex2_approx(fmaf(v[c][e].y, p.scale_log2, -lse));
            sum[c].z += ex2_approx(fmaf(v[c][e].z, p.scale_log2, -lse));
            sum[c].w += ex2_approx(fmaf(v[c][e].w, p.scale_log2, -lse));
          }
        }
    }
#pragma unroll
    for (int c = 0; c < SP; ++c) {
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        sum[c].x += __shfl_xor_sync(0xffffffffu, sum[c].x, off);
        sum[c].y += __shfl_xor_sync(0xffffffffu, sum[c].y, off);
        sum[c].z += __shfl_xor_sync(0xffffffffu, sum[c].z, off);
        sum[c].w += __shfl_xor_sync(0xffffffffu, sum[c].w, off);
      }
      const float mine = gl == 0 ? sum[c].x : gl == 1 ? sum[c].y : gl == 2 ? sum[c].z : sum[c].w;
      if (256 * c < left) score[256 * c] = w[c] + mine;
    }
  }
}

// The merge for many rows of few partials: LIVE_SUB lanes a row, four rows a warp side by side. A row's time is
// that of its dependent loads, whatever its partials (62496 rows of 2 to 4: the call 107 us with a warp a row, 71
// so; 16384 over 8192 + 500 keys: 132, 123; 16000 of about 6: 405, 394).
constexpr int LIVE_SUB = 8;
template <int D>
__global__ void __launch_bounds__(256, 4) live_merge_kernel(const __grid_constant__ LiveParams p) {
  constexpr int Q = D / 4 / LIVE_SUB;  // float4 a lane: number sl, sl + LIVE_SUB, ... of the row
  const int lane = threadIdx.x & 31, sl = lane % LIVE_SUB, first = lane - sl;
  const int64_t id = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LIVE_SUB;
  const bool live = id < (int64_t)p.n_tok * p.Hq;
  LParts a{0, 0, 0, 0}, o{0, 0, 0, 0};  // of the prefix, of the own cache
  bf16* dst = nullptr;
  if (live) {
    const int tok = (int)(id / p.Hq), hq = (int)(id - (int64_t)tok * p.Hq), hk = hq / p.G, gq = hq - hk * p.G;
    const int b = live_req_of(p, tok), i = tok - p.tok_begin[b], own = p.own_of[b];
    if (p.has_prefix) a = live_parts(p, 0, 0, hk, tok * p.G + gq);
    if (own >= 0) o = live_parts(p, 1, own, hk, i * p.G + gq);
    dst = p.o[b] + ((size_t)i * p.Hq + hq) * D;
  }
  pdl_wait();
  pdl_launch_dependents();
  const int total = a.count + o.count, most = __reduce_max_sync(0xffffffffu, total);
  auto lse_of = [&](int k) {
    return k >= total ? -INFINITY : k < a.count ? p.ws_lse[0][a.at(k)] : p.ws_lse[1][o.at(k - a.count)];
  };
  const float l0 = lse_of(sl);  // most rows have no more than a lane each
  float M = l0;
  for (int k0 = LIVE_SUB; k0 < most; k0 += LIVE_SUB) M = fmaxf(M, lse_of(k0 + sl));
#pragma unroll
  for (int off = LIVE_SUB / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float L = 0.f;
  float4 acc[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < most; k0 += LIVE_SUB) {
    const float l = k0 ? lse_of(k0 + sl) : l0, f = merge_weight(l, M);
    const unsigned wrote = __ballot_sync(0xffffffffu, l != -INFINITY) >> first;
    L += f;
    const int cnt = min(LIVE_SUB, most - k0);
#pragma unroll 2
    for (int c = 0; c < cnt; ++c) {
      const float fc = __shfl_sync(0xffffffffu, f, first + c);
      if ((wrote >> c) & 1u) {  // a partial that saw nothing was not written
        const int k = k0 + c;
        const float4* src = reinterpret_cast<const float4*>(k < a.count ? p.ws_o[0] + a.at(k) * D : p.ws_o[1] + o.at(k - a.count) * D) + sl;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const float4 v = __ldcg(src + q * LIVE_SUB);
          acc[q].x = fmaf(fc, v.x, acc[q].x);
          acc[q].y = fmaf(fc, v.y, acc[q].y);
          acc[q].z = fmaf(fc, v.z, acc[q].z);
          acc[q].w = fmaf(fc, v.w, acc[q].w);
        }
      }
    }
  }
#pragma unroll
  for (int off = LIVE_SUB / 2; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  if (!live) return;
  const float inv = L != 0.f ? 1.f / L : 0.f;
#pragma unroll
  for (int q = 0; q < Q; ++q)
    reinterpret_cast<uint2*>(dst)[sl + q * LIVE_SUB] =
        make_uint2(pack_bf16x2(acc[q].x * inv, acc[q].y * inv), pack_bf16x2(acc[q].z * inv, acc[q].w * inv));
}

// ------------------------------------------------------------------------------------------------
// bf16 [Hkv][cap][d] rows 0..rows-1 as a 3-D tensor (d, rows, Hkv); box 64 x 128 x 1, 128-byte swizzle.
// Rows beyond the last one read as zeros.
static bool live_map(CUtensorMap* m, const void* base, int d, int rows, int64_t cap, int Hkv) {
  auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tmap_encoder());
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)Hkv};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)cap * d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)LN, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int live_sms() {
  static const int n = [] {
    int dev = 0, v = 0;
    const bool ok = cudaGetDevice(&dev) == cudaSuccess &&
                    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
    return ok ? v : 152;
  }();
  return n;
}

static int64_t units_of(int64_t rows) { return (rows + LU - 1) / LU; }
static int slot_rows_of(int64_t rows) { return rows <= LM ? (int)(2 * rows) : LU; }
// CTAs for the prefix's and the own caches' costs: at most one per SM, none with a range below `least`, the
// cost of the kind's dearest tile (so that none holds less than a tile). With several units of prefix rows
// their number is a multiple of the units' (a last unit of up to LM rows counting half), where that leaves the
// longest range within a tenth of the shortest possible (2000 rows over 65536 keys: ranges cut at the same
// tiles read 526 MB from DRAM, others 2100 MB; 427 and 593 us when that was measured).
// They are shared by `weighed`, in which a unit of a head costs at least kLeastUnit: a piece of one tile takes as
// long as four of a longer one (224 rows over 54472 keys beside 28 own caches of up to 112: 58 us by the tiles
// alone, 44 with 4, 45.5 with 8; with 8 a batch of 4 over 3389 and up to 788 keys goes from 16.4 to 18.3).
constexpr int kLeastUnit = 4;
static void share_ctas(const int64_t (&cost)[2], const int64_t (&weighed)[2], const int (&least)[2], int prefix_rows,
                       int32_t (&n)[2]) {
  int most[2];
  for (int k = 0; k < 2; ++k) {
    const int64_t m = cost[k] / least[k];
    most[k] = cost[k] == 0 ? 0 : m < 1 ? 1 : m < live_sms() ? (int)m : live_sms();
  }
  n[0] = most[0];
  n[1] = most[1];
  const int units = (int)units_of(prefix_rows), half = prefix_rows - (units - 1) * LU <= LM;
  const int step = units < 2 ? 1 : 2 * units - half;  // in half units; twice as many CTAs without a half one
  if (most[0] == 0 || (most[0] + most[1] <= live_sms() && step == 1)) return;
  const int room = live_sms();
  // the shortest longest range; among equals the shortest ranges together
  struct Best {
    int64_t longest = INT64_MAX, sum = INT64_MAX;
    int at = 0;
    void take(int64_t l, int64_t s, int c) {
      if (l < longest || (l == longest && s < sum)) longest = l, sum = s, at = c;
    }
  } any, aligned;
  for (int c = 1; c <= most[0] && (most[1] == 0 || c < room); ++c) {
    const int o = most[1] < room - c ? most[1] : room - c;
    const int64_t p0 = (weighed[0] + c - 1) / c, p1 = o > 0 ? (weighed[1] + o - 1) / o : 0, longest = p0 > p1 ? p0 : p1;
    any.take(longest, p0 + p1, c);
    if ((half ? c : 2 * c) % step == 0) aligned.take(longest, p0 + p1, c);
  }
  const int at = aligned.at && aligned.longest * 10 <= any.longest * 11 ? aligned.at : any.at;
  n[0] = at;
  n[1] = most[1] < room - at ? most[1] : room - at;
}

static size_t pad256(size_t b) { return (b + 255) / 256 * 256; }

// Partials: slots of both kinds (a slot per CTA and unit); scores: every row's, in fp32.
size_t live_workspace_size(const vc_shape* s, int32_t max_rows, int32_t max_n, bool scored) {
  const int64_t G = s->Hq / s->Hkv, rows = max_rows * G, ctas = live_sms();
  const size_t per = (s->d + 1) * sizeof(float);
  size_t b = pad256((size_t)(ctas + s->B * s->Hkv * units_of(rows)) * slot_rows_of(rows) * per);
  if (scored)
    b += pad256((size_t)s->B * s->Hkv * rows * ((max_n + (int64_t)LN - 1) / LN * LN) * sizeof(float));
  else
    b += pad256((size_t)(ctas + s->Hkv * units_of(s->B * rows)) * slot_rows_of(s->B * rows) * per);
  return b + 256;
}

template <int D, bool SCORED>
static cudaError_t launch_live_t(const LiveParams& p, const LiveMaps& maps, cudaStream_t s) {
  static std::atomic<uint64_t> attr{0};
  if (p.n_cta[0] + p.n_cta[1] > 0) {
    cudaError_t e = raise_smem_limit(live_attn_kernel<D, SCORED>, LCfg<D>::SMEM, attr);
    if (e != cudaSuccess) return e;
    e = launch_pdl(live_attn_kernel<D, SCORED>, dim3(p.n_cta[0] + p.n_cta[1]), dim3(LTHREADS), LCfg<D>::SMEM, s, p, maps);
    if (e != cudaSuccess) return e;
  }
  if (p.merge_warps == 0) return launch_pdl(live_merge_kernel<D>, dim3(p.merge_blocks), dim3(256), 0, s, p);
  return launch_pdl(live_finish_kernel<D, SCORED>, dim3(p.merge_blocks + p.score_blocks), dim3(256), 0, s, p);
}

cudaError_t launch_live_attn(const LiveArgs& a, bool scored, cudaStream_t s, vc_status* st) {
  const int G = a.Hq / a.Hkv;
  LiveParams p;   // about 4 KB
  LiveMaps maps;  // about 8 KB: the tensor maps travel as kernel parameters
  memset(&p, 0, sizeof(p));
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = G;
  p.n_tok = a.n_tok;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)a.d));
  p.dev_status = a.dev_status;
  p.slot_rows[0] = p.slot_rows[1] = 1;
  int64_t cost[2] = {0, 0}, weighed[2] = {0, 0}, units[2] = {0, 0}, chunks = 0;
  int least[2] = {1, 1};
  size_t s_floats = 0;
  // adds the group of a key sequence; `b`: the request whose own cache it is, -1: the prefix
  auto add = [&](int b, int n, int n_rows, int tok_begin) {
    const int kind = b < 0 ? 0 : 1;
    LiveGroup& R = p.grp[p.n_grp];
    R.n = n;
    R.rows = n_rows * G;
    R.tok_begin = tok_begin;
    R.causal = kind;
    R.n_rows = n_rows;
    R.units = (int32_t)units_of(R.rows);
    R.tiles = (n + LN - 1) / LN;
    R.unit_begin = (int32_t)units[kind];
    p.cost_begin[p.n_grp] = (int32_t)cost[kind];
    if (R.rows > LM) least[kind] = 2;
    const int sr = slot_rows_of(R.rows);
    p.slot_rows[kind] = sr > p.slot_rows[kind] ? sr : p.slot_rows[kind];
    units[kind] += (int64_t)a.Hkv * R.units;
    // every unit but the last has LU rows
    const int64_t all = (int64_t)a.Hkv * R.tiles * (2 * R.units - (R.rows - (R.units - 1) * LU <= LM ? 1 : 0));
    const int64_t few = (int64_t)a.Hkv * R.units * kLeastUnit;
    cost[kind] += all;
    weighed[kind] += all > few ? all : few;
    if (scored) {
      chunks += (int64_t)a.Hkv * ((n + SCORE_KEYS - 1) / SCORE_KEYS);
      s_floats += (size_t)a.Hkv * R.rows * R.tiles * LN;
    }
    ++p.n_grp;
    // costs (and twice a unit's) and blocks are counted in 32 bits
    if (cost[kind] >= INT32_MAX / 2 || chunks >= INT32_MAX / 2 || units[kind] >= INT32_MAX / 2) *st = VC_ERR_UNSUPPORTED;
  };
  if (a.pn > 0) {
    p.has_prefix = 1;
    add(-1, a.pn, a.n_tok, 0);
  }
  for (int b = 0; b < a.B && *st == VC_OK; ++b) {
    const LiveReqDev& r = a.req[b];
    p.q[b] = r.q;
    p.o[b] = r.o;
    p.tok_begin[b] = r.tok_begin;
    p.own_of[b] = -1;
    if (r.n_rows == 0 || r.n == 0) continue;
    p.own_of[b] = p.n_grp;
    LiveGroup& R = p.grp[p.n_grp];
    R.score = r.score;
    R.cap = r.cap;
    add(b, r.n, r.n_rows, r.tok_begin);
  }
  const int64_t out_rows = (int64_t)a.n_tok * a.Hq;
  if (*st == VC_OK && out_rows + chunks >= INT32_MAX / 2) *st = VC_ERR_UNSUPPORTED;
  if (*st != VC_OK) return cudaSuccess;
  // Keys of a score block: fewer where 1024 leave SMs without two blocks, unless a block has little to do (us with
  // 1024 and with 256 keys: 6 heads of 128 rows and 14419 keys 95, 70; 48 of 32 and 957 26.9, 22.5; 16 of 5 and
  // 7009 22.9, 25.4)
  if (scored) {
    int keys = SCORE_KEYS;
    int most_rows = 0;
    for (int g = 0; g < p.n_grp; ++g) most_rows = p.grp[g].rows > most_rows ? p.grp[g].rows : most_rows;
    auto blocks = [&](int keys) {
      int64_t n = 0;
      for (int g = 0; g < p.n_grp; ++g) {
        p.chunk_begin[g] = (int32_t)n;
        n += (int64_t)a.Hkv * ((p.grp[g].n + keys - 1) / keys);
      }
      return n;
    };
    chunks = blocks(SCORE_KEYS);
    while (keys > 256 && chunks < 2 * live_sms() && keys * most_rows >= 16384) chunks = blocks(keys /= 2);
    p.score_shift = keys == 256 ? 8 : keys == 512 ? 9 : 10;
  }
  share_ctas(cost, weighed, least, p.has_prefix ? p.grp[0].rows : 0, p.n_cta);
  for (int kind = 0; kind < 2; ++kind)
    if (p.n_cta[kind] > 0) {
      p.cta_cost[kind] = (int32_t)(cost[kind] / p.n_cta[kind]);
      p.cta_more[kind] = (int32_t)(cost[kind] % p.n_cta[kind]);
    }
  // Warps a row of the merge: a row's partials, about two a CTA that holds part of its units, by fours (one
  // round trip each); no more than make a wave of blocks (288 rows with 76 partials: 41 us with a warp a row,
  // 27 with eight).
  int64_t parts = 0;
  for (int kind = 0; kind < 2; ++kind)
    if (units[kind]) parts += 2 * (1 + p.n_cta[kind] / units[kind]);
  int wpr = 1;
  while (wpr < 8 && parts > 4 * wpr && out_rows * wpr * 2 <= (int64_t)live_sms() * 4 * 8) wpr *= 2;
  // Several rows a warp where they are more than the warps of a wave and have few partials (with fewer rows both
  // take the same)
  const bool side = !scored && parts <= LIVE_SUB && out_rows > (int64_t)live_sms() * 4 * 8;
  p.merge_warps = side ? 0 : wpr;
  p.merge_blocks = (int32_t)(side ? (out_rows * LIVE_SUB + 255) / 256 : (out_rows * wpr + 7) / 8);
  p.score_blocks = (int32_t)chunks;
  uint8_t* at = static_cast<uint8_t*>(a.ws);
  size_t need = 0;
  auto take = [&](size_t bytes) {
    float* f = reinterpret_cast<float*>(at + need);
    need += pad256(bytes);
    return f;
  };
  if (!a.ws || (reinterpret_cast<uintptr_t>(a.ws) & 15u)) {
    *st = VC_ERR_WORKSPACE;
    return cudaSuccess;
  }
  for (int kind = 0; kind < 2; ++kind) {
    const size_t rows = units[kind] ? (size_t)(p.n_cta[kind] + units[kind]) * p.slot_rows[kind] : 0;
    p.ws_o[kind] = take(rows * (a.d + 1) * sizeof(float));
    p.ws_lse[kind] = p.ws_o[kind] + rows * a.d;
  }
  float* scores = take(s_floats * sizeof(float));
  if (need > a.ws_bytes) {
    *st = VC_ERR_WORKSPACE;
    return cudaSuccess;
  }
  // Partials and scores up to half of L2 are found there by the second kernel if the tiles do not push them
  // out (scored decode, 8 MB of scores: 50.9 us without the hint, 48.9 with it; 134 MB: 371.8 and 377.8)
  p.keep_ws = need <= (size_t)64 << 20;
  bool made = a.pn <= 0 || (live_map(&maps.tm[0][0], a.pk, a.d, a.pn, a.pcap, a.Hkv) &&
                            live_map(&maps.tm[0][1], a.pv, a.d, a.pn, a.pcap, a.Hkv));
  for (int b = 0; b < a.B && made; ++b) {
    const LiveReqDev& r = a.req[b];
    const int g = p.own_of[b];
    if (g >= 0)
      made = live_map(&maps.tm[g][0], r.k, a.d, r.n, r.cap, a.Hkv) && live_map(&maps.tm[g][1], r.v, a.d, r.n, r.cap, a.Hkv);
  }
  if (!made) {
    *st = VC_ERR_CUDA;
    return cudaSuccess;
  }
  for (int g = 0; g < p.n_grp && scored; ++g) {
    p.grp[g].s = scores;
    scores += (size_t)a.Hkv * p.grp[g].rows * p.grp[g].tiles * LN;
  }
  if (a.d == 128) return scored ? launch_live_t<128, true>(p, maps, s) : launch_live_t<128, false>(p, maps, s);
  return scored ? launch_live_t<64, true>(p, maps, s) : launch_live_t<64, false>(p, maps, s);
}

}  // namespace vc
