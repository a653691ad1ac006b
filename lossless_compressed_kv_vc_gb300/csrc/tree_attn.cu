// Attention of drafted trees, chains and single tokens over sequences in pages, on tcgen05 tensor cores.
//
// Token i of a request's n_rows tokens sees the rows of its sequence's context and the tokens its mask names:
//   s_t = q . k_t / sqrt(d),  o = sum_t 2^(s_t - lse) v_t  (log2 domain).
//
// Work decomposition. The rows of one KV head (tokens x G = Hq / Hkv heads) are cut into units of up to 256, the
// keys (context and tokens) into tiles of 128. Lengths live on the device, so the kernels themselves lay the
// plan down: one warp, a lane a request, adds up the tiles [request][head][unit][tile], and each CTA (one per SM:
// 8 softmax warps, 4 MMA issuers, 1 loader) takes an equal range of them by cost. A CTA's part of a unit of a head
// (a piece) leaves an (o, lse) partial; a second kernel merges a row's partials. Of a chain (no mask) each unit has
// the tiles up to the last key that it sees, so a prompt's upper half is not computed (32/8 heads of 128, 2048 tokens
// over no context: 112 us, 172 with all tiles; 69 with all that came since). Where every request has the same number U > 1 of full units, CTA c
// may take unit c % U in the c / U-th range of [request][head][tile], a lane, instead: the units of a head read a tile
// at about the same time, and it comes from DRAM once.
//
// Within a CTA two chains run side by side, each an issuer of S, one of P V and a warpgroup of softmax threads
// (a thread per query row): S = Q K^T into TMEM, softmax in registers, P (bf16) over S in TMEM, O += P V with P read
// from TMEM. The chains meet only in the ring of K and V tiles, so one's softmax runs while the tensor cores work for
// the other. A unit of more than 128 rows gives each chain 128 rows and every tile (a tile costs 2); one of up to 128
// rows gives both chains the same rows and a half of every tile (which costs 1), and at the end of a piece the two
// sums meet in TMEM, where a chain's warps reach the other's rows. A piece that is all of a unit writes the output
// itself. The loader's lanes fetch a tile page by page, each the pages that it looked up one tile before.
//
// S of 128 keys at a time would read Q from shared memory half as often, but leaves TMEM one S a chain: a tile then
// waits for the P V before it (8 trees of 64 over 32768 keys, 64/8 heads of 128: 499 us so, 395 with two S of 64 keys).
//
// What bounds it: up to about 130 rows of a KV head DRAM (16 trees of 25 over up to 16300 rows, 40/8 heads of 128:
// 946 MB in 154 us with the merge, 0.91 of the copy rate); above that each chain's loop S, softmax, P V, the next S
// (the case above: 369 us, 1.50 PFLOP/s, 0.79 of the bf16 rate, in a burst; 340 without exponentials and branches). Of a
// step's 1600 clocks a softmax warp spends 930 on its weights beside the other chain's warp, 135 on S from TMEM, 125 on P
// back to it, the rest on barriers and waits; the tensor cores need 1260 for both chains' step.
//
// What a query row may not see: keys get -infinity by the row's bits of the mask; value rows behind the last
// token (whatever the page holds there) are zeroed in shared memory, and where a step has a value row that is not
// finite and not for all, the threads add up the rows they see themselves. Tokens of a sequence whose last page
// others hold too have no rows there (vc_rope_pages has skipped them) and count for none.
#include "paged.cuh"
#include "tc05.cuh"

#include <cudaTypedefs.h>
#include <limits.h>
#include <math.h>
#include <string.h>
#include <type_traits>

namespace vc {

namespace {

constexpr int TM = 128;         // query rows of a chain
constexpr int TN = 128;         // keys per tile
constexpr int TS = 64;          // keys per step: S and P of half a tile, double-buffered
constexpr int TU = 2 * TM;      // query rows of a unit
// What a unit costs beside its tiles (Q, the first and last steps, the output), in the cost of 64 keys for 256 rows: about
// 5 us. The prompt above: 112 us with 0, 97 with 2, 89 with 4, 80 with 6, 76 with 10; 32 chunks of 60 tokens over 300
// keys 62, 53, 51, 50, 50; 16 trees of 25 over up to 16300 keys 169, 167, 171, 168, 172.
constexpr int TPIECE = 6;
// warps 0-3, 4-7 softmax of chains 0 and 1; 8, 9 issue their S; 10, 11 their P V; 12 TMA; 13 lays the plan down; 14
// and 15 make a warpgroup with them (registers are handed over by warpgroup)
constexpr int TTHREADS = 512;
// Registers a thread: launched with 128 (65536 / 512), then 176 in the softmax warpgroups and 80 in the others (with 64
// channels one word is spilled, with 128 none)
constexpr int TREG_SOFTMAX = 176, TREG_ISSUE = 80;
static_assert(256 * (TREG_SOFTMAX + TREG_ISSUE) <= 65536, "no more than the block was launched with");

// The kernel for few rows: 4 warps a CTA, 3 CTAs an SM (2 * 4 * 8 KB of shared memory each at 128 channels)
constexpr int FR = 16;          // query rows at most
constexpr int FK = 16;          // keys of a chunk
constexpr int FWARPS = 4, FCTAS = 3;

struct TreeParams {
  PagedDev kv;
  // what the plan reads lies together: 32 requests' own fields a line apart take the constant cache microseconds to
  // bring in, in every block of every launch
  int32_t seq[VC_MAX_BATCH], n_rows[VC_MAX_BATCH];
  int32_t tok_begin[VC_MAX_BATCH];   // first query token of each request, INT32_MAX behind the last one
  int32_t mask_words[VC_MAX_BATCH];
  const bf16* q[VC_MAX_BATCH];
  bf16* o[VC_MAX_BATCH];
  const uint32_t* mask[VC_MAX_BATCH];
  int32_t B, Hq, Hkv, G, n_tok;
  int32_t few;                       // 1: the kernel for few rows, whose tiles are chunks and whose CTAs are warps
  int32_t same;                      // full units of every head where all requests have as many, else 1
  uint32_t chains;                   // requests without a mask, a bit each
  int32_t n_cta;                     // CTAs
  int32_t least;                     // cost of the dearest tile: no CTA's range is shorter
  int32_t slot_rows;                 // rows of a partial's slot
  int32_t merge_warps;               // warps a row of the merge, 0: several rows a warp
  // A CTA's range begins inside one unit and ends inside one: partials of units that it takes up in their middle in
  // slot c, of those that it begins and does not end in slot n_cta + c
  float* ws_o;                       // [2 n_cta][slot_rows][d]
  float* ws_lse;                     // [2 n_cta][slot_rows], log2 domain, -inf: saw nothing
  float scale_log2;
  int32_t* dev_status;
};

struct TreeMaps {
  CUtensorMap kv[2];  // (d, page, pages * Hkv): box 64 x page x 1
};

// What follows from the lengths: in shared memory, laid down by one warp of every block.
struct TreePlan {
  int32_t cost_begin[VC_MAX_BATCH];  // of each request in the sequence of costs
  int32_t ctx[VC_MAX_BATCH], n[VC_MAX_BATCH];  // rows of context, and with the tokens' rows
  int32_t rows[VC_MAX_BATCH];        // query rows of a KV head
  int32_t total, ctas, each, more;   // cost; CTAs of a lane with work; a range's cost, and how many have one more
  int32_t lanes;                     // units of every head, each with CTAs of its own (c % lanes); 1: in one sequence
  uint32_t cut;                      // requests whose units end with the last key that they see, a bit each
};

// The page of a sequence's first token, which may hold rows of its context, is the sequence's alone. Those behind it
// always are, as a fork shares pages of context alone; and if this one is not, vc_pages_reserve had no page for the
// copy, and vc_rope_pages did not write there.
__device__ __forceinline__ int token_page(const PagedDev& kv, int seq, int ctx) { return __ldcg(kv.pages_of(seq) + (ctx >> kv.shift)); }
__device__ __forceinline__ bool holds_alone(const PagedDev& kv, int page) { return kv.has_page(page) && __ldcg(kv.refs + page) == 1; }

__device__ __forceinline__ int units_of(int rows) { return (rows + TU - 1) / TU; }
__device__ __forceinline__ int tiles_of(const TreeParams& p, int n) { return p.few ? (n + FK - 1) / FK : (n + TN - 1) / TN; }

// A chain's unit u, full, ends with token (256 u + 255) / G, which sees ctx more keys and itself: with
// b = floor((255 + G (ctx + 128)) / 128) these are floor((2 u + b) / G) tiles.
__device__ __forceinline__ int chain_b(int G, int ctx) { return (TU - 1 + G * (ctx + TN)) / TN; }
static_assert(TU == 2 * TN, "two tiles' rows a unit");
// Tiles of units 0 .. u - 1, the sum of those: it grows by 2 every G units, and within G units the remainder of b
// makes it one or two more from some unit on.
__device__ __forceinline__ int chain_tiles_before(int G, int ctx, int u) {
  const int b = chain_b(G, ctx), bq = b / G, br = b - bq * G, q = u / G, r = u - q * G;
  auto part = [&](int m) { return m * bq + max(0, m - (G - br + 1) / 2) + max(0, m - (2 * G - br + 1) / 2); };
  return q * part(G) + G * q * (q - 1) + part(r) + 2 * q * r;
}

__device__ __forceinline__ void tree_plan(const TreeParams& p, TreePlan* s, int lane, bool tell) {
  int n = 0, ctx = 0, cost = 0, cheap = 0, rows = 0, tiles = 0;
  bool chain = false;
  if (lane < p.B) {
    const int seq = p.seq[lane], tokens = p.n_rows[lane];
    const int held = min(max(__ldcg(p.kv.held + seq), 0), p.kv.max_pages), len = __ldcg(p.kv.len + seq), cap = held << p.kv.shift;
    ctx = min(max(len, 0), cap);
    n = (int)min((int64_t)cap, (int64_t)ctx + tokens);
    // two more dependent loads (2048 tokens over no context 68.4 to 69.0 us); the kernel for few rows makes them beside
    // its first keys, where they cost 0.2 us a call, and 0.7 here
    if (!p.few && n > ctx && !holds_alone(p.kv, token_page(p.kv, seq, ctx))) n = ctx;
    if (tell && (ctx != len || n - ctx != tokens)) set_status(p.dev_status, VC_DEV_PAGES);
    rows = tokens * p.G;
    tiles = tiles_of(p, n);
    const int u = units_of(rows), last = rows - (u - 1) * TU <= TM ? 1 : 2;
    cost = cheap = p.few ? tiles : tiles ? TPIECE * u + tiles * (2 * (u - 1) + last) : 0;
    chain = !p.few && u > 1 && ((p.chains >> lane) & 1u) && n - ctx == tokens && (int64_t)p.G * (ctx + TN) < INT_MAX / 2;
    if (chain) cheap = TPIECE * u + 2 * chain_tiles_before(p.G, ctx, u - 1) + tiles * last;
  }
  const int all = __reduce_add_sync(0xffffffffu, cost), least = __reduce_add_sync(0xffffffffu, cheap);
  // Lanes leave some CTAs without work and do not cut chains; they are taken where that costs up to 1/32 (us with lanes
  // and without, 64/8 heads of 128: trees of 64 over 32768 keys 386, 414; two chains of 256 over 32768 keys, 0.4% more
  // tiles, 384, 419; 32/8 heads: four of 512 over 16384, 1.2%, 414, 419, over 8192, 2.2%, 246, 236, over 4096, 4.3%,
  // 161, 147)
  const int used = p.n_cta / p.same * p.same;  // CTAs that have a lane
  const int lanes = p.same > 1 && (int64_t)all * p.n_cta * 32 <= (int64_t)least * used * 33 ? p.same : 1;
  cost = p.Hkv * (lanes > 1 && tiles ? TPIECE + 2 * tiles : cheap);
  const unsigned cut = __ballot_sync(0xffffffffu, chain && lanes == 1);
  int end = cost;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, end, off);
    if (lane >= off) end += o;
  }
  s->cost_begin[lane] = end - cost;
  s->ctx[lane] = ctx;
  s->n[lane] = n;
  s->rows[lane] = rows;
  if (lane == 31) {
    s->total = end;
    const int ctas = min(p.n_cta / lanes, max(end / p.least, end > 0));
    s->ctas = ctas;
    s->each = ctas ? end / ctas : 0;
    s->more = ctas ? end - ctas * s->each : 0;
    s->lanes = lanes;
    s->cut = cut;
  }
}

// Keys that unit u of request g's rows reads, and the cost of the units before it in its head's sequence.
__device__ __forceinline__ int unit_keys(const TreeParams& p, const TreePlan& s, int g, int u) {
  const bool less = ((s.cut >> g) & 1u) && (u + 1) * TU < s.rows[g];
  return less ? s.ctx[g] + ((u + 1) * TU - 1) / p.G + 1 : s.n[g];
}
__device__ __forceinline__ int cost_before(const TreeParams& p, const TreePlan& s, int g, int u) {
  if (s.lanes > 1 || p.few) return 0;
  return TPIECE * u + 2 * ((s.cut >> g) & 1u ? chain_tiles_before(p.G, s.ctx[g], u) : u * ((s.n[g] + TN - 1) / TN));
}
// Cost of a head of request g.
__device__ __forceinline__ int head_cost(const TreeParams& p, const TreePlan& s, int g) {
  const int tiles = tiles_of(p, s.n[g]), u = units_of(s.rows[g]);
  if (p.few) return tiles;
  return TPIECE + (s.lanes > 1 ? 2 * tiles : cost_before(p, s, g, u - 1) + tiles * (s.rows[g] - (u - 1) * TU <= TM ? 1 : 2));
}

// CTA c of a lane has the costs from cta_begin(c) on; x lies in those of cta_of(x).
__device__ __forceinline__ int cta_begin(const TreePlan& s, int c) { return c * s.each + min(c, s.more); }
__device__ __forceinline__ int cta_of(const TreePlan& s, int x) {
  const int e = s.more * (s.each + 1);
  return x < e ? x / (s.each + 1) : s.more + (x - e) / s.each;
}

// Steps of tile j of n keys: its second half only where it holds keys.
__device__ __forceinline__ int tree_steps(int n, int j) { return n - j * TN > TS ? 2 : 1; }

// A CTA's part of a unit of a head: tiles [j0, j1). Every role of the CTA walks through the same pieces.
struct TPiece {
  int g, hk, u, j0, j1;  // request, KV head, unit of its rows, tiles
  int rows, n, tiles;    // the unit's query rows, keys and tiles
  int at, end;           // cost at which the unit's tiles start, end of the CTA's range: a tile is the CTA's where it starts
  bool split;            // both chains hold the same rows, chain w takes half w of every tile

  __device__ __forceinline__ bool valid() const { return at < end; }
  __device__ __forceinline__ int cost() const { return split ? 1 : 2; }
  // chain 1 has none in the whole piece: a split unit's last, short tile
  __device__ __forceinline__ bool short_one() const { return split && j1 - j0 == 1 && tree_steps(n, j0) == 1; }
  __device__ __forceinline__ bool idle(int w) const { return w == 1 && short_one(); }
  // both chains have sums of the same rows
  __device__ __forceinline__ bool paired() const { return split && !short_one(); }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == tiles; }
  __device__ __forceinline__ void fit(const TreeParams& p, const TreePlan& s) {
    rows = min(TU, s.rows[g] - u * TU);
    n = unit_keys(p, s, g, u);
    tiles = (n + TN - 1) / TN;
    split = rows <= TM;
  }
  __device__ __forceinline__ void cut() { j1 = min(tiles, (end - at + cost() - 1) / cost()); }
  __device__ __forceinline__ void next(const TreeParams& p, const TreePlan& s) {
    at += cost() * tiles + TPIECE;
    if (!valid()) return;
    if (s.lanes > 1 || ++u == units_of(s.rows[g])) {
      if (s.lanes == 1) u = 0;
      if (++hk == p.Hkv) {
        hk = 0;
        do ++g;
        while (s.n[g] == 0);  // there is a further one: the range goes on
      }
    }
    fit(p, s);
    j0 = 0;
    cut();
  }
};

// Chain w's steps in a piece: step i holds the keys from beg + i * stride on, those before `full` are seen whole by
// every row of the chain.
struct TSteps {
  int beg, stride, count, full;
  int blind;  // the first key that some row of the chain does not see

  __device__ __forceinline__ TSteps(const TreeParams& p, const TreePlan& s, const TPiece& q, int w) {
    const int n = q.n, ctx = s.ctx[q.g];
    beg = q.j0 * TN + (q.split ? w * TS : 0);
    stride = q.split ? TN : TS;
    const int end = min(n, q.j1 * TN);
    count = end > beg ? (end - beg + stride - 1) / stride : 0;
    blind = p.mask[q.g] ? ctx : ctx + (q.u * TU + (q.split ? 0 : w * TM)) / p.G + 1;
    const int clear = min(blind, n) - TS - beg;
    full = min(count, clear >= 0 ? clear / stride + 1 : 0);
  }
};

template <int D>
struct TCfg {
  static constexpr int KB = D / 64;            // 64-channel (128-byte) blocks
  static constexpr int T_BYTES = KB * TN * 128;  // a K, V or Q tile
  // K and V tiles in flight or in use: a ring each, so that every role sees every phase of its barriers
  static constexpr int KST = D == 128 ? 3 : 5, VST = D == 128 ? 2 : 5;
  static constexpr int OFF_K = 2 * T_BYTES;    // behind a Q tile per chain
  static constexpr int OFF_V = OFF_K + KST * T_BYTES;
  static constexpr int OFF_BAR = OFF_V + VST * T_BYTES;
  static constexpr int BAR_BYTES = (2 * (KST + VST) + 24) * 8 + 32;
  static constexpr int OFF_SUM = OFF_BAR + BAR_BYTES;  // [2][TM] maxima and sums of the chains' rows
  static constexpr int SMEM = OFF_SUM + 2 * TM * 8 + (int)sizeof(TPiece) + (int)sizeof(TreePlan);
  static_assert(SMEM <= 227 * 1024, "one CTA's shared memory");
  static constexpr int OCOL = 4 * TS;          // TMEM: S (and P) of chain w at (2 w + step % 2) TS, O at OCOL + w D
  static constexpr uint32_t TCOLS = 512;
  static_assert(OCOL + 2 * D <= (int)TCOLS, "TMEM");
};

__device__ __forceinline__ TPiece tree_first(const TreeParams& p, const TreePlan& s) {
  TPiece q;
  const int c = blockIdx.x / s.lanes;
  const int beg = cta_begin(s, c);
  q.end = cta_begin(s, c + 1);
  q.g = 0;
  for (int b = 1; b < p.B; ++b)  // the last request that starts at or before; one without tiles starts where the next does
    if (s.cost_begin[b] <= beg) q.g = b;
  const int head = head_cost(p, s, q.g);
  int rem = beg - s.cost_begin[q.g];
  q.hk = rem / head;
  rem -= q.hk * head;
  q.u = blockIdx.x % s.lanes;
  if (s.lanes == 1) {  // the last unit that starts at or before
    int over = units_of(s.rows[q.g]);
    while (over - q.u > 1) {
      const int mid = (q.u + over) / 2;
      if (cost_before(p, s, q.g, mid) <= rem)
        q.u = mid;
      else
        over = mid;
    }
    rem -= cost_before(p, s, q.g, q.u);
  }
  q.fit(p, s);
  rem -= TPIECE;
  q.at = beg - rem;
  q.j0 = rem > 0 ? (rem + q.cost() - 1) / q.cost() : 0;
  q.cut();
  if (q.valid() && q.j0 >= q.j1) q.next(p, s);  // the range starts in a unit's last tile, which is the CTA's before
  return q;
}

// Bounded mbarrier wait by a whole warp, which goes on or gives up together (its collective instructions need every
// lane), also when another role of the CTA has aborted.
__device__ __forceinline__ bool twait_warp(uint64_t* bar, uint32_t parity, int32_t* st, volatile int* abort) {
  bool done = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, done)) return true;
  for (uint32_t it = 0; it < kSpinLimit && !done; ++it) {
    done = mbar_try_wait(bar, parity);
    if ((it & 31u) == 31u && *abort) break;
  }
  if (__all_sync(0xffffffffu, done)) return true;
  if (!*abort) set_status(st, VC_DEV_TIMEOUT);
  *abort = 1;
  return false;
}

// A value that all lanes of a warp share, known to be so.
template <typename T>
__device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }

// tcgen05.mma (A in shared memory, A in tensor memory) and commit by the lanes with `on`, without a branch.
__device__ __forceinline__ void mma_if(bool on, uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(bool on, uint32_t tmem_d, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void commit_if(bool on, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"((uint32_t)on)
      : "memory");
}

// Arrives where `on`, without a branch.
__device__ __forceinline__ void tarrive_if(uint64_t* bar, bool on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"((uint32_t)on)
      : "memory");
}

// The values of TMEM loads are there; nothing made of them moves before this.
template <int N>
__device__ __forceinline__ void arrived(uint32_t (&r)[N]) {
  tc05::wait_ld();
#pragma unroll
  for (int e = 0; e < N; ++e) asm volatile("" : "+r"(r[e]));
}

__device__ __forceinline__ bool broken_bf16x2(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Bits of the 64 keys from k0 on that a row sees: its words of the mask, shifted to the step; keys before the
// first token (node < 0) are context, keys from n on are not there.
__device__ __forceinline__ void mask_bits(const uint32_t* row, int words, int node, int left, uint32_t& lo, uint32_t& hi) {
  auto word = [&](int i) { return row && i < words ? row[i] : 0u; };
  uint64_t x;
  if (node >= 0) {
    const int w = node >> 5, sh = node & 31;
    const uint32_t a = word(w), b = word(w + 1), c = sh ? word(w + 2) : 0u;
    x = (uint64_t)__funnelshift_r(b, c, sh) << 32 | __funnelshift_r(a, b, sh);
  } else {  // -64 < node
    x = ((uint64_t)word(1) << 32 | word(0)) << -node | ((1ull << -node) - 1ull);
  }
  if (left < 64) x &= (1ull << left) - 1ull;
  lo = (uint32_t)x;
  hi = (uint32_t)(x >> 32);
}

template <int D>
__global__ void __launch_bounds__(TTHREADS, 1) tree_attn_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ TreeMaps maps) {
  using C = TCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem) & 1023u) {  // the swizzled layouts need 1024-byte aligned tiles
    pdl_wait();
    if (tid == 0) set_status(p.dev_status, VC_DEV_INTERNAL);
    return;
  }
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [KST] K tile landed
  uint64_t* kempty = kfull + C::KST;   // [KST] both chains' MMAs are done with it
  uint64_t* vfull = kempty + C::KST;   // [VST], the same for V
  uint64_t* vempty = vfull + C::VST;
  uint64_t* sfull = vempty + C::VST;  // [2][2] S of the chain's step in TMEM buffer step & 1
  uint64_t* pfull = sfull + 4;    // [2][2] the step's P in the same place (4 warps)
  uint64_t* ofull = pfull + 4;    // [2][2] its P V done: the buffer may take the S of two steps on
  uint64_t* qfull = ofull + 4;    // [2] the piece's Q tile in shared memory (4 warps)
  uint64_t* vbar = qfull + 2;     // [2] the chain's warps have looked through a V tile (4 warps)
  uint64_t* xbar = vbar + 2;      // [4] drain of an issuer's MMAs
  uint64_t* both = xbar + 4;      // [2] a paired piece: both chains' sums are there; they have been read (8 warps)
  // [2] the Q tile of the CTA's first piece (4 warps): for the loader, which holds back V for it. Of qfull it could miss
  // that phase: a chain that sees all of a first piece of one tile asks for its next queries without V.
  uint64_t* qfirst = both + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(qfirst + 2);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tslot + 1);
  // [2][2] by S buffer, as the barriers are: 1 + the chain's last step in it whose P V the softmax warps took. A
  // warp may be a step ahead of the others, and so ahead of the P V issuer, which reads a step's word once all
  // four have left the step; the word's next step needs the issuer's commit behind that.
  volatile uint32_t* s_odd = tslot + 2;
  float2* s_sum = reinterpret_cast<float2*>(smem + C::OFF_SUM);
  TPiece* s_first = reinterpret_cast<TPiece*>(s_sum + 2 * TM);  // the CTA's first piece
  TreePlan& plan = *reinterpret_cast<TreePlan*>(s_first + 1);

  if (warp == 12) {
    if (lane < 2) asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.kv[lane]) : "memory");
    tc05::alloc(tslot, C::TCOLS);
  }
  if (warp == 13) {
    pdl_wait();  // lengths are the kernel's before's
    tree_plan(p, &plan, lane, blockIdx.x == 0);
    __syncwarp();
    if (lane == 0) {
      if ((int)blockIdx.x / plan.lanes < plan.ctas)
        *s_first = tree_first(p, plan);
      else
        s_first->at = s_first->end = 0;
    }
  }
  if (tid == 0) {
    for (int i = 0; i < C::KST; ++i) {
      mbar_init(&kfull[i], 1);
      mbar_init(&kempty[i], 2);
    }
    for (int i = 0; i < C::VST; ++i) {
      mbar_init(&vfull[i], 1);
      mbar_init(&vempty[i], 2);
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
      mbar_init(&both[w], 8);
      mbar_init(&qfirst[w], 4);
      mbar_init(&xbar[w], 1);
      mbar_init(&xbar[2 + w], 1);
    }
    fence_mbar_init();
    *s_abort = 0;
  }
  tc05::fence_before();
  __syncthreads();
  tc05::fence_after();
  const uint32_t tmem = *tslot;
  pdl_wait();
  pdl_launch_dependents();

  // The chains' barriers are kept per S buffer: step s + 2 cannot complete a phase of one before step s's
  // has been waited for, while with one barrier for both, steps s and s + 1 could both pass unseen.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TREG_ISSUE));
    if (warp == 12) {
      // ---- TMA: tiles in order, K then V of each, a lane a page and 64-channel block -------------------
      TPiece q = *s_first;
      const uint64_t pol = l2_evict_first_policy();
      const int shift = p.kv.shift, per = TN >> shift;  // pages a tile
      const int kb = lane / per, pi = lane - kb * per;
      const bool mine = kb < C::KB;
      uint32_t it = 0, issued[2] = {0, 0};  // tiles; loads of K and of V on their way
      bool ok = true;
      for (; q.valid() && ok; q.next(p, plan)) {
        const int pages = (q.n + p.kv.rows() - 1) >> shift;
        const bool once = plan.lanes == 1 && plan.rows[q.g] <= TU;  // tiles that one CTA reads once leave L2 first
        const int32_t* table = p.kv.pages_of(p.seq[q.g]);
        auto look = [&](int j) { return mine && j * per + pi < pages ? table[j * per + pi] : 0; };
        int page = look(q.j0);
        if (it > 0)  // the next piece's queries on their way to L2 before the chains ask for them
          for (int r = lane; r < q.rows; r += 32) {
            const int row = q.u * TU + r, tok = row / p.G;
            const bf16* src = p.q[q.g] + ((size_t)tok * p.Hq + q.hk * p.G + (row - tok * p.G)) * D;
#pragma unroll
            for (int c = 0; c < D; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + c));
          }
        for (int j = q.j0; j < q.j1 && ok; ++j, ++it) {
          const int ahead = j + 1 < q.j1 ? look(j + 1) : 0;
          const int cnt = min(per, pages - j * per);  // pages of this tile: at least one
          const bool load = mine && pi < cnt;
          if (load && !p.kv.has_page(page)) {
            set_status(p.dev_status, VC_DEV_PAGES);
            page = p.kv.n_pages;  // beyond the map: reads as zeros
          }
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t ring = kv ? C::VST : C::KST, st = it % ring;
            uint64_t* full = kv ? vfull : kfull;
            if (it >= ring && !twait_warp(&(kv ? vempty : kempty)[st], (it / ring - 1) & 1, p.dev_status, s_abort)) {
              ok = false;
              break;
            }
            // All CTAs' rings together are 24 MB, 4 us of DRAM's time, and the first piece's Q would queue behind them
            // (16 x 1000 keys: 6.8 us for it): it goes ahead of all but the first tile of K.
            if (it == 0 && kv == 1 && (!twait_warp(&qfirst[0], 0, p.dev_status, s_abort) ||
                                       (!q.idle(1) && !twait_warp(&qfirst[1], 0, p.dev_status, s_abort)))) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(cnt << shift) * 128 * C::KB);
            __syncwarp();
            if (load) {
              uint8_t* dst = smem + (kv ? C::OFF_V : C::OFF_K) + st * C::T_BYTES + kb * (TN * 128) + ((pi << shift) * 128);
              if (once)
                tc05::tma_load_3d_hint(dst, &maps.kv[kv], kb * 64, 0, page * p.Hkv + q.hk, &full[st], pol);
              else
                tc05::tma_load_3d(dst, &maps.kv[kv], kb * 64, 0, page * p.Hkv + q.hk, &full[st]);
            }
            __syncwarp();
            ++issued[kv];
          }
          page = ahead;
        }
      }
      // what is on its way lands before the CTA leaves, whoever gave up (bounded)
      if (lane == 0)
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t ring = kv ? C::VST : C::KST, end = issued[kv];
          for (uint32_t i = end > ring ? end - ring : 0; i < end; ++i)
            mbar_wait_bounded(&(kv ? vfull : kfull)[i % ring], (i / ring) & 1, p.dev_status);
        }
      __syncwarp();
    } else if (warp < 12) {
      // ---- MMAs of chain w: S (warps 8, 9) a step ahead of the softmax, P V (10, 11) as soon as a step's P is there.
      // The whole warp goes through this and one lane issues: what the lanes share stays in uniform registers, where
      // the MMAs take their operands from.
      const int w = uniform(warp) & 1;
      const bool lead = lane == 0, of_s = uniform(warp) < 10;
      const uint32_t base = uniform(smem_u32(smem)), tm = uniform(tmem);
      const uint32_t tS = tm + 2 * w * TS, tO = tm + C::OCOL + w * D;
      constexpr uint32_t IDESC_S = tc05::idesc_bf16(TM, TS, false), IDESC_O = tc05::idesc_bf16(TM, D, true);
      const uint64_t dQ = tc05::sdesc_sw128(base + w * C::T_BYTES, 16, 1024), dK = tc05::sdesc_sw128(base + C::OFF_K, 16, 1024);
      const uint64_t dV = tc05::sdesc_sw128(base + C::OFF_V, TN * 128, 1024);
      uint64_t* full = of_s ? kfull : vfull;
      uint64_t* empty = of_s ? kempty : vempty;
      const uint32_t ring = of_s ? C::KST : C::VST;
      TPiece q = *s_first;
      uint32_t st = 0, ph = 0;  // stage and phase of the next tile
      uint32_t t = 0, u = 0;    // steps and pieces of the chain
      bool ok = true;
      for (; ok; q.next(p, plan)) {
        const int at = uniform(q.at), end = uniform(q.end);
        if (at >= end) break;
        const int whole = uniform(TSteps(p, plan, q, w).full);
        const int n = uniform(q.n), j0 = uniform(q.j0), j1 = uniform(q.j1), split = uniform((int)q.split);
        const int h0 = split ? w : 0, hmax = split ? w + 1 : 2;
        if (of_s && !(h0 >= tree_steps(n, j0) && j1 - j0 == 1)) {  // not idle
          ok = twait_warp(&qfull[w], u & 1, p.dev_status, s_abort);
          ++u;
        }
        int i = 0;  // steps of the piece
        for (int j = j0; j < j1 && ok; ++j) {
          ok = twait_warp(&full[st], ph, p.dev_status, s_abort);
          const int h1 = min(tree_steps(n, j), hmax);
          for (int h = h0; h < h1 && ok; ++h, ++t, ++i) {
            const uint32_t buf = 2 * w + (t & 1), tX = tS + (t & 1) * TS;
            if (of_s) {
              // the P V that read its P from this S buffer is done
              if (t > 1 && !twait_warp(&ofull[buf], ((t >> 1) - 1) & 1, p.dev_status, s_abort)) {
                ok = false;
                break;
              }
              tc05::fence_after();
              const uint64_t k = dK + ((st * C::T_BYTES + h * TS * 128) >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * (TN * 128) + (kk & 3) * 32) >> 4;
                mma_if(lead, tX, dQ + off, k + off, IDESC_S, kk > 0);
              }
              commit_if(lead, &sfull[buf]);
            } else {
              if (!twait_warp(&pfull[buf], (t >> 1) & 1, p.dev_status, s_abort)) {
                ok = false;
                break;
              }
              tc05::fence_after();
              if (i < whole || uniform(s_odd[buf]) != t + 1) {
                const uint64_t v = dV + ((st * C::T_BYTES + h * (TS / 16) * 2048) >> 4);
#pragma unroll
                for (int kk = 0; kk < TS / 16; ++kk) mma_ts_if(lead, tO, tX + kk * 8, v + kk * (2048 >> 4), IDESC_O, i > 0 || kk > 0);
              }
              commit_if(lead, &ofull[buf]);
            }
          }
          if (!ok) break;
          if (h0 < h1)
            commit_if(lead, &empty[st]);
          else if (lead)  // nothing in this tile, the unit's last, for the chain
            mbar_arrive(&empty[st]);
          __syncwarp();
          if (++st == ring) st = 0, ph ^= 1;
        }
      }
      // every MMA issued so far has completed before TMEM is released (bounded, even after an abort)
      commit_if(lead, &xbar[warp - 8]);
      mbar_wait_bounded(&xbar[warp - 8], 0, p.dev_status);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TREG_SOFTMAX));
    // ---- softmax of chain w: thread rt owns TMEM lane rt = row rt of the chain ----------------------
    const int w = warp >> 2, rt = tid & (TM - 1);
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + 2 * w * TS, tO = tmem + lane_off + C::OCOL + w * D;
    uint8_t* sQ = smem + w * C::T_BYTES;
    TPiece q = *s_first;
    uint32_t g = 0, t = 0, looked = 0, pairs = 0;
    // P V of step s done (and with it those before): asked for steps whose S has been read, so the phase
    // before on that buffer is over
    auto pv_done = [&](uint32_t s) { return twait_warp(&ofull[2 * w + (s & 1)], (s >> 1) & 1, p.dev_status, s_abort); };
    bool ok = true;
    // Q of the next piece with tiles for this chain, into its Q tile (the chain's S on the last one are all
    // done: their softmax is)
    auto fetch = [&]() {
      for (; q.valid(); g += q.j1 - q.j0, q.next(p, plan)) {
        if (q.idle(w)) continue;
        const int ru = q.split ? rt : w * TM + rt, row = q.u * TU + ru, tok = row / p.G;  // row of the unit, of the head
        const bf16* src = ru < q.rows ? p.q[q.g] + ((size_t)tok * p.Hq + q.hk * p.G + (row - tok * p.G)) * D : nullptr;  // this thread's row
        // the warp's 32 rows, a row's 16-byte pieces in neighbouring lanes (a lane per row would touch 32 lines a load)
        constexpr int PR = D / 8, RW = 32 / PR;  // pieces of a row, rows a load
        uint4 v[32 / RW];  // all on their way at once
#pragma unroll
        for (int i = 0; i < 32 / RW; ++i) {
          const bf16* from = reinterpret_cast<const bf16*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), i * RW + lane / PR));
          v[i] = from ? __ldcg(reinterpret_cast<const uint4*>(from) + lane % PR) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 32 / RW; ++i) {
          const int c = lane % PR, rr = (warp & 3) * 32 + i * RW + lane / PR;
          *reinterpret_cast<uint4*>(sQ + (c >> 3) * (TM * 128) + rr * 128 + (((c ^ rr) & 7) << 4)) = v[i];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&qfull[w]);
          if (g == 0) mbar_arrive(&qfirst[w]);
        }
        return;
      }
    };
    // the piece before: written once the next one's S are under way
    size_t part = 0;        // this row's partial
    bf16* out = nullptr;    // or its place in the output
    float m_run = 0.f, l_run = 0.f;
    bool row_ok = false, have = false, paired = false;
    while (ok) {
      fetch();
      if (have) {
        if (!pv_done(t - 1)) break;
        // weight of this chain's sum and of the other's
        float mine = l_run != 0.f ? 1.f / l_run : 0.f, theirs = 0.f, lse = l_run != 0.f ? m_run + log2f(l_run) : -INFINITY;
        if (paired) {
          s_sum[w * TM + rt] = make_float2(m_run, l_run);
          tc05::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&both[0]);
          if (!twait_warp(&both[0], pairs & 1, p.dev_status, s_abort)) break;
          const float2 o = s_sum[(w ^ 1) * TM + rt];
          const float M = fmaxf(m_run, o.x), mu = M == -INFINITY ? 0.f : M;  // rows that saw nothing: weights 0, or NaN
          mine = ex2_approx(m_run - mu);
          theirs = ex2_approx(o.x - mu);
          const float sum = w ? theirs * o.y + mine * l_run : mine * l_run + theirs * o.y;  // the same in both chains
          lse = sum != 0.f ? M + log2f(sum) : -INFINITY;
          const float inv = sum != 0.f ? 1.f / sum : 0.f;
          mine *= inv;
          theirs *= inv;
        }
        tc05::fence_after();
        // rows in the order of an MMA's accumulator: four lanes hold 8 neighbouring channels (whole 32-byte
        // sectors), where a lane per row would write 32 lines at a time; of paired chains each writes half the channels
        constexpr int NB = D / 32;  // blocks of 32 channels of a row
        const int cb0 = paired ? w * (NB / 2) : 0, nb = paired ? NB / 2 : NB;
        const uint32_t tX = tmem + lane_off + C::OCOL + (w ^ 1) * D;  // the other chain's O
        float* o_row0 = p.ws_o + (part - (rt & 31)) * D + cb0 * 32 + 2 * (lane & 3);  // of the warp's first row
        const unsigned rows_ok = __ballot_sync(0xffffffffu, row_ok);
        const bool direct = __any_sync(0xffffffffu, out != nullptr);
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh) {
          if (!((rows_ok >> (16 * hh)) & 0xffffu)) continue;
          const int r0 = hh * 16 + (lane >> 2);
          const uint32_t half = (uint32_t)(hh * 16) << 16;
          uint32_t r[NB][16];
#pragma unroll
          for (int c = 0; c < NB / 2; ++c) {  // warp-collective: every lane loads
            tc05::ld16x256_x4(tO + half + (cb0 + c) * 32, r[c]);
            tc05::ld16x256_x4((paired ? tX + cb0 * 32 : tO + (NB / 2) * 32) + half + c * 32, r[NB / 2 + c]);
          }
          float a[2], b[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            a[e] = __shfl_sync(0xffffffffu, mine, r0 + 8 * e);
            b[e] = __shfl_sync(0xffffffffu, paired ? theirs : mine, r0 + 8 * e);
          }
#pragma unroll
          for (int c = 0; c < NB; ++c) arrived(r[c]);
#pragma unroll
          for (int c = 0; c < NB / 2; ++c)
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float x = __uint_as_float(r[c][k]) * a[k >> 1 & 1], y = __uint_as_float(r[NB / 2 + c][k]) * b[k >> 1 & 1];
              r[c][k] = __float_as_uint(paired ? x + y : x);
              r[NB / 2 + c][k] = __float_as_uint(y);
            }
          if (direct) {
            bf16* to[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
              to[e] = reinterpret_cast<bf16*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), r0 + 8 * e)) +
                      cb0 * 32 + 8 * (lane & 1) + 2 * (lane & 2);
#pragma unroll
            for (int c = 0; c < NB; ++c) {
              if (c >= nb) continue;
#pragma unroll
              for (int k = 0; k < 4; k += 2)  // of two groups of 8 channels an even lane takes the first, with its neighbour's
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t x = pack_bf16x2(__uint_as_float(r[c][4 * k + 2 * e]), __uint_as_float(r[c][4 * k + 2 * e + 1]));
                  const uint32_t y = pack_bf16x2(__uint_as_float(r[c][4 * k + 4 + 2 * e]), __uint_as_float(r[c][4 * k + 5 + 2 * e]));
                  const uint32_t z = __shfl_xor_sync(0xffffffffu, lane & 1 ? x : y, 1);
                  if ((rows_ok >> (r0 + 8 * e)) & 1u) *reinterpret_cast<uint2*>(to[e] + c * 32 + 8 * k) = lane & 1 ? make_uint2(z, y) : make_uint2(x, z);
                }
            }
          } else {
#pragma unroll
            for (int c = 0; c < NB; ++c) {
              if (c >= nb) continue;
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if ((rows_ok >> (r0 + 8 * e)) & 1u)
                    *reinterpret_cast<uint2*>(o_row0 + (size_t)(r0 + 8 * e) * D + c * 32 + 8 * k) = make_uint2(r[c][4 * k + 2 * e], r[c][4 * k + 2 * e + 1]);
            }
          }
        }
        if (row_ok && !out && !(paired && w)) p.ws_lse[part] = lse;
        tc05::fence_before();
        if (paired) {  // neither chain's next P V before both have read
          __syncwarp();
          if (lane == 0) mbar_arrive(&both[1]);
          if (!twait_warp(&both[1], pairs & 1, p.dev_status, s_abort)) break;
          ++pairs;
        }
      }
      if (!q.valid()) break;
      have = true;
      paired = q.paired();
      const int ru = q.split ? rt : w * TM + rt;
      row_ok = ru < q.rows;
      const bool alive = __any_sync(0xffffffffu, row_ok);  // a warp without rows only keeps step
      const int row = q.u * TU + ru, tl = row / p.G;
      part = (size_t)(blockIdx.x + (q.j0 > 0 ? 0 : p.n_cta)) * p.slot_rows + ru;
      out = q.whole() && row_ok ? p.o[q.g] + ((size_t)tl * p.Hq + q.hk * p.G + (row - tl * p.G)) * D : nullptr;
      const int n = q.n, ctx = plan.ctx[q.g];
      const bool masked = p.mask[q.g] != nullptr;
      const int words = p.mask_words[q.g];
      const uint32_t* mrow = masked && row_ok ? p.mask[q.g] + (size_t)tl * words : nullptr;
      const TSteps steps(p, plan, q, w);
      m_run = -INFINITY, l_run = 0.f;
      // A step, with `tail` or without what only steps need that some row does not see whole: the others' loop is short,
      // and its registers go to the weights. The way back to them once a maximum has moved is a copy of its own, as a loop
      // around them keeps the compiler from overlapping them with what comes next (8 trees of 64 over 32768 keys, 64/8
      // heads: of 128 channels 378 us with one loop for all, 368 so; of 64 channels 340, 298). With 64 channels P also
      // goes to TMEM before it is known whether it stands: 275 us. With 128, where the tensor cores set the pace, that
      // costs more than it gives (382).
      constexpr bool EAGER = D == 64;
      auto step = [&](auto kind, int i) -> bool {
        constexpr bool tail = decltype(kind)::value;
        const uint32_t buf = 2 * w + (t & 1), tP = tS + (t & 1) * TS;
        if (!twait_warp(&sfull[buf], (t >> 1) & 1, p.dev_status, s_abort)) return false;
        tc05::fence_after();
        uint32_t see_lo = 0xffffffffu, see_hi = 0xffffffffu;  // keys of the step that the row sees
        if (alive) {
          float x[TS];
          {
            uint32_t lo[32], hi[32];
            tc05::ld32(tP, lo);
            tc05::ld32(tP + 32, hi);
            arrived(lo);
            arrived(hi);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(lo[e]), x[32 + e] = __uint_as_float(hi[e]);
          }
          if constexpr (tail) {
            const int k0 = steps.beg + i * steps.stride;
            if (masked) {
              mask_bits(mrow, words, k0 - ctx, n - k0, see_lo, see_hi);
            } else {
              const int last = min(ctx + tl, n - 1) - k0;
              see_lo = last >= 31 ? 0xffffffffu : last < 0 ? 0u : (2u << last) - 1u;
              see_hi = last >= 63 ? 0xffffffffu : last < 32 ? 0u : (2u << (last - 32)) - 1u;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (!((see_lo >> e) & 1u)) x[e] = -INFINITY;
              if (!((see_hi >> e) & 1u)) x[32 + e] = -INFINITY;
            }
          }
          // P = 2^(x scale - m), bf16, over S: the MMA wants both operands in one 16-bit type, and V is bf16 (its range
          // is not fp16's). A weight is off by 2^-8 of itself at most. Sums and lse take the weights unrounded.
          // m is the row's maximum when it was last looked for: as long as a step's weights add up to no more than
          // 2^10 it is kept (no weight is larger then, and a search in every step cost 15 us of 393 over 32768 keys).
          // Past that, and in the piece's first step, the maximum is found, O rescaled after the P V before, and P
          // computed again. TMEM loads and stores are warp-collective: the warp does it together.
          uint32_t r[TS / 2];
          float sum = 0.f;
          auto weights = [&] {
            const float mu = m_run == -INFINITY ? 0.f : m_run;
            const uint64_t sc = f2_pack(p.scale_log2, p.scale_log2), nm = f2_pack(-mu, -mu);
            uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int e = 0; e < TS / 2; ++e) {
              float a0, a1;
              f2_unpack(f2_fma(f2_pack(x[2 * e], x[2 * e + 1]), sc, nm), a0, a1);
              const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
              acc[e & 3] = f2_add(acc[e & 3], f2_pack(p0, p1));
              r[e] = pack_bf16x2(p0, p1);
            }
            float u0, u1;
            f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), u0, u1);
            sum = u0 + u1;
          };
          bool look = i == 0;
          if (!look) {
            weights();
            if constexpr (EAGER) tc05::st32(tP, r);  // ahead of the answer, which is rarely yes
            // a row that has seen nothing yet has no m: its weights say nothing of how large its scores are
            look = __any_sync(0xffffffffu, sum > 1024.f || m_run == -INFINITY);
          }
          if (look) {
            float top = -INFINITY;
#pragma unroll
            for (int e = 0; e < TS; e += 2) top = max3f(top, x[e], x[e + 1]);
            const float m_new = fmaxf(m_run, top * p.scale_log2);
            float f = 1.f;
            if (m_new > m_run) {
              f = ex2_approx(m_run - m_new);
              l_run *= f;
              m_run = m_new;
            }
            if (i > 0) {
              if (!pv_done(t - 1)) return false;
              tc05::fence_after();
#pragma unroll 1
              for (int cb = 0; cb < D / 32; ++cb) {
                uint32_t o[32];
                tc05::ld32(tO + cb * 32, o);
                arrived(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tc05::st32(tO + cb * 32, o);
              }
            }
            weights();
            if constexpr (EAGER) {
              tc05::wait_st();  // the P of before
              tc05::st32(tP, r);
            }
          }
          if constexpr (!EAGER) tc05::st32(tP, r);
          l_run += sum;
          tc05::wait_st();
        }
        // A step with keys that some rows do not see: a weight of 0 would carry an infinite or NaN value row to
        // them. Rows from n on, which nobody sees, are zeroed; if others hold such a value, the threads add up the
        // seen keys themselves.
        if constexpr (tail) {
          const int k0 = steps.beg + i * steps.stride, j = k0 / TN, h = k0 / TS & 1;
          const uint32_t gv = g + j - q.j0;
          // V has landed: the phase before is over (its P V are done), and its own cannot pass without this chain
          if (!twait_warp(&vfull[gv % C::VST], (gv / C::VST) & 1, p.dev_status, s_abort)) return false;
          uint8_t* sV = smem + C::OFF_V + (gv % C::VST) * C::T_BYTES;
          bool bad = false;
          const int kv = h * TS + (rt & (TS - 1));  // two threads look through each of the step's rows
          const bool there = j * TN + kv < n;
#pragma unroll
          for (int cc = 0; cc < D / 16; ++cc) {
            const int c = (rt / TS) * (D / 16) + cc;
            uint4* at = reinterpret_cast<uint4*>(sV + (c >> 3) * (TN * 128) + kv * 128 + (((c ^ kv) & 7) << 4));
            if (there) {
              const uint4 v = *at;
              bad |= broken_bf16x2(v.x) || broken_bf16x2(v.y) || broken_bf16x2(v.z) || broken_bf16x2(v.w);
            } else {
              *at = make_uint4(0, 0, 0, 0);  // by both chains where they share the tile
            }
          }
          if (bad) s_odd[buf] = t + 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&vbar[w]);
          if (!twait_warp(&vbar[w], looked & 1, p.dev_status, s_abort)) return false;
          ++looked;
          if (alive && s_odd[buf] == t + 1) {
            if (i > 0 && !pv_done(t - 1)) return false;
            tc05::fence_after();
#pragma unroll 1
            for (int cb = 0; cb < D / 32; ++cb) {
              uint32_t r[32];
              if (i > 0) {
                tc05::ld32(tO + cb * 32, r);
                arrived(r);
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = 0u;
              }
#pragma unroll 1
              for (int kp = 0; kp < TS / 2; ++kp) {  // two keys a column; rare, so kept small
                uint32_t pw[1] = {tc05::ld1(tP + kp)};
                arrived(pw);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int k = 2 * kp + e, kt = h * TS + k;
                  const bool sees = ((k < 32 ? see_lo : see_hi) >> (k & 31)) & 1u;
                  const float pk = __uint_as_float(e ? pw[0] & 0xffff0000u : pw[0] << 16);
#pragma unroll
                  for (int c = 0; c < 4; ++c) {
                    const int ch = cb * 4 + c;
                    const uint4 v = *reinterpret_cast<const uint4*>(sV + (ch >> 3) * (TN * 128) + kt * 128 + (((ch ^ kt) & 7) << 4));
                    const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                      const float val = __uint_as_float(y & 1 ? vw[y >> 1] & 0xffff0000u : vw[y >> 1] << 16);
                      const float a = __uint_as_float(r[c * 8 + y]);
                      r[c * 8 + y] = __float_as_uint(sees ? fmaf(pk, val, a) : a);
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
        tarrive_if(&pfull[buf], lane == 0);
        return true;
      };
      int i = 0;
#pragma unroll 1
      for (; ok && i < steps.full; ++i, ++t) ok = step(std::false_type(), i);
#pragma unroll 1
      for (; ok && i < steps.count; ++i, ++t) ok = step(std::true_type(), i);
      g += q.j1 - q.j0;
      if (!ok) break;
      q.next(p, plan);
    }
  }

  tc05::fence_before();
  __syncthreads();
  tc05::fence_after();
  if (warp == 12) tc05::dealloc(tmem, C::TCOLS);
}

// ---- few rows ---------------------------------------------------------------------------------------
// Up to 16 query rows of a KV head (single tokens, small trees): bound by reading K and V, so each warp works for
// itself, without a barrier: it takes an equal range of the chunks [request][head][16 keys], has three half chunks
// (K or V) on their way with 16-byte asynchronous copies into its own ring, and multiplies with mma.sync: S = Q K^T
// with Q in registers, P from S's accumulators as they lie, O += P V. The tcgen05 kernel's fixed part (tensor maps,
// TMEM, barriers, two chains' start and end) is what this one does without, and a page of 16 rows is as good as a
// larger one, where TMA boxes of 2 KB hold the other back. Measured with 32 ragged requests of up to 8200 rows, 32/8 heads of 128, call after call: 939 MB in 152 us with
// the merge, 6.2 TB/s. Equal ranges do not end together: SMs in the larger groups get up to 12% less of DRAM.
template <int D>
struct FCfg {
  static constexpr int HALF = FK * D * 2;             // bytes of a chunk's K or V
  static constexpr int SMEM = FWARPS * 4 * HALF;      // two chunks a warp
};

// Bits of the 16 keys from k0 on that row i of a request's tokens sees; node = k0 - ctx > -16; left: keys from k0 on, if any.
__device__ __forceinline__ uint32_t few_bits(const uint32_t* row, int words, bool masked, int tok, int node, int left) {
  uint32_t x;
  if (!masked) {
    const int last = tok - node;  // of the chunk's keys
    x = last >= 15 ? 0xffffu : last < 0 ? 0u : (2u << last) - 1u;
  } else {
    auto word = [&](int i) { return row && i < words ? row[i] : 0u; };
    if (node >= 0)
      x = __funnelshift_r(word(node >> 5), (node & 31) > 16 ? word((node >> 5) + 1) : 0u, node & 31);
    else
      x = word(0) << -node | ((1u << -node) - 1u);
  }
  return x & (left >= 16 ? 0xffffu : left > 0 ? (1u << left) - 1u : 0u);
}

template <int D>
__global__ void __launch_bounds__(FWARPS * 32, FCTAS) tree_few_kernel(const __grid_constant__ TreeParams p) {
  using C = FCfg<D>;
  constexpr int PC = D / 8;  // 16-byte pieces of a row
  extern __shared__ __align__(128) uint8_t few_smem[];
  __shared__ TreePlan plan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();  // behind the wait, when all CTAs are there: a merge waiting on an SM would keep one from it
  if (warp == 0) tree_plan(p, &plan, lane, blockIdx.x == 0);
  __syncthreads();
  const int wid = warp * gridDim.x + blockIdx.x;  // the first ones on different SMs
  if (wid >= plan.ctas) return;
  uint8_t* ring = few_smem + warp * 4 * C::HALF;  // K of chunk 0, V of chunk 0, K of chunk 1, V of chunk 1
  const int beg = cta_begin(plan, wid), end = cta_begin(plan, wid + 1);
  int g = 0;
  for (int b = 1; b < p.B; ++b)  // as in tree_first
    if (plan.cost_begin[b] <= beg) g = b;
  int rem = beg - plan.cost_begin[g], tiles = tiles_of(p, plan.n[g]);
  int hk = rem / tiles;
  rem -= hk * tiles;
  const int qrow = lane >> 2, qcol = 2 * (lane & 3);
  // where this lane's pieces of a half chunk lie in it: row lane / PC + i * 32 / PC
  constexpr int RS = 32 / PC;  // rows a load of the warp
  const int prow = lane / PC, pcol = lane % PC;
  for (int at = beg; at < end;) {
    const int n = plan.n[g], ctx = plan.ctx[g], j0 = rem, j1 = min(tiles, rem + end - at), rows = plan.rows[g];
    const int32_t* table = p.kv.pages_of(p.seq[g]);
    const bool masked = p.mask[g] != nullptr;
    const int words = p.mask_words[g];
    // pages of the chunks jb .. jb + 31, a lane each; those that are not the pool's count as none
    auto look = [&](int jb) {
      int page = -1;
      if (jb + lane < j1) {
        page = table[((jb + lane) * FK) >> p.kv.shift];
        if (!p.kv.has_page(page)) {
          set_status(p.dev_status, VC_DEV_PAGES);
          page = -1;
        }
      }
      return page;
    };
    int pages = look(j0), more = look(j0 + 32);  // those in use and the next ones
    const bool tokens = j1 * FK > ctx && n > ctx;
    const int tpage = tokens ? token_page(p.kv, p.seq[g], ctx) : 0;
    // Q, asked for ahead of all K and V, in A-fragment order: rows qrow and qrow + 8, channels 16 kk + qcol (+ 8)
    uint32_t qf[D / 16][4];
    int tok[2];
    const uint32_t* mrow[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = qrow + 8 * e;
      tok[e] = r < rows ? r / p.G : 0;
      mrow[e] = masked && r < rows ? p.mask[g] + (size_t)tok[e] * words : nullptr;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q[g] + ((size_t)tok[e] * p.Hq + hk * p.G + (r - tok[e] * p.G)) * D + qcol);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][e] = r < rows ? __ldcg(src + kk * 8) : 0u;
        qf[kk][2 + e] = r < rows ? __ldcg(src + kk * 8 + 4) : 0u;
      }
    }
    // half chunk `v` (0: K, 1: V) of chunk j into its place; one commit whether there is one or not
    auto load = [&](int j, int v) {
      const int page = __shfl_sync(0xffffffffu, pages, (j - j0) & 31);
      if (j < j1) {
        const int k0 = j * FK;
        uint8_t* dst = ring + ((j - j0) & 1) * 2 * C::HALF + v * C::HALF;
        const bf16* src = (v ? p.kv.v : p.kv.k) +
                          ((((int64_t)max(page, 0) * p.Hkv + hk) << p.kv.shift) + (k0 & (p.kv.rows() - 1))) * D + prow * D + pcol * 8;
#pragma unroll
        for (int i = 0; i < FK / RS; ++i) {
          const int r = prow + i * RS;
          cp_async16(dst + r * D * 2 + (((pcol & 8) | ((pcol ^ r) & 7)) << 4), src + i * RS * D, page >= 0 && k0 + r < n ? 16 : 0);
        }
      }
      cp_async_commit();
    };
    load(j0, 0);
    load(j0, 1);
    load(j0 + 1, 0);
    load(j0 + 1, 1);
    int seen = n;  // keys that count
    if (tokens && !holds_alone(p.kv, tpage)) {
      seen = ctx;
      set_status(p.dev_status, VC_DEV_PAGES);
    }
    const int blind = min(seen, masked ? ctx : ctx + 1);  // the first key that some row may not see
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
      const int k0 = j * FK;
      uint8_t* sK = ring + ((j - j0) & 1) * 2 * C::HALF;
      uint8_t* sV = sK + C::HALF;
      cp_async_wait<3>();  // K of this chunk is there: behind it its V and the next chunk's
      __syncwarp();
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        const int key = ((lane >> 4) << 3) + (lane & 7);
        const uint8_t* row = sK + key * D * 2;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int c = 2 * kk + ((lane >> 3) & 1);
          uint32_t b[4];
          ldsm_x4(b[0], b[1], b[2], b[3], row + (((c & 8) | ((c ^ key) & 7)) << 4));
          mma_bf16_16816(s[0], qf[kk], b[0], b[1]);
          mma_bf16_16816(s[1], qf[kk], b[2], b[3]);
        }
      }
      __syncwarp();  // K has been read by all
      if (((j - j0 + 2) & 31) == 0) pages = more;
      load(j + 2, 0);
      uint32_t see[2] = {0xffffu, 0xffffu};
      const bool tail = k0 + FK > blind;
      if (tail) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          see[e] = few_bits(mrow[e], words, masked, tok[e], k0 - ctx, seen - k0);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (!((see[e] >> (8 * t + qcol + i)) & 1u)) s[t][2 * e + i] = -INFINITY;
        }
      }
      // the running maximum moves when it is passed by more than 2^8 (or from -infinity), for the warp together
      float top[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        top[e] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2)) * p.scale_log2;
      }
      if (__any_sync(0xffffffffu, top[0] > m[0] + 8.f || top[1] > m[1] + 8.f)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float was = m[e];
          if (top[e] > was + 8.f) m[e] = top[e];
          const float f = was == m[e] ? 1.f : ex2_approx(was - m[e]);
          l[e] *= f;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            acc[i][2 * e] *= f;
            acc[i][2 * e + 1] *= f;
          }
        }
      }
      // P = 2^(s scale - m), rounded to bf16 for the product with V (its range is not fp16's); sums take it unrounded
      uint32_t pf[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mu = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float a = ex2_approx(fmaf(s[t][2 * e], p.scale_log2, -mu)), b = ex2_approx(fmaf(s[t][2 * e + 1], p.scale_log2, -mu));
          l[e] += a + b;
          pf[2 * t + e] = pack_bf16x2(a, b);
        }
      }
      cp_async_wait<3>();  // V of this chunk
      __syncwarp();
      bool odd = false;
      if (tail) {  // a value row that is not finite, and not for all
#pragma unroll
        for (int i = 0; i < FK / RS; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(sV + (i * 32 + lane) * 16);
          odd |= broken_bf16x2(v.x) || broken_bf16x2(v.y) || broken_bf16x2(v.z) || broken_bf16x2(v.w);
        }
        odd = __any_sync(0xffffffffu, odd);
      }
      if (!odd) {
        const int key = (((lane >> 3) & 1) << 3) + (lane & 7);
        const uint8_t* row = sV + key * D * 2;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int c = 2 * i + (lane >> 4);
          uint32_t b[4];
          ldsm_x4_t(b[0], b[1], b[2], b[3], row + (((c & 8) | ((c ^ key) & 7)) << 4));
          mma_bf16_16816(acc[2 * i], pf, b[0], b[1]);
          mma_bf16_16816(acc[2 * i + 1], pf, b[2], b[3]);
        }
      } else {  // the keys that a row sees, one by one
#pragma unroll 1
        for (int k = 0; k < FK; ++k) {
          const int from = (lane & ~3) | ((k & 7) >> 1);
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t x = __shfl_sync(0xffffffffu, k < 8 ? pf[e] : pf[2 + e], from);
            w[e] = __uint_as_float(k & 1 ? x & 0xffff0000u : x << 16);
          }
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(sV + k * D * 2 + (((i & 8) | ((i ^ k) & 7)) << 4) + qcol * 2);
            const float lo = __uint_as_float(v << 16), hi = __uint_as_float(v & 0xffff0000u);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if ((see[e] >> k) & 1u) {
                acc[i][2 * e] = fmaf(w[e], lo, acc[i][2 * e]);
                acc[i][2 * e + 1] = fmaf(w[e], hi, acc[i][2 * e + 1]);
              }
          }
        }
      }
      __syncwarp();
      load(j + 2, 1);
      if (((j - j0 + 2) & 31) == 0) more = look(j + 2 + 32);
    }
    cp_async_wait<0>();
    // the range's partial of this head: four lanes hold 8 neighbouring channels of a row
    const size_t part = (size_t)(wid + (j0 > 0 ? 0 : p.n_cta)) * p.slot_rows;
    const bool whole = j0 == 0 && j1 == tiles;  // then it is the output
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      const int r = qrow + 8 * e;
      if (r < rows) {
        const float inv = l[e] != 0.f ? 1.f / l[e] : 0.f;
        if (whole) {
          bf16* dst = p.o[g] + ((size_t)tok[e] * p.Hq + hk * p.G + (r - tok[e] * p.G)) * D + qcol;
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<uint32_t*>(dst + 8 * i) = pack_bf16x2(acc[i][2 * e] * inv, acc[i][2 * e + 1] * inv);
          continue;
        }
        float* dst = p.ws_o + (part + r) * D + qcol;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(dst + 8 * i) = make_float2(acc[i][2 * e] * inv, acc[i][2 * e + 1] * inv);
        if ((lane & 3) == 0) p.ws_lse[part + r] = l[e] != 0.f ? m[e] + log2f(l[e]) : -INFINITY;
      }
    }
    __syncwarp();
    at += j1 - j0;
    rem = 0;
    if (++hk == p.Hkv && at < end) {
      hk = 0;
      do ++g;
      while (plan.n[g] == 0);
      tiles = tiles_of(p, plan.n[g]);
    }
  }
}

// ---- merge ------------------------------------------------------------------------------------------
// Weight of a partial beside the largest lse M: 0 where it saw nothing; M stays -inf only beside a NaN.
__device__ __forceinline__ float part_weight(float l, float M) { return l == -INFINITY ? 0.f : M == -INFINITY ? NAN : exp2f(l - M); }

// Where a row's unit left its partials: `count` of them, number i at index at(i). One alone is the output already.
struct TParts {
  size_t first, base;
  int count, stride;  // stride: rows from a CTA's slot to that of the next one with the unit
  __device__ __forceinline__ size_t at(int i) const { return i ? base + (size_t)i * stride : first; }
};

// Output row `id` of the call (token, query head): its partials and its place.
template <int D>
__device__ __forceinline__ TParts tree_parts(const TreeParams& p, const TreePlan& plan, const int32_t* tok_begin, int64_t id, bf16*& dst) {
  const int tok = (int)(id / p.Hq), hq = (int)(id - (int64_t)tok * p.Hq), hk = hq / p.G;
  int b = 0;
#pragma unroll
  for (int k = VC_MAX_BATCH / 2; k > 0; k >>= 1)
    if (tok_begin[b + k] <= tok) b += k;
  const int i = tok - tok_begin[b], r = i * p.G + hq - hk * p.G;  // token of the request, row of the head
  dst = p.o[b] + ((size_t)i * p.Hq + hq) * D;
  const int rows = plan.rows[b], u = p.few ? 0 : r / TU;
  const int cost = p.few || rows - u * TU <= TM ? 1 : 2, tiles = tiles_of(p, p.few ? plan.n[b] : unit_keys(p, plan, b, u));
  TParts q{0, 0, 0, plan.lanes * p.slot_rows};
  if (tiles == 0) return q;
  const int at = plan.cost_begin[b] + hk * head_cost(p, plan, b) + cost_before(p, plan, b, u) + (p.few ? 0 : TPIECE);
  const int c0 = cta_of(plan, at), c1 = cta_of(plan, at + cost * (tiles - 1));  // of its first and last tile
  q.count = c1 - c0 + 1;
  q.base = (size_t)(c0 * plan.lanes + (plan.lanes > 1 ? u : 0)) * p.slot_rows + (r - u * TU);
  q.first = q.base + (size_t)p.n_cta * p.slot_rows;
  return q;
}

// Merge, o = sum_k 2^(lse_k - M) o_k / sum_k 2^(lse_k - M) over a row's partials. Few rows of many partials: one to
// eight warps a row, a lane per partial takes the weights, then the warp adds up the partials' channels, four loads
// in flight, the first four ahead of the weights. Bound by latency: it follows another kernel, so all that does not
// need that one's results is done before the wait. The plan is such: the attention kernels let this one start after
// their own wait, when whatever wrote the lengths has ended and is in L2, and they leave them as they are.
template <int D>
__global__ void __launch_bounds__(256, 4) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  constexpr int E = D / 32;  // channels a lane
  constexpr int PF = 4;      // partials in flight
  __shared__ TreePlan plan;
  __shared__ int32_t tok_begin[VC_MAX_BATCH];
  __shared__ float s_sum[8];
  __shared__ float s_acc[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wpr = p.merge_warps, part = warp % wpr;  // warps of a row, this one among them
  const int64_t id = (int64_t)blockIdx.x * (8 / wpr) + warp / wpr;
  bool live = id < (int64_t)p.n_tok * p.Hq;
  if (threadIdx.x < VC_MAX_BATCH) tok_begin[threadIdx.x] = p.tok_begin[threadIdx.x];
  if (warp == 0) tree_plan(p, &plan, lane, false);
  __syncthreads();
  TParts q{0, 0, 0, 0};
  bf16* dst = nullptr;
  if (live) q = tree_parts<D>(p, plan, tok_begin, id, dst);
  if (q.count == 1) {  // written by the piece itself: nothing to add up, the block's barrier is kept
    live = false;
    q.count = 0;
  }
  const int beg = q.count * part / wpr, end = q.count * (part + 1) / wpr;
  auto fetch = [&](float (&v)[E], int k) {
    const float* src = p.ws_o + q.at(k) * D + lane * E;
    if constexpr (E == 4)
      *reinterpret_cast<float4*>(v) = __ldcg(reinterpret_cast<const float4*>(src));
    else
      *reinterpret_cast<float2*>(v) = __ldcg(reinterpret_cast<const float2*>(src));
  };
  pdl_wait();
  pdl_launch_dependents();
  float ahead[PF][E];
#pragma unroll
  for (int c = 0; c < PF; ++c)
    if (beg + c < end) fetch(ahead[c], beg + c);
  auto lse_of = [&](int k, int end) { return k >= end ? -INFINITY : p.ws_lse[q.at(k)]; };
  float M = -INFINITY;
  for (int k0 = 0; k0 < q.count; k0 += 32) M = fmaxf(M, lse_of(k0 + lane, q.count));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float L = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int k0 = beg; k0 < end; k0 += 32) {
    const float l = lse_of(k0 + lane, end), f = part_weight(l, M);
    const unsigned wrote = __ballot_sync(0xffffffffu, l != -INFINITY);
    L += f;
    const int cnt = min(32, end - k0);
    for (int c0 = 0; c0 < cnt; c0 += PF) {
      float v[PF][E], fc[PF];
#pragma unroll
      for (int c = 0; c < PF; ++c) {
        fc[c] = __shfl_sync(0xffffffffu, f, c0 + c);  // c0 + c < 32; nothing was written beyond cnt
        const bool wr = (wrote >> (c0 + c)) & 1u;      // a partial that saw nothing was not written
        if (k0 + c0 == beg) {
#pragma unroll
          for (int e = 0; e < E; ++e) v[c][e] = wr ? ahead[c][e] : 0.f;
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) v[c][e] = 0.f;
          if (wr) fetch(v[c], k0 + c0 + c);
        }
      }
#pragma unroll
      for (int c = 0; c < PF; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(fc[c], v[c][e], acc[e]);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  if (wpr > 1) {  // the row's warps meet
#pragma unroll
    for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
    if (lane == 0) s_sum[warp] = L;
    __syncthreads();
    if (part != 0) return;
    for (int k = 1; k < wpr; ++k) {
      L += s_sum[warp + k];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += s_acc[warp + k][lane * E + e];
    }
  }
  if (!live) return;
  const float inv = L != 0.f ? 1.f / L : 0.f;
  dst += lane * E;
  uint32_t out[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = out[0];
}

// Many rows of few partials: TSUB lanes a row, four rows a warp side by side, one wave of blocks that go through the
// rows (each lays the plan down once).
constexpr int TSUB = 8;
template <int D>
__global__ void __launch_bounds__(256, 4) tree_merge_rows_kernel(const __grid_constant__ TreeParams p) {
  constexpr int Q = D / 4 / TSUB;  // float4 a lane: number sl, sl + TSUB, ... of the row
  __shared__ TreePlan plan;
  __shared__ int32_t tok_begin[VC_MAX_BATCH];
  const int lane = threadIdx.x & 31, sl = lane % TSUB, first = lane - sl;
  if (threadIdx.x < VC_MAX_BATCH) tok_begin[threadIdx.x] = p.tok_begin[threadIdx.x];
  if (threadIdx.x < 32) tree_plan(p, &plan, lane, false);
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const int64_t all = (int64_t)p.n_tok * p.Hq;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w * (32 / TSUB) < all; w += (int64_t)gridDim.x * 8) {
    const int64_t id = w * (32 / TSUB) + lane / TSUB;
    bool live = id < all;
    TParts q{0, 0, 0, 0};
    bf16* dst = nullptr;
    if (live) q = tree_parts<D>(p, plan, tok_begin, id, dst);
    if (q.count == 1) {  // written by the piece itself
      live = false;
      q.count = 0;
    }
    const int most = __reduce_max_sync(0xffffffffu, q.count);
    auto lse_of = [&](int k) { return k >= q.count ? -INFINITY : p.ws_lse[q.at(k)]; };
    const float l0 = lse_of(sl);  // most rows have no more than a lane each
    float M = l0;
    for (int k0 = TSUB; k0 < most; k0 += TSUB) M = fmaxf(M, lse_of(k0 + sl));
#pragma unroll
    for (int off = TSUB / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float L = 0.f;
    float4 acc[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < most; k0 += TSUB) {
      const float l = k0 ? lse_of(k0 + sl) : l0, f = part_weight(l, M);
      const unsigned wrote = __ballot_sync(0xffffffffu, l != -INFINITY) >> first;
      L += f;
      const int cnt = min(TSUB, most - k0);
#pragma unroll 2
      for (int c = 0; c < cnt; ++c) {
        const float fc = __shfl_sync(0xffffffffu, f, first + c);
        if ((wrote >> c) & 1u) {  // a partial that saw nothing was not written
          const float4* src = reinterpret_cast<const float4*>(p.ws_o + q.at(k0 + c) * D) + sl;
#pragma unroll
          for (int i = 0; i < Q; ++i) {
            const float4 v = __ldcg(src + i * TSUB);
            acc[i].x = fmaf(fc, v.x, acc[i].x);
            acc[i].y = fmaf(fc, v.y, acc[i].y);
            acc[i].z = fmaf(fc, v.z, acc[i].z);
            acc[i].w = fmaf(fc, v.w, acc[i].w);
          }
        }
      }
    }
#pragma unroll
    for (int off = TSUB / 2; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    if (!live) continue;
    const float inv = L != 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (int i = 0; i < Q; ++i)
      reinterpret_cast<uint2*>(dst)[sl + i * TSUB] =
          make_uint2(pack_bf16x2(acc[i].x * inv, acc[i].y * inv), pack_bf16x2(acc[i].z * inv, acc[i].w * inv));
  }
}

// ------------------------------------------------------------------------------------------------
// bf16 pages [n_pages][Hkv][page][d] as a 3-D tensor (d, page, n_pages * Hkv); box 64 x page x 1, 128-byte swizzle.
bool page_map(CUtensorMap* m, const void* base, int d, int page, int64_t heads) {
  auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tmap_encoder());
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)page, (cuuint64_t)heads};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)page * d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)page, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int tree_sms() {
  static const int n = [] {
    int dev = 0, v = 0;
    const bool ok = cudaGetDevice(&dev) == cudaSuccess &&
                    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
    return ok ? v : 152;
  }();
  return n;
}

int64_t host_units(int64_t rows) { return (rows + TU - 1) / TU; }
int few_warps() { return tree_sms() * FCTAS * FWARPS; }
int slot_rows_of(int64_t rows) { return rows <= TM ? (int)rows : TU; }

template <int D>
cudaError_t launch_tree_t(const TreeParams& p, const TreeMaps& maps, cudaStream_t s) {
  static std::atomic<uint64_t> attr{0}, few_attr{0};
  cudaError_t e;
  if (p.few) {
    e = raise_smem_limit(tree_few_kernel<D>, FCfg<D>::SMEM, few_attr);
    if (e != cudaSuccess) return e;
    e = launch_pdl(tree_few_kernel<D>, dim3(p.n_cta / FWARPS), dim3(FWARPS * 32), FCfg<D>::SMEM, s, p);
  } else {
    e = raise_smem_limit(tree_attn_kernel<D>, TCfg<D>::SMEM, attr);
    if (e != cudaSuccess) return e;
    e = launch_pdl(tree_attn_kernel<D>, dim3(p.n_cta), dim3(TTHREADS), TCfg<D>::SMEM, s, p, maps);
  }
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)p.n_tok * p.Hq;
  if (p.merge_warps) return launch_pdl(tree_merge_kernel<D>, dim3((unsigned)((rows * p.merge_warps + 7) / 8)), dim3(256), 0, s, p);
  const int64_t blocks = (rows * TSUB + 255) / 256, wave = 4 * tree_sms();
  return launch_pdl(tree_merge_rows_kernel<D>, dim3((unsigned)(blocks < wave ? blocks : wave)), dim3(256), 0, s, p);
}

}  // namespace

// Partials: two slots a CTA, or a warp for few rows; how many rows there are in all does not matter.
size_t tree_workspace_size(const vc_shape* s, int32_t max_rows) {
  const int64_t rows = (int64_t)max_rows * (s->Hq / s->Hkv);
  const int64_t few = 2 * few_warps() * (rows < FR ? rows : FR), many = 2 * tree_sms() * (int64_t)slot_rows_of(rows);
  return (size_t)(few > many ? few : many) * (s->d + 1) * sizeof(float) + 256;
}

cudaError_t launch_tree_attn(const TreeArgs& a, cudaStream_t s, vc_status* st) {
  TreeParams p;
  TreeMaps maps;
  memset(&p, 0, sizeof(p));
  const int G = a.Hq / a.Hkv;
  p.kv = a.kv;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = G;
  p.n_tok = a.n_tok;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)a.d));
  p.dev_status = a.dev_status;
  int most = 0;
  for (int b = 0; b < a.B; ++b) most = a.req[b].n_rows > most ? a.req[b].n_rows : most;
  // Up to 8 rows, or 16 where the table has room for no more than 4096 keys, for the kernel without tensor memory (us of it
  // and of the other, call after call: 32 x 1000 keys, 4 rows a head: 31.9, 41.8; 32 x 8200 from pages of 16: 150, 156, of
  // 128: 153, 148; 8 x 32768, 8 rows, from pages of 16: 170, 173, of 64: 174, 167. With 16 rows: 32 x 200 20.9, 27.1; 32 x
  // 1000 38.9, 41.9; 32 x 8200 160, 157; 1 x 100000 86, 72: each warp's partial is written and read again)
  p.few = (int64_t)most * G <= ((int64_t)a.kv.max_pages << a.kv.shift <= 4096 ? FR : FR / 2);
  const int64_t tiles = ((int64_t)a.kv.max_pages << a.kv.shift) / (p.few ? FK : TN) + 1;
  int64_t cost = 0, units = 0, same = host_units((int64_t)a.req[0].n_rows * G);
  p.slot_rows = 1;
  p.least = 1;
  for (int b = a.B; b < VC_MAX_BATCH; ++b) p.tok_begin[b] = INT32_MAX;
  for (int b = 0; b < a.B; ++b) {
    const TreeReqDev& r = a.req[b];
    p.seq[b] = r.seq;
    p.n_rows[b] = r.n_rows;
    p.tok_begin[b] = r.tok_begin;
    p.mask_words[b] = r.mask_words;
    p.q[b] = r.q;
    p.o[b] = r.o;
    p.mask[b] = r.mask;
    const int64_t rows = (int64_t)a.req[b].n_rows * G, u = host_units(rows);
    if (u != same || rows - (u - 1) * TU <= TM) same = 1;
    if (!r.mask) p.chains |= 1u << b;
    const int sr = p.few ? (int)rows : slot_rows_of(rows);
    p.slot_rows = sr > p.slot_rows ? sr : p.slot_rows;
    if (rows > TM) p.least = 2;
    units += u * a.Hkv;
    cost += (p.few ? tiles : u * (2 * tiles + TPIECE)) * a.Hkv;
  }
  // costs are counted in 32 bits
  if (cost >= INT32_MAX / 2 || units >= INT32_MAX / 2) {
    *st = VC_ERR_UNSUPPORTED;
    return cudaSuccess;
  }
  const int sms = tree_sms();
  p.same = same > 1 && same <= sms / 2 ? (int)same : 1;
  p.n_cta = p.few ? few_warps() : sms;
  const size_t rows = 2 * (size_t)p.n_cta * p.slot_rows;
  if (!a.ws || (reinterpret_cast<uintptr_t>(a.ws) & 15u) || rows * (a.d + 1) * sizeof(float) > a.ws_bytes) {
    *st = VC_ERR_WORKSPACE;
    return cudaSuccess;
  }
  p.ws_o = static_cast<float*>(a.ws);
  p.ws_lse = p.ws_o + rows * a.d;
  // Warps a row of the merge: a row's partials, one a CTA (or warp) that holds part of its unit, by fours (one round
  // trip each); no more than make a wave of blocks. Several rows a warp where they are more than the warps of a wave.
  const int64_t parts = 1 + p.n_cta / units, out_rows = (int64_t)a.n_tok * a.Hq, wave = (int64_t)sms * 4 * 8;
  p.merge_warps = 1;
  while (p.merge_warps < 8 && parts > 4 * p.merge_warps && out_rows * p.merge_warps * 2 <= wave) p.merge_warps *= 2;
  if (out_rows > wave) p.merge_warps = 0;
  const int64_t heads = (int64_t)a.kv.n_pages * a.Hkv;
  if (!p.few && (!page_map(&maps.kv[0], a.kv.k, a.d, 1 << a.kv.shift, heads) || !page_map(&maps.kv[1], a.kv.v, a.d, 1 << a.kv.shift, heads))) {
    *st = VC_ERR_CUDA;
    return cudaSuccess;
  }
  return a.d == 128 ? launch_tree_t<128>(p, maps, s) : launch_tree_t<64>(p, maps, s);
}

}  // namespace vc
