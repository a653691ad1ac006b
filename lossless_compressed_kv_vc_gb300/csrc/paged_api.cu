// C-ABI entry points of drafted trees over a cache of pages (vc_paged_kv): argument validation and launches.
// Validation failures return a status and launch nothing.
#include "paged.cuh"

#include <math.h>
#include <string.h>

using namespace vc;

namespace {

bool a16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool a4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The shape and the pool; fills the kernels' descriptor.
vc_status check_pool(const vc_shape* s, const vc_paged_kv* kv, PagedDev* out) {
  if (!s || s->B < 1 || s->B > VC_MAX_BATCH || s->Hkv < 1 || s->Hq < s->Hkv || s->Hq % s->Hkv != 0) return VC_ERR_INVALID;
  if (!kv || !a16(kv->k) || !a16(kv->v) || !a4(kv->refs) || !a4(kv->free_pages) || !a4(kv->n_free) || !a4(kv->table) ||
      !a4(kv->len) || !a4(kv->held) || !a4(kv->next) || kv->n_pages < 1 || kv->n_seq < 1 || kv->max_pages < 1)
    return VC_ERR_INVALID;
  if (s->Hkv > 65535) return VC_ERR_UNSUPPORTED;  // a grid's second dimension
  if (s->d != 64 && s->d != 128) return VC_ERR_UNSUPPORTED;
  int shift = 4;
  while (shift < 7 && kv->page != 1 << shift) ++shift;
  if (kv->page != 1 << shift) return VC_ERR_UNSUPPORTED;
  // heads' pages are numbered in 32 bits, with room for a page beyond the last one, and so are a sequence's rows with room for a tile beyond the last
  if (((int64_t)kv->n_pages + 1) * s->Hkv > INT32_MAX || (int64_t)kv->max_pages * kv->page > (int64_t(1) << 30))
    return VC_ERR_UNSUPPORTED;
  PagedDev d;
  d.k = static_cast<bf16*>(kv->k);
  d.v = static_cast<bf16*>(kv->v);
  d.refs = kv->refs;
  d.free_pages = kv->free_pages;
  d.n_free = kv->n_free;
  d.table = kv->table;
  d.len = kv->len;
  d.held = kv->held;
  d.next = kv->next;
  d.n_pages = kv->n_pages;
  d.shift = shift;
  d.n_seq = kv->n_seq;
  d.max_pages = kv->max_pages;
  *out = d;
  return VC_OK;
}

bool has_seq(const vc_paged_kv* kv, int32_t seq) { return seq >= 0 && seq < kv->n_seq; }

// Every request's sequence is in the pool, and no two name the same.
template <typename Req>
bool seqs_ok(const vc_paged_kv* kv, const Req* req, int B) {
  for (int b = 0; b < B; ++b) {
    if (!has_seq(kv, req[b].seq)) return false;
    for (int c = 0; c < b; ++c)
      if (req[c].seq == req[b].seq) return false;
  }
  return true;
}

vc_status done(cudaError_t e, cudaStream_t stream) {
  if (e != cudaSuccess) return VC_ERR_CUDA;
  note_cache_writer(stream);
  return VC_OK;
}

size_t compact_ints(int64_t n_pages) { return (size_t)(4 + 2 * (n_pages / 2 + 1) + n_pages); }

}  // namespace

extern "C" {

vc_status vc_pages_init(const vc_shape* shape, const vc_paged_kv* kv, cudaStream_t stream) {
  PagedDev d;
  const vc_status st = check_pool(shape, kv, &d);
  return st != VC_OK ? st : done(launch_pages_init(d, stream), stream);
}

size_t vc_pages_workspace_size(const vc_shape* shape, const vc_paged_kv* kv) {
  PagedDev d;
  if (check_pool(shape, kv, &d) != VC_OK) return 0;
  const size_t reserve = shape->B * sizeof(int4), compact = (compact_ints(kv->n_pages) * sizeof(int32_t) + 15) / 16 * 16;
  return reserve > compact ? reserve : compact;
}

vc_status vc_pages_reserve(const vc_shape* shape, const vc_paged_kv* kv, const vc_reserve_req* req, void* ws,
                           size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  ReserveParams p;
  memset(&p, 0, sizeof(p));
  const vc_status st = check_pool(shape, kv, &p.kv);
  if (st != VC_OK) return st;
  if (!req || !seqs_ok(kv, req, shape->B)) return VC_ERR_INVALID;
  for (int b = 0; b < shape->B; ++b) {
    if (req[b].rows < 0) return VC_ERR_INVALID;
    p.req[b] = req[b];
  }
  if (!a16(ws) || ws_bytes < shape->B * sizeof(int4)) return VC_ERR_WORKSPACE;
  p.copies = static_cast<int4*>(ws);
  p.B = shape->B;
  p.Hkv = shape->Hkv;
  p.dev_status = dev_status;
  return done(launch_reserve(p, shape->d, stream), stream);
}

vc_status vc_pages_fork(const vc_shape* shape, const vc_paged_kv* kv, const vc_fork_req* req, int32_t* dev_status,
                        cudaStream_t stream) {
  ForkParams p;
  memset(&p, 0, sizeof(p));
  const vc_status st = check_pool(shape, kv, &p.kv);
  if (st != VC_OK) return st;
  if (!req) return VC_ERR_INVALID;
  for (int b = 0; b < shape->B; ++b) {
    if (!has_seq(kv, req[b].src) || !has_seq(kv, req[b].dst)) return VC_ERR_INVALID;
    for (int c = 0; c < shape->B; ++c)
      if (req[c].src == req[b].dst || (c != b && req[c].dst == req[b].dst)) return VC_ERR_INVALID;
    p.req[b] = req[b];
  }
  p.dev_status = dev_status;
  return done(launch_fork(p, shape->B, stream), stream);
}

vc_status vc_pages_trim(const vc_shape* shape, const vc_paged_kv* kv, const vc_trim_req* req, int32_t* dev_status,
                        cudaStream_t stream) {
  TrimParams p;
  memset(&p, 0, sizeof(p));
  const vc_status st = check_pool(shape, kv, &p.kv);
  if (st != VC_OK) return st;
  if (!req || !seqs_ok(kv, req, shape->B)) return VC_ERR_INVALID;
  // pages given back are numbered in 32 bits, with room for a step of the block beyond the last one
  if ((int64_t)shape->B * kv->max_pages > INT32_MAX - 1024) return VC_ERR_UNSUPPORTED;
  for (int b = 0; b < shape->B; ++b) {
    if (req[b].rows < 0) return VC_ERR_INVALID;
    p.req[b] = req[b];
  }
  p.B = shape->B;
  p.dev_status = dev_status;
  return done(launch_trim(p, stream), stream);
}

vc_status vc_pages_compact(const vc_shape* shape, const vc_paged_kv* kv, void* ws, size_t ws_bytes, int32_t* dev_status,
                           cudaStream_t stream) {
  CompactParams p;
  memset(&p, 0, sizeof(p));
  const vc_status st = check_pool(shape, kv, &p.kv);
  if (st != VC_OK) return st;
  if (!a16(ws) || ws_bytes < compact_ints(kv->n_pages) * sizeof(int32_t)) return VC_ERR_WORKSPACE;
  const int64_t room = kv->n_pages / 2 + 1;
  p.Hkv = shape->Hkv;
  p.head = static_cast<int32_t*>(ws);
  p.hole = p.head + 4;
  p.from = p.hole + room;
  p.back = p.from + room;
  p.dev_status = dev_status;
  return done(launch_compact(p, shape->d, stream), stream);
}

// ---------------------------------------------------------------------------------------------
vc_status vc_rope_axes_init(const vc_rope* rope, int32_t n_axes, const int32_t* sections, int32_t dealt,
                            vc_rope_axes* out) {
  if (!rope || !sections || !out || n_axes < 1 || n_axes > VC_ROPE_MAX_AXES || (dealt != 0 && dealt != 1)) return VC_ERR_INVALID;
  if (rope->rot_dim < 16 || rope->rot_dim > 2 * VC_ROPE_MAX_PAIRS || rope->rot_dim % 16 != 0) return VC_ERR_UNSUPPORTED;
  const int pairs = rope->rot_dim / 2;
  int64_t sum = 0;
  int left[VC_ROPE_MAX_AXES];
  for (int a = 0; a < n_axes; ++a) {
    if (sections[a] < 0) return VC_ERR_INVALID;
    sum += left[a] = sections[a];
  }
  if (sum != pairs) return VC_ERR_INVALID;
  vc_rope_axes r;
  memset(&r, 0, sizeof(r));
  r.rope = *rope;
  r.n_axes = n_axes;
  for (int j = 0, a = 0; j < pairs; ++j) {
    while (left[a] == 0) a = (a + 1) % n_axes;
    --left[a];
    r.axis[j] = a;
    if (dealt) a = (a + 1) % n_axes;
  }
  *out = r;
  return VC_OK;
}

vc_status vc_rope_pages(const vc_shape* shape, const vc_rope_axes* axes, const vc_paged_kv* kv,
                        const vc_rope_page_req* req, int32_t* dev_status, cudaStream_t stream) {
  RopePageParams p;
  memset(&p, 0, sizeof(p));
  const vc_status st = check_pool(shape, kv, &p.kv);
  if (st != VC_OK) return st;
  if (!axes || !req || !seqs_ok(kv, req, shape->B)) return VC_ERR_INVALID;
  const vc_rope& rope = axes->rope;
  if (rope.layout != VC_ROPE_HALF && rope.layout != VC_ROPE_INTERLEAVED) return VC_ERR_INVALID;
  if (rope.rot_dim < 16 || rope.rot_dim > shape->d || rope.rot_dim % 16 != 0) return VC_ERR_UNSUPPORTED;
  if (!isfinite((float)rope.amp) || axes->n_axes < 1 || axes->n_axes > VC_ROPE_MAX_AXES) return VC_ERR_INVALID;
  // a token's 16-byte pieces are numbered in 32 bits, with room for a step beyond the last one
  if (((int64_t)shape->Hq + 2 * (int64_t)shape->Hkv) * (shape->d / 8) > (int64_t(1) << 30)) return VC_ERR_UNSUPPORTED;
  p.Hq = shape->Hq;
  p.Hkv = shape->Hkv;
  p.rot = rope.rot_dim;
  p.inter = rope.layout == VC_ROPE_INTERLEAVED;
  p.amp = (float)rope.amp;
  p.dev_status = dev_status;
  for (int j = 0; j < rope.rot_dim / 2; ++j) {
    if (!isfinite(rope.freq[j]) || axes->axis[j] < 0 || axes->axis[j] >= axes->n_axes) return VC_ERR_INVALID;
    p.turns[j] = rope.freq[j] / (2 * M_PI);
    p.axis[j / 32] |= (uint64_t)axes->axis[j] << (2 * (j % 32));
    static_assert(VC_ROPE_MAX_AXES <= 4 && VC_ROPE_MAX_PAIRS == 64, "two bits a pair");
  }
  int64_t total = 0;
  int n = 0;
  for (int b = 0; b < shape->B; ++b) {
    const vc_rope_page_req& r = req[b];
    if (r.n_rows < 0) return VC_ERR_INVALID;
    if (r.n_rows == 0) continue;
    const int64_t wq = (int64_t)shape->Hq * shape->d, wk = (int64_t)shape->Hkv * shape->d;
    if (!r.q != !r.q_out || (r.q && (!a16(r.q) || !a16(r.q_out))) || !a16(r.k) || !a16(r.v)) return VC_ERR_INVALID;
    const int64_t qs = r.q_stride ? r.q_stride : wq, ks = r.k_stride ? r.k_stride : wk, vs = r.v_stride ? r.v_stride : wk;
    // a token's heads do not reach into the next token's, and every token starts 16-byte aligned
    if (qs < wq || ks < wk || vs < wk || ((qs | ks | vs) & 7)) return VC_ERR_INVALID;
    if (r.q && r.q_out == r.q && qs != wq) return VC_ERR_INVALID;
    if (r.off && (!a4(r.off) || (r.off_stride != 0 && r.off_stride < r.n_rows))) return VC_ERR_INVALID;
    RopePageReqDev& e = p.req[n];
    e.q = static_cast<const bf16*>(r.q);
    e.k = static_cast<const bf16*>(r.k);
    e.v = static_cast<const bf16*>(r.v);
    e.q_stride = qs;
    e.k_stride = ks;
    e.v_stride = vs;
    e.off = r.off;
    e.off_stride = r.off_stride;
    e.q_out = static_cast<bf16*>(r.q_out);
    e.seq = r.seq;
    p.tok_begin[n++] = (int32_t)total;
    total += r.n_rows;
    if (total > (int64_t(1) << 30)) return VC_ERR_UNSUPPORTED;
  }
  while (n < VC_MAX_BATCH) p.tok_begin[n++] = INT32_MAX;
  p.n_tok = (int32_t)total;
  return total == 0 ? VC_OK : done(launch_rope_pages(p, shape->d, stream), stream);
}

// ---------------------------------------------------------------------------------------------
static vc_status check_trees(int32_t B, int32_t N_max, const void* parent, const void* n_nodes) {
  if (B < 1 || N_max < 1 || !a4(parent) || !a4(n_nodes)) return VC_ERR_INVALID;
  return N_max > VC_TREE_MAX_NODES || (int64_t)B * N_max > (int64_t(1) << 30) ? VC_ERR_UNSUPPORTED : VC_OK;
}

vc_status vc_tree_mask(int32_t B, int32_t N_max, const int32_t* parent, const int32_t* n_nodes, uint32_t* mask,
                       int32_t* depth, cudaStream_t stream) {
  const vc_status st = check_trees(B, N_max, parent, n_nodes);
  if (st != VC_OK) return st;
  if (!a4(mask) || (depth && !a4(depth))) return VC_ERR_INVALID;
  const TreeMaskArgs a{parent, n_nodes, mask, depth, B, N_max};
  return done(launch_tree_mask(a, stream), stream);
}

vc_status vc_tree_accept(int32_t B, int32_t N_max, int32_t V, const float* logits, const int32_t* token,
                         const int32_t* parent, const int32_t* n_nodes, int32_t* out_tokens, int32_t* path,
                         int32_t* n_acc, cudaStream_t stream) {
  const vc_status st = check_trees(B, N_max, parent, n_nodes);
  if (st != VC_OK) return st;
  if (V < 1 || !a4(logits) || !a4(token) || !a4(out_tokens) || !a4(path) || !a4(n_acc)) return VC_ERR_INVALID;
  const TreeAcceptArgs a{logits, token, parent, n_nodes, out_tokens, path, n_acc, B, N_max, V};
  return done(launch_tree_accept(a, stream), stream);
}

vc_status vc_tree_commit(const vc_shape* shape, const vc_paged_kv* kv, const vc_commit_req* req, int32_t* dev_status,
                         cudaStream_t stream) {
  CommitParams p;
  memset(&p, 0, sizeof(p));
  const vc_status st = check_pool(shape, kv, &p.kv);
  if (st != VC_OK) return st;
  if (!req || !seqs_ok(kv, req, shape->B)) return VC_ERR_INVALID;
  int n = 0;
  for (int b = 0; b < shape->B; ++b) {
    if (req[b].n_rows < 0 || (req[b].path && !a4(req[b].path)) || (req[b].n_acc && !a4(req[b].n_acc))) return VC_ERR_INVALID;
    if (req[b].n_rows > 0) p.req[n++] = req[b];
  }
  p.Hkv = shape->Hkv;
  p.dev_status = dev_status;
  return n == 0 ? VC_OK : done(launch_commit(p, n, shape->d, stream), stream);
}

// ---------------------------------------------------------------------------------------------
size_t vc_tree_workspace_size(const vc_shape* shape, int32_t max_rows) {
  if (!shape || shape->B < 1 || shape->B > VC_MAX_BATCH || shape->Hkv < 1 || shape->Hkv > 65535 || shape->Hq < shape->Hkv ||
      shape->Hq % shape->Hkv != 0 || (shape->d != 64 && shape->d != 128) || max_rows < 1)
    return 0;
  return tree_workspace_size(shape, max_rows);
}

vc_status vc_tree_attn(const vc_shape* shape, const vc_paged_kv* kv, const vc_tree_req* req, void* ws, size_t ws_bytes,
                       int32_t* dev_status, cudaStream_t stream) {
  TreeArgs a;
  memset(&a, 0, sizeof(a));
  vc_status st = check_pool(shape, kv, &a.kv);
  if (st != VC_OK) return st;
  if (!req) return VC_ERR_INVALID;
  int64_t total = 0;
  for (int b = 0; b < shape->B; ++b) {
    const vc_tree_req& r = req[b];
    if (!has_seq(kv, r.seq) || r.n_rows < 0) return VC_ERR_INVALID;
    if (r.n_rows == 0) continue;
    if (!a16(r.q) || !a16(r.o)) return VC_ERR_INVALID;
    if (r.mask && (!a4(r.mask) || r.mask_words < 0 || (int64_t)r.mask_words * 32 < r.n_rows)) return VC_ERR_INVALID;
    TreeReqDev& e = a.req[a.B++];
    e.q = static_cast<const bf16*>(r.q);
    e.o = static_cast<bf16*>(r.o);
    e.mask = r.mask;
    e.mask_words = r.mask_words;
    e.seq = r.seq;
    e.n_rows = r.n_rows;
    e.tok_begin = (int32_t)total;
    total += r.n_rows;
    // query rows are numbered in 32 bits
    if (total * shape->Hq > (int64_t(1) << 29)) return VC_ERR_UNSUPPORTED;
  }
  if (total == 0) return VC_OK;
  a.Hq = shape->Hq;
  a.Hkv = shape->Hkv;
  a.d = shape->d;
  a.n_tok = (int32_t)total;
  a.ws = ws;
  a.ws_bytes = ws_bytes;
  a.dev_status = dev_status;
  const cudaError_t e = launch_tree_attn(a, stream, &st);
  return st != VC_OK ? st : done(e, stream);
}

}  // extern "C"
