// C-ABI entry points of the caches that grow, are shared and shrink (vc_live_kv): argument validation
// and launches. Validation failures return a status and launch nothing.
#include "vc_internal.cuh"

#include <math.h>
#include <string.h>

using namespace vc;

namespace {

bool a16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool a4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

vc_status check_shape(const vc_shape* s) {
  if (!s || s->B < 1 || s->B > VC_MAX_BATCH || s->Hkv < 1 || s->Hq < s->Hkv || s->Hq % s->Hkv != 0) return VC_ERR_INVALID;
  if (s->Hkv > 65535) return VC_ERR_UNSUPPORTED;  // a grid's second dimension
  return s->d == 64 || s->d == 128 ? VC_OK : VC_ERR_UNSUPPORTED;
}

// The cache's own fields; score and pos, where present, are element-aligned.
bool kv_ok(const vc_live_kv& c) {
  return a16(c.k) && a16(c.v) && c.cap >= 1 && c.n >= 0 && c.n <= c.cap && (!c.score || a4(c.score)) &&
         (!c.pos || a4(c.pos));
}

// Kernels count a head's rows in 32 bits, with room for a tile beyond the last one.
constexpr int32_t kMaxRows = 1 << 30;

// Fills the requests of an attention call.
vc_status fill_live(const vc_shape* shape, const vc_live_req* req, bool scored, LiveArgs* a) {
  const int G = shape->Hq / shape->Hkv;
  int64_t total = 0;
  for (int b = 0; b < shape->B; ++b) {
    const vc_live_req& r = req[b];
    if (!kv_ok(r.kv) || r.n_rows < 0) return VC_ERR_INVALID;
    if (r.n_rows > 0 && (!a16(r.q) || !a16(r.o))) return VC_ERR_INVALID;
    if (scored && !r.kv.score) return VC_ERR_INVALID;
    if (r.kv.n > kMaxRows) return VC_ERR_UNSUPPORTED;
    if (scored && (int64_t)r.n_rows * G > VC_SCORED_MAX_ROWS) return VC_ERR_UNSUPPORTED;
    LiveReqDev& e = a->req[b];
    e.q = static_cast<const bf16*>(r.q);
    e.o = static_cast<bf16*>(r.o);
    e.k = static_cast<const bf16*>(r.kv.k);
    e.v = static_cast<const bf16*>(r.kv.v);
    e.score = r.kv.score;
    e.cap = r.kv.cap;
    e.n = r.kv.n;
    e.n_rows = r.n_rows;
    e.tok_begin = (int32_t)total;
    total += r.n_rows;
    // query rows of one KV head are numbered in 32 bits
    if (total * G > (int64_t(1) << 30)) return VC_ERR_UNSUPPORTED;
  }
  a->B = shape->B;
  a->Hq = shape->Hq;
  a->Hkv = shape->Hkv;
  a->d = shape->d;
  a->n_tok = (int32_t)total;
  return VC_OK;
}

vc_status run_live(LiveArgs& a, bool scored, void* ws, size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  if (a.n_tok == 0) return VC_OK;
  a.ws = ws;
  a.ws_bytes = ws_bytes;
  a.dev_status = dev_status;
  vc_status st = VC_OK;
  const cudaError_t e = launch_live_attn(a, scored, stream, &st);
  if (st != VC_OK) return st;
  if (e != cudaSuccess) return VC_ERR_CUDA;
  note_cache_writer(stream);  // o may be what a later step reads as its queries
  return VC_OK;
}

}  // namespace

extern "C" {

vc_status vc_rope_init(const vc_rope_config* c, vc_rope* out) {
  if (!c || !out) return VC_ERR_INVALID;
  if (c->kind < VC_ROPE_NONE || c->kind > VC_ROPE_BANDS) return VC_ERR_INVALID;
  if (c->layout != VC_ROPE_HALF && c->layout != VC_ROPE_INTERLEAVED) return VC_ERR_INVALID;
  if (!(c->base > 0) || !isfinite(c->base) || !isfinite((float)c->amp)) return VC_ERR_INVALID;
  if (c->kind != VC_ROPE_NONE && (!(c->factor > 0) || !isfinite(c->factor))) return VC_ERR_INVALID;
  if (c->kind == VC_ROPE_BANDS && (c->orig_ctx < 1 || !(c->low >= 0) || !(c->high > c->low) || !isfinite(c->high)))
    return VC_ERR_INVALID;
  const int rot = c->rot_dim;
  if (rot < 16 || rot > 2 * VC_ROPE_MAX_PAIRS || rot % 16 != 0) return VC_ERR_UNSUPPORTED;
  memset(out, 0, sizeof(*out));
  out->rot_dim = rot;
  out->layout = c->layout;
  out->amp = c->amp;
  const double base = c->kind == VC_ROPE_NTK ? c->base * pow(c->factor, (double)rot / (rot - 2)) : c->base;
  for (int j = 0; j < rot / 2; ++j) {
    double th = pow(base, -2.0 * j / rot);
    if (c->kind == VC_ROPE_LINEAR) th /= c->factor;
    if (c->kind == VC_ROPE_BANDS) {
      const double r = c->orig_ctx * th / (2 * M_PI);
      const double m = fmin(fmax((r - c->low) / (c->high - c->low), 0.0), 1.0);
      th = m * th + (1 - m) * th / c->factor;
    }
    out->freq[j] = th;
  }
  return VC_OK;
}

vc_status vc_rope_append(const vc_shape* shape, const vc_rope* rope, const vc_rope_req* req, cudaStream_t stream) {
  const vc_status st = check_shape(shape);
  if (st != VC_OK) return st;
  if (!rope || !req || (rope->layout != VC_ROPE_HALF && rope->layout != VC_ROPE_INTERLEAVED)) return VC_ERR_INVALID;
  if (rope->rot_dim < 16 || rope->rot_dim > shape->d || rope->rot_dim % 16 != 0) return VC_ERR_UNSUPPORTED;
  if (!isfinite((float)rope->amp)) return VC_ERR_INVALID;
  // a token's 16-byte pieces are numbered in 32 bits, with room for a step beyond the last one
  if (((int64_t)shape->Hq + 2 * (int64_t)shape->Hkv) * (shape->d / 8) > (int64_t(1) << 30)) return VC_ERR_UNSUPPORTED;
  RopeParams p;
  memset(&p, 0, sizeof(p));
  p.Hq = shape->Hq;
  p.Hkv = shape->Hkv;
  p.rot = rope->rot_dim;
  p.inter = rope->layout == VC_ROPE_INTERLEAVED;
  p.amp = (float)rope->amp;
  for (int j = 0; j < rope->rot_dim / 2; ++j) {
    if (!isfinite(rope->freq[j])) return VC_ERR_INVALID;
    p.turns[j] = rope->freq[j] / (2 * M_PI);
  }
  int64_t total = 0;
  for (int b = 0; b < shape->B; ++b) {
    const vc_rope_req& r = req[b];
    if (r.n_rows < 0 || !kv_ok(r.kv) || (int64_t)r.kv.n + r.n_rows > r.kv.cap) return VC_ERR_INVALID;
    if (r.n_rows == 0) continue;
    const int64_t wq = (int64_t)shape->Hq * shape->d, wk = (int64_t)shape->Hkv * shape->d;
    if (!r.q != !r.q_out || (r.q && (!a16(r.q) || !a16(r.q_out))) || !a16(r.k) || !a16(r.v)) return VC_ERR_INVALID;
    const int64_t qs = r.q_stride ? r.q_stride : wq, ks = r.k_stride ? r.k_stride : wk, vs = r.v_stride ? r.v_stride : wk;
    // a token's heads do not reach into the next token's, and every token starts 16-byte aligned
    if (qs < wq || ks < wk || vs < wk || ((qs | ks | vs) & 7)) return VC_ERR_INVALID;
    if (r.q && r.q_out == r.q && qs != wq) return VC_ERR_INVALID;
    if (r.pos ? !a4(r.pos) : (int64_t)r.pos0 + r.n_rows - 1 > INT32_MAX) return VC_ERR_INVALID;
    RopeReqDev& e = p.req[p.B];
    e.q = static_cast<const bf16*>(r.q);
    e.k = static_cast<const bf16*>(r.k);
    e.v = static_cast<const bf16*>(r.v);
    e.q_stride = qs;
    e.k_stride = ks;
    e.v_stride = vs;
    e.pos = r.pos;
    e.pos0 = r.pos0;
    e.q_out = static_cast<bf16*>(r.q_out);
    e.kc = static_cast<bf16*>(r.kv.k) + (size_t)r.kv.n * shape->d;
    e.vc = static_cast<bf16*>(r.kv.v) + (size_t)r.kv.n * shape->d;
    e.score = r.kv.score ? r.kv.score + r.kv.n : nullptr;
    e.cpos = r.kv.pos ? r.kv.pos + r.kv.n : nullptr;
    e.cap = r.kv.cap;
    e.tok_begin = (int32_t)total;
    total += r.n_rows;
    if (total > (int64_t(1) << 30)) return VC_ERR_UNSUPPORTED;
    ++p.B;
  }
  p.n_tok = (int32_t)total;
  if (total == 0) return VC_OK;
  if (launch_rope(p, shape->d, stream) != cudaSuccess) return VC_ERR_CUDA;
  note_cache_writer(stream);
  return VC_OK;
}

// ---------------------------------------------------------------------------------------------
size_t vc_prefix_workspace_size(const vc_shape* shape, int32_t max_rows) {
  if (check_shape(shape) != VC_OK || max_rows < 1) return 0;
  return live_workspace_size(shape, max_rows, 0, false);
}

size_t vc_scored_workspace_size(const vc_shape* shape, int32_t max_rows, int32_t max_n) {
  if (check_shape(shape) != VC_OK || max_rows < 1 || max_n < 0) return 0;
  if ((int64_t)max_rows * (shape->Hq / shape->Hkv) > VC_SCORED_MAX_ROWS) return 0;
  return live_workspace_size(shape, max_rows, max_n, true);
}

vc_status vc_prefix_attn(const vc_shape* shape, const vc_kv_full* prefix, const vc_live_req* req, void* ws,
                         size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  vc_status st = check_shape(shape);
  if (st != VC_OK) return st;
  if (!req) return VC_ERR_INVALID;
  LiveArgs a;
  memset(&a, 0, sizeof(a));
  if (prefix && prefix->ctx != 0) {
    if (!a16(prefix->k) || !a16(prefix->v) || prefix->ctx < 0 || prefix->cap < prefix->ctx) return VC_ERR_INVALID;
    if (prefix->ctx > kMaxRows) return VC_ERR_UNSUPPORTED;
    a.pk = static_cast<const bf16*>(prefix->k);
    a.pv = static_cast<const bf16*>(prefix->v);
    a.pcap = prefix->cap;
    a.pn = prefix->ctx;
  }
  st = fill_live(shape, req, false, &a);
  return st != VC_OK ? st : run_live(a, false, ws, ws_bytes, dev_status, stream);
}

vc_status vc_scored_attn(const vc_shape* shape, const vc_live_req* req, void* ws, size_t ws_bytes,
                         int32_t* dev_status, cudaStream_t stream) {
  vc_status st = check_shape(shape);
  if (st != VC_OK) return st;
  if (!req) return VC_ERR_INVALID;
  LiveArgs a;
  memset(&a, 0, sizeof(a));
  st = fill_live(shape, req, true, &a);
  return st != VC_OK ? st : run_live(a, true, ws, ws_bytes, dev_status, stream);
}

// ---------------------------------------------------------------------------------------------
// A head's plan: the number of moves (padded to 16 bytes), then as many destinations and sources as a
// budget of half the rows can need.
static size_t evict_plan_ints(int64_t n) { return (size_t)((n + 3) / 4 * 4 + 8); }

size_t vc_evict_workspace_size(const vc_shape* shape, int32_t max_n) {
  if (check_shape(shape) != VC_OK || max_n < 0) return 0;
  return (size_t)shape->B * shape->Hkv * evict_plan_ints(max_n) * sizeof(int32_t);
}

vc_status vc_evict_kv(const vc_shape* shape, const vc_evict_req* req, void* ws, size_t ws_bytes, int32_t* dev_status,
                      cudaStream_t stream) {
  const vc_status st = check_shape(shape);
  if (st != VC_OK) return st;
  if (!req) return VC_ERR_INVALID;
  EvictParams p;
  memset(&p, 0, sizeof(p));
  p.Hkv = shape->Hkv;
  p.dev_status = dev_status;
  size_t ints = 0;
  for (int b = 0; b < shape->B; ++b) {
    const vc_evict_req& r = req[b];
    if (!kv_ok(r.kv) || !r.kv.score || !r.kv.pos || r.keep < 1) return VC_ERR_INVALID;
    if (r.kv.n <= r.keep) continue;
    if (r.kv.n > kMaxRows) return VC_ERR_UNSUPPORTED;
    EvictReqDev& e = p.req[p.B++];
    e.k = static_cast<bf16*>(r.kv.k);
    e.v = static_cast<bf16*>(r.kv.v);
    e.score = r.kv.score;
    e.pos = r.kv.pos;
    e.plan = static_cast<int32_t*>(ws) + ints;  // checked against the workspace below
    e.cap = r.kv.cap;
    e.n = r.kv.n;
    e.keep = r.keep;
    e.sink = r.sink;
    e.recent_from = r.recent_from;
    e.room = r.keep < r.kv.n - r.keep ? r.keep : r.kv.n - r.keep;
    e.plan_stride = (int64_t)evict_plan_ints(r.kv.n);
    ints += (size_t)shape->Hkv * e.plan_stride;
  }
  if (p.B == 0) return VC_OK;
  if (!a16(ws) || ws_bytes < ints * sizeof(int32_t)) return VC_ERR_WORKSPACE;
  if (launch_evict(p, shape->d, stream) != cudaSuccess) return VC_ERR_CUDA;
  note_cache_writer(stream);
  return VC_OK;
}

}  // extern "C"
