// Attention of new rows over live caches and an optional shared prefix; with the scores of eviction.
//
// Row i of a request's n_rows rows sees every prefix row and own rows t <= n - n_rows + i:
//   s_t = q . k_t / sqrt(d),  o = sum_t 2^(s_t - lse) v_t  (log2 domain),  score[t] += sum_rows 2^(s_t - lse).
// One CTA takes one (token, query head): its warps stride over the keys with a running maximum and sum
// each and meet in shared memory; a second kernel takes the scores' sums, a warp per key.
#include "vc_internal.cuh"

#include <math.h>

namespace vc {

constexpr int kLiveWarps = 8;

template <int D>
__device__ __forceinline__ float row_dot(const float (&q)[D / 32], const bf16* k, int lane) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) s = fmaf(q[e], __bfloat162float(k[e * 32 + lane]), s);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}

__device__ __forceinline__ int live_req_of(const LiveArgs& p, int tok) {
  int b = 0;
#pragma unroll 1
  for (int i = 1; i < p.B; ++i)
    if (p.req[i].tok_begin <= tok) b = i;
  return b;
}

template <int D>
__global__ void __launch_bounds__(kLiveWarps * 32) live_rows_kernel(const __grid_constant__ LiveArgs p, float scale, float* lse) {
  constexpr int E = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int tok = blockIdx.x, hq = blockIdx.y, hk = hq / (p.Hq / p.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const LiveReqDev& r = p.req[live_req_of(p, tok)];
  const int i = tok - r.tok_begin;
  float q[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(r.q[((size_t)i * p.Hq + hq) * D + e * 32 + lane]) * scale;
    acc[e] = 0.f;
  }
  auto over = [&](const bf16* k, const bf16* v, int n) {
    for (int t = warp; t < n; t += kLiveWarps) {
      const float s = row_dot<D>(q, k + (size_t)t * D, lane);
      const float mn = fmaxf(m, s);
      const float f = m == -INFINITY ? 0.f : exp2f(m - mn), w = mn == -INFINITY ? 0.f : exp2f(s - mn);
      m = mn;
      l = l * f + w;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + w * __bfloat162float(v[(size_t)t * D + e * 32 + lane]);
    }
  };
  if (p.pn > 0) over(p.pk + (size_t)hk * p.pcap * D, p.pv + (size_t)hk * p.pcap * D, p.pn);
  over(r.k + (size_t)hk * r.cap * D, r.v + (size_t)hk * r.cap * D, r.n - r.n_rows + i + 1);
  __shared__ float sm[kLiveWarps], sl[kLiveWarps], so[kLiveWarps][D];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][e * 32 + lane] = acc[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kLiveWarps; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < kLiveWarps; ++w)
    if (sl[w] != 0.f) L += sl[w] * exp2f(sm[w] - M);
  for (int c = threadIdx.x; c < D; c += kLiveWarps * 32) {
    float o = 0.f;
    for (int w = 0; w < kLiveWarps; ++w)
      if (sl[w] != 0.f) o += so[w][c] * exp2f(sm[w] - M);
    r.o[((size_t)i * p.Hq + hq) * D + c] = __float2bfloat16(L != 0.f ? o / L : 0.f);
  }
  if (lse && threadIdx.x == 0) lse[(size_t)tok * p.Hq + hq] = L != 0.f ? M + log2f(L) : INFINITY;
}

template <int D>
__global__ void __launch_bounds__(256) live_score_kernel(const __grid_constant__ LiveArgs p, float scale, const float* lse) {
  constexpr int E = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int hk = blockIdx.y, G = p.Hq / p.Hkv, lane = threadIdx.x & 31;
  const LiveReqDev& r = p.req[blockIdx.z];
  for (int t = blockIdx.x * 8 + (threadIdx.x >> 5); t < r.n && r.n_rows > 0; t += gridDim.x * 8) {
    const bf16* k = r.k + ((size_t)hk * r.cap + t) * D;
    float w = 0.f;
    for (int i = max(0, t - (r.n - r.n_rows)); i < r.n_rows; ++i)
      for (int g = 0; g < G; ++g) {
        const size_t row = (size_t)i * p.Hq + hk * G + g;
        float q[E];
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] = __bfloat162float(r.q[row * D + e * 32 + lane]) * scale;
        w += exp2f(row_dot<D>(q, k, lane) - lse[(size_t)r.tok_begin * p.Hq + row]);
      }
    if (lane == 0) r.score[(size_t)hk * r.cap + t] += w;
  }
}

size_t live_workspace_size(const vc_shape* s, int32_t max_rows, int32_t max_n, bool scored) {
  return scored ? (size_t)s->B * max_rows * s->Hq * sizeof(float) + 16 : 16;
}

template <int D>
static cudaError_t launch_live_t(const LiveArgs& a, bool scored, cudaStream_t s) {
  const float scale = (float)(1.4426950408889634 / sqrt((double)D));
  float* lse = scored ? static_cast<float*>(a.ws) : nullptr;
  cudaError_t e = launch_pdl(live_rows_kernel<D>, dim3(a.n_tok, a.Hq), dim3(kLiveWarps * 32), 0, s, a, scale, lse);
  if (e != cudaSuccess || !scored) return e;
  int n = 1;
  for (int b = 0; b < a.B; ++b) n = a.req[b].n > n ? a.req[b].n : n;
  const int gx = (n + 7) / 8 < 1024 ? (n + 7) / 8 : 1024;
  return launch_pdl(live_score_kernel<D>, dim3(gx, a.Hkv, a.B), dim3(256), 0, s, a, scale, (const float*)lse);
}

cudaError_t launch_live_attn(const LiveArgs& a, bool scored, cudaStream_t s, vc_status* st) {
  const size_t need = scored ? (size_t)a.n_tok * a.Hq * sizeof(float) : 0;
  if (need && ((reinterpret_cast<uintptr_t>(a.ws) & 15u) || !a.ws || a.ws_bytes < need)) {
    *st = VC_ERR_WORKSPACE;
    return cudaSuccess;
  }
  return a.d == 128 ? launch_live_t<128>(a, scored, s) : launch_live_t<64>(a, scored, s);
}

}  // namespace vc
