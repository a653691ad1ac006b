// Rotary positions of new tokens, written to the cache.
//
// Pair j of a head's rotated channels (a, b) at position p becomes
//   (a c - b s, a s + b c),  c = amp cos(p theta_j), s = amp sin(p theta_j).
// The angle is taken in turns, p theta_j / 2 pi, in fp64 and reduced to [-1/2, 1/2] there, so that a far
// position loses nothing; cos and sin of the remainder are fp32 (cospi, sinpi).
//
// A CTA takes one token: its rot / 2 angles are computed once, in shared memory, for all of the token's
// query and key heads. It is a copy otherwise: every q, k and v element is read and written once, so it is
// bound by DRAM. A thread's first pieces are on their way while the angles are made (prompt chunks, 336 MB: 59.0
// us without that, 51.6 with it, 0.96 of the copy rate; with two or three items a thread in flight, and fewer
// CTAs on an SM for their registers, 60 and 58).
#include "vc_internal.cuh"

namespace vc {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ float2 bf2_unpack(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// One or two 16-byte pieces of a head: a group of eight channels and, in the half layout, its partner
// rot / 2 higher (`pair` pieces on); cs: the first of the group's pairs, -1: passes through.
struct RopeItem {
  const uint4* src;
  uint4* dst;
  int pair, cs;
};

template <int D>
__device__ __forceinline__ RopeItem rope_item(const RopeParams& p, const RopeReqDev& r, int t, int i, int per) {
  const int nq = r.q ? p.Hq * per : 0, nk = p.Hkv * per;
  RopeItem e;
  int c;
  if (i < nq) {
    const int h = i / per;
    c = i - h * per;
    e.src = reinterpret_cast<const uint4*>(r.q + t * r.q_stride + (int64_t)h * D);
    e.dst = reinterpret_cast<uint4*>(r.q_out + ((int64_t)t * p.Hq + h) * D);
  } else if (i < nq + nk) {
    const int h = (i - nq) / per;
    c = i - nq - h * per;
    e.src = reinterpret_cast<const uint4*>(r.k + t * r.k_stride + (int64_t)h * D);
    e.dst = reinterpret_cast<uint4*>(r.kc + (h * r.cap + t) * D);
  } else {
    const int h = (i - nq - nk) / (D / 8);
    c = (i - nq - nk) % (D / 8);
    e.src = reinterpret_cast<const uint4*>(r.v + t * r.v_stride + (int64_t)h * D) + c;
    e.dst = reinterpret_cast<uint4*>(r.vc + (h * r.cap + t) * D) + c;
    e.pair = 0;
    e.cs = -1;
    return e;
  }
  const int half = p.rot / 16;  // pieces of half the rotated channels
  if (p.inter) {
    e.pair = 0;
    e.cs = 8 * c < p.rot ? 4 * c : -1;
  } else {
    e.pair = c < half ? half : 0;
    e.cs = c < half ? 8 * c : -1;
    if (c >= half) c += half;  // passes through: pieces rot / 8 on
  }
  e.src += c;
  e.dst += c;
  return e;
}

__device__ __forceinline__ void rope_turn(const RopeItem& e, uint4& x, uint4& y, const float2* cs) {
  if (e.cs < 0) return;
  uint32_t *wx = reinterpret_cast<uint32_t*>(&x), *wy = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = bf2_unpack(wx[k]);
    if (e.pair) {
      const float2 b = bf2_unpack(wy[k]), t0 = cs[e.cs + 2 * k], t1 = cs[e.cs + 2 * k + 1];
      wx[k] = pack_bf16x2(a.x * t0.x - b.x * t0.y, a.y * t1.x - b.y * t1.y);
      wy[k] = pack_bf16x2(a.x * t0.y + b.x * t0.x, a.y * t1.y + b.y * t1.x);
    } else {
      const float2 t = cs[e.cs + k];
      wx[k] = pack_bf16x2(a.x * t.x - a.y * t.y, a.x * t.y + a.y * t.x);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs[VC_ROPE_MAX_PAIRS];
  const int tok = blockIdx.x;
  int b = 0;
#pragma unroll 1
  for (int i = 1; i < p.B; ++i)
    if (p.req[i].tok_begin <= tok) b = i;
  const RopeReqDev& r = p.req[b];
  const int t = tok - r.tok_begin;
  const int per = p.inter ? D / 8 : D / 8 - p.rot / 16;  // items of a rotated head
  const int n = ((r.q ? p.Hq : 0) + p.Hkv) * per + p.Hkv * (D / 8);
  static_assert(kRopeThreads >= VC_ROPE_MAX_PAIRS, "a pair a thread");
  const double turns = (int)threadIdx.x < p.rot / 2 ? p.turns[threadIdx.x] : 0.0;
  pdl_wait();
  const int at = r.pos ? r.pos[t] : r.pos0 + t;
  RopeItem e{nullptr, nullptr, 0, -1};
  uint4 x, y;
  auto load = [&](int i) {
    e = rope_item<D>(p, r, t, i, per);
    x = e.src[0];
    if (e.pair) y = e.src[e.pair];
  };
  if ((int)threadIdx.x < n) load(threadIdx.x);
  if ((int)threadIdx.x < p.rot / 2) {
    double turn = (double)at * turns;
    turn -= rint(turn);
    float sn, cn;
    sincospif((float)(2.0 * turn), &sn, &cn);
    cs[threadIdx.x] = make_float2(cn * p.amp, sn * p.amp);
  }
  for (int h = threadIdx.x; h < p.Hkv; h += kRopeThreads) {
    if (r.score) r.score[h * r.cap + t] = 0.f;
    if (r.cpos) r.cpos[h * r.cap + t] = at;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kRopeThreads) {
    if (i != (int)threadIdx.x) load(i);
    rope_turn(e, x, y, cs);
    e.dst[0] = x;
    if (e.pair) e.dst[e.pair] = y;
  }
}

cudaError_t launch_rope(const RopeParams& p, int d, cudaStream_t s) {
  auto kern = d == 128 ? rope_kernel<128> : rope_kernel<64>;
  return launch_pdl(kern, dim3(p.n_tok), dim3(kRopeThreads), 0, s, p);
}

}  // namespace vc
