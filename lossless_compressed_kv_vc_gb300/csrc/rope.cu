// Rotary positions of new tokens, written to the cache.
//
// Pair j of a head's rotated channels (a, b) at position p becomes
//   (a c - b s, a s + b c),  c = amp cos(p theta_j), s = amp sin(p theta_j).
// The angle is taken in turns, p theta_j / 2 pi, in fp64 and reduced to [-1/2, 1/2] there, so that a far
// position loses nothing; cos and sin of the remainder are fp32 (cospi, sinpi).
//
// A CTA takes one token: its rot / 2 angles are computed once, in shared memory, for all of the token's
// query and key heads. It is a copy otherwise: every q, k and v element is read and written once.
#include "vc_internal.cuh"

namespace vc {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ float2 bf2_unpack(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Rotates one item of a head of D channels: items 0 .. rot/16 - 1 of the half layout are the channel
// groups 8i..8i+7 with their partners rot/2 higher, the rest pass through; an item of the interleaved
// layout is a group of eight channels. cs: (cos, sin) of each pair.
template <int D>
__device__ __forceinline__ void rope_item(const bf16* src, bf16* dst, int item, int rot, bool inter, const float2* cs) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* o = reinterpret_cast<uint4*>(dst);
  if (inter) {
    uint4 x = s[item];
    if (8 * item < rot) {
      uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = bf2_unpack(w[e]), t = cs[4 * item + e];
        w[e] = pack_bf16x2(a.x * t.x - a.y * t.y, a.x * t.y + a.y * t.x);
      }
    }
    o[item] = x;
    return;
  }
  const int half = rot / 16;
  if (item >= half) {  // passes through: groups rot / 8 on
    o[item + half] = s[item + half];
    return;
  }
  uint4 x = s[item], y = s[item + half];
  uint32_t *wx = reinterpret_cast<uint32_t*>(&x), *wy = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = bf2_unpack(wx[e]), b = bf2_unpack(wy[e]);
    const float2 t0 = cs[8 * item + 2 * e], t1 = cs[8 * item + 2 * e + 1];
    wx[e] = pack_bf16x2(a.x * t0.x - b.x * t0.y, a.y * t1.x - b.y * t1.y);
    wy[e] = pack_bf16x2(a.x * t0.y + b.x * t0.x, a.y * t1.y + b.y * t1.x);
  }
  o[item] = x;
  o[item + half] = y;
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs[VC_ROPE_MAX_PAIRS];
  pdl_wait();
  const int tok = blockIdx.x;
  int b = 0;
#pragma unroll 1
  for (int i = 1; i < p.B; ++i)
    if (p.req[i].tok_begin <= tok) b = i;
  const RopeReqDev& r = p.req[b];
  const int t = tok - r.tok_begin;
  const int at = r.pos ? r.pos[t] : r.pos0 + t;
  for (int j = threadIdx.x; j < p.rot / 2; j += kRopeThreads) {
    double turn = (double)at * p.turns[j];
    turn -= rint(turn);
    float sn, cn;
    sincospif((float)(2.0 * turn), &sn, &cn);
    cs[j] = make_float2(cn * p.amp, sn * p.amp);
  }
  __syncthreads();
  const int per = p.inter ? D / 8 : D / 8 - p.rot / 16;  // items of a rotated head
  const int nq = r.q ? p.Hq * per : 0, nk = p.Hkv * per, nv = p.Hkv * (D / 8);
  for (int i = threadIdx.x; i < nq + nk + nv; i += kRopeThreads) {
    if (i < nq) {
      const int h = i / per;
      rope_item<D>(r.q + t * r.q_stride + (int64_t)h * D, r.q_out + ((int64_t)t * p.Hq + h) * D, i - h * per, p.rot, p.inter, cs);
    } else if (i < nq + nk) {
      const int h = (i - nq) / per;
      rope_item<D>(r.k + t * r.k_stride + (int64_t)h * D, r.kc + (h * r.cap + t) * D, i - nq - h * per, p.rot, p.inter, cs);
    } else {
      const int e = i - nq - nk, h = e / (D / 8), c = e % (D / 8);
      reinterpret_cast<uint4*>(r.vc + (h * r.cap + t) * D)[c] =
          reinterpret_cast<const uint4*>(r.v + t * r.v_stride + (int64_t)h * D)[c];
    }
  }
  for (int h = threadIdx.x; h < p.Hkv; h += kRopeThreads) {
    if (r.score) r.score[h * r.cap + t] = 0.f;
    if (r.cpos) r.cpos[h * r.cap + t] = at;
  }
}

cudaError_t launch_rope(const RopeParams& p, int d, cudaStream_t s) {
  auto kern = d == 128 ? rope_kernel<128> : rope_kernel<64>;
  return launch_pdl(kern, dim3(p.n_tok), dim3(kRopeThreads), 0, s, p);
}

}  // namespace vc
