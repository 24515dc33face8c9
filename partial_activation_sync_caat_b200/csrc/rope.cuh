// rope.cuh - rotary positions of q and k on every rank, with k and v optionally appended to a cache.
//
// Pair (a, b) of a head at position t turns by w = t f_j: (a cos w - b sin w, b cos w + a sin w),
// times mscale.  The same (token, pair) angles serve every head of every rank.
#pragma once

#include "ptx.cuh"

namespace caat {

constexpr int KR_THREADS = 256;
constexpr int KR_MAX_PAIRS = 128;  // rot <= 256

// Out-of-range device-resident arguments (slots, lengths): reported like the bounded waits' status,
// but kept apart from it, since waits give up when the status word is set.
__device__ int g_arg_status;

struct RopeTensor {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;
  int64_t in_rank, in_tok, out_rank, out_tok;  // strides, elements
  int heads;
};

struct RopeParams {
  RopeTensor q, k, v;          // v: heads = 0 unless appending
  const int32_t* positions;    // [T] or null
  const int64_t* slots;        // [T] or null; k.out_tok, v.out_tok then step over cache rows
  int64_t T, cache_rows;
  int P, dh, rot;
  float mscale;
  double turns[KR_MAX_PAIRS];  // f_j / (2 pi), negated for the backward
};

// One CTA per token.  Its first rot / 2 threads evaluate the token's angles: in double, since a
// position times a frequency has to keep its fraction of a turn (at position 10^6 a product rounded
// to fp32 is off by up to 0.03 rad), reduced to [-1/2, 1/2] turns and then passed on in fp32.
// Then the threads walk the 16-byte vectors of the token's heads on all ranks.
template <bool kInterleaved>
__global__ void __launch_bounds__(KR_THREADS) rope_kernel(const __grid_constant__ RopeParams prm) {
  __shared__ float2 cs[KR_MAX_PAIRS];
  const int64_t t = blockIdx.x;
  const int half = prm.rot >> 1;
  if (threadIdx.x < half) {
    const double pos = prm.positions ? static_cast<double>(prm.positions[t]) : static_cast<double>(t);
    const double turns = pos * prm.turns[threadIdx.x];
    float s, c;
    sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
    cs[threadIdx.x] = make_float2(prm.mscale * c, prm.mscale * s);
  }
  int64_t row = t;
  bool append = true;
  if (prm.slots) {
    row = prm.slots[t];
    append = row >= 0 && row < prm.cache_rows;
    if (!append && row != -1 && threadIdx.x == 0) atomicCAS(&g_arg_status, 0, (81 << 8) | 1);
  }
  __syncthreads();
  const int nrot = kInterleaved ? prm.rot >> 3 : prm.rot >> 4;  // rotated items of a head
  const int items = nrot + ((prm.dh - prm.rot) >> 3);           // and single vectors copied behind them
  for (int which = 0; which < 2; ++which) {
    const RopeTensor& x = which ? prm.k : prm.q;
    if (which && !append) break;
    const int64_t orow = (which && prm.slots) ? row : t;
    const int n = prm.P * x.heads * items;
    for (int i = threadIdx.x; i < n; i += KR_THREADS) {
      const int hr = i / items, it = i - hr * items;
      const int r = hr / x.heads, h = hr - r * x.heads;
      const __nv_bfloat16* src = x.in + r * x.in_rank + t * x.in_tok + h * prm.dh;
      __nv_bfloat16* dst = x.out + r * x.out_rank + orow * x.out_tok + h * prm.dh;
      if (it >= nrot) {
        const int e = prm.rot + 8 * (it - nrot);
        st_v4(dst + e, *reinterpret_cast<const uint4*>(src + e));
      } else if (kInterleaved) {
        const uint4 a = *reinterpret_cast<const uint4*>(src + 8 * it);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 z = cs[4 * it + e];
          const float x0 = bf16lo(w[e]), x1 = bf16hi(w[e]);
          o[e] = pack_bf16x2(x0 * z.x - x1 * z.y, x1 * z.x + x0 * z.y);
        }
        st_v4(dst + 8 * it, make_uint4(o[0], o[1], o[2], o[3]));
      } else {
        const uint4 a = *reinterpret_cast<const uint4*>(src + 8 * it);
        const uint4 b = *reinterpret_cast<const uint4*>(src + half + 8 * it);
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
        uint32_t oa[4], ob[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 z0 = cs[8 * it + 2 * e], z1 = cs[8 * it + 2 * e + 1];
          const float a0 = bf16lo(wa[e]), a1 = bf16hi(wa[e]), b0 = bf16lo(wb[e]), b1 = bf16hi(wb[e]);
          oa[e] = pack_bf16x2(a0 * z0.x - b0 * z0.y, a1 * z1.x - b1 * z1.y);
          ob[e] = pack_bf16x2(b0 * z0.x + a0 * z0.y, b1 * z1.x + a1 * z1.y);
        }
        st_v4(dst + 8 * it, make_uint4(oa[0], oa[1], oa[2], oa[3]));
        st_v4(dst + half + 8 * it, make_uint4(ob[0], ob[1], ob[2], ob[3]));
      }
    }
  }
  if (prm.v.heads && append) {
    const int vecs = prm.dh >> 3;
    const int n = prm.P * prm.v.heads * vecs;
    for (int i = threadIdx.x; i < n; i += KR_THREADS) {
      const int hr = i / vecs, e = 8 * (i - hr * vecs);
      const int r = hr / prm.v.heads, h = hr - r * prm.v.heads;
      const uint4 a = *reinterpret_cast<const uint4*>(prm.v.in + r * prm.v.in_rank + t * prm.v.in_tok + h * prm.dh + e);
      st_v4(prm.v.out + r * prm.v.out_rank + row * prm.v.out_tok + h * prm.dh + e, a);
    }
  }
}

}  // namespace caat
