// rope.cuh - rotary positions of q and k on every rank, with k and v optionally appended to a cache.
//
// Pair (a, b) of a head at position t turns by w = t f_j: (a cos w - b sin w, b cos w + a sin w),
// times mscale.  The same (token, pair) angles serve every head of every rank.
#pragma once

#include "ptx.cuh"

namespace caat {

constexpr int KR_THREADS = 256;
constexpr int KR_CTAS = 5;         // resident per SM, and launched (10 or 40 measured no faster)
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

// A CTA owns 256 kItems items (16-byte vectors, or pairs of vectors that turn together) of a token's heads
// on all ranks, and walks the tokens: what an item is does not depend on the token, so its addresses are
// worked out once.  Per token the loads go out first; meanwhile the first rot / 2 threads evaluate the
// token's angles: in double, since a position times a frequency has to keep its fraction of a turn (at
// position 10^6 a product rounded to fp32 is off by up to 0.03 rad), reduced to [-1/2, 1/2] turns and
// then passed on in fp32.  Bound by the memory: T=8192, 32 + 32 heads of 128, 268 MB in 50 us (5.4 TB/s).
// Two items a thread: 52 us against 57 with four (half of them idle at this size) in the same run.
template <bool kInterleaved, int kItems>
__global__ void __launch_bounds__(KR_THREADS, KR_CTAS) rope_kernel(const __grid_constant__ RopeParams prm) {
  __shared__ float2 cs[2][KR_MAX_PAIRS];
  const int half = prm.rot >> 1;
  const int nrot = kInterleaved ? prm.rot >> 3 : prm.rot >> 4;  // rotated items of a head
  const int items = nrot + ((prm.dh - prm.rot) >> 3);           // and single vectors copied behind them
  const int nq = prm.P * prm.q.heads * items, nk = prm.P * prm.k.heads * items;
  const int nv = prm.P * prm.v.heads * (prm.dh >> 3);
  const __nv_bfloat16* src[kItems];
  __nv_bfloat16* dst[kItems];
  int what[kItems];  // 0 q, 1 k, 2 v, -1 nothing; 4 set: turned, its first pair in the bits above
#pragma unroll
  for (int x = 0; x < kItems; ++x) {
    int i = (blockIdx.y * kItems + x) * KR_THREADS + threadIdx.x;
    what[x] = -1;
    src[x] = nullptr;
    dst[x] = nullptr;
    if (i >= nq + nk + nv) continue;
    const int which = i < nq ? 0 : i < nq + nk ? 1 : 2;
    const RopeTensor& t = which == 0 ? prm.q : which == 1 ? prm.k : prm.v;
    i -= which == 0 ? 0 : which == 1 ? nq : nq + nk;
    const int per = which == 2 ? prm.dh >> 3 : items;
    const int hr = i / per, it = i - hr * per;
    const int r = hr / t.heads, h = hr - r * t.heads;
    const bool turn = which != 2 && it < nrot;
    const int e = h * prm.dh + (which == 2 || turn ? 8 * it : prm.rot + 8 * (it - nrot));
    src[x] = t.in + r * t.in_rank + e;
    dst[x] = t.out + r * t.out_rank + e;
    what[x] = which | (turn ? 4 | (kInterleaved ? 4 : 8) * it << 3 : 0);
  }
  int buf = 0;
  for (int64_t t = blockIdx.x; t < prm.T; t += gridDim.x, buf ^= 1) {
    uint4 a[kItems], b[kItems];
#pragma unroll
    for (int x = 0; x < kItems; ++x) {
      if (what[x] < 0) continue;
      const int which = what[x] & 3;
      const __nv_bfloat16* p = src[x] + t * (which == 0 ? prm.q.in_tok : which == 1 ? prm.k.in_tok : prm.v.in_tok);
      a[x] = *reinterpret_cast<const uint4*>(p);
      if (!kInterleaved && (what[x] & 4)) b[x] = *reinterpret_cast<const uint4*>(p + half);
    }
    if (threadIdx.x < half) {
      const double pos = prm.positions ? static_cast<double>(prm.positions[t]) : static_cast<double>(t);
      const double turns = pos * prm.turns[threadIdx.x];
      float s, c;
      sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
      cs[buf][threadIdx.x] = make_float2(prm.mscale * c, prm.mscale * s);
    }
    int64_t row = t;  // of k_out and v_out
    bool append = true;
    if (prm.slots) {
      row = prm.slots[t];
      append = row >= 0 && row < prm.cache_rows;
      if (!append && row != -1 && threadIdx.x == 0) atomicCAS(&g_arg_status, 0, (81 << 8) | 1);
    }
    __syncthreads();  // (two buffers: a CTA is never two tokens ahead of one of its threads)
#pragma unroll
    for (int x = 0; x < kItems; ++x) {
      if (what[x] < 0) continue;
      const int which = what[x] & 3;
      if (which != 0 && !append) continue;
      __nv_bfloat16* p = dst[x] + (which == 0 ? t * prm.q.out_tok : row * (which == 1 ? prm.k.out_tok : prm.v.out_tok));
      if (!(what[x] & 4)) {
        st_v4(p, a[x]);
        continue;
      }
      const float2* z = &cs[buf][what[x] >> 3];
      const uint32_t wa[4] = {a[x].x, a[x].y, a[x].z, a[x].w};
      if (kInterleaved) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x0 = bf16lo(wa[e]), x1 = bf16hi(wa[e]);
          o[e] = pack_bf16x2(x0 * z[e].x - x1 * z[e].y, x1 * z[e].x + x0 * z[e].y);
        }
        st_v4(p, make_uint4(o[0], o[1], o[2], o[3]));
      } else {
        const uint32_t wb[4] = {b[x].x, b[x].y, b[x].z, b[x].w};
        uint32_t oa[4], ob[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 z0 = z[2 * e], z1 = z[2 * e + 1];
          const float a0 = bf16lo(wa[e]), a1 = bf16hi(wa[e]), b0 = bf16lo(wb[e]), b1 = bf16hi(wb[e]);
          oa[e] = pack_bf16x2(a0 * z0.x - b0 * z0.y, a1 * z1.x - b1 * z1.y);
          ob[e] = pack_bf16x2(b0 * z0.x + a0 * z0.y, b1 * z1.x + a1 * z1.y);
        }
        st_v4(p, make_uint4(oa[0], oa[1], oa[2], oa[3]));
        st_v4(p + half, make_uint4(ob[0], ob[1], ob[2], ob[3]));
      }
    }
  }
}

}  // namespace caat
