// attn_simple.cuh - causal attention, one warp per row on the CUDA cores.
//
// A lane holds 4 elements of the row (dh <= 128); the warp walks the visible keys with a running
// maximum and sum.  All arithmetic in fp32.
#pragma once

#include "ptx.cuh"
#include "rope.cuh"

namespace caat {

struct AttnView {            // a strided [P, T, heads, dh] operand
  const __nv_bfloat16* p;
  int64_t rank, tok;
};

struct AttnSimple {
  AttnView q, k, v;
  __nv_bfloat16* out;
  float* lse;
  int64_t Tq, Tk;
  int hq, hk, dh;
  float scale;
};

__device__ __forceinline__ float4 ld_row4(const __nv_bfloat16* p, int e, int dh) {
  if (e >= dh) return make_float4(0.f, 0.f, 0.f, 0.f);
  const uint2 w = *reinterpret_cast<const uint2*>(p + e);
  return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}

__device__ __forceinline__ void st_row4(__nv_bfloat16* p, int e, int dh, float4 f) {
  if (e < dh) *reinterpret_cast<uint2*>(p + e) = make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
}

__device__ __forceinline__ float warp_dot4(float4 a, float4 b) {
  float s = a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  return s;
}

__device__ __forceinline__ void axpy4(float4& o, float a, float4 x) {
  o.x = fmaf(a, x.x, o.x);
  o.y = fmaf(a, x.y, o.y);
  o.z = fmaf(a, x.z, o.z);
  o.w = fmaf(a, x.w, o.w);
}

struct AttnSimpleBwd {
  AttnSimple f;
  const __nv_bfloat16* dout;
  __nv_bfloat16 *dq, *dk, *dv;
  float* D;                  // [P, hq, Tq]
};

__global__ void __launch_bounds__(128) attn_simple_dq_kernel(AttnSimpleBwd b, int q0, int n, int k0, int m) {
  const AttnSimple& a = b.f;
  const int i = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31, e = 4 * lane;
  if (i >= n) return;
  const int h = blockIdx.y, r = blockIdx.z, kv = h / (a.hq / a.hk);
  const int64_t row = q0 + i, orow = ((r * a.Tq + row) * a.hq + h) * a.dh, srow = (int64_t(r) * a.hq + h) * a.Tq + row;
  const float4 q = ld_row4(a.q.p + r * a.q.rank + row * a.q.tok + h * a.dh, e, a.dh);
  const float4 g = ld_row4(b.dout + orow, e, a.dh);
  const float D = warp_dot4(g, ld_row4(a.out + orow, e, a.dh)), lse = a.lse[srow];
  if (lane == 0) b.D[srow] = D;
  float4 dq = make_float4(0.f, 0.f, 0.f, 0.f);
  const int seen = i + 1 + (m - n);
  for (int j = 0; j < seen; ++j) {
    const float4 k = ld_row4(a.k.p + r * a.k.rank + int64_t(k0 + j) * a.k.tok + kv * a.dh, e, a.dh);
    const float4 v = ld_row4(a.v.p + r * a.v.rank + int64_t(k0 + j) * a.v.tok + kv * a.dh, e, a.dh);
    const float p = expf(a.scale * warp_dot4(q, k) - lse);
    axpy4(dq, a.scale * p * (warp_dot4(g, v) - D), k);
  }
  st_row4(b.dq + orow, e, a.dh, dq);
}

__global__ void __launch_bounds__(128) attn_simple_dkv_kernel(AttnSimpleBwd b, int q0, int n, int k0, int m) {
  const AttnSimple& a = b.f;
  const int j = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31, e = 4 * lane;
  if (j >= m) return;
  const int kv = blockIdx.y, r = blockIdx.z, group = a.hq / a.hk;
  const float4 k = ld_row4(a.k.p + r * a.k.rank + int64_t(k0 + j) * a.k.tok + kv * a.dh, e, a.dh);
  const float4 v = ld_row4(a.v.p + r * a.v.rank + int64_t(k0 + j) * a.v.tok + kv * a.dh, e, a.dh);
  float4 dk = make_float4(0.f, 0.f, 0.f, 0.f), dv = dk;
  for (int h = kv * group; h < (kv + 1) * group; ++h) {
    for (int i = max(0, j - (m - n)); i < n; ++i) {
      const int64_t row = q0 + i, srow = (int64_t(r) * a.hq + h) * a.Tq + row;
      const float4 q = ld_row4(a.q.p + r * a.q.rank + row * a.q.tok + h * a.dh, e, a.dh);
      const float4 g = ld_row4(b.dout + ((r * a.Tq + row) * a.hq + h) * a.dh, e, a.dh);
      const float p = expf(a.scale * warp_dot4(q, k) - a.lse[srow]);
      axpy4(dv, p, g);
      axpy4(dk, a.scale * p * (warp_dot4(g, v) - b.D[srow]), q);
    }
  }
  const int64_t krow = ((r * a.Tk + k0 + j) * a.hk + kv) * a.dh;
  st_row4(b.dk + krow, e, a.dh, dk);
  st_row4(b.dv + krow, e, a.dh, dv);
}

// Decoding: one warp per (rank, sequence, head).
struct AttnSimpleDecode {
  AttnView q;
  const __nv_bfloat16 *k, *v;  // [P, B, capacity, hk, dh]
  const int32_t* lens;
  __nv_bfloat16* out;
  int64_t B, capacity;
  int hq, hk, dh;
  float scale;
};

__global__ void __launch_bounds__(32) attn_simple_decode_kernel(AttnSimpleDecode a) {
  const int64_t s = blockIdx.x;
  const int h = blockIdx.y, r = blockIdx.z, lane = threadIdx.x, e = 4 * lane, kv = h / (a.hq / a.hk);
  int len = a.lens[s];
  if (len < 0 || len > a.capacity) {
    if (lane == 0) atomicCAS(&g_arg_status, 0, (82 << 8) | 1);
    len = 0;
  }
  const float4 q = ld_row4(a.q.p + r * a.q.rank + s * a.q.tok + h * a.dh, e, a.dh);
  float top = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < len; ++j) {
    const int64_t row = (((r * a.B + s) * a.capacity + j) * a.hk + kv) * a.dh;
    const float x = a.scale * warp_dot4(q, ld_row4(a.k + row, e, a.dh));
    const float t = fmaxf(top, x);
    const float c = top == -INFINITY ? 0.f : expf(top - t), p = expf(x - t);
    sum = sum * c + p;
    o = make_float4(o.x * c, o.y * c, o.z * c, o.w * c);
    axpy4(o, p, ld_row4(a.v + row, e, a.dh));
    top = t;
  }
  const float inv = len > 0 ? 1.f / sum : 0.f;
  st_row4(a.out + ((r * a.B + s) * a.hq + h) * a.dh, e, a.dh, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
}

}  // namespace caat
