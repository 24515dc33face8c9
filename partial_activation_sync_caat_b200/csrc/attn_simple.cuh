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
