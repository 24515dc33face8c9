// attn_common.cuh - what the attention kernels share: the work list, tensor-memory operands, packed
// fp32 arithmetic.
#pragma once

#include "ptx.cuh"

namespace caat {

constexpr int KA_TILE = 128;               // queries (or keys) of one MMA tile
constexpr int KA_BOX_BYTES = 128 * 128;    // one TMA box: 128 rows x 64 bf16, 128-byte swizzle
constexpr uint64_t KA_DRAIN_NS = 1000000;  // error path only: let copies in flight land
constexpr float KA_LOG2E = 1.4426950408889634f;
constexpr float KA_LN2 = 0.6931471805599453f;

// One entry of a work list.  Forward and dq: `rows` queries from row q0 on, the first of which sees
// `first` keys of the sequence whose m keys start at row k0 (first <= 0: none); query i sees
// min(first + i, m) of them, and never fewer than 0.
struct AttnJob {
  int q0, rows, k0, first;
  int k_rows;  // dkv only
};

// Work lists travel in the launch's arguments when they fit, else through the workspace.
constexpr int KA_INLINE_JOBS = 160;
constexpr int KA_UPLOAD_JOBS = 200;
struct AttnJobList {
  const AttnJob* far;  // null: `near` holds them
  AttnJob near[KA_INLINE_JOBS];
};
struct AttnJobChunk {
  AttnJob job[KA_UPLOAD_JOBS];
};

// Division by a launch constant (n < 2^31) as a high product and a shift: with l = ceil(log2 d) and
// mul = floor(2^32 (2^l - d) / d) + 1, n / d = (mulhi(n, mul) + n) >> l.  (The compiler would otherwise
// keep each divisor's reciprocal in registers across the kernels' main loops.)
struct FastDiv {
  uint32_t d, mul, shift;
  void set(uint32_t div) {
    d = div;
    shift = 0;
    while ((uint64_t(1) << shift) < div) ++shift;
    mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - div)) / div + 1);
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
  }
};

__global__ void attn_upload_kernel(AttnJob* dst, int n, const __grid_constant__ AttnJobChunk c) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = c.job[i];
}

__device__ __forceinline__ void tma_load_4d(void* smem_dst, const void* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}

// One lane of the warp.  The MMA warps run their loops with all lanes, so that descriptors and addresses
// stay in uniform registers, and predicate the MMA instructions themselves with this.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

// D[tmem] (+)= A[smem] * B[smem]^T, by the lane with lead != 0.
__device__ __forceinline__ void umma_ss(uint32_t lead, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}

// The same with A in tensor memory: bf16, its rows in the lanes and two K neighbours per column.
__device__ __forceinline__ void umma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}

__device__ __forceinline__ void umma_arrive(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}

// Waits for the thread's tensor-memory loads into r.  The loads write their registers behind the
// compiler's back until then: listing them here keeps every use of them below the wait.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// The thread's lane of 32 columns.
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// MN-major operand of 128-row boxes (64 MN elements wide): as sw128_mnmajor_desc, the next 64 MN
// elements 16 KiB on.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc_128(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(KA_BOX_BYTES >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Two fp32 lanes in one instruction.
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^x of two values without the special-function unit: x = n + f with n the nearest whole number, 2^f
// by the polynomial of degree 5 that interpolates it at the 6 Chebyshev nodes of [-1/2, 1/2] (off by
// 1.0e-7 relative, 2.2e-7 = 2^-22 as evaluated in fp32), and 2^n put together in the exponent field.
// x below -126.5 gives 0, x is at most 126, NaN stays NaN.
__device__ __forceinline__ uint64_t ex2_poly_f32x2(uint64_t x) {
  float a, b;
  unpack_f32x2(x, a, b);
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(a));  // -127
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(b));
  const uint64_t c = pack_f32x2(a, b);
  const uint64_t t = add_f32x2(c, pack_f32x2(12582912.f, 12582912.f));  // 1.5 2^23: n in the low bits
  const uint64_t n = add_f32x2(t, pack_f32x2(-12582912.f, -12582912.f));
  const uint64_t f = fma_f32x2(n, pack_f32x2(-1.f, -1.f), c);
  uint64_t r = fma_f32x2(f, pack_f32x2(0.0013390863364571618f, 0.0013390863364571618f),
                         pack_f32x2(0.00967603191832481f, 0.00967603191832481f));
  r = fma_f32x2(r, f, pack_f32x2(0.05550357114219401f, 0.05550357114219401f));
  r = fma_f32x2(r, f, pack_f32x2(0.2402210748530825f, 0.2402210748530825f));
  r = fma_f32x2(r, f, pack_f32x2(0.6931471880262285f, 0.6931471880262285f));
  r = fma_f32x2(r, f, pack_f32x2(1.0000000754548972f, 1.0000000754548972f));
  unpack_f32x2(t, a, b);
  const uint32_t ea = (__float_as_uint(a) << 23) + 0x3F800000u, eb = (__float_as_uint(b) << 23) + 0x3F800000u;
  return mul_f32x2(r, pack_f32x2(__uint_as_float(ea), __uint_as_float(eb)));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Stores a warp's 32 rows of kChunks 16-byte pieces, lane = row, through a patch of shared memory (32
// kChunks 16 bytes), so that neighbouring lanes store neighbouring pieces of a row: a row a lane, each
// store instruction touches 32 rows and takes as many trips.  `rows` rows and `chunks` pieces exist.
template <int kChunks>
__device__ __forceinline__ void warp_store_rows(uint8_t* patch, const uint4 (&v)[kChunks], uint8_t* dst, int64_t stride,
                                                int rows, int chunks, int lane) {
  constexpr int kMask = kChunks < 8 ? kChunks - 1 : 7;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) *reinterpret_cast<uint4*>(patch + (lane * kChunks + (c ^ (lane & kMask))) * 16) = v[c];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int r = (i * 32 + lane) / kChunks, c = (i * 32 + lane) % kChunks;
    if (r < rows && c < chunks)
      st_v4(dst + r * stride + c * 16, *reinterpret_cast<const uint4*>(patch + (r * kChunks + (c ^ (r & kMask))) * 16));
  }
  __syncwarp();
}

// The long part of a wait, kept out of the loops: their code should stay short.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, uint64_t tmo, int site) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t n = 1;; ++n) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    if (__all_sync(0xFFFFFFFFu, done)) return true;
    if ((n & 63u) == 0u) {
      if (__any_sync(0xFFFFFFFFu, status_poll() != 0)) return false;
      if (__any_sync(0xFFFFFFFFu, globaltimer_ns() - t0 > tmo)) {
        status_raise(4, site);
        return false;
      }
    }
  }
}

// Bounded wait of a whole warp (uniform result).
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity, uint64_t tmo, int site) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  return wait_long(smem_u32(bar), parity, tmo, site);
}

// Warp-uniform bounded wait of all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t tmo, int site) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, tmo, site));
}

}  // namespace caat
