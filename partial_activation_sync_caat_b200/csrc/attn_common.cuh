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

// D[tmem] (+)= A[tmem] * B[smem]: A bf16, its rows in the lanes and two K neighbours per column.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
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

// Warp-uniform bounded wait of all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t tmo, int site) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, tmo, site));
}

}  // namespace caat
