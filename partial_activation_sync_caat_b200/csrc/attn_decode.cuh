// attn_decode.cuh - one new token per sequence against its cache, on every rank.
//
// Every byte of K and V is used once, so the read rate of the memory bounds it.  The work is the list of
// tiles (64 keys, of dh <= 64: 128) of all (sequence, rank, key head) segments; it is cut evenly over a fixed number of
// CTAs, whatever the lengths, so that one long sequence and many short ones alike keep all SMs
// reading.  A segment cut between CTAs leaves fp32 partial results (maximum, sum, sums of p v); the
// CTA that finishes the last of them joins them, in the order of the CTAs, so results do not change from
// run to run.  The counters it goes by are cleared by a kernel of one block that this one is launched
// behind without waiting (programmatic dependent launch: it waits before it counts).  A second kernel for that, launched
// early and waiting, measured 12 us more per call.
//
// Inside a CTA each of the 4 warps owns a quarter of a tile's keys and a ring of its own, filled with
// 16-byte asynchronous copies: no block-wide waits until a segment ends, when the warps' running
// maxima, sums and products are merged through shared memory.  Up to 16 query heads of the group share
// the tile as the 16 rows of the MMA (legacy mma.sync: the products are a small part of the time even
// with one head of the 16 rows in use: 64 keys x 128 elements of K and V are 32 KiB, about 1400 clocks of
// an SM's share of the memory rate, against 128 MMAs).  Keys past the length are never read: their rows
// are filled with zeros, their scores replaced by -inf.
#pragma once

#include "attn_common.cuh"
#include "rope.cuh"

namespace caat {

constexpr int KD_THREADS = 128;
// Keys of a tile per warp (4 warps): 32 KiB of K and V a tile at either width.
__host__ __device__ constexpr int kd_keys(int HD) { return HD == 64 ? 32 : 16; }
constexpr int KD_CTAS = 296;       // two per SM
constexpr int KD_MAX_B = 4096;
constexpr int KD_SMEM = 113 * 1024;

struct DecodeAttnParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;      // [P, B, capacity, hk, dh]
  const __nv_bfloat16* v;
  const int32_t* lens;
  __nv_bfloat16* out;          // [P, B, hq, dh]
  unsigned int* count;         // [CTAs], zero: parts of the segment that began in that CTA and are done
  float* part;                 // [CTAs][2][rows][dh + 2]: sums of p v, maximum (scaled, base 2), sum of p
  int64_t q_rank, q_tok;
  int64_t B, capacity;
  int P, hq, hk, dh, group;
  int rows;                    // min(group, 16)
  int n_gb;                    // blocks of 16 heads in a group
  int G;                       // segments of a sequence: P * hk * n_gb
  int stages;
  float scale;
};

// pre[b] = tiles of the sequences before b, pre[B] = all of them.  A length outside the cache counts as 0.
__device__ __forceinline__ void decode_prefix(const DecodeAttnParams& prm, int tile, int* pre, int* warp_sums) {
  const int B = static_cast<int>(prm.B);
  const int per = (B + KD_THREADS - 1) / KD_THREADS;
  const int b0 = threadIdx.x * per;
  int sum = 0;
  for (int b = b0; b < min(b0 + per, B); ++b) {
    const int len = __ldg(prm.lens + b);
    sum += (len > 0 && len <= prm.capacity) ? (len + tile - 1) / tile : 0;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int at = inc - sum;
  for (int w = 0; w < warp; ++w) at += warp_sums[w];
  for (int b = b0; b < min(b0 + per, B); ++b) {
    pre[b] = at;
    const int len = __ldg(prm.lens + b);
    at += (len > 0 && len <= prm.capacity) ? (len + tile - 1) / tile : 0;
  }
  if (b0 < B && b0 + per >= B) pre[B] = at;
  __syncthreads();
}

// The list is dealt in runs of equal length, the first `extra` CTAs one tile more.
struct DecodeDeal {
  int64_t each;
  int extra;
  __device__ __forceinline__ DecodeDeal(int64_t total, int ctas) : each(total / ctas), extra(static_cast<int>(total - each * ctas)) {}
  __device__ __forceinline__ int64_t begin(int cta) const { return cta * each + min(cta, extra); }
  __device__ __forceinline__ int owner(int64_t item) const {
    const int64_t longer = extra * (each + 1);
    return static_cast<int>(item < longer ? item / (each + 1) : extra + (item - longer) / each);
  }
};

__global__ void __launch_bounds__(KD_CTAS) attn_decode_clear_kernel(unsigned int* count) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  count[threadIdx.x] = 0;
}

// A tile of the work list: sequence, segment of the sequence, tile of the segment.
struct DecodeCursor {
  int b, g, t, tiles;
  __device__ __forceinline__ void seek(const DecodeAttnParams& prm, const int* pre, int64_t item) {
    int lo = 0, hi = static_cast<int>(prm.B);  // pre[lo] G <= item < pre[hi] G
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (int64_t(pre[mid]) * prm.G <= item) lo = mid;
      else hi = mid;
    }
    b = lo;
    tiles = pre[b + 1] - pre[b];
    const int64_t in = item - int64_t(pre[b]) * prm.G;
    g = static_cast<int>(in / tiles);
    t = static_cast<int>(in - int64_t(g) * tiles);
  }
  __device__ __forceinline__ void next(const DecodeAttnParams& prm, const int* pre) {
    if (++t < tiles) return;
    t = 0;
    if (++g < prm.G) return;
    g = 0;
    do {
      ++b;
    } while (b < prm.B && pre[b + 1] == pre[b]);
    if (b < prm.B) tiles = pre[b + 1] - pre[b];
  }
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Two floats of another CTA's shared memory (a shared::cluster address).
__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Joins the parts of a segment that CTAs z0..z1 left; z0, where it begins, in its slot 1, the others in
// their slot 0.  A warp a row: its lanes fetch the parts' maxima and sums side by side.
__device__ __noinline__ void decode_join(const DecodeAttnParams& prm, int z0, int z1, int b, int rank, int head0, int rows,
                                         int warp, int lane) {
  const int64_t stride = int64_t(prm.rows) * (prm.dh + 2);
  for (int r = warp; r < rows; r += KD_THREADS / 32) {
    const float* p0 = prm.part + r * (prm.dh + 2);
    auto part = [&](int z) { return p0 + (2 * int64_t(z) + (z == z0)) * stride; };
    float M = -INFINITY;
    for (int z = z0 + lane; z <= z1; z += 32) M = fmaxf(M, __ldcg(part(z) + prm.dh));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, d));
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int z = z0; z <= z1; z += 32) {  // in the order of the CTAs
      float2 ml = make_float2(-INFINITY, 0.f);
      if (z + lane <= z1) ml = __ldcg(reinterpret_cast<const float2*>(part(z + lane) + prm.dh));
      const float f = ex2(ml.x - base), fl = f * ml.y;
      const int n = min(32, z1 + 1 - z);
      for (int i0 = 0; i0 < n; i0 += 8) {  // 8 parts' loads at once
        float2 v[8][2];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            v[i][e] = i0 + i < n && 2 * lane + 64 * e < prm.dh
                          ? __ldcg(reinterpret_cast<const float2*>(part(z + i0 + i) + 2 * lane + 64 * e))
                          : make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float fi = __shfl_sync(0xFFFFFFFFu, f, i0 + i);
          L += __shfl_sync(0xFFFFFFFFu, fl, i0 + i);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            o[2 * e] = fmaf(fi, v[i][e].x, o[2 * e]);
            o[2 * e + 1] = fmaf(fi, v[i][e].y, o[2 * e + 1]);
          }
        }
      }
    }
    const float inv = 1.f / L;
    __nv_bfloat16* dst = prm.out + ((rank * prm.B + b) * prm.hq + head0 + r) * prm.dh + 2 * lane;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (2 * lane + 64 * e < prm.dh) *reinterpret_cast<uint32_t*>(dst + 64 * e) = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
  }
}

// A warp's share of a segment: the query rows as MMA fragments, the running maximum and sum of the
// thread's two rows (r0, r0 + 8) and the sums of p v.
template <int HD>
struct DecodeWarp {
  static constexpr int kKeys = kd_keys(HD);
  static constexpr int kRow = HD * 2;  // bytes of a key's row in shared memory
  uint32_t qa[HD / 16][4];
  float o[HD / 8][4];
  float m[2], l[2];
  int lane, r0;

  __device__ __forceinline__ void begin(const __nv_bfloat16* q, int rows, int dh) {
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 8 * (e & 1), d = 16 * kk + 8 * (e >> 1) + 2 * (lane & 3);
        qa[kk][e] = (r < rows && d < dh) ? *reinterpret_cast<const uint32_t*>(q + r * dh + d) : 0u;
      }
#pragma unroll
    for (int x = 0; x < HD / 8; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[x][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // The warp's keys of a tile, `live` of them before the sequence's end; K rows at ks, V rows at vs.
  __device__ __forceinline__ void tile(uint32_t ks, uint32_t vs, int live, float c) {
    float s[kKeys / 8][4] = {};
    const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;  // ldmatrix row and chunk of the lane
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk)
#pragma unroll
      for (int x = 0; x < kKeys / 16; ++x) {
        uint32_t b[4];
        ldmatrix_x4(ks + (16 * x + kr) * kRow + (((2 * kk + kc) ^ (kr & 7)) << 4), b);
        mma_16816(s[2 * x], qa[kk], b[0], b[1]);
        mma_16816(s[2 * x + 1], qa[kk], b[2], b[3]);
      }
    float top[2] = {m[0], m[1]};
#pragma unroll
    for (int x = 0; x < kKeys / 8; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[x][e] *= c;
        if (live < kKeys) {
          const int key = 8 * x + 2 * (lane & 3) + (e & 1);
          s[x][e] = key < live ? s[x][e] : -INFINITY;
        }
        top[e >> 1] = fmaxf(top[e >> 1], s[x][e]);
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 1));
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 2));
    }
    // the maximum only moves when exceeded by 2^8: p stays below 256, the quotient is the same
    if (__any_sync(0xFFFFFFFFu, top[0] - m[0] > 8.f || top[1] - m[1] > 8.f)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f = top[e] > m[e] ? ex2(m[e] - top[e]) : 1.f;
        m[e] = top[e];
        l[e] *= f;
#pragma unroll
        for (int x = 0; x < HD / 8; ++x) {
          o[x][2 * e] *= f;
          o[x][2 * e + 1] *= f;
        }
      }
    }
    uint32_t pa[kKeys / 16][4];
#pragma unroll
    for (int x = 0; x < kKeys / 8; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float base = m[e] == -INFINITY ? 0.f : m[e];
        const float p0 = ex2(s[x][2 * e] - base), p1 = ex2(s[x][2 * e + 1] - base);
        l[e] += p0 + p1;
        pa[x >> 1][2 * (x & 1) + e] = pack_bf16x2(p0, p1);
      }
    const int vr = (lane & 7) + (((lane >> 3) & 1) << 3), vc = lane >> 4;
#pragma unroll
    for (int y = 0; y < kKeys / 16; ++y)
#pragma unroll
      for (int x = 0; x < HD / 16; ++x) {
        uint32_t b[4];
        ldmatrix_x4_trans(vs + (16 * y + vr) * kRow + (((2 * x + vc) ^ (vr & 7)) << 4), b);
        mma_16816(o[2 * x], pa[y], b[0], b[1]);
        mma_16816(o[2 * x + 1], pa[y], b[2], b[3]);
      }
  }

  // This warp's results into merge [4][all_rows][HD] and ml [4][all_rows][2].
  __device__ __forceinline__ void publish(float* merge, float* ml, int warp, int rows, int all_rows) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
      l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
      const int r = r0 + 8 * e;
      if (r < rows) {
        float* row = merge + (warp * all_rows + r) * HD;
#pragma unroll
        for (int x = 0; x < HD / 8; ++x)
          *reinterpret_cast<float2*>(row + 8 * x + 2 * (lane & 3)) = make_float2(o[x][2 * e], o[x][2 * e + 1]);
        if ((lane & 3) == 0) {
          ml[(warp * all_rows + r) * 2] = m[e];
          ml[(warp * all_rows + r) * 2 + 1] = l[e];
        }
      }
    }
  }
};

// The four warps' results of elements d, d + 1 of row r: maximum, sum, sums of p v.
template <int HD>
__device__ __forceinline__ void decode_merge(const float* merge, const float* ml, int all_rows, int r, int d, float& M, float& L,
                                             float& x0, float& x1) {
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < 4; ++w) M = fmaxf(M, ml[(w * all_rows + r) * 2]);
  const float base = M == -INFINITY ? 0.f : M;
  L = x0 = x1 = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = ex2(ml[(w * all_rows + r) * 2] - base);
    const float2 x = *reinterpret_cast<const float2*>(merge + (w * all_rows + r) * HD + d);
    L = fmaf(f, ml[(w * all_rows + r) * 2 + 1], L);
    x0 = fmaf(f, x.x, x0);
    x1 = fmaf(f, x.y, x1);
  }
}

__device__ __forceinline__ void cp_async_wait_stages(int stages) {  // all but the stages - 1 newest groups
  switch (stages) {
    case 2: cp_async_wait<1>(); break;
    case 3: cp_async_wait<2>(); break;
    case 4: cp_async_wait<3>(); break;
    default: cp_async_wait<4>(); break;
  }
}

// A lane's copies of a tile: one 16-byte piece of every kStep-th of the warp's keys.  `ahead`: keys left
// from the lane's first one on (0 where its piece lies past dh).
template <int HD>
__device__ __forceinline__ void decode_copy(uint32_t dst, const __nv_bfloat16* kp, const __nv_bfloat16* vp, int64_t tok, int ahead,
                                            const __nv_bfloat16* any, int lane) {
  constexpr int kKeys = kd_keys(HD), kRow = HD * 2, kChunks = HD / 8, kStep = 32 / kChunks;
  const int chunk = lane % kChunks;
#pragma unroll
  for (int i = 0; i < kKeys / kStep; ++i) {
    const int r = i * kStep + lane / kChunks;
    const bool in = i * kStep < ahead;
    const uint32_t d = dst + r * kRow + ((chunk ^ (r & 7)) << 4);
    cp_async_16(d, in ? kp + i * kStep * tok : any, in ? 16 : 0);
    cp_async_16(d + kKeys * kRow, in ? vp + i * kStep * tok : any, in ? 16 : 0);
  }
}

template <int HD>
__global__ void __launch_bounds__(KD_THREADS, 2) attn_decode_kernel(const __grid_constant__ DecodeAttnParams prm) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  constexpr int kKeys = kd_keys(HD);           // a warp's keys of a tile
  constexpr int kTile = 4 * kKeys;
  constexpr int kRow = HD * 2;                 // bytes of a key's row in shared memory
  constexpr int kStage = 2 * kKeys * kRow;     // a warp's keys of K and of V
  constexpr int kChunks = HD / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem_raw + warp * prm.stages * kStage;
  float* merge = reinterpret_cast<float*>(smem_raw + 4 * prm.stages * kStage);  // [4][rows][HD]
  float* ml = merge + 4 * prm.rows * HD;                                        // [4][rows][2]
  int* pre = reinterpret_cast<int*>(ml + 4 * prm.rows * 2);                     // [B + 1]
  int* warp_sums = pre + prm.B + 1;
  __shared__ int last_part;

  decode_prefix(prm, kTile, pre, warp_sums);
  // sequences without keys
  for (int64_t b = blockIdx.x; b < prm.B; b += gridDim.x) {
    if (pre[b + 1] != pre[b]) continue;
    if (threadIdx.x == 0 && __ldg(prm.lens + b) != 0) atomicCAS(&g_arg_status, 0, (82 << 8) | 1);
    const int n = prm.hq * prm.dh / 8;
    for (int r = 0; r < prm.P; ++r)
      for (int i = threadIdx.x; i < n; i += KD_THREADS)
        st_v4(prm.out + (r * prm.B + b) * prm.hq * prm.dh + 8 * i, make_uint4(0, 0, 0, 0));
  }
  // (two tiles a CTA at least: parts cost time to join)
  const int64_t total = int64_t(pre[prm.B]) * prm.G;
  const int active = static_cast<int>(min(int64_t(gridDim.x), (total + 1) / 2));
  if (static_cast<int>(blockIdx.x) >= active) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const DecodeDeal deal(total, active);
  const int64_t i0 = deal.begin(blockIdx.x), i1 = deal.begin(blockIdx.x + 1);
  if (i0 == i1) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }

  DecodeCursor ld, at;
  ld.seek(prm, pre, i0);
  at = ld;
  int64_t todo = i1 - i0;
  // segment g of a sequence: head block fastest, then key head, then rank
  auto split_g = [&](int g, int& rank, int& kvh, int& gb) {
    gb = g % prm.n_gb;
    const int x = g / prm.n_gb;
    rank = x / prm.hk;
    kvh = x - rank * prm.hk;
  };
  // Each lane copies one 16-byte piece of every kStep-th key; its pointers and the keys left behind its
  // first one are carried from tile to tile and set up again only where a segment begins.
  const int my_key = warp * kKeys + lane / kChunks, my_chunk = lane % kChunks;
  const bool my_part = my_chunk * 8 < prm.dh;
  const int64_t tok = int64_t(prm.hk) * prm.dh;
  const __nv_bfloat16 *kp = prm.k, *vp = prm.v;
  int ahead = 0;
  bool fresh_ld = true;
  auto load = [&](int stage) {
    if (todo > 0) {
      if (fresh_ld) {
        int rank, kvh, gb;
        split_g(ld.g, rank, kvh, gb);
        const int key = ld.t * kTile + my_key;
        const int64_t off = ((rank * prm.B + ld.b) * prm.capacity + key) * tok + int64_t(kvh) * prm.dh + my_chunk * 8;
        kp = prm.k + off;
        vp = prm.v + off;
        ahead = my_part ? __ldg(prm.lens + ld.b) - key : 0;
        fresh_ld = false;
      }
      const uint32_t dst = smem_u32(ring + stage * kStage);
      decode_copy<HD>(dst, kp, vp, tok, ahead, prm.k, lane);
      kp += kTile * tok;
      vp += kTile * tok;
      ahead -= kTile;
      --todo;
      fresh_ld = ld.t + 1 == ld.tiles;
      ld.next(prm, pre);
    }
    cp_async_commit();
  };

  for (int s = 0; s < prm.stages - 1; ++s) load(s);
  const float c = prm.scale * KA_LOG2E;
  DecodeWarp<HD> w;
  w.lane = lane;
  w.r0 = lane >> 2;
  int rank = 0, kvh = 0, gb = 0, rows = 0, head0 = 0, len = 0;
  bool fresh = true;
  int stage = 0, ld_stage = prm.stages - 1;
  for (int64_t left = i1 - i0; left > 0; --left) {
    if (fresh) {
      split_g(at.g, rank, kvh, gb);
      rows = min(prm.group - 16 * gb, 16);
      head0 = kvh * prm.group + 16 * gb;
      len = __ldg(prm.lens + at.b);
      w.begin(prm.q + rank * prm.q_rank + at.b * prm.q_tok + int64_t(head0) * prm.dh, rows, prm.dh);
      fresh = false;
    }
    load(ld_stage);
    ld_stage = ld_stage + 1 == prm.stages ? 0 : ld_stage + 1;
    cp_async_wait_stages(prm.stages);
    __syncwarp();
    const uint32_t ks = smem_u32(ring + stage * kStage), vs = ks + kKeys * kRow;
    const int live = len - (at.t * kTile + warp * kKeys);
    if (live > 0) w.tile(ks, vs, live, c);
    __syncwarp();
    stage = stage + 1 == prm.stages ? 0 : stage + 1;

    const bool ends = at.t + 1 == at.tiles;
    if (ends || left == 1) {
      // the CTA's part of the segment: merge the four warps
      w.publish(merge, ml, warp, rows, prm.rows);
      __syncthreads();
      const bool starts_here = left + at.t <= i1 - i0;  // the segment's first tile is this CTA's
      const bool complete = ends && starts_here;
      float* part = prm.part + (int64_t(blockIdx.x) * 2 + (starts_here ? 1 : 0)) * prm.rows * (prm.dh + 2);
      for (int i = threadIdx.x; i < rows * (HD / 2); i += KD_THREADS) {
        const int r = i / (HD / 2), d = 2 * (i % (HD / 2));
        if (d >= prm.dh) continue;
        float M, L, x0, x1;
        decode_merge<HD>(merge, ml, prm.rows, r, d, M, L, x0, x1);
        if (complete) {
          const float inv = 1.f / L;
          *reinterpret_cast<uint32_t*>(prm.out + ((rank * prm.B + at.b) * prm.hq + head0 + r) * prm.dh + d) =
              pack_bf16x2(x0 * inv, x1 * inv);
        } else {
          float* p = part + r * (prm.dh + 2);
          *reinterpret_cast<float2*>(p + d) = make_float2(x0, x1);
          if (d == 0) *reinterpret_cast<float2*>(p + prm.dh) = make_float2(M, L);
        }
      }
      __syncthreads();
      if (!complete) {
        const int64_t begin = i1 - left - at.t;
        const int z0 = starts_here ? blockIdx.x : deal.owner(begin), z1 = deal.owner(begin + at.tiles - 1);
        if (threadIdx.x == 0) {
          __threadfence();
          asm volatile("griddepcontrol.wait;" ::: "memory");  // the counters are cleared
          last_part = atomicAdd(prm.count + z0, 1u) == static_cast<unsigned int>(z1 - z0);
          __threadfence();
        }
        __syncthreads();
        if (last_part) decode_join(prm, z0, z1, at.b, rank, head0, rows, warp, lane);
      }
      fresh = true;
    }
    at.next(prm, pre);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (every block, so that the clearing never outlives this kernel)
}

// The same with a cluster of CTAs per segment instead of the even deal: each CTA takes an equal part of the
// segment's tiles, and the parts are joined through distributed shared memory, so that there is one
// launch and no workspace.  The deal is kept for what this does badly: contexts so long that one
// sequence's part would outlast all others, and short parts in more clusters than fit the SMs at once.
template <int HD>
__global__ void __launch_bounds__(KD_THREADS, 2) attn_decode_cluster_kernel(const __grid_constant__ DecodeAttnParams prm, int ctas) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  constexpr int kKeys = kd_keys(HD);
  constexpr int kTile = 4 * kKeys;
  constexpr int kRow = HD * 2;
  constexpr int kStage = 2 * kKeys * kRow;
  constexpr int kChunks = HD / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem_raw + warp * prm.stages * kStage;
  float* merge = reinterpret_cast<float*>(smem_raw + 4 * prm.stages * kStage);  // [4][rows][HD]
  float* ml = merge + 4 * prm.rows * HD;                                        // [4][rows][2], then this CTA's [rows][2]
  const int part = blockIdx.x % ctas;
  const int64_t seg = blockIdx.x / ctas;
  // a sequence's segments are neighbours: (sequence, rank, key head, block of heads)
  const int64_t b = seg / prm.G;
  const int g = static_cast<int>(seg - b * prm.G);
  const int gb = g % prm.n_gb, x = g / prm.n_gb, rank = x / prm.hk, kvh = x - rank * prm.hk;
  const int rows = min(prm.group - 16 * gb, 16), head0 = kvh * prm.group + 16 * gb;
  const int asked = __ldg(prm.lens + b);
  const int len = asked > 0 && asked <= prm.capacity ? asked : 0;
  __nv_bfloat16* out = prm.out + ((rank * prm.B + b) * prm.hq + head0) * prm.dh;
  if (len == 0) {  // (the whole cluster)
    if (asked != 0 && g == 0 && threadIdx.x == 0 && part == 0) atomicCAS(&g_arg_status, 0, (82 << 8) | 1);
    if (part == 0)
      for (int i = threadIdx.x; i < rows * prm.dh / 8; i += KD_THREADS) st_v4(out + 8 * i, make_uint4(0, 0, 0, 0));
    return;
  }
  const int tiles = (len + kTile - 1) / kTile;
  const int t0 = static_cast<int>(int64_t(tiles) * part / ctas), t1 = static_cast<int>(int64_t(tiles) * (part + 1) / ctas);

  const int my_key = warp * kKeys + lane / kChunks, my_chunk = lane % kChunks;
  const int64_t tok = int64_t(prm.hk) * prm.dh;
  const int64_t off = ((rank * prm.B + b) * prm.capacity + t0 * kTile + my_key) * tok + int64_t(kvh) * prm.dh + my_chunk * 8;
  const __nv_bfloat16 *kp = prm.k + off, *vp = prm.v + off;
  int ahead = my_chunk * 8 < prm.dh ? len - t0 * kTile - my_key : 0;
  int todo = t1 - t0;
  auto load = [&](int stage) {
    if (todo > 0) {
      decode_copy<HD>(smem_u32(ring + stage * kStage), kp, vp, tok, ahead, prm.k, lane);
      kp += kTile * tok;
      vp += kTile * tok;
      ahead -= kTile;
      --todo;
    }
    cp_async_commit();
  };
  for (int s = 0; s < prm.stages - 1; ++s) load(s);
  const float c = prm.scale * KA_LOG2E;
  DecodeWarp<HD> w;
  w.lane = lane;
  w.r0 = lane >> 2;
  w.begin(prm.q + rank * prm.q_rank + b * prm.q_tok + int64_t(head0) * prm.dh, rows, prm.dh);
  int stage = 0, ld_stage = prm.stages - 1;
  for (int t = t0; t < t1; ++t) {
    load(ld_stage);
    ld_stage = ld_stage + 1 == prm.stages ? 0 : ld_stage + 1;
    cp_async_wait_stages(prm.stages);
    __syncwarp();
    const uint32_t ks = smem_u32(ring + stage * kStage);
    const int live = len - (t * kTile + warp * kKeys);
    if (live > 0) w.tile(ks, ks + kKeys * kRow, live, c);
    __syncwarp();
    stage = stage + 1 == prm.stages ? 0 : stage + 1;
  }
  w.publish(merge, ml, warp, rows, prm.rows);
  __syncthreads();
  float* cta_ml = ml + 4 * prm.rows * 2;
  for (int i = threadIdx.x; i < rows * (HD / 2); i += KD_THREADS) {
    const int r = i / (HD / 2), d = 2 * (i % (HD / 2));
    float M, L, x0, x1;
    decode_merge<HD>(merge, ml, prm.rows, r, d, M, L, x0, x1);
    if (ctas == 1) {
      const float inv = 1.f / L;
      if (d < prm.dh) *reinterpret_cast<uint32_t*>(out + r * prm.dh + d) = pack_bf16x2(x0 * inv, x1 * inv);
    } else {
      *reinterpret_cast<float2*>(merge + r * HD + d) = make_float2(x0, x1);  // over warp 0's, read by this thread alone
      if (d == 0) {
        cta_ml[2 * r] = M;
        cta_ml[2 * r + 1] = L;
      }
    }
  }
  if (ctas == 1) return;
  cluster_sync();
  for (int i = part * KD_THREADS + threadIdx.x; i < rows * (HD / 2); i += ctas * KD_THREADS) {
    const int r = i / (HD / 2), d = 2 * (i % (HD / 2));
    if (d >= prm.dh) continue;
    const uint32_t at_ml = smem_u32(cta_ml + 2 * r), at_x = smem_u32(merge + r * HD + d);
    float2 pm[8], px[8];
#pragma unroll
    for (int z = 0; z < 8; ++z)
      if (z < ctas) {
        pm[z] = ld_cluster_f32x2(mapa_shared(at_ml, z));
        px[z] = ld_cluster_f32x2(mapa_shared(at_x, z));
      }
    float M = -INFINITY, L = 0.f, x0 = 0.f, x1 = 0.f;
#pragma unroll
    for (int z = 0; z < 8; ++z)
      if (z < ctas) M = fmaxf(M, pm[z].x);
    const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int z = 0; z < 8; ++z)
      if (z < ctas) {
        const float f = ex2(pm[z].x - base);
        L = fmaf(f, pm[z].y, L);
        x0 = fmaf(f, px[z].x, x0);
        x1 = fmaf(f, px[z].y, x1);
      }
    const float inv = 1.f / L;
    *reinterpret_cast<uint32_t*>(out + r * prm.dh + d) = pack_bf16x2(x0 * inv, x1 * inv);
  }
  cluster_sync();  // nobody leaves while its results are read
}

}  // namespace caat
