// attn_bwd.cuh - gradients of the packed causal attention on the tensor cores.
//
//   p_ij = 2^(c s_ij - lse_i log2(e)),  dP = dO V^T,  D_i = sum_d dO_id O_id,  dS = p (dP - D)
//   dQ = scale dS K,   dV = p^T dO,   dK = scale dS^T Q
//
// Two kernels, so that every sum has one owner and a fixed order (one kernel that walks the scores
// once would have to add dQ into memory from every key block, in an order that changes from run to
// run): dq walks the keys of a query tile and also leaves D for the second; dkv walks the queries of
// a key tile.  The scores and dP are computed in both: 7 products of 128 x 128 x dh per pair of
// tiles instead of 5.
//
// p and dS are rounded to bf16 to be operands of the products (their A operand, read from tensor
// memory); the scale is applied once to the fp32 sums.  Masked scores are replaced, never added to;
// operand rows of another sequence that meet p = 0 or dS = 0 in a product are zeroed in shared memory
// first, since 0 times a NaN or an infinity is NaN.
#pragma once

#include "attn_common.cuh"

namespace caat {

constexpr int KB2_THREADS = 384;  // dkv: warps 0-7 elementwise, 8 MMA, 9 TMA, 10 scrubbing, 11 idle
constexpr int KB2_QT = 64;        // queries per step of the dkv kernel

struct BwdAttnParams {
  const __nv_bfloat16* out;   // [P, Tq, hq, dh]
  const __nv_bfloat16* dout;
  const float* lse;           // [P, hq, Tq]
  float* D;                   // [P, hq, Tq]
  __nv_bfloat16 *dq, *dk, *dv;
  float* part;                // [2][splits][P, Tk, hk, dh] partial dk, dv (splits > 1)
  int64_t Tq, Tk;
  int P, hq, hk, dh, group;
  int per_job;                // grid units per job
  int splits;                 // CTAs that share the queries of a key tile
  float scale;
  uint64_t timeout_ns;
  AttnJobList jobs;
};

template <int HD>
struct DqCfg {
  static constexpr int kBoxes = HD / 64;
  static constexpr int kTileBytes = kBoxes * KA_BOX_BYTES;        // Q or dO: 128 queries
  static constexpr int kKeys = HD;                                // keys of a block
  static constexpr int kBox = kKeys * 128;                        // K or V: a block of 64 elements
  static constexpr int kBlockBytes = kBoxes * kBox;
  static constexpr int kHalves = kKeys / 64;                      // a thread has one row and 64 keys
  static constexpr int kEw = 4 * kHalves;                         // elementwise warps; behind them MMA, TMA, scrubbing, idle
  static constexpr int kThreads = 32 * (kEw + 4);
  static constexpr int kCtas = HD == 128 ? 1 : 2;                 // per SM
  static constexpr int kTmem = 512 / kCtas;                       // columns: S | dP | dQ | dS of even blocks | of odd blocks
  // A K block is held until the product with dS, one block longer than its V block.
  static constexpr int kK = HD == 128 ? 3 : 5;
  static constexpr int kV = HD == 128 ? 2 : 4;
  static constexpr int kSlots = kK + kV;
  static constexpr int kSmem = 1024 + 2 * kTileBytes + kSlots * kBlockBytes + 2 * KA_TILE * 4 + 512;
  static __device__ __forceinline__ int k_slot(int j) { return j % kK; }
  static __device__ __forceinline__ int v_slot(int j) { return kK + j % kV; }
};

// One CTA: 128 queries of one head.  All elementwise warps work on one block at a time; they copy S and dP to
// registers and free them at once, so that the next block's two products run meanwhile, and the product with
// K follows when dS is written.  Of dh <= 64, two CTAs of half the size share an SM (blocks of 64 keys, half
// of the tensor memory): one's start, end and waits are hidden by the other (packed sequences of 5 to 2048 tokens, 32 heads: 81 us to 68).
//
// Where the tile sees 128 keys at most, the sum of p dP over them is D without the rounding of the stored
// output, whose share of the error is largest in such rows (dq of 5 to 2048 tokens off by 0.0025 relative
// without this, 0.0024 with; the rounding of dq itself is 0.0017).  A pass over the blocks ahead of the others
// finds it.
//
// dS has a barrier per buffer.  A warp frees S and dP before it has written its dS, so the next block's scores
// may be there, and a fast warp be done with that block too, before a slow one has arrived for this: on one
// barrier the fast warp's second arrival would count for the slow one's first, and the product would read 32 rows
// that nobody has written.  A warp's next arrival on the same barrier, two blocks on, is behind the scores of
// that block, which need every warp to have freed the block in between, and each does so after its arrival here.
template <int HD>
__global__ void __launch_bounds__(DqCfg<HD>::kThreads, DqCfg<HD>::kCtas)
    attn_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ BwdAttnParams prm) {
  using Cfg = DqCfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];  // (a known address: no registers spent on it)
  uint8_t* sQ = smem;
  uint8_t* sG = smem + Cfg::kTileBytes;
  uint8_t* sRing = smem + 2 * Cfg::kTileBytes;
  float* sD = reinterpret_cast<float*>(sRing + Cfg::kSlots * Cfg::kBlockBytes);  // [2][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sD + 2 * KA_TILE);
  uint64_t* q_full = bars;
  uint64_t* full = q_full + 1;             // [slots]
  uint64_t* empty = full + Cfg::kSlots;    // [slots]
  uint64_t* sd_full = empty + Cfg::kSlots;
  uint64_t* sd_free = sd_full + 1;         // elementwise warps
  uint64_t* ds_full = sd_free + 1;         // [2 dS buffers] elementwise warps
  uint64_t* k_raw = ds_full + 2;           // the last key block has arrived, to be scrubbed
  uint64_t* scrubbed = k_raw + 1;
  uint64_t* dq_done = scrubbed + 1;
  uint64_t* d_full = dq_done + 1;          // elementwise warps
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(d_full + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled tiles would not line up
    if (threadIdx.x == 0) status_raise(2, 90);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int ji = blockIdx.x / prm.per_job;
  const int rh = blockIdx.x - ji * prm.per_job;
  const int rank = rh / prm.hq;
  const int head = rh - rank * prm.hq;
  const int kvh = head / prm.group;
  const AttnJob job = prm.jobs.far ? prm.jobs.far[ji] : prm.jobs.near[ji];
  const int m_seen = max(job.first + job.rows - 1, 0);
  const int n_blk = (m_seen + Cfg::kKeys - 1) / Cfg::kKeys;
  const int n_pre = m_seen <= KA_TILE ? n_blk : 0;        // blocks of the pass for D
  const int n_all = n_pre + n_blk;
  const bool ragged = (m_seen & (Cfg::kKeys - 1)) != 0;  // the last block reaches past the sequence's keys

  // The TMA warp sets up the barriers and sends the first loads off before the block meets; the elementwise
  // warps' loads for D go out before that, too.
  const uint64_t pol_q = policy_evict_first(), pol_kv = policy_evict_last();
  auto load_kv = [&](int i) {
    const int j = i >> 1;
    const int slot = (i & 1) ? Cfg::v_slot(j) : Cfg::k_slot(j);
    uint64_t* bar = &full[slot];
    if (ragged && i == 2 * (n_all - 1)) {
      bar = k_raw;
      mbar_arrive(&full[slot]);
    }
    mbar_arrive_expect_tx(bar, Cfg::kBlockBytes);
    for (int b = 0; b < Cfg::kBoxes; ++b)
      tma_load_4d(sRing + slot * Cfg::kBlockBytes + b * Cfg::kBox, (i & 1) ? &tmV : &tmK, bar, 64 * b, kvh,
                  job.k0 + (j < n_pre ? j : j - n_pre) * Cfg::kKeys, rank, pol_kv);
  };
  if (warp == Cfg::kEw + 1 && lane == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < Cfg::kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(sd_full, 1);
    mbar_init(sd_free, Cfg::kEw);
    for (int b = 0; b < 2; ++b) mbar_init(&ds_full[b], Cfg::kEw);
    mbar_init(k_raw, 1);
    mbar_init(scrubbed, 1);
    mbar_init(dq_done, 1);
    mbar_init(d_full, Cfg::kEw);
    fence_mbar_init();
    if (n_blk > 0) {
      mbar_arrive_expect_tx(q_full, 2 * Cfg::kTileBytes);
      for (int b = 0; b < Cfg::kBoxes; ++b) tma_load_4d(sQ + b * KA_BOX_BYTES, &tmQ, q_full, 64 * b, head, job.q0, rank, pol_q);
      load_kv(0);
      for (int b = 0; b < Cfg::kBoxes; ++b) tma_load_4d(sG + b * KA_BOX_BYTES, &tmG, q_full, 64 * b, head, job.q0, rank, pol_q);
      load_kv(1);
    }
  }
  constexpr int kLanes = HD / 8;  // of a row, for D; a warp's rows: 8 times as many as it has at once
  uint4 d_o[8], d_g[8];
  if (warp < Cfg::kEw && n_pre == 0) {
    const int e = 8 * (lane % kLanes);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = (8 * warp + i) * (32 / kLanes) + lane / kLanes;
      const bool in = r < job.rows && e < prm.dh;
      const int64_t off = ((rank * prm.Tq + job.q0 + r) * prm.hq + head) * prm.dh + e;
      d_o[i] = in ? ld_nc_v4(prm.out + off) : make_uint4(0, 0, 0, 0);
      d_g[i] = in ? ld_nc_v4(prm.dout + off) : make_uint4(0, 0, 0, 0);
    }
  }
  if (warp == Cfg::kEw) {
    tmem_alloc(tmem_holder, Cfg::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = Cfg::kCtas == 1 ? 0 : *tmem_holder;  // all 512 columns: the allocation starts at the first
  const uint64_t tmo = prm.timeout_ns;
  constexpr uint32_t kDP = Cfg::kKeys, kDQ = 2 * Cfg::kKeys, kDS = kDQ + HD;  // tensor memory columns

  if (warp >= Cfg::kEw) {
    if constexpr (HD == 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == Cfg::kEw + 1) {
      if (lane == 0 && n_blk > 0) {
        bool ok = true;
        for (int i = 2; i < 2 * n_all && ok; ++i) {
          const int j = i >> 1;
          const int slot = (i & 1) ? Cfg::v_slot(j) : Cfg::k_slot(j);
          ok = mbar_wait(&empty[slot], ((j / ((i & 1) ? Cfg::kV : Cfg::kK)) & 1) ^ 1, tmo, 111);
          if (ok) load_kv(i);
        }
        if (!ok) spin_ns(KA_DRAIN_NS);
      }
    } else if (warp == Cfg::kEw) {
      if (n_blk > 0) {
        const uint32_t lead = elect_one();
        constexpr uint32_t id_s = idesc_bf16_f32(KA_TILE, Cfg::kKeys);
        constexpr uint32_t id_q = idesc_bf16_f32_major(KA_TILE, HD, false, true);
        constexpr uint32_t kBlock16 = Cfg::kBlockBytes >> 4;
        const uint64_t dQ = sw128_kmajor_desc(smem_u32(sQ)), dG = sw128_kmajor_desc(smem_u32(sG));
        const uint64_t dR = sw128_kmajor_desc(smem_u32(sRing)), dRt = sw128_mnmajor_desc_128(smem_u32(sRing));
        int ks = 0, vs = 0;            // slots of the next K and V block, and their phases
        uint32_t kp = 0, vp = 0;
        auto scores = [&](int j) {
          if (!lane_wait(&full[ks], kp, tmo, 112)) return false;
          if (ragged && j == n_all - 1 && !lane_wait(scrubbed, 0, tmo, 113)) return false;
          const uint64_t dk = dR + ks * kBlock16;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * KA_BOX_BYTES + (kk & 3) * 32) >> 4;
            umma_ss(lead, tmem, dQ + off, dk + (((kk >> 2) * Cfg::kBox + (kk & 3) * 32) >> 4), id_s, kk > 0);
          }
          if (!lane_wait(&full[Cfg::kK + vs], vp, tmo, 114)) return false;
          const uint64_t dv = dR + (Cfg::kK + vs) * kBlock16;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * KA_BOX_BYTES + (kk & 3) * 32) >> 4;
            umma_ss(lead, tmem + kDP, dG + off, dv + (((kk >> 2) * Cfg::kBox + (kk & 3) * 32) >> 4), id_s, kk > 0);
          }
          // also the completion of the product with dS two blocks back, whose buffer comes next
          umma_arrive(lead, sd_full);
          umma_arrive(lead, &empty[Cfg::kK + vs]);
          if (++ks == Cfg::kK) { ks = 0; kp ^= 1; }
          if (++vs == Cfg::kV) { vs = 0; vp ^= 1; }
          return true;
        };
        bool ok = lane_wait(q_full, 0, tmo, 115) && scores(0);
        int kq = 0;  // slot of the block whose dS comes next
        for (int j = 0; j < n_all && ok; ++j) {
          if (j + 1 < n_all) {
            ok = lane_wait(sd_free, j & 1, tmo, 116);
            if (!ok) break;
            tc_fence_after();
            ok = scores(j + 1);
            if (!ok) break;
          }
          if (j >= n_pre) {
            const int i = j - n_pre;
            ok = lane_wait(&ds_full[i & 1], (i >> 1) & 1, tmo, 117);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dk = dRt + kq * kBlock16;
#pragma unroll
            for (int kk = 0; kk < Cfg::kKeys / 16; ++kk)
              umma_ts(lead, tmem + kDQ, tmem + kDS + (i & 1) * (Cfg::kKeys / 2) + 8 * kk, dk + (kk * 2048 >> 4), id_q,
                      (i > 0 || kk > 0) ? 1u : 0u);
          }
          umma_arrive(lead, &empty[kq]);
          if (++kq == Cfg::kK) kq = 0;
        }
        umma_arrive(lead, dq_done);
        lane_wait(dq_done, 0, tmo, 118);
      }
    } else if (warp == Cfg::kEw + 2 && ragged) {
      if (warp_wait(k_raw, 0, tmo, 119)) {
        uint8_t* k = sRing + Cfg::k_slot(n_all - 1) * Cfg::kBlockBytes;
        const int live = m_seen - (n_blk - 1) * Cfg::kKeys;
        for (int b = 0; b < Cfg::kBoxes; ++b)
          for (int x = live * 8 + lane; x < Cfg::kKeys * 8; x += 32)
            reinterpret_cast<uint4*>(k + b * Cfg::kBox)[x] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(scrubbed);
      }
    }
  } else {
    if constexpr (HD == 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int w = warp >> 2;  // which half of the block's keys, and of dQ's columns at the end
    const int q = warp & 3;
    const int row = q * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const bool mine = row < job.rows;
    const int64_t grow = job.q0 + row;
    const int64_t srow = (int64_t(rank) * prm.hq + head) * prm.Tq + grow;
    float D = 0.f;
    if (n_pre == 0) {
      // (a row a lane, the loads touched 32 rows each and took 12,000 clocks)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t wa[4] = {d_o[i].x, d_o[i].y, d_o[i].z, d_o[i].w}, wb[4] = {d_g[i].x, d_g[i].y, d_g[i].z, d_g[i].w};
        float part = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          part = fmaf(bf16lo(wa[u]), bf16lo(wb[u]), part);
          part = fmaf(bf16hi(wa[u]), bf16hi(wb[u]), part);
        }
#pragma unroll
        for (int e = kLanes / 2; e > 0; e >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, e);
        if (lane % kLanes == 0) sD[(8 * warp + i) * (32 / kLanes) + lane / kLanes] = part;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * Cfg::kEw) : "memory");
      D = sD[row];
      if (mine && w == 0) prm.D[srow] = D;
    }
    const float c = prm.scale * KA_LOG2E;
    float nl = mine ? -prm.lse[srow] * KA_LOG2E : 0.f;
    if (nl == INFINITY) nl = 0.f;  // a row that sees no key: all its scores are masked
    const uint64_t c2 = pack_f32x2(c, c), nl2 = pack_f32x2(nl, nl);
    const int vis = job.first + row;
    bool ok = true;
    uint64_t sum2 = 0;
    for (int j = 0; j < n_all; ++j) {
      ok = warp_wait(sd_full, j & 1, tmo, 120);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[64], g[64];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        tmem_ld_32x32b_x32(lanes + 64 * w + 32 * x, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * x));
        tmem_ld_32x32b_x32(lanes + kDP + 64 * w + 32 * x, *reinterpret_cast<uint32_t(*)[32]>(g + 32 * x));
      }
      tmem_wait_ld(g);
      tmem_wait_ld(s);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sd_free);
      const int key0 = (j < n_pre ? j : j - n_pre) * Cfg::kKeys + 64 * w;
      const int seen = vis - key0;
      const bool cut = job.first + q * 32 - key0 < 64;
      if (cut) {
        // unseen: s = -inf makes p = 0, and dP = 0 keeps dS = p (dP - D) from being 0 times a NaN
#pragma unroll
        for (int y = 0; y < 64; ++y) {
          s[y] = y < seen ? s[y] : 0xFF800000u;
          g[y] = y < seen ? g[y] : 0u;
        }
      }
      auto prob = [&](int y) {
        float a, b;
        unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[2 * y]), __uint_as_float(s[2 * y + 1])), c2, nl2), a, b);
        return pack_f32x2(ex2(a), ex2(b));
      };
      auto dp = [&](int y) { return pack_f32x2(__uint_as_float(g[2 * y]), __uint_as_float(g[2 * y + 1])); };
      if (j < n_pre) {
#pragma unroll
        for (int y = 0; y < 32; ++y) sum2 = fma_f32x2(prob(y), dp(y), sum2);
        if (j + 1 < n_pre) continue;
        float a, b;
        unpack_f32x2(sum2, a, b);
        D = a + b;
        if constexpr (Cfg::kHalves == 2) {
          sD[w * KA_TILE + row] = D;
          __syncwarp();
          if (lane == 0) mbar_arrive(d_full);
          ok = warp_wait(d_full, 0, tmo, 122);
          if (!ok) break;
          D = sD[row] + sD[KA_TILE + row];
        }
        if (mine && w == 0) prm.D[srow] = D;
        continue;
      }
      const uint64_t nd2 = pack_f32x2(-D, -D);
      uint32_t p[32];
#pragma unroll
      for (int y = 0; y < 32; ++y) {
        float x0, x1;
        unpack_f32x2(mul_f32x2(prob(y), add_f32x2(dp(y), nd2)), x0, x1);
        p[y] = pack_bf16x2(x0, x1);
      }
      const int buf = (j - n_pre) & 1;
      tmem_st_32x32b_x32(lanes + kDS + buf * (Cfg::kKeys / 2) + 32 * w, p);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ds_full[buf]);
    }
    if (ok && n_blk > 0) ok = warp_wait(dq_done, 0, tmo, 121);
    tc_fence_after();
    if (ok) {
      // every product is done: the Q tile's place serves to turn the rows
      const int e = 64 * w;
      uint4 v[8];
#pragma unroll
      for (int x = 0; x < 64; x += 32) {
        uint32_t o[32];
        if (n_blk > 0) {
          tmem_ld_32x32b_x32(lanes + kDQ + e + x, o);
          tmem_wait_ld(o);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t u[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            u[z] = n_blk > 0 ? pack_bf16x2(__uint_as_float(o[8 * y + 2 * z]) * prm.scale, __uint_as_float(o[8 * y + 2 * z + 1]) * prm.scale) : 0u;
          v[x / 8 + y] = make_uint4(u[0], u[1], u[2], u[3]);
        }
      }
      const int64_t base = ((rank * prm.Tq + job.q0 + q * 32) * prm.hq + head) * prm.dh + e;
      warp_store_rows(sQ + warp * 4096, v, reinterpret_cast<uint8_t*>(prm.dq + base), int64_t(prm.hq) * prm.dh * 2,
                      job.rows - q * 32, (prm.dh - e) / 8, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == Cfg::kEw) tmem_dealloc(tmem, Cfg::kTmem);
}

template <int HD>
struct DkvCfg {
  static constexpr int kBoxes = HD / 64;
  static constexpr int kTileBytes = kBoxes * KA_BOX_BYTES;         // K or V: 128 keys
  static constexpr int kQBox = KB2_QT * 128;                       // 64 queries x 64 elements
  static constexpr int kQBytes = kBoxes * kQBox;                   // Q or dO: 64 queries
  static constexpr int kStages = HD == 128 ? 4 : 8;
  static constexpr int kBufs = HD == 128 ? 2 : 3;                  // (S^T | dP^T) in tensor memory beside dV and dK
  static constexpr int kSmem = 1024 + 2 * kTileBytes + kStages * (2 * kQBytes + 2 * KB2_QT * 4) + 512;
};

// One CTA: 128 keys of one key head, against its share (1 / splits) of the queries of the group's
// heads, 64 at a time.  Tensor memory: (S^T | dP^T) of two steps (dh <= 64: three) | dV | dK, S^T and
// dP^T with the keys in the lanes; p^T and dS^T are written over them and are the A operands of the
// two sums.  Warps 0-3 take the even steps, 4-7 the odd ones: while one set computes, the tensor
// cores run the other step's products.  Warp 10 passes on every tile of Q and dO: it zeroes the rows
// behind the sequence's last query and puts lse and D beside the tile.
//
// Job: `rows` queries from row q0 on see keys of the tile that starts at row k0 and has k_rows keys:
// query x sees key y when x >= y + first.
template <int HD>
__global__ void __launch_bounds__(KB2_THREADS, 1)
    attn_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ BwdAttnParams prm) {
  using Cfg = DkvCfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];  // (a known address: no registers spent on it)
  uint8_t* sK = smem;
  uint8_t* sV = smem + Cfg::kTileBytes;
  uint8_t* sQ = smem + 2 * Cfg::kTileBytes;
  uint8_t* sG = sQ + Cfg::kStages * Cfg::kQBytes;
  float* sL = reinterpret_cast<float*>(sG + Cfg::kStages * Cfg::kQBytes);  // [stages][2][64]: -lse log2(e), -D
  uint64_t* bars = reinterpret_cast<uint64_t*>(sL + Cfg::kStages * 2 * KB2_QT);
  uint64_t* kv_full = bars;
  uint64_t* raw = kv_full + 1;             // [stages] TMA
  uint64_t* full = raw + Cfg::kStages;     // [stages] passed on by warp 10
  uint64_t* empty = full + Cfg::kStages;   // [stages]
  uint64_t* sd_full = empty + Cfg::kStages;  // [bufs]
  uint64_t* pd_full = sd_full + Cfg::kBufs;  // [bufs] 4 warps
  uint64_t* done = pd_full + Cfg::kBufs;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled tiles would not line up
    if (threadIdx.x == 0) status_raise(2, 90);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int ji = blockIdx.x / prm.per_job;
  int rest = blockIdx.x - ji * prm.per_job;
  const int split = rest % prm.splits;
  rest /= prm.splits;
  const int rank = rest / prm.hk;
  const int kvh = rest - rank * prm.hk;
  const AttnJob job = prm.jobs.far ? prm.jobs.far[ji] : prm.jobs.near[ji];
  const int nt = (job.rows + KB2_QT - 1) / KB2_QT;
  const int total = nt * prm.group;
  const int it0 = static_cast<int>(int64_t(total) * split / prm.splits);
  const int n = static_cast<int>(int64_t(total) * (split + 1) / prm.splits) - it0;

  const uint64_t pol_kv = policy_evict_first(), pol_q = policy_evict_last();
  auto load_q = [&](int i) {
    const int st = i % Cfg::kStages, h = (it0 + i) / nt, x = (it0 + i) - h * nt;
    mbar_arrive_expect_tx(&raw[st], 2 * Cfg::kQBytes);
    for (int b = 0; b < Cfg::kBoxes; ++b) {
      tma_load_4d(sQ + st * Cfg::kQBytes + b * Cfg::kQBox, &tmQ, &raw[st], 64 * b, kvh * prm.group + h,
                  job.q0 + x * KB2_QT, rank, pol_q);
      tma_load_4d(sG + st * Cfg::kQBytes + b * Cfg::kQBox, &tmG, &raw[st], 64 * b, kvh * prm.group + h,
                  job.q0 + x * KB2_QT, rank, pol_q);
    }
  };
  if (threadIdx.x == 9 * 32) {  // the TMA warp sends the first loads off before the block meets
    mbar_init(kv_full, 1);
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(&raw[s], 1);
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < Cfg::kBufs; ++b) {
      mbar_init(&sd_full[b], 1);
      mbar_init(&pd_full[b], 4);
    }
    mbar_init(done, 1);
    fence_mbar_init();
    if (n > 0) {
      mbar_arrive_expect_tx(kv_full, 2 * Cfg::kTileBytes);
      for (int b = 0; b < Cfg::kBoxes; ++b) tma_load_4d(sK + b * KA_BOX_BYTES, &tmK, kv_full, 64 * b, kvh, job.k0, rank, pol_kv);
      load_q(0);
      for (int b = 0; b < Cfg::kBoxes; ++b) tma_load_4d(sV + b * KA_BOX_BYTES, &tmV, kv_full, 64 * b, kvh, job.k0, rank, pol_kv);
    }
  }
  if (warp == 8) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns: the allocation starts at the first
  const uint64_t tmo = prm.timeout_ns;
  constexpr uint32_t kDV = Cfg::kBufs * 2 * KB2_QT, kDK = kDV + HD;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 9) {
      if (lane == 0 && n > 0) {
        bool ok = true;
        for (int i = 1; i < n && ok; ++i) {
          ok = mbar_wait(&empty[i % Cfg::kStages], ((i / Cfg::kStages) & 1) ^ 1, tmo, 131);
          if (ok) load_q(i);
        }
        if (!ok) spin_ns(KA_DRAIN_NS);
      }
    } else if (warp == 8) {
      if (n > 0) {
        const uint32_t lead = elect_one();
        constexpr uint32_t id_s = idesc_bf16_f32(KA_TILE, KB2_QT);
        constexpr uint32_t id_g = idesc_bf16_f32_major(KA_TILE, HD, false, true);
        constexpr uint32_t kQ16 = Cfg::kQBytes >> 4;
        const uint64_t dK = sw128_kmajor_desc(smem_u32(sK)), dV = sw128_kmajor_desc(smem_u32(sV));
        const uint64_t dQ = sw128_kmajor_desc(smem_u32(sQ)), dG = sw128_kmajor_desc(smem_u32(sG));
        const uint64_t dQt = sw128_mnmajor_desc(smem_u32(sQ)), dGt = sw128_mnmajor_desc(smem_u32(sG));
        int ss = 0, st = 0;  // stages of the next scores and of the next sums
        uint32_t sp = 0, buf = 0, bp = 0;
        auto scores = [&](uint32_t buf) {
          if (!lane_wait(&full[ss], sp, tmo, 132)) return false;
          const uint64_t q = dQ + ss * kQ16, g = dG + ss * kQ16;
          const uint32_t d = tmem + buf * 2 * KB2_QT;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            umma_ss(lead, d, dK + (((kk >> 2) * KA_BOX_BYTES + (kk & 3) * 32) >> 4),
                    q + (((kk >> 2) * Cfg::kQBox + (kk & 3) * 32) >> 4), id_s, kk > 0);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            umma_ss(lead, d + KB2_QT, dV + (((kk >> 2) * KA_BOX_BYTES + (kk & 3) * 32) >> 4),
                    g + (((kk >> 2) * Cfg::kQBox + (kk & 3) * 32) >> 4), id_s, kk > 0);
          umma_arrive(lead, &sd_full[buf]);
          if (++ss == Cfg::kStages) { ss = 0; sp ^= 1; }
          return true;
        };
        bool ok = lane_wait(kv_full, 0, tmo, 133);
#pragma unroll 1
        for (int i = -Cfg::kBufs; i < n && ok; ++i) {
          if (i >= 0) {
            ok = lane_wait(&pd_full[buf], bp, tmo, 134);
            if (!ok) break;
            tc_fence_after();
            const uint64_t q = dQt + st * kQ16, g = dGt + st * kQ16;
            const uint32_t a = tmem + buf * 2 * KB2_QT;
#pragma unroll
            for (int kk = 0; kk < KB2_QT / 16; ++kk)
              umma_ts(lead, tmem + kDV, a + 8 * kk, g + (kk * 2048 >> 4), id_g, (i > 0 || kk > 0) ? 1u : 0u);
#pragma unroll
            for (int kk = 0; kk < KB2_QT / 16; ++kk)
              umma_ts(lead, tmem + kDK, a + KB2_QT + 8 * kk, q + (kk * 2048 >> 4), id_g, (i > 0 || kk > 0) ? 1u : 0u);
            umma_arrive(lead, &empty[st]);
            if (++st == Cfg::kStages) st = 0;
          }
          if (i + Cfg::kBufs < n) ok = scores(buf);
          if (++buf == Cfg::kBufs) {
            buf = 0;
            if (i >= 0) bp ^= 1;
          }
        }
        umma_arrive(lead, done);
        lane_wait(done, 0, tmo, 135);
      }
    } else if (warp == 10) {
      asm volatile("griddepcontrol.wait;" ::: "memory");  // D is there (and no CTA ends before the dq kernel)
      for (int i = 0; i < n; ++i) {
        const int st = i % Cfg::kStages;
        const uint32_t ph = (i / Cfg::kStages) & 1;
        const int h = (it0 + i) / nt, x = ((it0 + i) - h * nt) * KB2_QT;
        const int live = min(job.rows - x, KB2_QT);
        const int64_t srow = (int64_t(rank) * prm.hq + kvh * prm.group + h) * prm.Tq + job.q0 + x;
        float v[4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int y = lane + 32 * u;
          v[u] = y < live ? -prm.lse[srow + y] * KA_LOG2E : 0.f;
          v[2 + u] = y < live ? -prm.D[srow + y] : 0.f;
        }
        if (!warp_wait(&raw[st], ph, tmo, 136)) break;
        float* l = sL + st * 2 * KB2_QT;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          l[lane + 32 * u] = v[u];
          l[KB2_QT + lane + 32 * u] = v[2 + u];
        }
        if (live < KB2_QT) {
          for (int b = 0; b < Cfg::kBoxes; ++b)
            for (int y = live * 8 + lane; y < KB2_QT * 8; y += 32) {
              reinterpret_cast<uint4*>(sQ + st * Cfg::kQBytes + b * Cfg::kQBox)[y] = make_uint4(0, 0, 0, 0);
              reinterpret_cast<uint4*>(sG + st * Cfg::kQBytes + b * Cfg::kQBox)[y] = make_uint4(0, 0, 0, 0);
            }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int w = warp >> 2;
    const int q = warp & 3;
    const int row = q * 32 + lane;  // key
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const float c = prm.scale * KA_LOG2E;
    const uint64_t c2 = pack_f32x2(c, c);
    bool ok = true;
    int x0 = n > 0 ? ((it0 + w) % nt) * KB2_QT : 0;  // the step's first query
    int buf = w;
    uint32_t bp = 0;
    for (int i = w; i < n; i += 2) {
      const int st = i % Cfg::kStages;
      ok = warp_wait(&full[st], (i / Cfg::kStages) & 1, tmo, 137) && warp_wait(&sd_full[buf], bp, tmo, 138);
      if (!ok) break;
      tc_fence_after();
      const uint32_t base = lanes + buf * 2 * KB2_QT;
      uint32_t s[64], g[64];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        tmem_ld_32x32b_x32(base + 32 * x, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * x));
        tmem_ld_32x32b_x32(base + KB2_QT + 32 * x, *reinterpret_cast<uint32_t(*)[32]>(g + 32 * x));
      }
      tmem_wait_ld(g);
      tmem_wait_ld(s);
      const int lo = row + job.first - x0;    // the key is seen from this query of the step on
      const int hi = job.rows - x0;           // queries of the step
      const bool cut = hi < KB2_QT || q * 32 + 31 + job.first > x0;
      if (cut) {
        // unseen: s = -inf makes p = 0, and dP = 0 keeps dS = p (dP - D) from being 0 times a NaN
#pragma unroll
        for (int y = 0; y < KB2_QT; ++y) {
          const bool see = y >= lo && y < hi;
          s[y] = see ? s[y] : 0xFF800000u;
          g[y] = see ? g[y] : 0u;
        }
      }
      const float4* l = reinterpret_cast<const float4*>(sL + st * 2 * KB2_QT);
      uint32_t pp[32], pd[32];
#pragma unroll
      for (int y = 0; y < 16; ++y) {  // four queries at a time
        const float4 nl = l[y], nd = l[16 + y];
        float a[4], d[4];
        unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[4 * y]), __uint_as_float(s[4 * y + 1])), c2, pack_f32x2(nl.x, nl.y)), a[0], a[1]);
        unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[4 * y + 2]), __uint_as_float(s[4 * y + 3])), c2, pack_f32x2(nl.z, nl.w)), a[2], a[3]);
#pragma unroll
        for (int u = 0; u < 4; ++u) a[u] = ex2(a[u]);
        unpack_f32x2(mul_f32x2(pack_f32x2(a[0], a[1]), add_f32x2(pack_f32x2(__uint_as_float(g[4 * y]), __uint_as_float(g[4 * y + 1])), pack_f32x2(nd.x, nd.y))), d[0], d[1]);
        unpack_f32x2(mul_f32x2(pack_f32x2(a[2], a[3]), add_f32x2(pack_f32x2(__uint_as_float(g[4 * y + 2]), __uint_as_float(g[4 * y + 3])), pack_f32x2(nd.z, nd.w))), d[2], d[3]);
        pp[2 * y] = pack_bf16x2(a[0], a[1]);
        pp[2 * y + 1] = pack_bf16x2(a[2], a[3]);
        pd[2 * y] = pack_bf16x2(d[0], d[1]);
        pd[2 * y + 1] = pack_bf16x2(d[2], d[3]);
      }
      tmem_st_32x32b_x32(base, pp);
      tmem_st_32x32b_x32(base + KB2_QT, pd);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pd_full[buf]);
      if ((buf += 2) >= Cfg::kBufs) {
        buf -= Cfg::kBufs;
        bp ^= 1;
      }
      x0 += 2 * KB2_QT;
      while (x0 >= nt * KB2_QT) x0 -= nt * KB2_QT;  // the next head
    }
    if (ok && n > 0) ok = warp_wait(done, 0, tmo, 139);
    tc_fence_after();
    if (ok) {
      // warps 0-3 store dV, 4-7 dK
      const float f = w ? prm.scale : 1.f;
      const int64_t krow = ((rank * prm.Tk + job.k0 + q * 32) * prm.hk + kvh) * prm.dh;
      const int64_t all = prm.P * prm.Tk * prm.hk * prm.dh, stride = int64_t(prm.hk) * prm.dh;
      const int rows = job.k_rows - q * 32;
      float* pdst = prm.part + (w * prm.splits + split) * all + krow;
      __nv_bfloat16* dst = (w ? prm.dk : prm.dv) + krow;
      uint8_t* patch = sQ + warp * 4096;  // every product is done
#pragma unroll 1
      for (int x = 0; x < HD; x += 32) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld_32x32b_x32(lanes + (w ? kDK : kDV) + x, o);
          tmem_wait_ld(o);
        }
#pragma unroll
        for (int y = 0; y < 32; ++y) o[y] = n > 0 ? __float_as_uint(__uint_as_float(o[y]) * f) : 0u;
        if (prm.splits > 1) {
          uint4 v[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) v[y] = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
          warp_store_rows(patch, v, reinterpret_cast<uint8_t*>(pdst + x), stride * 4, rows, (prm.dh - x) / 4, lane);
        } else {
          uint4 v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t u[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) u[z] = pack_bf16x2(__uint_as_float(o[8 * y + 2 * z]), __uint_as_float(o[8 * y + 2 * z + 1]));
            v[y] = make_uint4(u[0], u[1], u[2], u[3]);
          }
          warp_store_rows(patch, v, reinterpret_cast<uint8_t*>(dst + x), stride * 2, rows, (prm.dh - x) / 8, lane);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// dk, dv of a job's keys from the partial sums, added in the order of the splits.  Each thread has one
// 16-byte piece of dk or dv, four splits' loads in flight (packed 4096 tokens, 4 ranks of one key head of 64,
// 3 splits, 25 MB: 9.3 to 10.2 us between events; with two pieces a thread, one after another, 11.1).
__global__ void __launch_bounds__(256) attn_dkv_join_kernel(const __grid_constant__ BwdAttnParams prm) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const AttnJob job = prm.jobs.far ? prm.jobs.far[blockIdx.x] : prm.jobs.near[blockIdx.x];
  const int rank = blockIdx.y, w = blockIdx.z & 1;
  const int vecs = prm.hk * prm.dh / 4;  // a key's row over all heads
  const int64_t all = prm.P * prm.Tk * prm.hk * prm.dh;
  const int64_t base = (rank * prm.Tk + job.k0) * prm.hk * prm.dh;
  for (int i = threadIdx.x + (blockIdx.z >> 1) * 256; i < job.k_rows * vecs; i += 256 * (gridDim.z >> 1)) {
    const float4* src = reinterpret_cast<const float4*>(prm.part + w * prm.splits * all + base) + i;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int z = 0; z < prm.splits; ++z) {
      const float4 v = __ldcs(src + z * (all / 4));
      s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
    *reinterpret_cast<uint2*>((w ? prm.dk : prm.dv) + base + 4 * i) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

}  // namespace caat
