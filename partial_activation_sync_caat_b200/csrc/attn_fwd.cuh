// attn_fwd.cuh - causal attention over packed sequences on the tensor cores.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(c (s_ij - m_i)),  s = q k^T,  c = scale log2(e)
//
// over the visible keys, in one pass over the keys with a running maximum m_i.  A CTA owns two tiles of
// 128 queries that share their keys (two heads of a group, or 256 rows of one head) and walks the
// keys 128 at a time:
//   warp 8   issues the MMAs: S_t = Q_t K_j^T into tensor memory, O_t += P_t V_j with P_t read from
//            tensor memory (bf16, over the columns of S_t) and V_j from shared memory, MN-major
//   warp 9   TMA: Q once, then K_j and V_j through a ring
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread owns a row, so maximum and sum need no shuffles
//   warps 10, 11    scrub V blocks that some row does not see whole (below)
// While one tile's softmax runs, the tensor cores work on the other's two products.
//
// The maximum is only moved (and O rescaled, by the softmax warps themselves, which then wait for the
// tile's last product) when a block exceeds it by more than 2^8 in the scaled domain: p stays below
// 256, far from the range of bf16 and of the fp32 sums, and the quotient does not depend on m.
//
// Masked keys: s is replaced by -inf before the maximum, so whatever q k^T held there is gone; but
// p = 0 times a NaN or an infinity of V would be NaN in the product.  So blocks that reach past some
// row's last visible key have the rows behind the sequence's keys zeroed in shared memory, and their
// other values that are not finite replaced by 0 and written down (per column: the first such key),
// to be added to the rows that see them at the end.
#pragma once

#include "attn_common.cuh"

namespace caat {

constexpr int KF_THREADS = 384;
constexpr int KF_NONE = 0x7FFFFFFF;
constexpr int KF_ODD = 3;  // key blocks that 256 consecutive rows' last visible keys fall into

template <int HD>
struct FwdCfg {
  static constexpr int kBoxes = HD / 64;
  static constexpr int kTileBytes = kBoxes * KA_BOX_BYTES;      // one Q, K or V tile
  static constexpr int kSlots = HD == 128 ? 5 : 10;             // ring of K and V tiles
  static constexpr int kSmem = 1024 + 2 * kTileBytes + kSlots * kTileBytes + 3 * HD * 4 + 512;
};

struct FwdParams {
  __nv_bfloat16* out;   // [P, Tq, hq, dh]
  float* lse;           // [P, hq, Tq] or null
  int64_t Tq;
  int hq, hk, dh, group;
  int pair_heads;       // 1: the tiles are heads 2h, 2h + 1 of the same rows; 0: rows 0-127, 128-255 of a job
  int n_heads;          // grid units per job and rank: hq / 2 or hq
  int per_job;          // P * n_heads
  float scale;
  uint64_t timeout_ns;
  AttnJobList jobs;
};

template <int HD>
__global__ void __launch_bounds__(KF_THREADS, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ FwdParams prm) {
  using Cfg = FwdCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + 2 * Cfg::kTileBytes;
  int* odd = reinterpret_cast<int*>(sRing + Cfg::kSlots * Cfg::kTileBytes);  // [3][HD]: first NaN, +inf, -inf key
  uint64_t* bars = reinterpret_cast<uint64_t*>(odd + 3 * HD);
  uint64_t* q_full = bars;                   // [2]
  uint64_t* full = q_full + 2;               // [slots]
  uint64_t* empty = full + Cfg::kSlots;      // [slots]
  uint64_t* s_full = empty + Cfg::kSlots;    // [2]
  uint64_t* p_full = s_full + 2;             // [2] 4 warps
  uint64_t* pv_done = p_full + 2;            // [2]
  uint64_t* v_full = pv_done + 2;            // [KF_ODD] V blocks to scrub have arrived
  uint64_t* scrubbed = v_full + KF_ODD;      // [KF_ODD] 2 warps
  uint64_t* all_scrubbed = scrubbed + KF_ODD;  // 2 warps
  uint64_t* mma_done = all_scrubbed + 1;
  int* any_odd = reinterpret_cast<int*>(mma_done + 1);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(any_odd + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int ji = blockIdx.x / prm.per_job;
  const int rh = blockIdx.x - ji * prm.per_job;
  const int rank = rh / prm.n_heads;
  const int hu = rh - rank * prm.n_heads;
  const AttnJob job = prm.jobs.far ? prm.jobs.far[ji] : prm.jobs.near[ji];
  const bool ph = prm.pair_heads != 0;
  const int head0 = ph ? 2 * hu : hu;
  const int kvh = head0 / prm.group;
  // rows of each tile, the first row's visible keys and the blocks of keys the tile needs
  const int rows[2] = {min(job.rows, KA_TILE), ph ? job.rows : max(job.rows - KA_TILE, 0)};
  const int first[2] = {job.first, ph ? job.first : job.first + KA_TILE};
  int n_blk[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) n_blk[t] = rows[t] > 0 ? max(first[t] + rows[t] - 1 + KA_TILE - 1, 0) / KA_TILE : 0;
  const int n_max = max(n_blk[0], n_blk[1]);
  // the keys end where the last row's view ends; blocks from j_odd on are not seen whole by row 0
  const int m_seen = max(rows[1] > 0 ? first[1] + rows[1] - 1 : 0, first[0] + rows[0] - 1);
  const int j_odd = max(job.first, 0) / KA_TILE;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&pv_done[t], 1);
    }
    for (int s = 0; s < Cfg::kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < KF_ODD; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&scrubbed[s], 2);
    }
    mbar_init(all_scrubbed, 2);
    mbar_init(mma_done, 1);
    *any_odd = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  for (int i = threadIdx.x; i < 3 * HD; i += KF_THREADS) odd[i] = KF_NONE;
  if (warp == 8) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint64_t tmo = prm.timeout_ns;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 9) {
      // -------------------------------------------------------------- TMA
      if (lane == 0) {
        const uint64_t pol_q = policy_evict_first();
        const uint64_t pol_kv = policy_evict_last();
        bool ok = true, issued = false;
        for (int t = 0; t < 2; ++t) {
          if (n_blk[t] == 0) continue;
          mbar_arrive_expect_tx(&q_full[t], Cfg::kTileBytes);
          for (int b = 0; b < Cfg::kBoxes; ++b)
            tma_load_4d(sQ + t * Cfg::kTileBytes + b * KA_BOX_BYTES, &tmQ, &q_full[t], 64 * b, ph ? head0 + t : head0,
                        job.q0 + (ph ? 0 : t * KA_TILE), rank, pol_q);
          issued = true;
        }
        for (int i = 0; i < 2 * n_max && ok; ++i) {
          const int slot = i % Cfg::kSlots;
          if (!mbar_wait(&empty[slot], ((i / Cfg::kSlots) & 1) ^ 1, tmo, 91)) {
            ok = false;
            break;
          }
          // a block to scrub goes to the scrubbing warps first, which pass it on to the MMA warp
          uint64_t* bar = &full[slot];
          if ((i & 1) && (i >> 1) >= j_odd) {
            bar = &v_full[(i >> 1) - j_odd];
            mbar_arrive(&full[slot]);
          }
          mbar_arrive_expect_tx(bar, Cfg::kTileBytes);
          for (int b = 0; b < Cfg::kBoxes; ++b)
            tma_load_4d(sRing + slot * Cfg::kTileBytes + b * KA_BOX_BYTES, (i & 1) ? &tmV : &tmK, bar, 64 * b, kvh,
                        job.k0 + (i >> 1) * KA_TILE, rank, pol_kv);
          issued = true;
        }
        if (!ok && issued) spin_ns(KA_DRAIN_NS);
      }
    } else if (warp == 8) {
      // -------------------------------------------------------------- MMA
      if (lane == 0 && n_max > 0) {
        constexpr uint32_t id_s = idesc_bf16_f32(KA_TILE, KA_TILE);
        constexpr uint32_t id_o = idesc_bf16_f32_major(KA_TILE, HD, false, true);
        auto s_mma = [&](int t, int j) {
          const uint32_t qa = smem_u32(sQ + t * Cfg::kTileBytes);
          const uint32_t ka = smem_u32(sRing + ((2 * j) % Cfg::kSlots) * Cfg::kTileBytes);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t off = (kk >> 2) * KA_BOX_BYTES + (kk & 3) * 32;
            umma_bf16(tmem + t * KA_TILE, sw128_kmajor_desc(qa + off), sw128_kmajor_desc(ka + off), id_s, kk > 0);
          }
          umma_commit(&s_full[t]);
        };
        auto wait_tile = [&](int i, int site) {
          return mbar_wait(&full[i % Cfg::kSlots], (i / Cfg::kSlots) & 1, tmo, site);
        };
        bool ok = wait_tile(0, 92);
        for (int t = 0; t < 2 && ok; ++t) {
          if (n_blk[t] == 0) continue;
          ok = mbar_wait(&q_full[t], 0, tmo, 93);
          if (ok) s_mma(t, 0);
        }
        if (ok) umma_commit(&empty[0]);
        for (int j = 0; j < n_max && ok; ++j) {
          if (!wait_tile(2 * j + 1, 94)) { ok = false; break; }
          if (j >= j_odd && !mbar_wait(&scrubbed[j - j_odd], 0, tmo, 95)) { ok = false; break; }
          if (j + 1 < n_max && !wait_tile(2 * j + 2, 96)) { ok = false; break; }
          const uint32_t va = smem_u32(sRing + ((2 * j + 1) % Cfg::kSlots) * Cfg::kTileBytes);
          for (int t = 0; t < 2; ++t) {
            if (j >= n_blk[t]) continue;
            if (!mbar_wait(&p_full[t], j & 1, tmo, 97)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < KA_TILE / 16; ++kk)
              umma_bf16_ts(tmem + 2 * KA_TILE + t * HD, tmem + t * KA_TILE + 8 * kk, sw128_mnmajor_desc_128(va + kk * 2048),
                           id_o, (j > 0 || kk > 0) ? 1u : 0u);
            umma_commit(&pv_done[t]);
            if (j + 1 < n_blk[t]) s_mma(t, j + 1);
          }
          if (!ok) break;
          umma_commit(&empty[(2 * j + 1) % Cfg::kSlots]);
          if (j + 1 < n_max) umma_commit(&empty[(2 * j + 2) % Cfg::kSlots]);
        }
        umma_commit(mma_done);
        mbar_wait(mma_done, 0, tmo, 98);
      }
    } else {
      // -------------------------------------------------------------- scrubbing V
      for (int j = j_odd; j < n_max; ++j) {
        const int i = 2 * j + 1;
        if (!warp_wait(&v_full[j - j_odd], 0, tmo, 99)) break;
        uint8_t* v = sRing + (i % Cfg::kSlots) * Cfg::kTileBytes;
        const int live = m_seen - j * KA_TILE;  // keys of this block that some row sees
        for (int x = threadIdx.x - 320; x < Cfg::kTileBytes / 16; x += 64) {
          const int box = x >> 10, key = (x >> 3) & 127, chunk = (x & 7) ^ (key & 7);
          uint4* p = reinterpret_cast<uint4*>(v) + x;
          if (key >= live) {
            *p = make_uint4(0, 0, 0, 0);
            continue;
          }
          const uint4 w = *p;
          uint32_t e[4] = {w.x, w.y, w.z, w.w};
          bool hit = false;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            hit |= (e[u] & 0x7F80u) == 0x7F80u || (e[u] & 0x7F800000u) == 0x7F800000u;
          if (hit) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const uint32_t b = (e[u >> 1] >> (16 * (u & 1))) & 0xFFFFu;
              if ((b & 0x7F80u) != 0x7F80u) continue;
              const int kind = (b & 0x7Fu) ? 0 : (b & 0x8000u) ? 2 : 1;
              atomicMin(&odd[kind * HD + 64 * box + 8 * chunk + u], j * KA_TILE + key);
              e[u >> 1] &= (u & 1) ? 0x0000FFFFu : 0xFFFF0000u;
            }
            *any_odd = 1;
            *p = make_uint4(e[0], e[1], e[2], e[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&scrubbed[j - j_odd]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(all_scrubbed);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = warp >> 2;
    const int q = warp & 3;
    const int row = q * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t tS = tmem + lane_base + t * KA_TILE;
    const uint32_t tO = tmem + lane_base + 2 * KA_TILE + t * HD;
    const int nb = n_blk[t];
    const int my_first = t ? first[1] : first[0];
    const int vis = my_first + row;  // visible keys (rows past the tile's end see what they like)
    const float c = prm.scale * KA_LOG2E;
    const uint64_t c2 = pack_f32x2(c, c);
    float m = -INFINITY, mc = 0.f;
    uint64_t sum2 = 0;  // two partial sums
    bool ok = true;
    for (int j = 0; j < nb; ++j) {
      ok = warp_wait(&s_full[t], j & 1, tmo, 100 + t);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[128];
#pragma unroll
      for (int x = 0; x < 4; ++x) tmem_ld_32x32b_x32(tS + 32 * x, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * x));
      tmem_wait_ld();
      const int seen = vis - j * KA_TILE;
      if (my_first + q * 32 - j * KA_TILE < KA_TILE) {  // some row of the warp does not see the whole block
#pragma unroll
        for (int x = 0; x < 128; ++x) s[x] = x < seen ? s[x] : 0xFF800000u;
      }
      float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int x = 0; x < 128; ++x) mx[x & 3] = fmaxf(mx[x & 3], __uint_as_float(s[x]));
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      const bool move = (top - m) * c > 8.0f;  // m = -inf and a visible score: inf > 8; both -inf: no
      if (__any_sync(0xFFFFFFFFu, move)) {
        float f = 1.f;
        if (move) {
          f = ex2((m - top) * c);
          m = top;
          mc = m * c;
        }
        const uint64_t f2 = pack_f32x2(f, f);
        sum2 = mul_f32x2(sum2, f2);
        if (j > 0) {
          ok = warp_wait(&pv_done[t], (j - 1) & 1, tmo, 102 + t);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int x = 0; x < HD; x += 32) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + x, o);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
            tmem_st_32x32b_x32(tO + x, o);
          }
        }
      }
      const uint64_t nm2 = pack_f32x2(-mc, -mc);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t p[32];
#pragma unroll
        for (int y = 0; y < 32; ++y) {
          const int e = 64 * x + 2 * y;
          float a, b;
          unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, nm2), a, b);
          a = ex2(a);
          b = ex2(b);
          sum2 = add_f32x2(sum2, pack_f32x2(a, b));
          p[y] = pack_bf16x2(a, b);
        }
        tmem_st_32x32b_x32(tS + 32 * x, p);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[t]);
    }
    if (ok && nb > 0) ok = warp_wait(&pv_done[t], (nb - 1) & 1, tmo, 104 + t);
    if (ok && n_max > 0) ok = warp_wait(all_scrubbed, 0, tmo, 106);
    tc_fence_after();
    if (ok) {
      float s0, s1;
      unpack_f32x2(sum2, s0, s1);
      const float sum = s0 + s1;
      const bool live = nb > 0 && vis > 0;
      const float inv = live ? 1.f / sum : 0.f;
      const bool mine = row < (t ? rows[1] : rows[0]);
      const int head = ph ? head0 + t : head0;
      const int64_t grow = job.q0 + (ph ? 0 : t * KA_TILE) + row;
      __nv_bfloat16* dst = prm.out + ((rank * prm.Tq + grow) * prm.hq + head) * prm.dh;
      const bool patch = *reinterpret_cast<volatile int*>(any_odd) != 0;
#pragma unroll
      for (int x = 0; x < HD; x += 32) {
        uint32_t o[32];
        if (nb > 0) {
          tmem_ld_32x32b_x32(tO + x, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int y = 0; y < 32; ++y) o[y] = live ? __float_as_uint(__uint_as_float(o[y]) * inv) : 0u;
        if (patch) {
          for (int y = 0; y < 32; ++y) {
            float f = __uint_as_float(o[y]);
            if (odd[x + y] < vis) f = __uint_as_float(0x7FC00000u);
            if (odd[HD + x + y] < vis) f += INFINITY;
            if (odd[2 * HD + x + y] < vis) f -= INFINITY;
            o[y] = __float_as_uint(f);
          }
        }
        if (mine) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            if (x + 8 * y < prm.dh) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16x2(__uint_as_float(o[8 * y + 2 * e]), __uint_as_float(o[8 * y + 2 * e + 1]));
              st_v4(dst + x + 8 * y, make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
        }
      }
      if (mine && prm.lse)
        prm.lse[(int64_t(rank) * prm.hq + head) * prm.Tq + grow] = live ? (mc + log2f(sum)) * KA_LN2 : -INFINITY;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

}  // namespace caat
