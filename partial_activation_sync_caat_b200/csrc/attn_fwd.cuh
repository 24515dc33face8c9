// attn_fwd.cuh - causal attention over packed sequences on the tensor cores.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(c (s_ij - m_i)),  s = q k^T,  c = scale log2(e)
//
// over the visible keys, in one pass over the keys with a running maximum m_i.  A persistent CTA takes
// units of two tiles of 128 queries that share their keys (two heads of a group, or 256 rows of one
// head) and walks a unit's keys in blocks of 128, each in two steps of 64.  Of dh <= 64 it has one tile, and
// two CTAs share an SM: they start and end their units apart (4 to 10% on prompts of 128 to 1500 tokens
// against a CTA of two tiles, 2% at 8192).  Warps (one tile: 4 fewer in front):
//   warps 8, 11  issue the MMAs of tile 0, 1: S_t = Q_t K_j^T into tensor memory, O_t += P_t V_j with P_t
//            read from tensor memory (bf16, over the columns of S_t) and V_j from shared memory, MN-major
//   warp 9   TMA of the K and V blocks through a ring that runs on from unit to unit
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread owns a row, so maximum and sum need no shuffles
//   warp 10  scrubs V blocks that some row does not see whole (below); TMA of the next unit's Q
// Each tile has two S buffers, and its scores run two steps ahead of its products: the softmax of a step
// starts when the last one is done, without waiting for any product.  (Steps of 128 keys with one S
// buffer a tile, all that tensor memory holds beside O, measured 3600 clocks per block and pair of
// tiles against 2050 of products: softmax, 2170, and products, 1300, took turns.)  One MMA warp for
// both tiles could not keep up: a wait costs it 150 clocks, a product 90, 64 scores 260.
//
// The units are ordered by their length, longest first, and dealt to the CTAs back and forth (0..G-1,
// G-1..0, ...), which evens out their sums without a counter in memory.
//
// The maximum is only moved when a score exceeds it by more than 2^8 in the scaled domain: p stays below
// 256, far from the range of bf16 and of the fp32 sums, and the quotient does not depend on m.  When
// it moves (mostly: in a unit's first step) the softmax warps rescale O themselves, once the tile's last
// product is done.
//
// Masked keys: s is replaced by -inf before the maximum, so whatever q k^T held there is gone; but
// p = 0 times a NaN or an infinity of V would be NaN in the product.  So blocks that reach past some
// row's last visible key have the rows behind the sequence's keys zeroed in shared memory, and their
// other values that are not finite replaced by 0 and written down (per column: the first such key),
// to be added to the rows that see them at the end.
#pragma once

#include "attn_common.cuh"

namespace caat {

// Every 8th pair of exponentials comes from a polynomial on the FMA units: the special-function units
// (16 per clock and SM) bound a step.  T=8192, 32 heads, on a cool part: none 482 us, every 8th 461-472, every 4th
// 464-474; at the power cap every 8th takes 554-563, and none, every 4th and every 16th 2-3% more.
constexpr int KF_POLY = 8;
constexpr int KF_STEP = 64;  // keys of a step
constexpr int KF_ODD = 8;  // barriers of blocks to scrub: more than V blocks fit in the ring

template <int HD>
struct FwdCfg {
  static constexpr int kBoxes = HD / 64;
  static constexpr int kTileBytes = kBoxes * KA_BOX_BYTES;      // one Q, K or V tile
  static constexpr int kTiles = HD == 128 ? 2 : 1;              // of queries
  static constexpr int kCtas = 3 - kTiles;                      // per SM
  static constexpr int kSlots = HD == 128 ? 5 : 6;              // ring of K and V tiles
  static constexpr int kSoft = 4 * kTiles;                      // softmax warps; behind them MMA, K and V, Q and scrubbing, MMA
  static constexpr int kThreads = 32 * (kSoft + 4);
  static constexpr int kTmem = 512 / kCtas;                     // columns
  static constexpr int kSmem = kTiles * kTileBytes + kSlots * kTileBytes + 2 * HD * 4 + 512;
};

struct FwdParams {
  __nv_bfloat16* out;   // [P, Tq, hq, dh]
  float* lse;           // [P, hq, Tq] or null
  int64_t Tq;
  int hq, hk, dh;
  int pair_heads;       // 1: the tiles are heads 2h, 2h + 1 of the same rows; 0: rows 0-127, 128-255 of a job
  FastDiv group_div;
  FastDiv n_heads;      // units per job and rank: hq / 2 or hq
  FastDiv per_job;      // P * n_heads
  int n_units;
  float scale;
  uint64_t timeout_ns;
  AttnJobList jobs;
};

// The CTA's k-th unit of n_units, -1 if there is none (nor any later one).
__device__ __forceinline__ int dealt_unit(int k, int n_units) {
  const int64_t g = gridDim.x, b = blockIdx.x;
  const int64_t i = k * g + ((k & 1) ? g - 1 - b : b);
  return i < n_units ? static_cast<int>(i) : -1;
}

// What the MMA warp needs of a unit.
struct FwdSpan {
  int nb[2], n_blk, j_odd;
  __device__ __forceinline__ bool get(const FwdParams& prm, int k) {
    const int i = dealt_unit(k, prm.n_units);
    if (i < 0) return false;
    const int ji = prm.per_job.div(i);
    const AttnJob* jobs = prm.jobs.far ? prm.jobs.far : prm.jobs.near;
    const int first = jobs[ji].first, rows = jobs[ji].rows;
    const int more = prm.pair_heads ? rows : rows - KA_TILE;  // queries of tile 1
    const int last1 = prm.pair_heads ? first : first + KA_TILE;
    nb[0] = max(first + min(rows, KA_TILE) - 1 + KF_STEP - 1, 0) / KF_STEP;
    nb[1] = more > 0 ? max(last1 + more - 1 + KF_STEP - 1, 0) / KF_STEP : 0;
    n_blk = (max(nb[0], nb[1]) + 1) / 2;
    j_odd = max(first, 0) / KA_TILE;
    return true;
  }
};

struct FwdUnit {
  int rank, head0, kvh;
  int q0, k0;
  int rows[2], first[2], nb[2];  // of each tile: queries, keys the first of them sees, steps of 64 keys
  int n_blk;   // blocks of 128 keys
  int m_seen;  // keys that the last query sees: the sequence's keys end there
  int j_odd;   // blocks from here on are not seen whole by the first query
  __device__ __forceinline__ bool get(const FwdParams& prm, int k) {
    const int i = dealt_unit(k, prm.n_units);
    if (i < 0) return false;
    const int ji = prm.per_job.div(i), rh = i - ji * static_cast<int>(prm.per_job.d);
    rank = prm.n_heads.div(rh);
    const int hu = rh - rank * static_cast<int>(prm.n_heads.d);
    const AttnJob job = prm.jobs.far ? prm.jobs.far[ji] : prm.jobs.near[ji];
    const bool ph = prm.pair_heads != 0;
    head0 = ph ? 2 * hu : hu;
    kvh = prm.group_div.div(head0);
    q0 = job.q0;
    k0 = job.k0;
    rows[0] = min(job.rows, KA_TILE);
    rows[1] = ph ? job.rows : max(job.rows - KA_TILE, 0);
    first[0] = job.first;
    first[1] = ph ? job.first : job.first + KA_TILE;
#pragma unroll
    for (int t = 0; t < 2; ++t) nb[t] = rows[t] > 0 ? max(first[t] + rows[t] - 1 + KF_STEP - 1, 0) / KF_STEP : 0;
    n_blk = (max(nb[0], nb[1]) + 1) / 2;
    m_seen = job.first + job.rows - 1;
    j_odd = max(job.first, 0) / KA_TILE;
    return true;
  }
};

template <int HD>
__global__ void __launch_bounds__(FwdCfg<HD>::kThreads, FwdCfg<HD>::kCtas)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ FwdParams prm) {
  using Cfg = FwdCfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];  // (a known address: no registers spent on it)
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + Cfg::kTiles * Cfg::kTileBytes;
  // [2][HD], by the unit's parity: the first key (from block j_odd on) whose value is NaN, +inf, -inf,
  // 10 bits each, 1023: none
  uint32_t* odd = reinterpret_cast<uint32_t*>(sRing + Cfg::kSlots * Cfg::kTileBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(odd + 2 * HD);
  uint64_t* q_full = bars;                   // [2]
  uint64_t* q_empty = q_full + 2;            // [2]
  uint64_t* full = q_empty + 2;              // [slots]
  uint64_t* empty = full + Cfg::kSlots;      // [slots]
  uint64_t* s_full = empty + Cfg::kSlots;    // [2 tiles][2 buffers]
  uint64_t* p_full = s_full + 4;             // [2 tiles][2 buffers] 4 warps
  uint64_t* pv_done = p_full + 4;            // [2 tiles][2 buffers]
  uint64_t* o_free = pv_done + 4;            // [2] 4 warps
  uint64_t* v_full = o_free + 2;             // [KF_ODD] V blocks to scrub have arrived
  uint64_t* scrubbed = v_full + KF_ODD;      // [KF_ODD]
  uint64_t* scrub_done = scrubbed + KF_ODD;  // [2] all of a unit's
  uint64_t* epi_done = scrub_done + 2;       // [2] softmax warps
  uint64_t* mma_done = epi_done + 2;
  volatile int* any_odd = reinterpret_cast<int*>(mma_done + 1);  // [2]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled tiles would not line up
    if (threadIdx.x == 0) status_raise(2, 90);
    return;
  }
  const bool ph = prm.pair_heads != 0;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_empty[t], 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&s_full[2 * t + b], 1);
        mbar_init(&p_full[2 * t + b], 4);
        mbar_init(&pv_done[2 * t + b], 1);
      }
      mbar_init(&o_free[t], 4);
      mbar_init(&scrub_done[t], 1);
      mbar_init(&epi_done[t], Cfg::kSoft);
      any_odd[t] = 0;
    }
    for (int s = 0; s < Cfg::kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], Cfg::kTiles);
    }
    for (int s = 0; s < KF_ODD; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&scrubbed[s], 1);
    }
    mbar_init(mma_done, Cfg::kTiles);
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  for (int i = threadIdx.x; i < 2 * HD; i += Cfg::kThreads) odd[i] = 0x3FFFFFFFu;
  const int role = warp - Cfg::kSoft;
  if (role == 0) {
    tmem_alloc(tmem_holder, Cfg::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = Cfg::kCtas == 1 ? 0 : *tmem_holder;  // all 512 columns: the allocation starts at the first
  constexpr uint32_t kO = Cfg::kTiles * KA_TILE;
  const uint64_t tmo = prm.timeout_ns;
  FwdUnit u;

  if (role >= 0) {
    if constexpr (Cfg::kCtas == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (role == 1) {
      // -------------------------------------------------------------- TMA: K and V
      if (lane == 0) {
        const uint64_t pol_kv = policy_evict_last();
        bool ok = true, issued = false;
        int i = 0, ns = 0;  // ring position, blocks to scrub so far
        for (int k = 0; ok && u.get(prm, k); ++k) {
          for (int x = 0; x < 2 * u.n_blk; ++x, ++i) {
            const int slot = i % Cfg::kSlots;
            ok = mbar_wait(&empty[slot], ((i / Cfg::kSlots) & 1) ^ 1, tmo, 91);
            if (!ok) break;
            // a block to scrub goes to the scrubbing warp first, which passes it on to the MMA warp
            uint64_t* bar = &full[slot];
            if ((x & 1) && (x >> 1) >= u.j_odd) {
              bar = &v_full[ns++ % KF_ODD];
              mbar_arrive(&full[slot]);
            }
            mbar_arrive_expect_tx(bar, Cfg::kTileBytes);
            for (int b = 0; b < Cfg::kBoxes; ++b)
              tma_load_4d(sRing + slot * Cfg::kTileBytes + b * KA_BOX_BYTES, (x & 1) ? &tmV : &tmK, bar, 64 * b, u.kvh,
                          u.k0 + (x >> 1) * KA_TILE, u.rank, pol_kv);
            issued = true;
          }
        }
        if (!ok && issued) spin_ns(KA_DRAIN_NS);
      }
    } else if (role != 2) {
      // -------------------------------------------------------------- MMA: the first of tile 0, the last of tile 1
      const int t = Cfg::kTiles == 1 || role == 0 ? 0 : 1;
      const uint32_t lead = elect_one();
      constexpr uint32_t id_s = idesc_bf16_f32(KA_TILE, KF_STEP);
      constexpr uint32_t id_o = idesc_bf16_f32_major(KA_TILE, HD, false, true);
      const uint64_t dQ = sw128_kmajor_desc(smem_u32(sQ + t * Cfg::kTileBytes)), dK = sw128_kmajor_desc(smem_u32(sRing));
      const uint64_t dV = sw128_mnmajor_desc_128(smem_u32(sRing));
      int slot = 0;       // ring slot, and phase, of the next block to use
      uint32_t phase = 0;
      auto wait_block = [&](int site) { return lane_wait(&full[slot], phase, tmo, site); };
      auto next_slot = [&] {
        if (++slot == Cfg::kSlots) {
          slot = 0;
          phase ^= 1;
        }
      };
      uint32_t np = 0, ns = 0, no = 0;  // the tile's products, scores, units so far
      int n_scrub = 0;
      auto scores = [&](int k_slot, int h) {
        const uint32_t buf = ns++ & 1;
        const uint64_t b = dK + static_cast<uint32_t>(k_slot * (Cfg::kTileBytes >> 4) + h * (KF_STEP * 128 >> 4));
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * KA_BOX_BYTES + (kk & 3) * 32) >> 4;
          umma_ss(lead, tmem + t * KA_TILE + buf * KF_STEP, dQ + off, b + off, id_s, kk > 0);
        }
        umma_arrive(lead, &s_full[2 * t + buf]);
      };
      FwdSpan u;
      const bool idle = Cfg::kTiles == 1 && role != 0;
      bool ok = !idle;
      for (int k = 0; ok && u.get(prm, k); ++k) {
        if (u.n_blk == 0) continue;
        const int nb = t ? u.nb[1] : u.nb[0];
        // the unit's first two steps of scores; the softmax warps may still store the last unit's output
        ok = wait_block(93) && (nb == 0 || lane_wait(&q_full[t], no & 1, tmo, 94));
        if (!ok) break;
        if (nb > 0) scores(slot, 0);
        if (nb > 1) scores(slot, 1);
        if (nb == 1 || nb == 2) umma_arrive(lead, &q_empty[t]);
        umma_arrive(lead, &empty[slot]);
        next_slot();
        for (int blk = 0; blk < u.n_blk && ok; ++blk) {
          ok = wait_block(95);
          const int v = slot;
          next_slot();
          if (ok && blk >= u.j_odd) {
            ok = lane_wait(&scrubbed[n_scrub % KF_ODD], (n_scrub / KF_ODD) & 1, tmo, 96);
            ++n_scrub;
          }
          const bool more = blk + 1 < u.n_blk;
          const int kn = slot;  // the next block's keys: scores run two steps ahead
          if (more) {
            ok = ok && wait_block(97);
            next_slot();
          }
          // O is free once the tile's last unit has been stored
          if (blk == 0 && nb > 0 && ok) ok = lane_wait(&o_free[t], (no++ & 1) ^ 1, tmo, 98);
#pragma unroll 1
          for (int h = 0; h < 2 && ok; ++h) {
            const int j = 2 * blk + h;
            if (j >= nb) break;
            const uint32_t buf = np & 1;
            ok = lane_wait(&p_full[2 * t + buf], (np >> 1) & 1, tmo, 99);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b = dV + static_cast<uint32_t>(v * (Cfg::kTileBytes >> 4) + h * (KF_STEP * 128 >> 4));
#pragma unroll
            for (int kk = 0; kk < KF_STEP / 16; ++kk)
              umma_ts(lead, tmem + kO + t * HD, tmem + t * KA_TILE + buf * KF_STEP + 8 * kk, b + (kk * 2048 >> 4), id_o,
                      (j > 0 || kk > 0) ? 1u : 0u);
            umma_arrive(lead, &pv_done[2 * t + buf]);
            ++np;
            if (j + 2 < nb) {
              scores(kn, h);
              if (j + 3 == nb) umma_arrive(lead, &q_empty[t]);
            }
          }
          if (!ok) break;
          umma_arrive(lead, &empty[v]);
          if (more) umma_arrive(lead, &empty[kn]);
        }
      }
      if (!idle) {
        umma_arrive(lead, mma_done);
        lane_wait(mma_done, 0, tmo, 99);
      }
    } else {
      // -------------------------------------------------------------- TMA of Q; scrubbing V
      const uint64_t pol_q = policy_evict_first();
      int nq[2] = {0, 0};
      bool issued = false;
      auto load_q = [&](const FwdUnit& w) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (w.nb[t] == 0) continue;
          if (!warp_wait(&q_empty[t], (nq[t]++ & 1) ^ 1, tmo, 92)) return false;
          if (lane == 0) {
            mbar_arrive_expect_tx(&q_full[t], Cfg::kTileBytes);
            for (int b = 0; b < Cfg::kBoxes; ++b)
              tma_load_4d(sQ + t * Cfg::kTileBytes + b * KA_BOX_BYTES, &tmQ, &q_full[t], 64 * b, ph ? w.head0 + t : w.head0,
                          w.q0 + (ph ? 0 : t * KA_TILE), w.rank, pol_q);
          }
          issued = true;
        }
        return true;
      };
      int i = 0, ns = 0;
      bool have = u.get(prm, 0);
      bool ok = !have || load_q(u);
      for (int k = 0; ok && have; ++k) {
        const int par = k & 1;
        uint32_t* od = odd + par * HD;
        if (k >= 2) {
          ok = warp_wait(&epi_done[par], ((k >> 1) - 1) & 1, tmo, 100);
          if (!ok) break;
          if (any_odd[par]) {
            for (int x = lane; x < HD; x += 32) od[x] = 0x3FFFFFFFu;
            __syncwarp();
            if (lane == 0) any_odd[par] = 0;
          }
          __syncwarp();
        }
        for (int j = u.j_odd; j < u.n_blk; ++j, ++ns) {
          ok = warp_wait(&v_full[ns % KF_ODD], (ns / KF_ODD) & 1, tmo, 101);
          if (!ok) break;
          uint4* v = reinterpret_cast<uint4*>(sRing + ((i + 2 * j + 1) % Cfg::kSlots) * Cfg::kTileBytes);
          const int live = u.m_seen - j * KA_TILE;  // keys of this block that some row sees
          // a value times 0 is 0 unless it is not finite: one packed multiply-add per pair finds those
          __nv_bfloat162 acc = __floats2bfloat162_rn(0.f, 0.f);
          const __nv_bfloat162 zero = acc;
#pragma unroll 8
          for (int x = lane; x < Cfg::kTileBytes / 16; x += 32) {
            if (((x >> 3) & 127) >= live) {
              v[x] = make_uint4(0, 0, 0, 0);
            } else {
              const uint4 w = v[x];
              const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&e[y]), zero, acc);
            }
          }
          const bool clean = __low2float(acc) == 0.f && __high2float(acc) == 0.f;
          for (int x = clean ? Cfg::kTileBytes : lane; x < Cfg::kTileBytes / 16; x += 32) {
            const int box = x >> 10, key = (x >> 3) & 127, chunk = (x & 7) ^ (key & 7);
            const uint4 w = v[x];
            uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const uint32_t b = (e[y >> 1] >> (16 * (y & 1))) & 0xFFFFu;
              if ((b & 0x7F80u) != 0x7F80u) continue;
              const int shift = (b & 0x7Fu) ? 0 : (b & 0x8000u) ? 20 : 10;
              const uint32_t at = static_cast<uint32_t>((j - u.j_odd) * KA_TILE + key);
              uint32_t* word = &od[64 * box + 8 * chunk + y];
              uint32_t old = *reinterpret_cast<volatile uint32_t*>(word);
              while (((old >> shift) & 1023u) > at) {
                const uint32_t was = atomicCAS(word, old, (old & ~(1023u << shift)) | (at << shift));
                if (was == old) break;
                old = was;
              }
              e[y >> 1] &= (y & 1) ? 0x0000FFFFu : 0xFFFF0000u;
              any_odd[par] = 1;
            }
            v[x] = make_uint4(e[0], e[1], e[2], e[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&scrubbed[ns % KF_ODD]);
        }
        if (!ok) break;
        i += 2 * u.n_blk;
        __syncwarp();
        if (lane == 0) mbar_arrive(&scrub_done[par]);
        // the next Q tile's place is free once the unit's last scores are done, which need its scrubbed blocks
        have = u.get(prm, k + 1);
        ok = !have || load_q(u);
      }
      if (!ok && issued) spin_ns(KA_DRAIN_NS);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    if constexpr (Cfg::kCtas == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int t = warp >> 2;
    const int q = warp & 3;
    const int row = q * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t tS0 = tmem + lane_base + t * KA_TILE;
    const uint32_t tO = tmem + lane_base + kO + t * HD;
    const float c = prm.scale * KA_LOG2E;
    const uint64_t c2 = pack_f32x2(c, c);
    bool ok = true;
    int np = 0;  // steps so far
    // Product i is done.  A barrier per buffer: when step i + 1 has its scores, product i - 2 is done and
    // i + 2 cannot have begun, so the phase waited for is either running or the last one.
    auto product_done = [&](int i) { return warp_wait(&pv_done[2 * t + (i & 1)], (i >> 1) & 1, tmo, 104 + t); };
    for (int k = 0; ok && u.get(prm, k); ++k) {
      const int nb = t ? u.nb[1] : u.nb[0];
      const int my_first = t ? u.first[1] : u.first[0];
      const int vis = my_first + row;  // visible keys (rows past the tile's end see what they like)
      float m = -INFINITY, mc = 0.f;
      uint64_t sum2 = 0;  // two partial sums
      for (int j = 0; j < nb; ++j, ++np) {
        const uint32_t tS = tS0 + (np & 1) * KF_STEP;
        ok = warp_wait(&s_full[2 * t + (np & 1)], (np >> 1) & 1, tmo, 102 + t);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[64];
        tmem_ld_32x32b_x32(tS, *reinterpret_cast<uint32_t(*)[32]>(s));
        tmem_ld_32x32b_x32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
        tmem_wait_ld(s);
        const int seen = vis - j * KF_STEP;
        if (my_first + q * 32 - j * KF_STEP < KF_STEP) {  // some row of the warp does not see the whole step
#pragma unroll
          for (int x = 0; x < 64; ++x) s[x] = x < seen ? s[x] : 0xFF800000u;
        }
        float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 64; x += 2)
          mx[(x >> 1) & 3] = max3(mx[(x >> 1) & 3], __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
        const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
        const bool move = (top - m) * c > 8.0f;  // m = -inf and a visible score: inf > 8; both -inf: no
        if (__any_sync(0xFFFFFFFFu, move)) {
          const float f = move ? ex2((m - top) * c) : 1.f;
          m = move ? top : m;
          mc = m == -INFINITY ? 0.f : m * c;
          sum2 = mul_f32x2(sum2, pack_f32x2(f, f));
          if (j > 0) {
            ok = product_done(np - 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < HD; x += 16) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(tO + x, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_st_32x32b_x16(tO + x, o);
            }
          }
        }
        const uint64_t nm2 = pack_f32x2(-mc, -mc);
        uint64_t acc = 0;
        uint32_t p[32];
#pragma unroll
        for (int y = 0; y < 32; ++y) {
          const uint64_t a2 = fma_f32x2(pack_f32x2(__uint_as_float(s[2 * y]), __uint_as_float(s[2 * y + 1])), c2, nm2);
          uint64_t& part = (y & 1) ? acc : sum2;
          float a, b;
          if (y % KF_POLY == 1) {
            const uint64_t r = ex2_poly_f32x2(a2);
            part = add_f32x2(part, r);
            unpack_f32x2(r, a, b);
          } else {
            unpack_f32x2(a2, a, b);
            a = ex2(a);
            b = ex2(b);
            part = add_f32x2(part, pack_f32x2(a, b));
          }
          p[y] = pack_bf16x2(a, b);
        }
        sum2 = add_f32x2(sum2, acc);
        tmem_st_32x32b_x32(tS, p);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * t + (np & 1)]);
      }
      if (ok && nb > 0) ok = product_done(np - 1);
      if (ok) ok = warp_wait(&scrub_done[k & 1], (k >> 1) & 1, tmo, 108);
      if (!ok) break;
      tc_fence_after();
      int again = k;  // looked up once more, rather than kept in registers over the blocks
      asm volatile("" : "+r"(again));
      u.get(prm, again);
      float sum_a, sum_b;
      unpack_f32x2(sum2, sum_a, sum_b);
      const float sum = sum_a + sum_b;
      const bool live = nb > 0 && vis > 0;
      const float inv = live ? 1.f / sum : 0.f;
      const bool mine = row < (t ? u.rows[1] : u.rows[0]);
      const int head = ph ? u.head0 + t : u.head0;
      const int64_t grow = u.q0 + (ph ? 0 : t * KA_TILE) + row;
      __nv_bfloat16* dst = prm.out + ((u.rank * prm.Tq + grow) * prm.hq + head) * prm.dh;
      const bool patch = any_odd[k & 1] != 0;
      const int odd_vis = vis - u.j_odd * KA_TILE;
#pragma unroll 1
      for (int x = 0; x < HD; x += 32) {
        uint32_t o[32];
        if (nb > 0) {
          tmem_ld_32x32b_x32(tO + x, o);
          tmem_wait_ld(o);
        }
#pragma unroll
        for (int y = 0; y < 32; ++y) o[y] = live ? __float_as_uint(__uint_as_float(o[y]) * inv) : 0u;
        if (patch) {
          const uint32_t* od = odd + (k & 1) * HD + x;
#pragma unroll
          for (int y = 0; y < 32; ++y) {
            auto sees = [&](int shift) {
              const int at = static_cast<int>((od[y] >> shift) & 1023u);
              return at != 1023 && at < odd_vis;
            };
            float f = __uint_as_float(o[y]);
            if (sees(0)) f = __uint_as_float(0x7FC00000u);
            if (sees(10)) f += INFINITY;
            if (sees(20)) f -= INFINITY;
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
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (nb > 0) mbar_arrive(&o_free[t]);
        mbar_arrive(&epi_done[k & 1]);
      }
      if (mine && prm.lse)
        prm.lse[(int64_t(u.rank) * prm.hq + head) * prm.Tq + grow] = live ? (mc + log2f(sum)) * KA_LN2 : -INFINITY;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (role == 0) tmem_dealloc(tmem, Cfg::kTmem);
}

}  // namespace caat
