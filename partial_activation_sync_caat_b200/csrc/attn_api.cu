// attn_api.cu - host side of the attention block's calls in include/caat.h (rotary positions, packed
// causal attention and its gradients, decoding): argument validation, work lists and launches.
// The device code lives in the *.cuh files included below.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include "caat.h"
#include "host_common.h"
#include "ptx.cuh"
#include "attn_bwd.cuh"
#include "attn_decode.cuh"
#include "attn_fwd.cuh"
#include "rope.cuh"

namespace caat {
namespace host {

bool attn_take_status(int* v) {
  int w = 0, g = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbol(&w, g_status_word, sizeof(int)) != cudaSuccess ||
      cudaMemcpyToSymbol(g_status_word, &zero, sizeof(int)) != cudaSuccess ||
      cudaMemcpyFromSymbol(&g, g_arg_status, sizeof(int)) != cudaSuccess ||
      cudaMemcpyToSymbol(g_arg_status, &zero, sizeof(int)) != cudaSuccess)
    return false;
  *v = w ? w : g;
  return true;
}

}  // namespace host
}  // namespace caat

namespace {

using caat::host::Recorder;

constexpr size_t kDecodeCounters = 2048;  // 4 bytes per CTA
static_assert(caat::KD_CTAS * 4 <= kDecodeCounters, "one counter per CTA");
constexpr int64_t kMaxRows = int64_t(1) << 30;  // tokens of a buffer, rows of a sequence's cache
// A warp may wait through a whole sequence (for its last block, 64 keys each 1,000 to 2,000 clocks): within the
// waits' limit of 2 s.
constexpr int kMaxSequence = 1 << 25;
constexpr int64_t kMaxCacheRows = int64_t(1) << 36;  // of all sequences: far more than fit the memory

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// A [P, T, heads, dh] operand: strides as given, or contiguous for (0, 0).
struct View {
  const caat_bf16* p = nullptr;
  int64_t rank = 0, tok = 0;
  uintptr_t lo = 0, hi = 0;  // bytes it spans
};

caat_status make_view(View* v, const caat_bf16* p, int64_t s_rank, int64_t s_tok, int P, int64_t T, int heads, int dh) {
  v->p = p;
  const int64_t row = int64_t(heads) * dh;
  v->rank = s_rank;
  v->tok = s_tok;
  if (s_rank == 0 && s_tok == 0) {
    v->tok = row;
    v->rank = T * row;
  }
  if (!p) return CAAT_ERR_INVALID_ARG;
  if (v->tok < row || v->rank < (P > 1 ? row : 0)) return CAAT_ERR_INVALID_ARG;
  // a tensor map's strides are below 2^40 bytes; T tokens of 2^31 elements stay inside 64 bits
  if (v->tok > (int64_t(1) << 31) || v->rank > (int64_t(1) << 38)) return CAAT_ERR_UNSUPPORTED;
  if (v->tok % 8 != 0 || v->rank % 8 != 0 || !aligned16(p)) return CAAT_ERR_UNSUPPORTED;
  v->lo = reinterpret_cast<uintptr_t>(p);
  v->hi = v->lo + 2 * static_cast<uintptr_t>((P - 1) * v->rank + (T - 1) * v->tok + row);
  return CAAT_OK;
}

struct Range {
  uintptr_t lo, hi;
};
Range range_of(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + bytes};
}
bool meet(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
Range range_of(const View& v) { return {v.lo, v.hi}; }

// Whether a row of `a` shares elements with one of `b`, two [P, T] tensors of rows of row_a and row_b elements with
// the same strides, or with another row of `a` itself (b the same).  What counts is how far rows are apart: for
// each difference in rank, the nearest row of `b` that ends behind the start of one of `a`.
bool rows_meet(const View& a, int64_t row_a, const View& b, int64_t row_b, int P, int64_t T) {
  const int64_t apart = (static_cast<int64_t>(b.lo) - static_cast<int64_t>(a.lo)) / 2;
  for (int r = 1 - P; r < P; ++r) {
    if (&a == &b && r == 0) continue;  // tokens of a rank are at least a row apart
    const int64_t at = apart + r * a.rank, d = -row_b - at;  // b's row at at + t tok; the first t with t tok > d
    const int64_t t = std::max((d >= 0 ? d / a.tok : -((-d + a.tok - 1) / a.tok)) + 1, 1 - T);
    if (t < T && at + t * a.tok < row_a) return true;
  }
  return false;
}

caat_status check_heads(int P, int hq, int hk, int dh, float scale) {
  if (P < 1 || P > CAAT_MAX_P || hq < 1 || hk < 1 || dh < 1) return CAAT_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return CAAT_ERR_INVALID_ARG;
  if (hq % hk != 0) return CAAT_ERR_INVALID_ARG;
  if (dh % 8 != 0 || dh > 128 || hq > 1024) return CAAT_ERR_UNSUPPORTED;
  return CAAT_OK;
}

caat_status check_offsets(const int32_t* cu, int n_seq, int64_t T) {
  if (cu[0] < 0) return CAAT_ERR_INVALID_ARG;
  for (int i = 0; i < n_seq; ++i)
    if (cu[i + 1] < cu[i]) return CAAT_ERR_INVALID_ARG;
  if (cu[n_seq] > T) return CAAT_ERR_INVALID_ARG;
  for (int i = 0; i < n_seq; ++i)
    if (cu[i + 1] - cu[i] > kMaxSequence) return CAAT_ERR_UNSUPPORTED;
  return CAAT_OK;
}

// One-time kernel attributes, per device and context.
caat_status attn_setup(int* sms) {
  const caat_status s = caat::host::device_sms(sms);
  if (s != CAAT_OK) return s;
  static std::mutex mu;
  static CUcontext done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return CAAT_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  const CUcontext ctx = caat::host::context();
  if (done[dev] == ctx && ctx) return CAAT_OK;
  auto smem = [](auto* kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
  };
  if (!smem(caat::attn_fwd_kernel<64>, caat::FwdCfg<64>::kSmem) || !smem(caat::attn_fwd_kernel<128>, caat::FwdCfg<128>::kSmem) ||
      !smem(caat::attn_dq_kernel<64>, caat::DqCfg<64>::kSmem) || !smem(caat::attn_dq_kernel<128>, caat::DqCfg<128>::kSmem) ||
      !smem(caat::attn_decode_kernel<64>, caat::KD_SMEM) || !smem(caat::attn_decode_kernel<128>, caat::KD_SMEM) ||
      !smem(caat::attn_decode_cluster_kernel<64>, caat::KD_SMEM) || !smem(caat::attn_decode_cluster_kernel<128>, caat::KD_SMEM) ||
      !smem(caat::attn_dkv_kernel<64>, caat::DkvCfg<64>::kSmem) || !smem(caat::attn_dkv_kernel<128>, caat::DkvCfg<128>::kSmem))
    return CAAT_ERR_CUDA;
  done[dev] = ctx;
  return CAAT_OK;
}

// Tensor map of a [P, T, heads, dh] operand as (dh, heads, T, P) in boxes of 64 elements x box_rows
// tokens of one head, 128-byte swizzle; elements past dh and tokens past T read as zeros.
caat_status heads_map(CUtensorMap* map, const View& v, int P, int64_t T, int heads, int dh, int box_rows = caat::KA_TILE) {
  const caat::host::EncodeTiledFn fn = caat::host::tensor_map_encoder();
  if (!fn) return CAAT_ERR_CUDA;
  const cuuint64_t dims[4] = {cuuint64_t(dh), cuuint64_t(heads), cuuint64_t(T), cuuint64_t(P)};
  const int64_t rank = P > 1 ? v.rank : v.tok;  // one rank: never stepped over
  const cuuint64_t strides[3] = {cuuint64_t(dh) * 2, cuuint64_t(v.tok) * 2, cuuint64_t(rank) * 2};
  const cuuint32_t box[4] = {64, 1, cuuint32_t(box_rows), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<caat_bf16*>(v.p), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CAAT_OK : CAAT_ERR_CUDA;
}

// Most entries a work list of `step` rows each can have.
int64_t max_jobs(int64_t T, int n_seq, int step) { return T / step + n_seq; }

size_t list_bytes(int64_t jobs) { return jobs <= caat::KA_INLINE_JOBS ? 0 : align256(size_t(jobs) * sizeof(caat::AttnJob)); }

// Queries of each sequence cut into jobs of `step` rows, those with the most keys first: the last jobs
// to start are then the shortest, which evens out when the SMs run dry.
void query_jobs(const int32_t* cu_q, const int32_t* cu_k, int n_seq, int step, std::vector<caat::AttnJob>& jobs) {
  jobs.clear();
  for (int s = 0; s < n_seq; ++s) {
    const int n = cu_q[s + 1] - cu_q[s], m = cu_k[s + 1] - cu_k[s];
    for (int i = 0; i < n; i += step) jobs.push_back({cu_q[s] + i, std::min(step, n - i), cu_k[s], i + 1 + (m - n), 0});
  }
  std::stable_sort(jobs.begin(), jobs.end(),
                   [](const caat::AttnJob& a, const caat::AttnJob& b) { return a.first + a.rows > b.first + b.rows; });
}

// Keys of each sequence in tiles of 128, each with the queries that see any of them, most first.
void key_jobs(const int32_t* cu_q, const int32_t* cu_k, int n_seq, std::vector<caat::AttnJob>& jobs) {
  jobs.clear();
  for (int s = 0; s < n_seq; ++s) {
    const int n = cu_q[s + 1] - cu_q[s], m = cu_k[s + 1] - cu_k[s];
    for (int j = 0; j < m; j += caat::KA_TILE) {
      const int sees = j - (m - n);  // the first query that sees key j, if not before the sequence's first
      const int i0 = std::min(std::max(sees, 0), n);
      jobs.push_back({cu_q[s] + i0, n - i0, cu_k[s] + j, sees - i0, std::min(caat::KA_TILE, m - j)});
    }
  }
  std::stable_sort(jobs.begin(), jobs.end(), [](const caat::AttnJob& a, const caat::AttnJob& b) { return a.rows > b.rows; });
}

// CTAs that share the queries of a key tile (their fp32 sums are then joined by another kernel): enough
// for two waves of the 148 SMs when ranks, key heads and tiles alone do not give them, but with 8 steps of 64
// queries each at least (34 tokens, 4 ranks of 4 heads: 26.7 us with 16 empty or short parts, 16.4 without;
// 606 tokens 45.1 | 28.7).  (148, here and below, and not the device's count: the workspace's size goes by the
// same rules, and may be asked for where there is no GPU.)
int dkv_splits(int64_t Tq, int64_t Tk, int P, int hq, int hk) {
  const int64_t units = std::max<int64_t>(Tk / caat::KA_TILE, 1) * P * hk;
  const int64_t steps = (Tq / caat::KB2_QT + 1) * (hq / hk);
  return static_cast<int>(std::min({int64_t(16), (2 * 148 + units - 1) / units, std::max<int64_t>(steps / 8, 1)}));
}

struct BwdLayout {
  size_t D, q_list, k_list, part, total;
  int splits;
};

BwdLayout bwd_layout(int64_t Tq, int64_t Tk, int n_seq, int P, int hq, int hk, int dh) {
  BwdLayout L{};
  L.splits = dkv_splits(Tq, Tk, P, hq, hk);
  L.D = 0;
  L.q_list = align256(size_t(P) * hq * Tq * 4);
  L.k_list = L.q_list + list_bytes(max_jobs(Tq, n_seq, caat::KA_TILE));
  L.part = L.k_list + list_bytes(max_jobs(Tk, n_seq, caat::KA_TILE));
  L.total = L.part + (L.splits > 1 ? align256(size_t(2) * L.splits * P * Tk * hk * dh * 4) : 0);
  return L;
}

// CTAs per segment (sequence, rank, key head, 16 query heads) of the decode kernel with a cluster for each, 0
// for the kernel that deals tiles evenly.  Clusters are as large as it takes for two CTAs per SM and for
// parts of 2048 keys at most, so that a ragged batch's longest sequence ends with the others.  They start
// slowly when more of them come than the SMs hold at once, which only parts of 1 MiB make up for (us,
// clusters | even deal; dh 128: 32 segments of 2048 keys 8.6 | 15.5, of 8192 26.2 | 35.8; 512 of 256 keys
// with 2 CTAs each 34.2 | 19.0, of 8192 with 4 301 | 331; 2048 of 256 keys, one CTA each, 47.9 | 54.4).  Few
// segments leave SMs idle, which costs less than the deal's parts and second launch while a CTA has 16
// tiles or fewer (dh 128: one segment of 600 keys 8.2 | 10.3, of 4096 10.3 | 14.3, of 8192 14.9 | 18.4;
// 30 of 148 keys 8.2 | 16.6).
int decode_cluster(int64_t B, int64_t capacity, int P, int hq, int hk, int dh) {
  const int64_t segs = B * P * hk * ((hq / hk + 15) / 16);
  const int tile = 4 * caat::kd_keys(dh <= 64 ? 64 : 128);
  int c = 1;
  while (c < 8 && (capacity > 2048 * c || (segs * c < 2 * 148 && 2 * c * tile <= capacity))) c *= 2;
  if (capacity > 2048 * c || (segs * c < 148 && capacity > int64_t(16) * tile * c) || segs * c > INT32_MAX) return 0;
  return c == 1 || segs * c <= 4 * 148 || capacity / c * dh * 4 >= (1 << 20) ? c : 0;
}

// The list into the launch's arguments, or through `dst` in the workspace (queued on the stream).
caat_status place_jobs(const std::vector<caat::AttnJob>& jobs, caat::AttnJobList* list, void* dst, cudaStream_t st) {
  if (jobs.size() <= size_t(caat::KA_INLINE_JOBS)) {
    list->far = nullptr;
    std::copy(jobs.begin(), jobs.end(), list->near);
    return CAAT_OK;
  }
  caat::AttnJob* far = static_cast<caat::AttnJob*>(dst);
  list->far = far;
  static thread_local caat::AttnJobChunk chunk;
  for (size_t i = 0; i < jobs.size(); i += caat::KA_UPLOAD_JOBS) {
    const size_t n = std::min(jobs.size() - i, size_t(caat::KA_UPLOAD_JOBS));
    std::copy(jobs.begin() + i, jobs.begin() + i + n, chunk.job);
    caat::attn_upload_kernel<<<1, caat::KA_UPLOAD_JOBS, 0, st>>>(far + i, static_cast<int>(n), chunk);
    if (cudaGetLastError() != cudaSuccess) return CAAT_ERR_CUDA;
  }
  return CAAT_OK;
}

caat_status launch_attn_forward(const caat_attn_args* a, const int32_t* cu_k, const View& q, const View& k, const View& v) {
  int sms = 0;
  caat_status s = attn_setup(&sms);
  if (s != CAAT_OK) return s;
  const int group = a->heads_q / a->heads_k;
  static thread_local std::vector<caat::AttnJob> jobs;
  static thread_local caat::FwdParams prm;
  // A CTA has one tile (dh <= 64), or two.  Two heads of a group on the same 128 rows when the group is
  // even: both tiles then need the same key blocks, and a short sequence wastes less than with 256 rows of
  // one head.
  query_jobs(a->cu_q, cu_k, a->n_seq, caat::KA_TILE, jobs);
  if (jobs.empty()) return CAAT_OK;
  // Where one tile a CTA does not fill the SMs, the second stays empty: a tile alone takes fewer clocks a step
  // (4 heads of 128 on 4096 tokens: 60.5 us with two tiles a CTA, 47.6 with one; 8 on 2048: 35.0 | 28.1).
  const bool two = a->dh > 64 && int64_t(jobs.size()) * a->P * a->heads_q > sms;
  prm.pair_heads = two && group % 2 == 0 ? 1 : 0;
  if (two && !prm.pair_heads) query_jobs(a->cu_q, cu_k, a->n_seq, 2 * caat::KA_TILE, jobs);
  prm.out = reinterpret_cast<__nv_bfloat16*>(a->out);
  prm.lse = a->lse;
  prm.Tq = a->Tq;
  prm.hq = a->heads_q;
  prm.hk = a->heads_k;
  prm.dh = a->dh;
  const int n_heads = prm.pair_heads ? a->heads_q / 2 : a->heads_q;
  prm.group_div.set(group);
  prm.n_heads.set(n_heads);
  prm.per_job.set(a->P * n_heads);
  prm.scale = a->scale;
  prm.timeout_ns = caat::host::wait_limit_ns();
  const int64_t units = int64_t(jobs.size()) * a->P * n_heads;
  if (units > INT32_MAX) return CAAT_ERR_UNSUPPORTED;
  prm.n_units = static_cast<int>(units);
  const int64_t grid = std::min<int64_t>(units, (a->dh > 64 ? caat::FwdCfg<128>::kCtas : caat::FwdCfg<64>::kCtas) * int64_t(sms));
  CUtensorMap mq, mk, mv;
  if ((s = heads_map(&mq, q, a->P, a->Tq, a->heads_q, a->dh)) != CAAT_OK) return s;
  // no keys at all: every row is empty and neither map is used
  if ((s = heads_map(&mk, a->Tk ? k : q, a->P, a->Tk ? a->Tk : 1, a->Tk ? a->heads_k : 1, a->dh)) != CAAT_OK) return s;
  if ((s = heads_map(&mv, a->Tk ? v : q, a->P, a->Tk ? a->Tk : 1, a->Tk ? a->heads_k : 1, a->dh)) != CAAT_OK) return s;
  if ((s = place_jobs(jobs, &prm.jobs, a->workspace, a->stream)) != CAAT_OK) return s;
  Recorder rec;
  rec.begin(a->timing, a->stream);
  if (a->dh <= 64)
    caat::attn_fwd_kernel<64><<<static_cast<unsigned>(grid), caat::FwdCfg<64>::kThreads, caat::FwdCfg<64>::kSmem, a->stream>>>(mq, mk, mv, prm);
  else
    caat::attn_fwd_kernel<128><<<static_cast<unsigned>(grid), caat::FwdCfg<128>::kThreads, caat::FwdCfg<128>::kSmem, a->stream>>>(mq, mk, mv, prm);
  if (cudaGetLastError() != cudaSuccess) return CAAT_ERR_CUDA;
  rec.after_kernel(a->stream);
  return CAAT_OK;
}

caat_status launch_attn_backward(const caat_attn_bwd_args* a, const int32_t* cu_k, const View& q, const View& k, const View& v) {
  int sms = 0;
  caat_status s = attn_setup(&sms);
  if (s != CAAT_OK) return s;
  const int P = a->P, hq = a->heads_q, hk = a->heads_k, dh = a->dh;
  const BwdLayout L = bwd_layout(a->Tq, a->Tk, a->n_seq, P, hq, hk, dh);
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  static thread_local std::vector<caat::AttnJob> jobs;
  static thread_local caat::BwdAttnParams prm;
  prm.out = reinterpret_cast<const __nv_bfloat16*>(a->out);
  prm.dout = reinterpret_cast<const __nv_bfloat16*>(a->dout);
  prm.lse = a->lse;
  prm.D = reinterpret_cast<float*>(ws + L.D);
  prm.dq = reinterpret_cast<__nv_bfloat16*>(a->dq);
  prm.dk = reinterpret_cast<__nv_bfloat16*>(a->dk);
  prm.dv = reinterpret_cast<__nv_bfloat16*>(a->dv);
  prm.part = reinterpret_cast<float*>(ws + L.part);
  prm.Tq = a->Tq;
  prm.Tk = a->Tk;
  prm.P = P;
  prm.hq = hq;
  prm.hk = hk;
  prm.dh = dh;
  prm.group = hq / hk;
  prm.splits = L.splits;
  prm.scale = a->scale;
  prm.timeout_ns = caat::host::wait_limit_ns();
  const View& any = a->Tq ? q : k;  // a side without rows is never read
  View g = any;
  if (a->Tq) {
    g.p = a->dout;
    g.tok = int64_t(hq) * dh;
    g.rank = a->Tq * g.tok;
  }
  const int64_t Tq = a->Tq ? a->Tq : 1, Tk = a->Tk ? a->Tk : 1;
  const int hq_m = a->Tq ? hq : 1, hk_m = a->Tk ? hk : 1;
  CUtensorMap mq, mg, mk, mv, mq64, mg64, mk64, mv64;
  if ((s = heads_map(&mq, any, P, Tq, hq_m, dh)) != CAAT_OK || (s = heads_map(&mg, g, P, Tq, hq_m, dh)) != CAAT_OK ||
      (s = heads_map(&mk, a->Tk ? k : any, P, Tk, hk_m, dh)) != CAAT_OK ||
      (s = heads_map(&mv, a->Tk ? v : any, P, Tk, hk_m, dh)) != CAAT_OK ||
      (s = heads_map(&mq64, any, P, Tq, hq_m, dh, caat::KB2_QT)) != CAAT_OK ||
      (s = heads_map(&mg64, g, P, Tq, hq_m, dh, caat::KB2_QT)) != CAAT_OK)
    return s;
  if (dh <= 64 && ((s = heads_map(&mk64, a->Tk ? k : any, P, Tk, hk_m, dh, caat::DqCfg<64>::kKeys)) != CAAT_OK ||
                   (s = heads_map(&mv64, a->Tk ? v : any, P, Tk, hk_m, dh, caat::DqCfg<64>::kKeys)) != CAAT_OK))
    return s;
  Recorder rec;
  rec.begin(a->timing, a->stream);
  query_jobs(a->cu_q, cu_k, a->n_seq, caat::KA_TILE, jobs);
  const bool dq_ran = !jobs.empty();
  if (dq_ran) {
    prm.per_job = P * hq;
    const int64_t grid = int64_t(jobs.size()) * prm.per_job;
    if (grid > INT32_MAX) return CAAT_ERR_UNSUPPORTED;
    if ((s = place_jobs(jobs, &prm.jobs, ws + L.q_list, a->stream)) != CAAT_OK) return s;
    if (dh <= 64)
      caat::attn_dq_kernel<64><<<static_cast<unsigned>(grid), caat::DqCfg<64>::kThreads, caat::DqCfg<64>::kSmem, a->stream>>>(mq, mg, mk64, mv64, prm);
    else
      caat::attn_dq_kernel<128><<<static_cast<unsigned>(grid), caat::DqCfg<128>::kThreads, caat::DqCfg<128>::kSmem, a->stream>>>(mq, mg, mk, mv, prm);
    if (cudaGetLastError() != cudaSuccess) return CAAT_ERR_CUDA;
    rec.after_kernel(a->stream);
  }
  key_jobs(a->cu_q, cu_k, a->n_seq, jobs);
  if (!jobs.empty()) {
    prm.per_job = P * hk * L.splits;
    const int64_t grid = int64_t(jobs.size()) * prm.per_job;
    if (grid > INT32_MAX) return CAAT_ERR_UNSUPPORTED;
    if ((s = place_jobs(jobs, &prm.jobs, ws + L.k_list, a->stream)) != CAAT_OK) return s;
    // Launched behind dq without waiting for its end (its CTAs set up, load and multiply, and wait where they
    // need D), and the join likewise: 34 tokens 16.4 us | 14.4, packed sequences of 5 to 2048 tokens 139.8 | 135.1.
    // (Not behind an upload.)
    cudaLaunchAttribute behind[1];
    behind[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    behind[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(caat::KB2_THREADS, 1, 1);
    cfg.dynamicSmemBytes = dh <= 64 ? caat::DkvCfg<64>::kSmem : caat::DkvCfg<128>::kSmem;
    cfg.stream = a->stream;
    cfg.attrs = behind;
    cfg.numAttrs = dq_ran && !prm.jobs.far ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, dh <= 64 ? caat::attn_dkv_kernel<64> : caat::attn_dkv_kernel<128>, mq64, mg64, mk, mv, prm) != cudaSuccess)
      return CAAT_ERR_CUDA;
    rec.after_kernel(a->stream);
    if (L.splits > 1) {
      const int pieces = (caat::KA_TILE * hk * dh / 4 + 255) / 256;
      cfg.gridDim = dim3(static_cast<unsigned>(jobs.size()), P, 2 * std::min(pieces, 1024));
      cfg.blockDim = dim3(256, 1, 1);
      cfg.dynamicSmemBytes = 0;
      cfg.numAttrs = 1;
      if (cudaLaunchKernelEx(&cfg, caat::attn_dkv_join_kernel, prm) != cudaSuccess) return CAAT_ERR_CUDA;
      rec.after_kernel(a->stream);
    }
  }
  return CAAT_OK;
}

}  // namespace

extern "C" {

caat_status caat_rope_frequencies(int rot, double theta, int scaling, double factor, double trained_length,
                                  double* inv_freq, float* mscale_out) {
  if (!inv_freq || rot < 2 || rot > 2 * caat::KR_MAX_PAIRS || rot % 2 != 0) return CAAT_ERR_INVALID_ARG;
  if (!(theta > 1.0) || !std::isfinite(theta)) return CAAT_ERR_INVALID_ARG;
  if (scaling < CAAT_ROPE_SCALING_NONE || scaling > CAAT_ROPE_SCALING_YARN) return CAAT_ERR_INVALID_ARG;
  if (scaling != CAAT_ROPE_SCALING_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return CAAT_ERR_INVALID_ARG;
  if (scaling == CAAT_ROPE_SCALING_NTK && rot < 4) return CAAT_ERR_INVALID_ARG;
  if (scaling == CAAT_ROPE_SCALING_YARN && (!(trained_length > 0.0) || !std::isfinite(trained_length)))
    return CAAT_ERR_INVALID_ARG;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (scaling == CAAT_ROPE_SCALING_NTK) theta *= std::pow(factor, double(rot) / (rot - 2));
  if (!std::isfinite(theta)) return CAAT_ERR_INVALID_ARG;
  for (int j = 0; j < rot / 2; ++j) {
    double f = std::pow(theta, -2.0 * j / rot);
    if (scaling == CAAT_ROPE_SCALING_LINEAR) f /= factor;
    if (scaling == CAAT_ROPE_SCALING_YARN) {
      const double turns = trained_length * f / kTwoPi;
      const double keep = std::min(1.0, std::max(0.0, (turns - 1.0) / (32.0 - 1.0)));
      f *= keep + (1.0 - keep) / factor;
    }
    inv_freq[j] = f;
  }
  if (mscale_out) *mscale_out = scaling == CAAT_ROPE_SCALING_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return CAAT_OK;
}

caat_status caat_rope(const caat_rope_args* a) {
  if (!a) return CAAT_ERR_INVALID_ARG;
  if (a->P < 1 || a->P > CAAT_MAX_P || a->T < 0 || a->heads_q < 0 || a->heads_k < 0 || a->dh < 1 || a->rot < 1 ||
      a->rot > a->dh || !std::isfinite(a->mscale))
    return CAAT_ERR_INVALID_ARG;
  if (a->flags & ~(CAAT_ROPE_FLAG_INTERLEAVED | CAAT_ROPE_FLAG_BACKWARD)) return CAAT_ERR_INVALID_ARG;
  const bool inter = (a->flags & CAAT_ROPE_FLAG_INTERLEAVED) != 0;
  if (a->dh % 8 != 0 || a->dh > 256 || a->rot % (inter ? 8 : 16) != 0) return CAAT_ERR_UNSUPPORTED;
  if (a->T > kMaxRows || a->heads_q > 1024 || a->heads_k > 1024) return CAAT_ERR_UNSUPPORTED;
  const bool append = a->slots != nullptr;
  if (append && (a->cache_rows < 0 || a->heads_k == 0)) return CAAT_ERR_INVALID_ARG;
  if (append && a->cache_rows > kMaxCacheRows) return CAAT_ERR_UNSUPPORTED;
  if (!a->inv_freq) return CAAT_ERR_INVALID_ARG;
  for (int j = 0; j < a->rot / 2; ++j)
    if (!std::isfinite(a->inv_freq[j])) return CAAT_ERR_INVALID_ARG;
  if (a->T == 0 || (a->heads_q == 0 && a->heads_k == 0)) return CAAT_OK;

  static thread_local caat::RopeParams prm;
  std::memset(&prm, 0, sizeof(prm));
  Range in[5], out[3];
  View read[3];  // the tensors of in[], their rows, and whether they are turned in place
  int64_t row_of[3];
  bool written[3];
  int n_in = 0, n_out = 0;
  auto tensor = [&](caat::RopeTensor* x, const caat_bf16* p, caat_bf16* o, int64_t s_rank, int64_t s_tok, int heads,
                    bool to_cache) -> caat_status {
    View v;
    const caat_status s = make_view(&v, p, s_rank, s_tok, a->P, a->T, heads, a->dh);
    if (s != CAAT_OK) return s;
    if (!o) return CAAT_ERR_INVALID_ARG;
    if (!aligned16(o)) return CAAT_ERR_UNSUPPORTED;
    const int64_t row = int64_t(heads) * a->dh, rows = to_cache ? a->cache_rows : a->T;
    const bool same = o == p && !to_cache;
    x->in = reinterpret_cast<const __nv_bfloat16*>(p);
    x->out = reinterpret_cast<__nv_bfloat16*>(o);
    x->in_rank = v.rank;
    x->in_tok = v.tok;
    x->out_rank = same ? v.rank : rows * row;
    x->out_tok = same ? v.tok : row;
    x->heads = heads;
    read[n_in] = v;
    row_of[n_in] = row;
    written[n_in] = same;
    in[n_in++] = range_of(v);
    if (!same) out[n_out++] = range_of(o, static_cast<size_t>(a->P) * rows * row * 2);
    return CAAT_OK;
  };
  caat_status s = CAAT_OK;
  if (a->heads_q) s = tensor(&prm.q, a->q, a->q_out, a->q_stride_rank, a->q_stride_token, a->heads_q, false);
  if (s == CAAT_OK && a->heads_k)
    s = tensor(&prm.k, a->k, a->k_out, a->k_stride_rank, a->k_stride_token, a->heads_k, append);
  if (s == CAAT_OK && append) s = tensor(&prm.v, a->v, a->v_out, a->v_stride_rank, a->v_stride_token, a->heads_k, true);
  if (s != CAAT_OK) return s;
  for (int i = 0; i < n_in; ++i) {
    if (!written[i]) continue;
    // in place: no row may lie on another one, of this tensor or of the others (slices of one projection lie
    // side by side within the same tokens)
    const View& w = read[i];
    if (rows_meet(w, row_of[i], w, row_of[i], a->P, a->T)) return CAAT_ERR_INVALID_ARG;
    for (int j = 0; j < n_in; ++j) {
      if (j == i || !meet(in[i], in[j])) continue;
      const View& r = read[j];
      if ((a->T > 1 && w.tok != r.tok) || (a->P > 1 && w.rank != r.rank) || rows_meet(w, row_of[i], r, row_of[j], a->P, a->T))
        return CAAT_ERR_INVALID_ARG;
    }
    out[n_out++] = in[i];
  }
  const int tensors = n_in;
  if (a->positions) in[n_in++] = range_of(a->positions, size_t(a->T) * 4);
  if (append) in[n_in++] = range_of(a->slots, size_t(a->T) * 8);
  const int apart = n_out - static_cast<int>(std::count(written, written + tensors, true));
  for (int o = 0; o < n_out; ++o) {
    for (int i = o < apart ? 0 : tensors; i < n_in; ++i)  // (in place against the tensors: above)
      if (meet(out[o], in[i])) return CAAT_ERR_INVALID_ARG;
    for (int i = 0; i < std::min(o, apart); ++i)
      if (meet(out[o], out[i])) return CAAT_ERR_INVALID_ARG;
  }
  if ((reinterpret_cast<uintptr_t>(a->positions) & 3u) || (reinterpret_cast<uintptr_t>(a->slots) & 7u))
    return CAAT_ERR_UNSUPPORTED;
  int sms = 0;
  s = caat::host::device_sms(&sms);
  if (s != CAAT_OK) return s;
  prm.positions = a->positions;
  prm.slots = a->slots;
  prm.T = a->T;
  prm.cache_rows = a->cache_rows;
  prm.P = a->P;
  prm.dh = a->dh;
  prm.rot = a->rot;
  prm.mscale = a->mscale;
  constexpr double kInvTwoPi = 0.15915494309189533576888376337251;
  for (int j = 0; j < a->rot / 2; ++j)
    prm.turns[j] = (a->flags & CAAT_ROPE_FLAG_BACKWARD ? -kInvTwoPi : kInvTwoPi) * a->inv_freq[j];
  Recorder rec;
  rec.begin(a->timing, a->stream);
  const int per_head = a->rot / (inter ? 8 : 16) + (a->dh - a->rot) / 8;
  const int64_t items = int64_t(a->P) * ((prm.q.heads + prm.k.heads) * per_head + prm.v.heads * (a->dh / 8));
  // Two items a thread keep more loads in flight for many tokens; for few, one a thread spreads them over
  // more SMs, and where a token has no more than 256 the second would be nobody's (T=3001, 176 items a
  // token: 8.2 us | 9.1 in one run; 8.2 to 10.2 from run to run, as calls this short end in steps of 2 us).
  const bool few = items <= caat::KR_THREADS || a->T * ((items + 511) / 512) < 4 * int64_t(sms);
  const int per_cta = caat::KR_THREADS * (few ? 1 : 2);
  const unsigned gy = static_cast<unsigned>((items + per_cta - 1) / per_cta);
  const unsigned gx = static_cast<unsigned>(std::min<int64_t>(a->T, std::max<int64_t>(1, (caat::KR_CTAS * int64_t(sms) + gy - 1) / gy)));
  auto kernel = inter ? (few ? caat::rope_kernel<true, 1> : caat::rope_kernel<true, 2>)
                      : (few ? caat::rope_kernel<false, 1> : caat::rope_kernel<false, 2>);
  kernel<<<dim3(gx, gy), caat::KR_THREADS, 0, a->stream>>>(prm);
  if (cudaGetLastError() != cudaSuccess) return CAAT_ERR_CUDA;
  rec.after_kernel(a->stream);
  return CAAT_OK;
}

size_t caat_attn_workspace_size(int64_t Tq, int64_t Tk, int n_seq, int P, int heads_q, int heads_k, int dh,
                                int variant) {
  if (check_heads(P, heads_q, heads_k, dh, 1.f) != CAAT_OK || Tq < 0 || Tk < 0 || Tq > kMaxRows || Tk > kMaxRows)
    return SIZE_MAX;
  switch (variant) {
    case CAAT_VARIANT_ATTN: return n_seq < 0 ? SIZE_MAX : list_bytes(max_jobs(Tq, n_seq, caat::KA_TILE));
    case CAAT_VARIANT_ATTN_BWD: return n_seq < 0 ? SIZE_MAX : bwd_layout(Tq, Tk, n_seq, P, heads_q, heads_k, dh).total;
    case CAAT_VARIANT_ATTN_DECODE:
      if (decode_cluster(Tq, Tk, P, heads_q, heads_k, dh) > 0) return 0;
      return kDecodeCounters + align256(size_t(caat::KD_CTAS) * 2 * std::min(heads_q / heads_k, 16) * (dh + 2) * 4);
  }
  return SIZE_MAX;
}

caat_status caat_attn_forward(const caat_attn_args* a) {
  if (!a) return CAAT_ERR_INVALID_ARG;
  caat_status s = check_heads(a->P, a->heads_q, a->heads_k, a->dh, a->scale);
  if (s != CAAT_OK) return s;
  if (a->Tq < 0 || a->Tk < 0 || a->n_seq < 0 || a->flags != 0) return CAAT_ERR_INVALID_ARG;
  if (a->Tq > kMaxRows || a->Tk > kMaxRows) return CAAT_ERR_UNSUPPORTED;
  if (a->n_seq == 0 || a->Tq == 0) return CAAT_OK;
  if (!a->cu_q) return CAAT_ERR_INVALID_ARG;
  const int32_t* cu_k = a->cu_k ? a->cu_k : a->cu_q;
  if ((s = check_offsets(a->cu_q, a->n_seq, a->Tq)) != CAAT_OK) return s;
  if ((s = check_offsets(cu_k, a->n_seq, a->Tk)) != CAAT_OK) return s;
  View q, k, v;
  if ((s = make_view(&q, a->q, a->q_stride_rank, a->q_stride_token, a->P, a->Tq, a->heads_q, a->dh)) != CAAT_OK) return s;
  if (a->Tk > 0) {
    if ((s = make_view(&k, a->k, a->k_stride_rank, a->k_stride_token, a->P, a->Tk, a->heads_k, a->dh)) != CAAT_OK) return s;
    if ((s = make_view(&v, a->v, a->v_stride_rank, a->v_stride_token, a->P, a->Tk, a->heads_k, a->dh)) != CAAT_OK) return s;
  }
  if (!a->out) return CAAT_ERR_INVALID_ARG;
  if (!aligned16(a->out) || (reinterpret_cast<uintptr_t>(a->lse) & 3u)) return CAAT_ERR_UNSUPPORTED;
  const Range out = range_of(a->out, size_t(a->P) * a->Tq * a->heads_q * a->dh * 2);
  const Range lse = range_of(a->lse, a->lse ? size_t(a->P) * a->Tq * a->heads_q * 4 : 0);
  if (meet(lse, out) || meet(lse, range_of(q)) || meet(lse, range_of(k)) || meet(lse, range_of(v)))
    return CAAT_ERR_INVALID_ARG;
  if (meet(out, range_of(q)) || meet(out, range_of(k)) || meet(out, range_of(v))) return CAAT_ERR_INVALID_ARG;
  const size_t need = caat_attn_workspace_size(a->Tq, a->Tk, a->n_seq, a->P, a->heads_q, a->heads_k, a->dh, CAAT_VARIANT_ATTN);
  if (need > 0 && (!a->workspace || a->ws_bytes < need || (reinterpret_cast<uintptr_t>(a->workspace) & 255u)))
    return CAAT_ERR_WORKSPACE;
  try {
    return launch_attn_forward(a, cu_k, q, k, v);
  } catch (const std::bad_alloc&) {
    return CAAT_ERR_CUDA;
  }
}

caat_status caat_attn_backward(const caat_attn_bwd_args* a) {
  if (!a) return CAAT_ERR_INVALID_ARG;
  caat_status s = check_heads(a->P, a->heads_q, a->heads_k, a->dh, a->scale);
  if (s != CAAT_OK) return s;
  if (a->Tq < 0 || a->Tk < 0 || a->n_seq < 0 || a->flags != 0) return CAAT_ERR_INVALID_ARG;
  if (a->Tq > kMaxRows || a->Tk > kMaxRows) return CAAT_ERR_UNSUPPORTED;
  if (a->n_seq == 0 || (a->Tq == 0 && a->Tk == 0)) return CAAT_OK;
  if (!a->cu_q) return CAAT_ERR_INVALID_ARG;
  const int32_t* cu_k = a->cu_k ? a->cu_k : a->cu_q;
  if ((s = check_offsets(a->cu_q, a->n_seq, a->Tq)) != CAAT_OK) return s;
  if ((s = check_offsets(cu_k, a->n_seq, a->Tk)) != CAAT_OK) return s;
  View q, k, v;
  Range in[6], out[3];
  int n_in = 0, n_out = 0;
  if (a->Tq > 0) {
    if ((s = make_view(&q, a->q, a->q_stride_rank, a->q_stride_token, a->P, a->Tq, a->heads_q, a->dh)) != CAAT_OK) return s;
    if (!a->out || !a->dout || !a->lse || !a->dq) return CAAT_ERR_INVALID_ARG;
    if (!aligned16(a->out) || !aligned16(a->dout) || !aligned16(a->dq) || (reinterpret_cast<uintptr_t>(a->lse) & 3u))
      return CAAT_ERR_UNSUPPORTED;
    const size_t bytes = size_t(a->P) * a->Tq * a->heads_q * a->dh * 2;
    in[n_in++] = range_of(q);
    in[n_in++] = range_of(a->out, bytes);
    in[n_in++] = range_of(a->dout, bytes);
    in[n_in++] = range_of(a->lse, size_t(a->P) * a->Tq * a->heads_q * 4);
    out[n_out++] = range_of(a->dq, bytes);
  }
  if (a->Tk > 0) {
    if ((s = make_view(&k, a->k, a->k_stride_rank, a->k_stride_token, a->P, a->Tk, a->heads_k, a->dh)) != CAAT_OK) return s;
    if ((s = make_view(&v, a->v, a->v_stride_rank, a->v_stride_token, a->P, a->Tk, a->heads_k, a->dh)) != CAAT_OK) return s;
    if (!a->dk || !a->dv) return CAAT_ERR_INVALID_ARG;
    if (!aligned16(a->dk) || !aligned16(a->dv)) return CAAT_ERR_UNSUPPORTED;
    const size_t bytes = size_t(a->P) * a->Tk * a->heads_k * a->dh * 2;
    in[n_in++] = range_of(k);
    in[n_in++] = range_of(v);
    out[n_out++] = range_of(a->dk, bytes);
    out[n_out++] = range_of(a->dv, bytes);
  }
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i)
      if (meet(out[o], in[i])) return CAAT_ERR_INVALID_ARG;
    for (int i = 0; i < o; ++i)
      if (meet(out[o], out[i])) return CAAT_ERR_INVALID_ARG;
  }
  const size_t need =
      caat_attn_workspace_size(a->Tq, a->Tk, a->n_seq, a->P, a->heads_q, a->heads_k, a->dh, CAAT_VARIANT_ATTN_BWD);
  if (need > 0 && (!a->workspace || a->ws_bytes < need || (reinterpret_cast<uintptr_t>(a->workspace) & 255u)))
    return CAAT_ERR_WORKSPACE;
  try {
    return launch_attn_backward(a, cu_k, q, k, v);
  } catch (const std::bad_alloc&) {
    return CAAT_ERR_CUDA;
  }
}

caat_status caat_attn_decode(const caat_attn_decode_args* a) {
  if (!a) return CAAT_ERR_INVALID_ARG;
  caat_status s = check_heads(a->P, a->heads_q, a->heads_k, a->dh, a->scale);
  if (s != CAAT_OK) return s;
  if (a->B < 0 || a->capacity < 0 || a->flags != 0) return CAAT_ERR_INVALID_ARG;
  if (a->capacity > kMaxRows || a->B > caat::KD_MAX_B || a->B * a->capacity > kMaxCacheRows) return CAAT_ERR_UNSUPPORTED;
  if (a->B == 0) return CAAT_OK;
  View q;
  if ((s = make_view(&q, a->q, a->q_stride_rank, a->q_stride_token, a->P, a->B, a->heads_q, a->dh)) != CAAT_OK) return s;
  if (!a->lens || !a->out || (a->capacity > 0 && (!a->k_cache || !a->v_cache))) return CAAT_ERR_INVALID_ARG;
  if (!aligned16(a->k_cache) || !aligned16(a->v_cache) || !aligned16(a->out) || (reinterpret_cast<uintptr_t>(a->lens) & 3u))
    return CAAT_ERR_UNSUPPORTED;
  const Range out = range_of(a->out, size_t(a->P) * a->B * a->heads_q * a->dh * 2);
  const size_t cache = size_t(a->P) * a->B * a->capacity * a->heads_k * a->dh * 2;
  if (meet(out, range_of(q)) || meet(out, range_of(a->k_cache, cache)) || meet(out, range_of(a->v_cache, cache)) ||
      meet(out, range_of(a->lens, size_t(a->B) * 4)))
    return CAAT_ERR_INVALID_ARG;
  const size_t need = caat_attn_workspace_size(a->B, a->capacity, 0, a->P, a->heads_q, a->heads_k, a->dh, CAAT_VARIANT_ATTN_DECODE);
  if (need > 0 && (!a->workspace || a->ws_bytes < need || (reinterpret_cast<uintptr_t>(a->workspace) & 255u)))
    return CAAT_ERR_WORKSPACE;
  int sms = 0;
  if ((s = attn_setup(&sms)) != CAAT_OK) return s;
  caat::DecodeAttnParams p{};
  p.q = reinterpret_cast<const __nv_bfloat16*>(a->q);
  p.k = reinterpret_cast<const __nv_bfloat16*>(a->k_cache);
  p.v = reinterpret_cast<const __nv_bfloat16*>(a->v_cache);
  p.lens = a->lens;
  p.out = reinterpret_cast<__nv_bfloat16*>(a->out);
  p.q_rank = q.rank;
  p.q_tok = q.tok;
  p.B = a->B;
  p.capacity = a->capacity;
  p.P = a->P;
  p.hq = a->heads_q;
  p.hk = a->heads_k;
  p.dh = a->dh;
  p.group = a->heads_q / a->heads_k;
  p.rows = std::min(p.group, 16);
  p.n_gb = (p.group + 15) / 16;
  p.G = a->P * a->heads_k * p.n_gb;
  p.scale = a->scale;
  const int HD = a->dh <= 64 ? 64 : 128;
  const int tile = 4 * caat::kd_keys(HD);
  const int stage = tile * 2 * HD * 2, merge = 4 * p.rows * (HD + 2) * 4;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.blockDim = dim3(caat::KD_THREADS, 1, 1);
  cfg.stream = a->stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  Recorder rec;
  rec.begin(a->timing, a->stream);
  cudaError_t e;
  const int cluster = decode_cluster(a->B, a->capacity, a->P, a->heads_q, a->heads_k, a->dh);
  if (cluster > 0) {
    const int own = p.rows * 2 * 4;  // the CTA's maxima and sums
    p.stages = std::min(5, (caat::KD_SMEM - merge - own) / stage);
    cfg.gridDim = dim3(static_cast<unsigned>(a->B * p.G * cluster), 1, 1);
    cfg.dynamicSmemBytes = p.stages * stage + merge + own;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    e = HD == 64 ? cudaLaunchKernelEx(&cfg, caat::attn_decode_cluster_kernel<64>, p, cluster)
                 : cudaLaunchKernelEx(&cfg, caat::attn_decode_cluster_kernel<128>, p, cluster);
  } else {
    p.count = static_cast<unsigned int*>(a->workspace);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) + kDecodeCounters);
    const int index = static_cast<int>(a->B + 5) * 4;
    p.stages = std::min(5, (caat::KD_SMEM - merge - index) / stage);
    const int64_t most = int64_t(p.G) * a->B * ((a->capacity + tile - 1) / tile);
    cfg.gridDim = dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(caat::KD_CTAS, most))), 1, 1);
    cfg.dynamicSmemBytes = p.stages * stage + merge + index;
    caat::attn_decode_clear_kernel<<<1, caat::KD_CTAS, 0, a->stream>>>(p.count);
    if (cudaGetLastError() != cudaSuccess) return CAAT_ERR_CUDA;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    e = HD == 64 ? cudaLaunchKernelEx(&cfg, caat::attn_decode_kernel<64>, p)
                 : cudaLaunchKernelEx(&cfg, caat::attn_decode_kernel<128>, p);
  }
  if (e != cudaSuccess) return CAAT_ERR_CUDA;
  rec.after_kernel(a->stream);
  return CAAT_OK;
}

}  // extern "C"
