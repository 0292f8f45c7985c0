// api_dense.cu -- the C ABI of the full-attention operators over packed and
// paged keys and values: argument validation, workspace layout, launches.
#include <math.h>

#include "api_common.h"
#include "kernels.h"

namespace msa {
namespace {

// CTAs of the persistent kernels, at most; sizes the partial results in the
// workspace without asking the device (a B200 has 148 SMs)
constexpr int kMaxCtas = 160;
// a unit of the prefill is split only when it has more than four key tiles
constexpr int kSplitKeys = 4 * 128;
constexpr int kMaxHeadsPerGroup = 128;  // a token's heads of one group fill at most one row tile

int grid_ctas() {
  const int n = sm_count();
  return n < kMaxCtas ? n : kMaxCtas;
}

// index_dim, top_k and block_size are not read
msa_status_t check_dense_cfg(const msa_config_t* c) {
  if (!c) return MSA_ERR_INVALID_ARG;
  if (c->num_heads <= 0 || c->num_groups <= 0 || c->head_dim <= 0) return MSA_ERR_INVALID_ARG;
  if (c->num_heads % c->num_groups != 0) return MSA_ERR_INVALID_ARG;
  if (!(c->softmax_scale > 0.f) || !isfinite(c->softmax_scale)) return MSA_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return MSA_ERR_UNSUPPORTED;
  if (c->num_heads > 4096 || c->num_heads / c->num_groups > kMaxHeadsPerGroup)
    return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

msa_status_t check_rows(const msa_config_t* c, int64_t T, int32_t B) {
  if (T < 1 || B < 1) return MSA_ERR_INVALID_ARG;
  if (T >= (int64_t(1) << 26) || B >= (1 << 24)) return MSA_ERR_UNSUPPORTED;
  // unit numbers (tile pairs x groups) are 32-bit
  if ((T + B + 4 * kMaxCtas) * c->num_groups >= (int64_t(1) << 31)) return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

msa_status_t check_cache(const msa_config_t* c, const msa_paged_kv_t* kv, PagedCache* out) {
  if (!kv || !kv->k || !kv->v || !kv->block_table) return MSA_ERR_INVALID_ARG;
  if (!aligned16(kv->k) || !aligned16(kv->v) || (reinterpret_cast<uintptr_t>(kv->block_table) & 3))
    return MSA_ERR_INVALID_ARG;
  if (kv->num_pages < 1 || kv->table_stride < 1) return MSA_ERR_INVALID_ARG;
  const int ps = kv->page_size;
  if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256) return MSA_ERR_UNSUPPORTED;
  const int64_t page = (int64_t)ps * c->num_groups * c->head_dim;
  if (kv->page_stride < page || kv->page_stride % 8 != 0) return MSA_ERR_INVALID_ARG;
  if (kv->num_pages >= (int64_t(1) << 31) - 1 || kv->page_stride >= (int64_t(1) << 38) ||
      (int64_t)kv->table_stride * ps > (int64_t(1) << 30))
    return MSA_ERR_UNSUPPORTED;
  out->k = kv->k;
  out->v = kv->v;
  out->block_table = kv->block_table;
  out->num_pages = kv->num_pages;
  out->page_stride = kv->page_stride;
  out->page_size = ps;
  out->table_stride = kv->table_stride;
  return MSA_OK;
}

// prefill workspace: header (error word, unit counts) | units | split list |
// partial outputs | partial maxima and sums
struct PrefillWs {
  size_t units, splits, part_o, part_ml, total;
  int32_t max_units, max_slots;
};
PrefillWs prefill_ws(const msa_config_t* c, int64_t T, int32_t B, bool paged) {
  PrefillWs w;
  const int64_t U = 2 * dense_tile_tokens(c->num_heads, c->num_groups);
  w.max_slots = paged || T > kSplitKeys ? 2 * kMaxCtas : 0;
  w.max_units = (int32_t)(T / U + B + w.max_slots);
  size_t off = kHeader;
  w.units = off;
  off += align256((size_t)w.max_units * sizeof(DenseUnit));
  w.splits = off;
  off += align256((size_t)w.max_slots * sizeof(DenseSplit));
  w.part_o = off;
  off += (size_t)w.max_slots * 256 * c->head_dim * sizeof(float);
  w.part_ml = off;
  off += (size_t)w.max_slots * 256 * sizeof(float2);
  w.total = off;
  return w;
}
constexpr size_t kCountsOffset = 128;  // within the header

// decode workspace: header | tickets | partials
struct DecodeWs {
  size_t tickets, part, total;
};
DecodeWs decode_ws(const msa_config_t* c, int32_t B) {
  DecodeWs w;
  size_t off = kHeader;
  w.tickets = off;
  off += align256((size_t)B * dense_decode_chunks(c->num_heads, c->num_groups) * 4);
  w.part = off;
  off += (size_t)kMaxCtas * 2 * kDenseDecodeWarps *
         dense_decode_partial_floats(c->num_heads, c->num_groups, c->head_dim) * 4;
  w.total = off;
  return w;
}

msa_status_t run_prefill(const msa_config_t* cfg, DensePrefillLaunch& p, const PrefillWs& w,
                         void* ws, cudaStream_t s, int* launches) {
  p.H = cfg->num_heads;
  p.G = cfg->num_groups;
  p.d = cfg->head_dim;
  p.scale = cfg->softmax_scale;
  p.units = at<DenseUnit>(ws, w.units);
  p.splits = at<DenseSplit>(ws, w.splits);
  p.counts = at<int32_t>(ws, kCountsOffset);
  p.part_o = at<float>(ws, w.part_o);
  p.part_ml = at<float2>(ws, w.part_ml);
  p.max_units = w.max_units;
  p.max_slots = w.max_slots;
  p.err = at<uint32_t>(ws, 0);
  p.grid = grid_ctas();
  return cuda_status(launch_dense_prefill(p, s, launches));
}

}  // namespace

msa_status_t dense_workspace_size(const msa_config_t* cfg, msa_op_t op, int64_t n_tokens,
                                  int32_t batch, size_t* bytes) {
  msa_status_t st = check_dense_cfg(cfg);
  if (st != MSA_OK) return st;
  if (!bytes) return MSA_ERR_INVALID_ARG;
  if ((st = check_rows(cfg, n_tokens, batch)) != MSA_OK) return st;
  if (op == MSA_OP_ROPE_APPEND)
    *bytes = kHeader;
  else if (op == MSA_OP_DENSE_DECODE)
    *bytes = decode_ws(cfg, batch).total;
  else
    *bytes = prefill_ws(cfg, n_tokens, batch, op == MSA_OP_DENSE_PREFILL_PAGED).total;
  return MSA_OK;
}

}  // namespace msa

using namespace msa;

extern "C" {

msa_status_t msa_rope_append_paged(const msa_config_t* cfg, const void* q, int64_t q_stride,
                                   const void* k, int64_t k_stride, const void* v,
                                   int64_t v_stride, const float* inv_freq, int32_t rot_dim,
                                   int32_t interleaved, const msa_paged_kv_t* cache,
                                   const int64_t* cu_seqlens, const int32_t* seq_lens, int32_t B,
                                   int64_t T, void* q_out, void* ws, size_t ws_bytes,
                                   msa_stream_t stream) {
  set_launch_count(0);
  msa_status_t st = check_dense_cfg(cfg);
  if (st != MSA_OK) return st;
  if ((st = check_rows(cfg, T, B)) != MSA_OK) return st;
  if (!k || !v || (!inv_freq && rot_dim != 0) || !cu_seqlens || !seq_lens ||
      (q == nullptr) != (q_out == nullptr))
    return MSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
      (reinterpret_cast<uintptr_t>(inv_freq) & 3) || (reinterpret_cast<uintptr_t>(cu_seqlens) & 7) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3))
    return MSA_ERR_INVALID_ARG;
  const int64_t hd = (int64_t)cfg->num_heads * cfg->head_dim;
  const int64_t gd = (int64_t)cfg->num_groups * cfg->head_dim;
  if ((q && (q_stride < hd || q_stride % 8 != 0)) || k_stride < gd || k_stride % 8 != 0 ||
      v_stride < gd || v_stride % 8 != 0)
    return MSA_ERR_INVALID_ARG;
  if (q && q == q_out && q_stride != hd && T > 1) return MSA_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > cfg->head_dim) return MSA_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0) return MSA_ERR_UNSUPPORTED;
  RopeAppendLaunch p{};
  if ((st = check_cache(cfg, cache, &p.cache)) != MSA_OK) return st;
  if (!ws || ws_bytes < kHeader || !aligned16(ws)) return MSA_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.inv_freq = inv_freq;
  p.rot = rot_dim;
  p.interleaved = interleaved;
  p.cu = cu_seqlens;
  p.seq_lens = seq_lens;
  p.B = B;
  p.H = cfg->num_heads;
  p.G = cfg->num_groups;
  p.d = cfg->head_dim;
  p.T = T;
  p.q_out = q_out;
  p.err = at<uint32_t>(ws, 0);
  p.num_sms = sm_count();
  st = cuda_status(launch_rope_append(p, s));
  set_launch_count(1);
  return st;
}

msa_status_t msa_dense_prefill_varlen(const msa_config_t* cfg, const void* q, const void* k,
                                      const void* v, const int64_t* cu_seqlens, int32_t B,
                                      void* out, void* ws, size_t ws_bytes, msa_stream_t stream) {
  set_launch_count(0);
  msa_status_t st = check_dense_cfg(cfg);
  if (st != MSA_OK) return st;
  if (!q || !k || !v || !out || !cu_seqlens || B < 1) return MSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return MSA_ERR_INVALID_ARG;
  if (cu_seqlens[0] != 0) return MSA_ERR_INVALID_ARG;
  for (int32_t b = 0; b < B; ++b)
    if (cu_seqlens[b + 1] < cu_seqlens[b]) return MSA_ERR_INVALID_ARG;
  const int64_t T = cu_seqlens[B];
  if ((st = check_rows(cfg, T, B)) != MSA_OK) return st;
  if (!ws || !aligned16(ws) || ws_bytes < prefill_ws(cfg, T, B, false).total)
    return MSA_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t hd = (size_t)cfg->num_heads * cfg->head_dim * 2;
  const size_t gd = (size_t)cfg->num_groups * cfg->head_dim * 2;
  int launches = 0;
  // the offsets travel as a kernel parameter: up to 1024 sequences a pass
  static thread_local DenseOffsets off;
  for (int32_t b0 = 0; b0 < B && st == MSA_OK; b0 += kDenseMaxSeqs) {
    const int32_t n = B - b0 < kDenseMaxSeqs ? B - b0 : kDenseMaxSeqs;
    const int64_t t0 = cu_seqlens[b0], rows = cu_seqlens[b0 + n] - t0;
    if (rows == 0) continue;
    for (int32_t i = 0; i <= n; ++i) off.cu[i] = cu_seqlens[b0 + i] - t0;
    DensePrefillLaunch p{};
    p.q = static_cast<const uint8_t*>(q) + t0 * hd;
    p.k = static_cast<const uint8_t*>(k) + t0 * gd;
    p.v = static_cast<const uint8_t*>(v) + t0 * gd;
    p.out = static_cast<uint8_t*>(out) + t0 * hd;
    p.offsets = &off;
    p.B = n;
    p.T = rows;
    p.clear_err = launches == 0;
    PrefillWs w = prefill_ws(cfg, rows, n, false);
    st = run_prefill(cfg, p, w, ws, s, &launches);
  }
  set_launch_count(launches);
  return st;
}

msa_status_t msa_dense_prefill_paged(const msa_config_t* cfg, const void* q,
                                     const msa_paged_kv_t* cache, const int64_t* cu_seqlens,
                                     const int32_t* seq_lens, int32_t B, int64_t T, void* out,
                                     void* ws, size_t ws_bytes, msa_stream_t stream) {
  set_launch_count(0);
  msa_status_t st = check_dense_cfg(cfg);
  if (st != MSA_OK) return st;
  if ((st = check_rows(cfg, T, B)) != MSA_OK) return st;
  if (!q || !out || !cu_seqlens || !seq_lens) return MSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(cu_seqlens) & 7) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3))
    return MSA_ERR_INVALID_ARG;
  DensePrefillLaunch p{};
  if ((st = check_cache(cfg, cache, &p.cache)) != MSA_OK) return st;
  PrefillWs w = prefill_ws(cfg, T, B, true);
  if (!ws || !aligned16(ws) || ws_bytes < w.total) return MSA_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.clear_err = 1;
  // no sequence can be long enough to be split: no pass that joins parts
  if ((int64_t)p.cache.table_stride * p.cache.page_size <= kSplitKeys) w.max_slots = 0;
  static const DenseOffsets kNoOffsets = {};
  p.q = q;
  p.out = out;
  p.offsets = &kNoOffsets;
  p.cu = cu_seqlens;
  p.seq_lens = seq_lens;
  p.B = B;
  p.T = T;
  int launches = 0;
  st = run_prefill(cfg, p, w, ws, s, &launches);
  set_launch_count(launches);
  return st;
}

msa_status_t msa_dense_decode_paged(const msa_config_t* cfg, const void* q,
                                    const msa_paged_kv_t* cache, const int32_t* seq_lens,
                                    int32_t B, void* out, void* ws, size_t ws_bytes,
                                    msa_stream_t stream) {
  set_launch_count(0);
  msa_status_t st = check_dense_cfg(cfg);
  if (st != MSA_OK) return st;
  if ((st = check_rows(cfg, B, B)) != MSA_OK) return st;
  if (!q || !out || !seq_lens) return MSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(seq_lens) & 3))
    return MSA_ERR_INVALID_ARG;
  DenseDecodeLaunch p{};
  if ((st = check_cache(cfg, cache, &p.cache)) != MSA_OK) return st;
  const DecodeWs w = decode_ws(cfg, B);
  if (!ws || !aligned16(ws) || ws_bytes < w.total) return MSA_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.q = q;
  p.seq_lens = seq_lens;
  p.B = B;
  p.H = cfg->num_heads;
  p.G = cfg->num_groups;
  p.d = cfg->head_dim;
  p.scale = cfg->softmax_scale;
  p.out = out;
  p.tickets = at<int32_t>(ws, w.tickets);
  p.part = at<float>(ws, w.part);
  p.err = at<uint32_t>(ws, 0);
  p.clear_words = (int64_t)(w.part / 4);
  p.grid = grid_ctas();
  st = cuda_status(launch_dense_decode(p, s));
  set_launch_count(2);
  return st;
}

}  // extern "C"
