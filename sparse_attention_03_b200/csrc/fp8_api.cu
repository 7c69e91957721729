// C entry points of the paged 8-bit caches: argument checks, workspace carving
// and kernel dispatch. The operations are defined in include/lsa.h.
#include <algorithm>

#include "api.h"
#include "common.cuh"
#include "fp8.h"

namespace lsa {
namespace {

// Regions of one block of R rows of lsa_fp8_forward.
struct ForwardPlan {
  size_t scores, hist, idx, count, pos, index, topk, mla, total;
  size_t topk_bytes, mla_bytes;
};

ForwardPlan forward_plan(const lsa_config* c, int R, int64_t max_len) {
  ForwardPlan p;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  p.scores = take((size_t)R * max_len * sizeof(float));
  p.hist = take((size_t)R * kTopkHistStride * sizeof(uint32_t));
  p.idx = take((size_t)R * c->index_topk * sizeof(int32_t));
  p.count = take((size_t)R * sizeof(int32_t));
  p.pos = take((size_t)R * sizeof(int32_t));
  p.index = take(fp8_index_ws_bytes(R));
  p.topk_bytes = topk_ws(R, max_len);
  p.topk = take(p.topk_bytes);
  p.mla_bytes = fp8_mla_ws_bytes(R, c->cli_factor, c->index_topk);
  p.mla = take(p.mla_bytes);
  p.total = o;
  return p;
}

lsa_status check_rows(const char* fn, int32_t n_rows, int32_t n_seq, const int32_t* seq_of_row, int32_t n_pages,
                      int32_t max_pages, int64_t max_len) {
  if (n_rows < 0 || n_seq < 1 || max_len < 1 || max_pages < 1)
    return set_error(LSA_ERR_INVALID, "%s: need n_rows >= 0, n_seq >= 1, max_pages >= 1, max_len >= 1", fn);
  if (n_pages < 1 || n_pages > kMaxPages)
    return set_error(LSA_ERR_INVALID, "%s: need 1 <= n_pages <= %d", fn, kMaxPages);
  if (max_len > INT32_MAX) return set_error(LSA_ERR_INVALID, "%s: max_len exceeds 2^31 - 1", fn);
  if (!seq_of_row && n_rows > n_seq)
    return set_error(LSA_ERR_INVALID, "%s: seq_of_row is NULL with more rows than sequences", fn);
  return LSA_OK;
}

lsa_status check_subs(const char* fn, int n_sub, const lsa_bf16* const* q, const void* const* lat,
                      lsa_bf16* const* out) {
  if (!q || !lat || !out) return set_error(LSA_ERR_INVALID, "%s: NULL array argument", fn);
  for (int z = 0; z < n_sub; ++z) {
    if (!q[z] || !lat[z] || !out[z]) return set_error(LSA_ERR_INVALID, "%s: NULL pointer for sub-block %d", fn, z);
    if (!aligned16(q[z]) || !aligned16(lat[z]) || !aligned16(out[z]))
      return set_error(LSA_ERR_INVALID, "%s: sub-block %d arrays must be 16-byte aligned", fn, z);
  }
  return LSA_OK;
}

char* align_ws(void* ws, size_t bytes, size_t* avail) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(ws), p = (b + kAlign - 1) & ~uintptr_t(kAlign - 1);
  *avail = ws ? bytes - std::min(bytes, (size_t)(p - b)) : 0;
  return ws ? reinterpret_cast<char*>(p) : nullptr;
}

PagedRows paged_rows(int32_t n_rows, int32_t n_seq, const int32_t* seq_of_row, const int32_t* pos,
                     const int32_t* block_table, int32_t max_pages, int32_t n_pages, int64_t max_len) {
  PagedRows r;
  r.seq_of_row = seq_of_row;
  r.pos = pos;
  r.block_table = block_table;
  r.n_rows = n_rows;
  r.n_seq = n_seq;
  r.max_pages = max_pages;
  r.n_pages = n_pages;
  r.max_len = max_len;
  r.err = device_error_word();
  return r;
}

}  // namespace

size_t fp8_workspace_size(const lsa_config* c, int op, int n_rows, int n_seq, int64_t max_len) {
  if (op == LSA_OP_FP8_INDEX) return fp8_index_ws_bytes(n_rows) + kAlign;
  if (op == LSA_OP_FP8_MLA) return fp8_mla_ws_bytes(n_rows, c->cli_factor, max_len) + kAlign;
  if (max_len <= c->index_topk) return fp8_mla_ws_bytes(n_rows, c->cli_factor, max_len) + kAlign;
  return forward_plan(c, prefill_block_rows(n_rows, max_len), max_len).total + kAlign;
}

}  // namespace lsa

using namespace lsa;

extern "C" {

lsa_status lsa_page_plan(int32_t n_seq, const int32_t* cached, const int32_t* fresh, const int32_t* free_pages,
                         int32_t n_free, int32_t* block_table, int32_t max_pages, int32_t n_rows,
                         int32_t* seq_of_row, int32_t* pos, int32_t* slot, int32_t* totals, void* stream) {
  const char* fn = "lsa_page_plan";
  if (n_seq < 1 || n_free < 0 || max_pages < 1 || n_rows < 0)
    return set_error(LSA_ERR_INVALID, "%s: need n_seq >= 1, n_free >= 0, max_pages >= 1, n_rows >= 0", fn);
  if (n_seq > LSA_PLAN_MAX_SEQ)
    return set_error(LSA_ERR_UNSUPPORTED, "%s: at most %d requests", fn, LSA_PLAN_MAX_SEQ);
  if (!cached || !fresh || !block_table || !totals || (n_free > 0 && !free_pages) ||
      (n_rows > 0 && (!seq_of_row || !pos || !slot)))
    return set_error(LSA_ERR_INVALID, "%s: NULL array argument", fn);
  PagePlanArgs a;
  a.cached = cached;
  a.fresh = fresh;
  a.free_pages = free_pages;
  a.block_table = block_table;
  a.seq_of_row = seq_of_row;
  a.pos = pos;
  a.slot = slot;
  a.totals = totals;
  a.n_seq = n_seq;
  a.n_free = n_free;
  a.max_pages = max_pages;
  a.n_rows = n_rows;
  a.err = device_error_word();
  return cuda_status(launch_page_plan(a, (cudaStream_t)stream), fn);
}

lsa_status lsa_fp8_append(const lsa_config* c, int32_t n_rows, const int32_t* slot, int32_t n_sub,
                          const lsa_bf16* const* latent, int64_t latent_ld, void* const* latent_pages,
                          const lsa_bf16* k_idx, int64_t k_ld, void* key_pages, int32_t n_pages, void* stream) {
  const char* fn = "lsa_fp8_append";
  lsa_status s = check_cfg(c, fn);
  if (s != LSA_OK) return s;
  if (n_rows < 0 || n_sub < 0 || n_sub > 2)
    return set_error(LSA_ERR_INVALID, "%s: need n_rows >= 0 and n_sub in 0..2", fn);
  if (n_pages < 1 || n_pages > kMaxPages)
    return set_error(LSA_ERR_INVALID, "%s: need 1 <= n_pages <= %d", fn, kMaxPages);
  if (n_sub == 0 && !k_idx && !key_pages) return set_error(LSA_ERR_INVALID, "%s: nothing to append", fn);
  if (n_sub > 0 && (latent_ld < kDLat || latent_ld % 8))
    return set_error(LSA_ERR_INVALID, "%s: latent_ld must be a multiple of 8, at least %d", fn, kDLat);
  if ((k_idx == nullptr) != (key_pages == nullptr))
    return set_error(LSA_ERR_INVALID, "%s: k_idx and key_pages go together", fn);
  if (k_idx && (k_ld < kDi || k_ld % 8))
    return set_error(LSA_ERR_INVALID, "%s: k_ld must be a multiple of 8, at least %d", fn, kDi);
  if (n_rows == 0) return LSA_OK;
  if (!slot || (n_sub > 0 && (!latent || !latent_pages)))
    return set_error(LSA_ERR_INVALID, "%s: NULL array argument", fn);
  Fp8AppendArgs a = {};
  for (int z = 0; z < n_sub; ++z) {
    if (!latent[z] || !latent_pages[z]) return set_error(LSA_ERR_INVALID, "%s: NULL pointer for sub-block %d", fn, z);
    if (!aligned16(latent[z]) || !aligned16(latent_pages[z]))
      return set_error(LSA_ERR_INVALID, "%s: sub-block %d arrays must be 16-byte aligned", fn, z);
    a.src[z] = latent[z];
    a.dst[z] = static_cast<uint8_t*>(latent_pages[z]);
    a.ld[z] = latent_ld;
  }
  if (!aligned16(k_idx) || !aligned16(key_pages))
    return set_error(LSA_ERR_INVALID, "%s: k_idx and key_pages must be 16-byte aligned", fn);
  a.src[2] = k_idx;
  a.dst[2] = static_cast<uint8_t*>(key_pages);
  a.ld[2] = k_ld;
  a.slot = slot;
  a.n_rows = n_rows;
  a.n_pages = n_pages;
  a.err = device_error_word();
  return cuda_status(launch_fp8_append(a, (cudaStream_t)stream), fn);
}

lsa_status lsa_fp8_index_scores(const lsa_config* c, int32_t n_rows, int32_t n_seq, const int32_t* seq_of_row,
                                const int32_t* pos, const lsa_bf16* q_idx, const float* w, const void* key_pages,
                                int32_t n_pages, const int32_t* block_table, int32_t max_pages, int64_t max_len,
                                float* scores, int64_t ld, uint32_t* topk_hist, void* ws, size_t ws_bytes,
                                void* stream) {
  const char* fn = "lsa_fp8_index_scores";
  lsa_status s = check_cfg(c, fn);
  if (s != LSA_OK) return s;
  s = check_rows(fn, n_rows, n_seq, seq_of_row, n_pages, max_pages, max_len);
  if (s != LSA_OK) return s;
  if (ld < max_len) return set_error(LSA_ERR_INVALID, "%s: need ld >= max_len", fn);
  if (n_rows == 0) return LSA_OK;
  if (!pos || !q_idx || !w || !key_pages || !block_table || !scores)
    return set_error(LSA_ERR_INVALID, "%s: NULL array argument", fn);
  if (!aligned16(q_idx) || !aligned16(w) || !aligned16(key_pages))
    return set_error(LSA_ERR_INVALID, "%s: q_idx, w and key_pages must be 16-byte aligned", fn);
  if (topk_hist && !aligned16(topk_hist))
    return set_error(LSA_ERR_INVALID, "%s: topk_hist must be 16-byte aligned", fn);
  size_t avail;
  char* base = align_ws(ws, ws_bytes, &avail);
  const size_t need = fp8_index_ws_bytes(n_rows);
  if (avail < need) return set_error(LSA_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need + kAlign);
  Fp8IndexArgs a;
  a.rows = paged_rows(n_rows, n_seq, seq_of_row, pos, block_table, max_pages, n_pages, max_len);
  a.q_idx = q_idx;
  a.w = w;
  a.key_pages = static_cast<const uint8_t*>(key_pages);
  a.n_init = c->index_init_tokens;
  a.n_loc = c->index_local_tokens;
  a.topk = c->index_topk;
  a.scores = scores;
  a.ld = ld;
  a.hist = topk_hist;
  a.top_pos = nullptr;
  a.ws = base;
  return cuda_status(launch_fp8_index(a, (cudaStream_t)stream), fn);
}

lsa_status lsa_fp8_sparse_mla(const lsa_config* c, int32_t n_sub, int32_t n_rows, int32_t n_seq,
                              const int32_t* seq_of_row, const int32_t* pos, const lsa_bf16* const* q_abs,
                              const void* const* latent_pages, int32_t n_pages, const int32_t* block_table,
                              int32_t max_pages, const int32_t* idx, const int32_t* count, int64_t max_len,
                              lsa_bf16* const* out, float* const* lse, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "lsa_fp8_sparse_mla";
  lsa_status s = check_cfg(c, fn);
  if (s != LSA_OK) return s;
  if (n_sub < 1 || n_sub > c->cli_factor)
    return set_error(LSA_ERR_INVALID, "%s: n_sub must be in 1..cli_factor", fn);
  s = check_rows(fn, n_rows, n_seq, seq_of_row, n_pages, max_pages, max_len);
  if (s != LSA_OK) return s;
  if (n_rows == 0) return LSA_OK;
  if (!pos || !block_table || (idx && !count)) return set_error(LSA_ERR_INVALID, "%s: NULL array argument", fn);
  s = check_subs(fn, n_sub, q_abs, latent_pages, out);
  if (s != LSA_OK) return s;
  Fp8MlaArgs a = {};
  a.rows = paged_rows(n_rows, n_seq, seq_of_row, pos, block_table, max_pages, n_pages, max_len);
  for (int z = 0; z < n_sub; ++z) {
    a.q[z] = q_abs[z];
    a.lat[z] = static_cast<const uint8_t*>(latent_pages[z]);
    a.out[z] = out[z];
    a.lse[z] = lse ? lse[z] : nullptr;
  }
  a.idx = idx;
  a.count = count;
  a.n_sub = n_sub;
  a.topk = c->index_topk;
  a.scale = c->softmax_scale;
  a.ws = align_ws(ws, ws_bytes, &a.ws_bytes);
  return cuda_status(launch_fp8_mla(a, (cudaStream_t)stream), fn);
}

lsa_status lsa_fp8_forward(const lsa_config* c, int32_t n_rows, int32_t n_seq, const int32_t* seq_of_row,
                           const int32_t* pos, int64_t max_len, const lsa_bf16* q_idx, const float* w,
                           const void* key_pages, const lsa_bf16* const* q_abs, const void* const* latent_pages,
                           int32_t n_pages, const int32_t* block_table, int32_t max_pages, lsa_bf16* const* out,
                           float* const* lse, int32_t* idx_out, int32_t* count_out, void* ws, size_t ws_bytes,
                           void* stream) {
  const char* fn = "lsa_fp8_forward";
  lsa_status s = check_cfg(c, fn);
  if (s != LSA_OK) return s;
  s = check_rows(fn, n_rows, n_seq, seq_of_row, n_pages, max_pages, max_len);
  if (s != LSA_OK) return s;
  if ((idx_out == nullptr) != (count_out == nullptr))
    return set_error(LSA_ERR_INVALID, "%s: idx_out and count_out go together", fn);
  if (n_rows == 0) return LSA_OK;
  const int cli = c->cli_factor;
  if (!pos || !block_table) return set_error(LSA_ERR_INVALID, "%s: NULL array argument", fn);
  s = check_subs(fn, cli, q_abs, latent_pages, out);
  if (s != LSA_OK) return s;
  if (max_len <= c->index_topk)  // no index pass: every row is dense
    return lsa_fp8_sparse_mla(c, cli, n_rows, n_seq, seq_of_row, pos, q_abs, latent_pages, n_pages, block_table,
                              max_pages, nullptr, nullptr, max_len, out, lse, ws, ws_bytes, stream);
  if (!q_idx || !w || !key_pages) return set_error(LSA_ERR_INVALID, "%s: NULL indexer argument", fn);
  if (!aligned16(q_idx) || !aligned16(w) || !aligned16(key_pages))
    return set_error(LSA_ERR_INVALID, "%s: q_idx, w and key_pages must be 16-byte aligned", fn);
  size_t avail;
  char* base = align_ws(ws, ws_bytes, &avail);
  int R = prefill_block_rows(n_rows, max_len);
  while (R > 1 && forward_plan(c, R, max_len).total > avail) R = R > 64 ? R / 64 * 32 : R / 2;
  const ForwardPlan p = forward_plan(c, R, max_len);
  if (p.total > avail)
    return set_error(LSA_ERR_WORKSPACE, "%s: workspace %zu below the minimum %zu", fn, ws_bytes, p.total + kAlign);
  const cudaStream_t st = (cudaStream_t)stream;
  for (int r0 = 0; r0 < n_rows; r0 += R) {
    const int nr = std::min(R, n_rows - r0);
    // without seq_of_row, row r0 + i is sequence r0 + i: the table's rows shift along
    PagedRows rows = paged_rows(nr, seq_of_row ? n_seq : n_seq - r0, seq_of_row ? seq_of_row + r0 : nullptr, pos + r0,
                                seq_of_row ? block_table : block_table + (int64_t)r0 * max_pages, max_pages, n_pages,
                                max_len);
    Fp8IndexArgs a;
    a.rows = rows;
    a.q_idx = q_idx + (int64_t)r0 * kHi * kDi;
    a.w = w + (int64_t)r0 * kHi;
    a.key_pages = static_cast<const uint8_t*>(key_pages);
    a.n_init = c->index_init_tokens;
    a.n_loc = c->index_local_tokens;
    a.topk = c->index_topk;
    a.scores = reinterpret_cast<float*>(base + p.scores);
    a.ld = max_len;
    // The streaming indexer builds the top-k's histogram from the scores in registers;
    // rows short enough that the top-k holds all their scores gain nothing from it.
    const bool hist = fp8_index_streams(nr, rows.n_seq, max_len) &&
                      max_len - c->index_init_tokens - c->index_local_tokens > kTopkShortMid;
    a.hist = hist ? reinterpret_cast<uint32_t*>(base + p.hist) : nullptr;
    a.top_pos = reinterpret_cast<int32_t*>(base + p.pos);  // a padding row selects nothing, whatever its position says
    a.ws = base + p.index;
    s = cuda_status(launch_fp8_index(a, st), fn);
    if (s != LSA_OK) return s;
    int32_t* idx = idx_out ? idx_out + (int64_t)r0 * c->index_topk : reinterpret_cast<int32_t*>(base + p.idx);
    int32_t* count = count_out ? count_out + r0 : reinterpret_cast<int32_t*>(base + p.count);
    s = run_topk(c, nr, a.top_pos, max_len, a.scores, max_len, idx, count, base + p.topk, p.topk_bytes, st,
                 a.hist);
    if (s != LSA_OK) return s;
    Fp8MlaArgs m = {};
    m.rows = rows;
    for (int z = 0; z < cli; ++z) {
      m.q[z] = q_abs[z] + (int64_t)r0 * kH * kDLat;
      m.lat[z] = static_cast<const uint8_t*>(latent_pages[z]);
      m.out[z] = out[z] + (int64_t)r0 * kH * kDV;
      m.lse[z] = lse && lse[z] ? lse[z] + (int64_t)r0 * kH : nullptr;
    }
    m.idx = idx;
    m.count = count;
    m.n_sub = cli;
    m.topk = c->index_topk;
    m.scale = c->softmax_scale;
    m.ws = base + p.mla;
    m.ws_bytes = p.mla_bytes;
    s = cuda_status(launch_fp8_mla(m, st), fn);
    if (s != LSA_OK) return s;
  }
  return LSA_OK;
}

}  // extern "C"
