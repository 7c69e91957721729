// Internal launchers of the paged 8-bit cache operators (host side; the C entry
// points are in fp8_api.cu). Not part of the C-ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kernels.h"

namespace lsa {

constexpr int kPage = LSA_PAGE_TOKENS;             // tokens of a page
constexpr int kLatRow = LSA_FP8_LATENT_ROW;        // bytes of a latent row: 576 codes, scale, padding
constexpr int kKeyPage = LSA_FP8_KEY_PAGE;         // bytes of a key page: 64 x 128 codes, 64 scales
constexpr int kMaxPages = (1 << 25) - 1;           // pages of a pool: every slot fits an int32

struct PagePlanArgs {
  const int32_t *cached, *fresh, *free_pages;
  int32_t *block_table, *seq_of_row, *pos, *slot, *totals;
  int n_seq, n_free, max_pages, n_rows;
  int* err;
};
cudaError_t launch_page_plan(const PagePlanArgs& a, cudaStream_t st);

struct Fp8AppendArgs {
  const uint16_t* src[3];   // latent sub-blocks, then the index keys (null: absent)
  uint8_t* dst[3];
  int64_t ld[3];            // elements between source rows
  const int32_t* slot;
  int n_rows, n_pages;
  int* err;
};
cudaError_t launch_fp8_append(const Fp8AppendArgs& a, cudaStream_t st);

// Rows and pages, as every reader of the paged caches gets them.
struct PagedRows {
  const int32_t* seq_of_row;  // null: row r is sequence r
  const int32_t* pos;
  const int32_t* block_table;
  int n_rows, n_seq, max_pages, n_pages;
  int64_t max_len;
  int* err;
};

struct Fp8IndexArgs {
  PagedRows rows;
  const uint16_t* q_idx;
  const float* w;
  const uint8_t* key_pages;
  int n_init, n_loc, topk;
  float* scores;
  int64_t ld;
  uint32_t* hist;  // top-k histograms (zeroed by the launcher), or null
  int32_t* top_pos;  // or null: gets the rows' last visible key for the top-k, -1 for a row without keys
  void* ws;        // fp8_index_ws_bytes, 256-byte aligned
};
size_t fp8_index_ws_bytes(int n_rows);
// Whether these rows take the streaming form, which builds histograms on the way.
bool fp8_index_streams(int n_rows, int n_seq, int64_t max_len);
cudaError_t launch_fp8_index(const Fp8IndexArgs& a, cudaStream_t st);

struct Fp8MlaArgs {
  PagedRows rows;
  const uint16_t* q[kMaxSub];
  const uint8_t* lat[kMaxSub];
  uint16_t* out[kMaxSub];
  float* lse[kMaxSub];
  const int32_t *idx, *count;
  int n_sub, topk;
  float scale;
  void* ws;
  size_t ws_bytes;
};
size_t fp8_mla_ws_bytes(int n_rows, int n_sub, int64_t max_list);
cudaError_t launch_fp8_mla(const Fp8MlaArgs& a, cudaStream_t st);

// The three operations of lsa_workspace_size that belong to the paged caches.
size_t fp8_workspace_size(const lsa_config* c, int op, int n_rows, int n_seq, int64_t max_len);

}  // namespace lsa
