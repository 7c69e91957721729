// Host-side pieces shared by the C-ABI's translation units (argument checks,
// workspace carving and the top-k step). Not part of the C-ABI.
#pragma once

#include "kernels.h"

namespace lsa {

constexpr size_t kAlign = 256;  // alignment of the regions carved from a workspace
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// LSA_OK, or LSA_ERR_CUDA with the CUDA error's message recorded.
lsa_status cuda_status(cudaError_t e, const char* fn);
// The top-k's workspace for these rows (max_len 0: the base layout only).
size_t topk_ws(int n_rows, int64_t max_len = 0);
// Rows of one block of scores (the scores of a block stay within a fixed budget).
int prefill_block_rows(int n_rows, int64_t max_len);
// The flat top-k over a score block, with its workspace carved from ws.
lsa_status run_topk(const lsa_config* c, int n_rows, const int32_t* pos, int64_t max_len, const float* scores,
                    int64_t ld, int32_t* idx, int32_t* count, void* ws, size_t ws_bytes, cudaStream_t st,
                    uint32_t* hist_ext = nullptr);

}  // namespace lsa
