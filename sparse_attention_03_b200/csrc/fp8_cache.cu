// Paged 8-bit caches: the page plan (block tables and slot maps from request
// lengths) and the quantising append.
#include "common.cuh"
#include "fp8.cuh"
#include "launch.h"

namespace lsa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr uint32_t kSat = 0x7fffffffu;  // sums saturate here (associative for non-negative terms)

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }

// Exclusive block-wide prefix sum (saturating) of one value per thread.
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x = sat_add(x, y);
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t s = warp_sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s = sat_add(s, y);
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  uint32_t before = __shfl_up_sync(0xffffffffu, x, 1);
  if (lane == 0) before = 0;
  if (warp > 0) before = sat_add(before, warp_sums[warp - 1]);
  __syncthreads();
  return before;
}

// The request that owns item i: the last s with pref[s] <= i (pref is exclusive,
// n + 1 entries, i < pref[n]); requests without items are passed over.
__device__ __forceinline__ int owner(const uint32_t* pref, int n, uint32_t i) {
  int lo = 0, hi = n;  // pref[lo] <= i < pref[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Every CTA forms the prefix sums of rows and pages over all requests in shared
// memory (8 bytes a request, at most 128 KB read per CTA, from L2), then the CTAs
// share the rows and the pages: item i finds its request by bisection. One
// launch; nothing is exchanged between CTAs. Bound by latency: 64 requests of a
// token each 4.0 us, 254317 rows of 1000 requests 6.
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(PagePlanArgs a) {
  extern __shared__ uint32_t sh[];
  __shared__ uint32_t warp_sums[32];
  uint32_t* rows = sh;                  // [n_seq + 1]
  uint32_t* pages = sh + a.n_seq + 1;   // [n_seq + 1]
  pdl_wait();
  const bool report = blockIdx.x == 0;
  // A table may be wider than the largest pool: what is beyond has no page, and positions stay in 32 bits.
  const int64_t room = min64(a.max_pages, kMaxPages) * kPage;
  for (int s = threadIdx.x; s < a.n_seq; s += kPlanThreads) {
    const int64_t c = a.cached[s], f = a.fresh[s];
    uint32_t nr = 0, np = 0;
    if (c < 0 || f < 0 || c + f > room) {
      if (report) flag_error(a.err, LSA_DEVERR_POS);
    } else {
      nr = (uint32_t)f;
      np = (uint32_t)((c + f + kPage - 1) / kPage - (c + kPage - 1) / kPage);
    }
    rows[s] = nr;
    pages[s] = np;
  }
  __syncthreads();
  const int per = (a.n_seq + kPlanThreads - 1) / kPlanThreads;
  const int s0 = min((int)threadIdx.x * per, a.n_seq), s1 = min(s0 + per, a.n_seq);
  uint32_t tr = 0, tp = 0;
  for (int s = s0; s < s1; ++s) {
    tr = sat_add(tr, rows[s]);
    tp = sat_add(tp, pages[s]);
  }
  uint32_t br = block_prefix(tr, warp_sums), bp = block_prefix(tp, warp_sums);
  for (int s = s0; s < s1; ++s) {
    const uint32_t nr = rows[s], np = pages[s];
    rows[s] = br;
    pages[s] = bp;
    br = sat_add(br, nr);
    bp = sat_add(bp, np);
  }
  if (s1 == a.n_seq && s0 < s1) {
    rows[a.n_seq] = br;
    pages[a.n_seq] = bp;
  }
  __syncthreads();
  const uint32_t n_rows = rows[a.n_seq], n_pages = pages[a.n_seq];
  if (report && threadIdx.x == 0) {
    a.totals[0] = (int)n_rows;
    a.totals[1] = (int)n_pages;
    if (n_rows > (uint32_t)a.n_rows) flag_error(a.err, LSA_DEVERR_COUNT);
    if (n_pages > (uint32_t)a.n_free) flag_error(a.err, LSA_DEVERR_PAGE);
  }
  // A page taken from the free list: -1 when there is none left or its number is out of range.
  auto take = [&](uint32_t i) {
    const int p = i < (uint32_t)a.n_free ? a.free_pages[i] : -1;
    if (i < (uint32_t)a.n_free && !page_ok(p, kMaxPages)) flag_error(a.err, LSA_DEVERR_PAGE);
    return page_ok(p, kMaxPages) ? p : -1;
  };
  const int64_t stride = (int64_t)gridDim.x * kPlanThreads, first = (int64_t)blockIdx.x * kPlanThreads + threadIdx.x;
  for (int64_t i = first; i < n_pages; i += stride) {
    const int s = owner(pages, a.n_seq, (uint32_t)i);
    const int col = (a.cached[s] + kPage - 1) / kPage + (int)((uint32_t)i - pages[s]);
    a.block_table[(int64_t)s * a.max_pages + col] = take((uint32_t)i);
  }
  for (int64_t i = first; i < a.n_rows; i += stride) {
    int s = -1, p = -1, slot = -1;
    if (i < n_rows) {
      s = owner(rows, a.n_seq, (uint32_t)i);
      const int c = a.cached[s], col0 = (c + kPage - 1) / kPage;
      p = c + (int)((uint32_t)i - rows[s]);
      const int col = p / kPage;
      int page;
      if (col < col0) {  // the request's last page had room
        page = a.block_table[(int64_t)s * a.max_pages + col];
        if (!page_ok(page, kMaxPages)) {
          flag_error(a.err, LSA_DEVERR_PAGE);
          page = -1;
        }
      } else {
        page = take(pages[s] + (uint32_t)(col - col0));
      }
      if (page >= 0) slot = page * kPage + p % kPage;
    }
    a.seq_of_row[i] = s;
    a.pos[i] = p;
    a.slot[i] = slot;
  }
}

// A warp quantises four vectors of N bf16 at once: their 4 N / 8 chunks of 16
// bytes go round the lanes (288 chunks of a latent: nine full loads a lane, all in
// flight; one row a warp leaves the third of three loads three quarters idle).
// Largest magnitudes on the bit patterns, then a multiply and a conversion per
// element. Bound by the latency of a warp's one chain, slot -> loads -> maxima ->
// stores (top stall: long scoreboard; DRAM 31 %, ALU 55 %, issue 0.55): a warp loads
// nothing under its own stores. 16384 rows (2 sub-blocks and the key, 63 MB, which
// stay in L2 from call to call) 15.8 us, 4.0 TB/s; one row a warp took 25. 64 rows:
// 4.3 us, a launch.
constexpr int kRowsPerWarp = 4;

template <int N>
struct Quant4 {
  static constexpr int kRowChunks = N / 8, kLoads = kRowsPerWarp * kRowChunks / 32;
  static_assert(kRowsPerWarp * kRowChunks % 32 == 0, "whole loads");
  uint4 v[kLoads];
  int e[kRowsPerWarp];       // scale exponents
  uint32_t m[kRowsPerWarp];  // largest magnitudes (bf16 bits)

  // rows: bit r set where row r is there
  __device__ __forceinline__ void load(const uint16_t* __restrict__ src, int64_t ld, uint32_t rows, int lane) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = lane + 32 * i, r = c / kRowChunks;
      v[i] = rows >> r & 1 ? __ldg(reinterpret_cast<const uint4*>(src + r * ld) + (c - r * kRowChunks)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) m[r] = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t x = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(0, v[i].x), v[i].y), v[i].z), v[i].w);
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r)
        if (r >= 32 * i / kRowChunks && r <= (32 * i + 31) / kRowChunks)  // the rows that this load touches
          m[r] = __vmaxu2(m[r], (lane + 32 * i) / kRowChunks == r ? x : 0);
    }
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
      m[r] = fold_max(m[r]);
      e[r] = bf16_finite(m[r]) ? scale_exponent(m[r]) : 0;
    }
  }
  // The row's scale (NaN for one with an infinity or NaN, whose codes are zeros).
  __device__ __forceinline__ float scale(int r) const { return bf16_finite(m[r]) ? pow2i(e[r]) : __uint_as_float(0x7fc00000u); }
  template <typename F>
  __device__ __forceinline__ void store(uint32_t rows, int lane, F row_codes) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = lane + 32 * i, r = c / kRowChunks;
      int er = 0;
      bool fin = true;
#pragma unroll
      for (int k = 0; k < kRowsPerWarp; ++k)
        if (k >= 32 * i / kRowChunks && k <= (32 * i + 31) / kRowChunks && k == r) {
          er = e[k];
          fin = bf16_finite(m[k]);
        }
      if (rows >> r & 1)
        *reinterpret_cast<uint2*>(row_codes(r) + 8 * (c - r * kRowChunks)) = fin ? quant8(v[i], pow2i(-er)) : make_uint2(0, 0);
    }
  }
};

constexpr int kAppendWarps = 4;

// Grid y: the arrays of the call (latent sub-blocks, index keys); four rows a warp.
__global__ void __launch_bounds__(kAppendWarps * 32) fp8_append_kernel(Fp8AppendArgs a) {
  pdl_wait();
  const int lane = threadIdx.x & 31, y = blockIdx.y;
  const int64_t r0 = ((int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5)) * kRowsPerWarp;
  if (r0 >= a.n_rows || !a.src[y]) return;
  int slot = -1;  // lane r < 4: row r0 + r's
  if (lane < kRowsPerWarp && r0 + lane < a.n_rows) {
    slot = a.slot[r0 + lane];
    if (slot < -1 || slot >= (int64_t)a.n_pages * kPage) {
      flag_error(a.err, LSA_DEVERR_PAGE);
      slot = -1;
    }
  }
  const uint32_t rows = __ballot_sync(0xffffffffu, slot >= 0);
  if (rows == 0) return;
  int at[kRowsPerWarp];
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) at[r] = __shfl_sync(0xffffffffu, slot, r);
  auto slot_of = [&](int r) { return r == 0 ? at[0] : r == 1 ? at[1] : r == 2 ? at[2] : at[3]; };
  if (y < 2) {
    Quant4<kDLat> q;
    q.load(a.src[y] + r0 * a.ld[y], a.ld[y], rows, lane);
    auto row = [&](int r) { return a.dst[y] + (int64_t)slot_of(r) * kLatRow; };
    q.store(rows, lane, row);
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r)
      if (lane == r && (rows >> r & 1))
        *reinterpret_cast<uint4*>(row(r) + kDLat) = make_uint4(__float_as_uint(q.scale(r)), q.m[r] == 0 ? 1u : 0u, 0, 0);
  } else {
    Quant4<kDi> q;
    q.load(a.src[2] + r0 * a.ld[2], a.ld[2], rows, lane);
    auto page = [&](int r) { return a.dst[2] + (int64_t)(slot_of(r) / kPage) * kKeyPage; };
    q.store(rows, lane, [&](int r) { return page(r) + (slot_of(r) % kPage) * kDi; });
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r)
      if (lane == r && (rows >> r & 1))
        *reinterpret_cast<float*>(page(r) + kPage * kDi + 4 * (slot_of(r) % kPage)) = q.scale(r);
  }
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanArgs& a, cudaStream_t st) {
  const size_t smem = 2 * ((size_t)a.n_seq + 1) * sizeof(uint32_t);
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               2 * (LSA_PLAN_MAX_SEQ + 1) * (int)sizeof(uint32_t));
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  // one item per thread up to a wave of the SMs, then strided
  const int64_t ctas = (max64(a.n_rows, a.n_seq) + kPlanThreads - 1) / kPlanThreads;
  const cudaError_t e = launch_pdl(page_plan_kernel, dim3((unsigned)max64(1, min64(ctas, 148))), dim3(kPlanThreads),
                                   smem, st, a);
  count_launches(1);
  return e;
}

cudaError_t launch_fp8_append(const Fp8AppendArgs& a, cudaStream_t st) {
  constexpr int kRowsPerCta = kAppendWarps * kRowsPerWarp;
  const unsigned nx = (unsigned)(((int64_t)a.n_rows + kRowsPerCta - 1) / kRowsPerCta);
  const cudaError_t e = launch_pdl(fp8_append_kernel, dim3(nx, 3), dim3(kAppendWarps * 32), 0, st, a);
  count_launches(1);
  return e;
}

}  // namespace lsa
