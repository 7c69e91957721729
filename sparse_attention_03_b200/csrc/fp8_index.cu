// Lightning indexer over paged 8-bit keys.
//
//   score[r, j] = sk[j] * sum_h (w[r,h] * sq[r,h]) * max(0, q8[r,h] . k8[j])
//
// (scales are positive, so they leave the ReLU; a scale that is NaN counts as a
// product of zero, as max(0, NaN) does in the bf16 indexer). Products of e4m3
// codes on tcgen05 kind::f8f6f4 with fp32 accumulators: keys as M = 128, heads
// as N, K = 128 in four instructions. Legacy mma.sync runs e4m3 at less than its
// bf16 rate here (224 against 351 TFLOP/s, measured) and would hold the
// streaming form at half of the memory rate.
//
// Two kernels. A row of its own (decode) is bound by the key stream: 132 bytes a
// key against 180 of ~730 cycles a 128-key tile for the products (16 x 128K keys:
// 49 us, 5.8 TB/s; 64 x 16K to 32K: 38 us; one row x 8K: 5 us, latency). Rows that
// share their keys (a prompt's chunk) are bound by the tensor cores and the
// ReLU-weighted sum over them: 16 rows at a time, N = 128 (4 rows x 32 heads). The
// host takes the form that costs less (use_blocks).
//
// A tile is two pages of 64 keys, each one TMA copy of 8 KB (the 128-byte
// swizzle) and one bulk copy of its 64 scales into a ring of their own (the
// epilogue reads them after the tile's stage is free again).
#include "fp8.cuh"
#include "launch.h"
#include "tc.cuh"

namespace lsa {
namespace {

constexpr int kTile = 128;
constexpr uint32_t kTileBytes = kTile * kDi;  // 16 KB
constexpr int kScaleRing = 16;                // tiles: more than the stages and accumulators between producer and epilogue

// The scales of a tile's keys, and which of its two pages are there.
struct __align__(16) TileScales {  // bulk copies land on 16-byte boundaries
  float s[kTile];
  int ok[2];
};
static_assert(sizeof(TileScales) % 16 == 0 && (kPage * 4) % 16 == 0 && (kPage * kDi) % 16 == 0 && kKeyPage % 16 == 0,
              "bulk copies: addresses and sizes in 16 bytes");

// One tile's copies, issued by one thread: the pages' codes into `dst` on `full`
// and their scales into `sc` on `sfull`. page < 0: not in the pool, or past the
// keys that are visible; nothing is copied for it and what is in its place is
// never used.
__device__ __forceinline__ void load_tile(const CUtensorMap* map, const uint8_t* key_pages, int page0, int page1,
                                          uint8_t* dst, TileScales* sc, uint64_t* full, uint64_t* sfull) {
  const int n = (page0 >= 0) + (page1 >= 0);
  sc->ok[0] = page0 >= 0;
  sc->ok[1] = page1 >= 0;
  mbar_expect_tx(full, n * kPage * kDi);
  mbar_expect_tx(sfull, n * kPage * 4);
  if (page0 >= 0) {
    tma_load_3d(dst, map, 0, 0, page0, full);
    bulk_load(sc->s, key_pages + (int64_t)page0 * kKeyPage + kPage * kDi, kPage * 4, sfull);
  }
  if (page1 >= 0) {
    tma_load_3d(dst + kPage * kDi, map, 0, 0, page1, full);
    bulk_load(sc->s + kPage, key_pages + (int64_t)page1 * kKeyPage + kPage * kDi, kPage * 4, sfull);
  }
}

// A batch of pages looked up by the producer warp, a lane each: pages first ..
// first + 31 of the sequence (-1: past the visible keys, or outside the pool).
__device__ __forceinline__ int lookup_pages(const PagedRows& rows, int seq, int64_t nvis, int64_t first, int lane) {
  const int64_t p = first + lane;
  if (p * kPage >= nvis) return -1;
  const int page = rows.block_table[(int64_t)seq * rows.max_pages + p];
  if (page_ok(page, rows.n_pages)) return page;
  flag_error(rows.err, LSA_DEVERR_PAGE);
  return -1;
}

__device__ __forceinline__ float score_value(float s, float sk) { return sk == sk ? s * sk : 0.f; }

// s += w * (x0, x1), two fp32 in one register pair; and the sum of two such pairs.
__device__ __forceinline__ void fma_pair(unsigned long long& s, unsigned long long w, float x0, float x1) {
  asm("{\n .reg .b64 x;\n mov.b64 x, {%2, %3};\n fma.rn.f32x2 %0, %1, x, %0;\n}\n" : "+l"(s) : "l"(w), "f"(x0), "f"(x1));
}
__device__ __forceinline__ float sum_pairs(unsigned long long a, unsigned long long b) {
  float x, y;
  asm("{\n .reg .b64 t;\n add.rn.f32x2 t, %2, %3;\n mov.b64 {%0, %1}, t;\n}\n" : "=f"(x), "=f"(y) : "l"(a), "l"(b));
  return x + y;
}

// One row's 32 weights for ReLU-weighted sums: volatile, so that they are asked for
// where this stands, while a tcgen05.ld is under way.
__device__ __forceinline__ void load_weights(ulonglong2 (&w)[8], const float* row) {
  const uint32_t p = smem_u32(row);
#pragma unroll
  for (int i = 0; i < 8; ++i) asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];\n" : "=l"(w[i].x), "=l"(w[i].y) : "r"(p + i * 16));
}

// The row's sum of w max(0, x), two heads an instruction (packed fp32 pairs).
__device__ __forceinline__ float weighted_sum(const uint32_t (&v)[32], const ulonglong2 (&w)[8]) {
  unsigned long long s0 = 0, s1 = 0;
#pragma unroll
  for (int h = 0; h < 32; h += 4) {
    fma_pair(s0, w[h / 4].x, fmaxf(__uint_as_float(v[h]), 0.f), fmaxf(__uint_as_float(v[h + 1]), 0.f));
    fma_pair(s1, w[h / 4].y, fmaxf(__uint_as_float(v[h + 2]), 0.f), fmaxf(__uint_as_float(v[h + 3]), 0.f));
  }
  return sum_pairs(s0, s1);
}

// Quantises one head's 128 query elements over a half warp (8 elements a lane,
// sub = lane & 15): the codes and the scale (NaN vectors: zeros and 0).
__device__ __forceinline__ uint2 quant_head(uint4 v, float& scale) {
  uint32_t m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(0, v.x), v.y), v.z), v.w);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
  m = max(m & 0xffffu, m >> 16);
  const bool fin = bf16_finite(m);
  const int e = fin ? scale_exponent(m) : 0;
  scale = fin ? pow2i(e) : 0.f;
  return fin ? quant8(v, pow2i(-e)) : make_uint2(0, 0);
}

// ---------------------------------------------------------------- rows of their own

constexpr int kStages = 5;      // 80 KB of keys in flight a CTA, two CTAs an SM
constexpr int kAcc = 4;         // accumulators of 32 columns
constexpr int kDecThreads = 10 * 32;

struct RowInfo {
  int row, seq;
  int t0, t1;    // its tiles [t0, t1) of this CTA (row -1: no more)
  int64_t nvis;
};

struct __align__(1024) DecodeSmem {
  uint8_t a[kStages][kTileBytes];
  uint8_t q[2][kHi * kDi];
  TileScales sc[kScaleRing];
  float w[2][kHi];
  RowInfo info[4];
  unsigned long long sums[kDecThreads];
  unsigned long long total;
  int start_row, start_tile;
  uint64_t full[kStages], empty[kStages], sfull[kScaleRing], tfull[kAcc], tempty[kAcc], qfull[2], qempty[2], rfull[4],
      rempty[4];
  uint32_t tmem_base;
  int abort_flag;
  uint32_t hist[2048];
};

__device__ __forceinline__ int64_t row_tiles(const PagedRows& rows, int r) {
  return (paged_geom(rows, r, false).nvis + kTile - 1) / kTile;
}

// The four epilogue warps' barrier with an OR.
__device__ __forceinline__ bool epilogue_any(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %1, 0;\n bar.red.or.pred p, 1, 128, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// At exit after a wait that gave up: none of this CTA's copies may be in flight
// into its shared memory. The last tiles' barriers, each with a limit of its own.
template <int STAGES>
__device__ __forceinline__ void drain_copies(uint64_t* full, uint64_t* sfull, uint32_t issued) {
  const long long t0 = global_ns();
  for (uint32_t i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
    while (!mbar_try_wait(&full[i % STAGES], (i / STAGES) & 1) ||
           (sfull && !mbar_try_wait(&sfull[i % kScaleRing], (i / kScaleRing) & 1)))
      if (global_ns() - t0 > kWaitLimitNs) return;
}

// Persistent: every CTA sums the rows' tiles and takes an equal share of them
// (tiles of consecutive rows). Warps: producer, MMA, four for the epilogue (a
// thread = a key), four for the rows' queries.
template <bool HIST>
__global__ void __launch_bounds__(kDecThreads, 2)
    fp8_index_rows_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ Fp8IndexArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) flag_error(a.rows.err, LSA_DEVERR_TIMEOUT);
    return;
  }
  DecodeSmem& sm = *reinterpret_cast<DecodeSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < kScaleRing; ++i) mbar_init(&sm.sfull[i], 1);
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(&sm.tfull[i], 1);
      mbar_init(&sm.tempty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.qfull[i], 4);
      mbar_init(&sm.qempty[i], 1 + 4);  // its products (a commit) and the epilogue's warps
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.rfull[i], 1);
      mbar_init(&sm.rempty[i], 4 + 1 + 4);
    }
    sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::);
  }
  if (warp == 1) tmem_alloc(&sm.tmem_base, kAcc * kHi);
  if (HIST)
    for (int i = tid; i < 2048; i += kDecThreads) sm.hist[i] = 0;
  pdl_wait();

  // This CTA's share of all rows' tiles.
  const int n_rows = a.rows.n_rows, per = (n_rows + kDecThreads - 1) / kDecThreads;
  const int r0 = min(tid * per, n_rows), r1 = min(r0 + per, n_rows);
  unsigned long long mine = 0;
  for (int r = r0; r < r1; ++r) {
    const int64_t nvis = paged_geom(a.rows, r, blockIdx.x == 0).nvis;
    if (a.top_pos && blockIdx.x == 0) a.top_pos[r] = (int)(nvis - 1);
    mine += (unsigned long long)((nvis + kTile - 1) / kTile);
  }
  sm.sums[tid] = mine;
  __syncthreads();
  if (warp == 0) {  // exclusive prefix over the 320 threads, ten a lane
    unsigned long long s = 0;
    for (int i = 0; i < 10; ++i) s += sm.sums[lane * 10 + i];
    unsigned long long x = s;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) sm.total = x;
    x -= s;
    for (int i = 0; i < 10; ++i) {
      const unsigned long long v = sm.sums[lane * 10 + i];
      sm.sums[lane * 10 + i] = x;
      x += v;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const unsigned long long total = sm.total;
  const unsigned long long first = total * blockIdx.x / gridDim.x, last = total * (blockIdx.x + 1) / gridDim.x;
  const unsigned long long before = sm.sums[tid];
  if (first < last && first >= before && first < before + mine) {
    unsigned long long at = before;
    for (int r = r0; r < r1; ++r) {
      const unsigned long long n = (unsigned long long)row_tiles(a.rows, r);
      if (first < at + n) {
        sm.start_row = r;
        sm.start_tile = (int)(first - at);
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;
  const bool work = first < last;

  if (work && warp == 0) {
    // ---------------- producer (and the rows' order, for the other roles) ----------------
    unsigned long long left = last - first;
    int t0 = sm.start_tile;
    uint32_t g = 0, k = 0;
    bool ok = true;
    for (int r = sm.start_row; ok; ++r) {
      RowInfo in = {-1, 0, 0, 0, 0};
      if (left > 0 && r < n_rows) {
        const PagedGeom geo = paged_geom(a.rows, r, false);
        in.row = r;
        in.seq = geo.seq;
        in.nvis = geo.nvis;
        in.t0 = t0;
        in.t1 = (int)((geo.nvis + kTile - 1) / kTile);
        if ((unsigned long long)(in.t1 - in.t0) > left) in.t1 = in.t0 + (int)left;
        t0 = 0;
        if (in.t0 >= in.t1) continue;  // a row without keys
      }
      ok = k < 4 || mbar_wait_fast(&sm.rempty[k & 3], ((k >> 2) - 1) & 1, abort_flag);
      if (!ok) break;
      __syncwarp();
      if (lane == 0) {
        sm.info[k & 3] = in;
        mbar_arrive(&sm.rfull[k & 3]);
      }
      __syncwarp();
      ++k;
      if (in.row < 0) break;
      left -= in.t1 - in.t0;
      int pages = 0;
      for (int t = in.t0; t < in.t1; ++t, ++g) {
        const int in_batch = (t - in.t0) & 15;
        if (in_batch == 0) pages = lookup_pages(a.rows, in.seq, in.nvis, 2 * (int64_t)t, lane);
        const int p0 = __shfl_sync(0xffffffffu, pages, 2 * in_batch), p1 = __shfl_sync(0xffffffffu, pages, 2 * in_batch + 1);
        const int s = g % kStages;
        if (g >= kStages && !mbar_wait_fast(&sm.empty[s], ((g / kStages) - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        __syncwarp();
        if (lane == 0)
          load_tile(&map, a.key_pages, p0, p1, sm.a[s], &sm.sc[g % kScaleRing], &sm.full[s], &sm.sfull[g % kScaleRing]);
        __syncwarp();
      }
    }
    if (*abort_flag) drain_copies<kStages>(sm.full, sm.sfull, g);
  } else if (work && warp == 1) {
    // ---------------- MMA ----------------
    const uint32_t leader = elect_one();
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      if (!mbar_wait_fast(&sm.rfull[k & 3], (k >> 2) & 1, abort_flag)) break;
      const int n = sm.info[k & 3].row < 0 ? 0 : sm.info[k & 3].t1 - sm.info[k & 3].t0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.rempty[k & 3]);
      if (n == 0 || !mbar_wait_fast(&sm.qfull[k & 1], (k >> 1) & 1, abort_flag)) break;
      const uint64_t bd = sw128_desc(smem_u32(sm.q[k & 1]));
      for (int i = 0; i < n; ++i, ++g) {
        const int s = g % kStages, acc = g % kAcc;
        if (!mbar_wait_fast(&sm.full[s], (g / kStages) & 1, abort_flag) ||
            (g >= kAcc && !mbar_wait_fast(&sm.tempty[acc], ((g / kAcc) - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        const uint64_t ad = sw128_desc(smem_u32(sm.a[s]));
#pragma unroll
        for (int c = 0; c < kDi / 32; ++c)
          umma_f8(tmem + acc * kHi, ad + (c * 32 >> 4), bd + (c * 32 >> 4), f8_idesc(kHi, false), c > 0 ? 1u : 0u, leader);
        if (leader) {
          umma_commit(&sm.tfull[acc]);
          umma_commit(&sm.empty[s]);
          if (i + 1 == n) umma_commit(&sm.qempty[k & 1]);
        }
        __syncwarp();
      }
    }
  } else if (work && warp < 6) {
    // ---------------- epilogue ----------------
    const int quarter = warp & 3;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    uint32_t g = 0;
    bool ok = true;  // after a wait that gave up the loops run on without storing
    for (uint32_t k = 0;; ++k) {
      ok = ok && mbar_wait_fast(&sm.rfull[k & 3], (k >> 2) & 1, abort_flag);
      if (epilogue_any(!ok)) break;  // all four warps or none: they meet at the histogram
      const RowInfo in = sm.info[k & 3];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.rempty[k & 3]);
      if (in.row < 0) break;
      ok = mbar_wait_fast(&sm.qfull[k & 1], (k >> 1) & 1, abort_flag);
      float w[kHi];
#pragma unroll
      for (int h = 0; h < kHi; ++h) w[h] = sm.w[k & 1][h];
      const bool hist_row = HIST && in.nvis > a.topk;
      float* __restrict__ out = a.scores + (int64_t)in.row * a.ld;
      for (int t = in.t0; t < in.t1; ++t, ++g) {
        const int acc = g % kAcc, sr = g % kScaleRing;
        ok = ok && mbar_wait_fast(&sm.sfull[sr], (g / kScaleRing) & 1, abort_flag);
        const float sk = sm.sc[sr].s[quarter * 32 + lane];
        const bool there = sm.sc[sr].ok[quarter >> 1] != 0;
        ok = ok && mbar_wait_fast(&sm.tfull[acc], (g / kAcc) & 1, abort_flag);
        __syncwarp();
        tc_fence_after();
        float v[kHi];
        tmem_ld32(tmem + lanes + acc * kHi, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.tempty[acc]);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int h = 0; h < kHi; h += 2) {
          s0 = fmaf(w[h], fmaxf(v[h], 0.f), s0);
          s1 = fmaf(w[h + 1], fmaxf(v[h + 1], 0.f), s1);
        }
        const int64_t j = (int64_t)t * kTile + quarter * 32 + lane;
        if (ok && j < in.nvis) {
          const bool forced = j < a.n_init || j >= in.nvis - a.n_loc;
          const float x = there ? score_value(s0 + s1, sk) : -INFINITY;
          out[j] = forced ? INFINITY : x;
          if (HIST && hist_row && !forced) atomicAdd(&sm.hist[score_key(x) >> 21], 1u);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.qempty[k & 1]);
      if (HIST) {  // the row's share of its histogram
        asm volatile("bar.sync 1, 128;\n" ::: "memory");
        if (hist_row) {
          uint32_t* hr = a.hist + (int64_t)in.row * kTopkHistStride;
          for (int i = (warp - 2) * 32 + lane; i < 2048; i += 128)
            if (sm.hist[i]) {
              atomicAdd(&hr[i], sm.hist[i]);
              sm.hist[i] = 0;
            }
        }
        asm volatile("bar.sync 1, 128;\n" ::: "memory");
      }
    }
  } else if (work) {
    // ---------------- queries (warps 6..9: heads 8 (warp - 6) ..) ----------------
    const int h0 = (warp - 6) * 8 + (lane >> 4), sub = lane & 15;
    for (uint32_t k = 0;; ++k) {
      if (!mbar_wait_fast(&sm.rfull[k & 3], (k >> 2) & 1, abort_flag)) break;
      const int r = sm.info[k & 3].row;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.rempty[k & 3]);
      if (r < 0) break;
      uint4 v[4];
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = h0 + 2 * i;
        v[i] = __ldg(reinterpret_cast<const uint4*>(a.q_idx + ((int64_t)r * kHi + h) * kDi) + sub);
        w[i] = __ldg(a.w + (int64_t)r * kHi + h);
      }
      if (k >= 2 && !mbar_wait_fast(&sm.qempty[k & 1], ((k >> 1) - 1) & 1, abort_flag)) break;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = h0 + 2 * i;
        float scale;
        const uint2 c = quant_head(v[i], scale);
        *reinterpret_cast<uint2*>(sm.q[k & 1] + h * kDi + (((sub >> 1) ^ (h & 7)) << 4) + (sub & 1) * 8) = c;
        if (sub == 0) sm.w[k & 1][h] = scale == 0.f ? 0.f : w[i] * scale;
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.qfull[k & 1]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm.abort_flag) flag_error(a.rows.err, LSA_DEVERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kAcc * kHi);
  }
}

// ---------------------------------------------------------------- rows that share keys

constexpr int kRows = 16;                     // rows of a block
constexpr int kBStages = 6;
constexpr int kEpiWarps = 16;
constexpr int kGroups = 4;                    // accumulators of 128 columns: 4 rows x 32 heads, four warps each
static_assert(kRows / kEpiWarps == 1, "a warp sums four rows of a quarter of the keys");
constexpr int kProducer = kEpiWarps, kMma = kEpiWarps + 1;  // their warps (the products': two)
constexpr int kBlkWarps = kEpiWarps + 3, kBlkThreads = kBlkWarps * 32;
constexpr uint32_t kGroupBytes = 128 * kDi;   // 4 rows x 32 heads x 128 codes: 16 KB

struct __align__(1024) BlockSmem {
  uint8_t b[kGroups][kGroupBytes];
  uint8_t a[kBStages][kTileBytes];
  TileScales sc[kScaleRing];
  __align__(16) float w[kRows][kHi];
  int64_t nvis[kRows];
  int seq[kRows];
  // runs of rows of one sequence: its rows [run_r0, run_r1) of the block, its tiles, the cost of one
  int run_r0[kRows], run_r1[kRows], run_tiles[kRows], run_cost[kRows], n_runs;
  long long sums[kBlkWarps], start_at;
  int start_block;
  uint64_t full[kBStages], empty[kBStages], tfull[kGroups], tempty[kGroups], qfull;
  uint32_t tmem_base;
  int abort_flag;
};

// The tiles that a block of rows takes: the runs of rows of one sequence, each up to
// its furthest visible key. A tile costs its load and the groups of four rows that
// the run has a part in. seq[i], nvis[i]: row i's sequence (-1: none) and keys.
template <typename F>
__device__ __forceinline__ void block_runs(const int* seq, const int64_t* nvis, F&& run) {
  for (int i = 0; i < kRows;) {
    int e = i + 1;
    int64_t most = nvis[i];
    for (; e < kRows && seq[e] == seq[i]; ++e) most = max64(most, nvis[e]);
    if (seq[i] >= 0 && most > 0) run(i, e, (int)((most + kTile - 1) / kTile), 2 + (e - 1) / 4 - i / 4);
    i = e;
  }
}

// The codes and weights of all rows' queries, a half warp a head, and the cost of
// every block's tiles (a CTA has the 16 heads of half a row: every 32nd takes a block).
__global__ void __launch_bounds__(256) fp8_index_query_kernel(const __grid_constant__ Fp8IndexArgs a, uint8_t* codes,
                                                              float* wq, int* block_cost) {
  pdl_wait();
  const int64_t head = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4;
  const int sub = threadIdx.x & 15;
  const bool live = head < (int64_t)a.rows.n_rows * kHi;
  const uint4 v = live ? __ldg(reinterpret_cast<const uint4*>(a.q_idx + head * kDi) + sub) : make_uint4(0, 0, 0, 0);
  if (blockIdx.x % (2 * kRows) == 0 && threadIdx.x < 32) {
    __shared__ int seq[kRows];
    __shared__ int64_t nvis[kRows];
    const int block = blockIdx.x / (2 * kRows), r = block * kRows + threadIdx.x;
    if (threadIdx.x < kRows) {
      PagedGeom g = {-1, true, 0};
      if (r < a.rows.n_rows) g = paged_geom(a.rows, r, true);
      seq[threadIdx.x] = g.seq;
      nvis[threadIdx.x] = g.nvis;
      if (a.top_pos && r < a.rows.n_rows) a.top_pos[r] = (int)(g.nvis - 1);
    }
    __syncwarp();
    if (threadIdx.x == 0) {
      int n = 0;
      block_runs(seq, nvis, [&](int, int, int tiles, int cost) { n += tiles * cost; });
      block_cost[block] = n;
    }
    __syncwarp();
  }
  float scale;
  const uint2 c = quant_head(v, scale);
  if (!live) return;
  *reinterpret_cast<uint2*>(codes + head * kDi + sub * 8) = c;
  if (sub == 0) wq[head] = scale == 0.f ? 0.f : a.w[head] * scale;
}

// Walks the CTA's tiles [t0, t1) of the block's runs, one after the other.
struct RunCursor {
  int run, tile;
  __device__ __forceinline__ void start(const BlockSmem& sm, int t) {
    run = 0;
    tile = t;
    while (run < sm.n_runs && tile >= sm.run_tiles[run]) tile -= sm.run_tiles[run++];
  }
  __device__ __forceinline__ void next(const BlockSmem& sm) {
    ++tile;
    while (run < sm.n_runs && tile >= sm.run_tiles[run]) {
      tile = 0;
      ++run;
    }
  }
};

// How many of the block's tiles begin before cost x (from the block's begin).
__device__ __forceinline__ int tiles_before(const BlockSmem& sm, long long x) {
  int n = 0;
  for (int r = 0; r < sm.n_runs && x > 0; ++r) {
    const int cost = sm.run_cost[r], all = sm.run_tiles[r] * cost;
    n += x >= all ? sm.run_tiles[r] : ((int)x + cost - 1) / cost;
    x -= all;
  }
  return n;
}

// Persistent: the tiles of all blocks of 16 rows (the furthest rows' block first)
// make one list, of which every CTA takes an equal share (by cost), block after
// block. Warps: sixteen for the epilogue, TMA producer, two for the products (with
// one, the issue and its waits held them: 302 us). A tile's products are four
// accumulators of 4 rows x 32 heads, each with its own four epilogue warps (a thread
// = a key), so a group's sums wait for nobody else's. Rows of several sequences (a
// block that straddles prompts, or has a few rows of each) take their sequences'
// tiles one after the other, with the groups that have a row of the sequence.
//
// 4096 rows x 16K keys: 280 us back to back, 1.72 PFLOP/s (318 as single calls). Two
// things hold it. Without the sums and the stores it takes 197 us, twice the
// products' own 1030 cycles a tile: an accumulator has no second buffer and is given
// back only after four rounds of load, wait and sum, so the tensor cores wait for it
// (the pipe is active 40 %). And the sums (a maximum a product, an FMA for two, eight
// loads of weights a row and key quarter: ~70 instructions, 16 rows a scheduler and
// tile) need 1150 issue cycles a tile, 64 % of the slots. Accumulators of 256
// columns took 301 us, eight epilogue warps 365, x + |x| for half of the maxima 291.
__global__ void __launch_bounds__(kBlkThreads, 1)
    fp8_index_block_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ Fp8IndexArgs a, const float* wq, const int* block_cost) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) flag_error(a.rows.err, LSA_DEVERR_TIMEOUT);
    return;
  }
  BlockSmem& sm = *reinterpret_cast<BlockSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_blocks = (a.rows.n_rows + kRows - 1) / kRows;
  if (tid == 0) {
    for (int s = 0; s < kBStages; ++s) {
      mbar_init(&sm.full[s], 2);  // load_tile's two announcements
      mbar_init(&sm.empty[s], 2);  // both MMA warps
    }
    for (int b = 0; b < kGroups; ++b) {
      mbar_init(&sm.tfull[b], 2);  // the products' commit, and the MMA warp's own arrival
      mbar_init(&sm.tempty[b], kEpiWarps / kGroups);
    }
    mbar_init(&sm.qfull, 1);
    sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::);
  }
  if (warp == kMma) tmem_alloc(&sm.tmem_base, 512);
  pdl_wait();
  // This CTA's share [lo, hi) of the list: block n_blocks - 1 first. A thread sums
  // `per` consecutive blocks, a warp its threads, and the thread in whose part lo
  // lies walks it.
  const int per = (n_blocks + kBlkThreads - 1) / kBlkThreads;
  const int b0 = min(tid * per, n_blocks), b1 = min(b0 + per, n_blocks);  // places in the list
  long long part = 0;
  for (int b = b0; b < b1; ++b) part += block_cost[n_blocks - 1 - b];
  long long before = part;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, before, off);
    if (lane >= off) before += o;
  }
  if (lane == 31) sm.sums[warp] = before;
  before -= part;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long total = 0;
  for (int i = 0; i < kBlkWarps; ++i) {
    if (i == warp) before += total;
    total += sm.sums[i];
  }
  const long long lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
  if (lo < hi && before <= lo && lo < before + part) {
    int b = b0;
    long long at = before;
    for (; lo >= at + block_cost[n_blocks - 1 - b]; ++b) at += block_cost[n_blocks - 1 - b];
    sm.start_at = at;
    sm.start_block = n_blocks - 1 - b;
  }
  __syncthreads();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;
  int block = sm.start_block;
  uint32_t g = 0;       // tiles of the CTA before this block's
  uint32_t turns = 0;   // parity of the warp's uses of an accumulator (an MMA warp: a bit for each of two)
  if (lo >= hi) block = -1;

  uint32_t seg = 0;
  for (long long at = sm.start_at; block >= 0 && at < hi; at += block_cost[block--]) {
    if (block_cost[block] == 0) continue;  // padding
    const int row0 = block * kRows;
    if (tid < kRows) {
      PagedGeom geom = {-1, true, 0};
      if (row0 + tid < a.rows.n_rows) geom = paged_geom(a.rows, row0 + tid, false);
      sm.seq[tid] = geom.seq;
      sm.nvis[tid] = geom.nvis;
    }
    for (int i = tid; i < kRows * kHi; i += kBlkThreads)
      sm.w[i / kHi][i % kHi] = row0 + i / kHi < a.rows.n_rows ? wq[(int64_t)row0 * kHi + i] : 0.f;
    if (warp == 0) {
      __syncwarp();
      if (lane == 0) {
        int n = 0;
        block_runs(sm.seq, sm.nvis, [&](int r0, int r1, int tiles, int cost) {
          sm.run_r0[n] = r0;
          sm.run_r1[n] = r1;
          sm.run_cost[n] = cost;
          sm.run_tiles[n++] = tiles;
        });
        sm.n_runs = n;
      }
    }
    __syncthreads();
    const int first_tile = tiles_before(sm, lo - at), n_tiles = tiles_before(sm, hi - at) - first_tile;
    if (n_tiles == 0) {  // none begins in this share
      __syncthreads();
      continue;
    }
    RunCursor cur;
    cur.start(sm, first_tile);
    if (warp == kProducer) {
      // ---------------- producer ----------------
      if (lane == 0) {  // the last block's products have been read: the queries' place is free
        mbar_expect_tx(&sm.qfull, kGroups * kGroupBytes);
        for (int q = 0; q < kGroups; ++q) tma_load_2d(sm.b[q], &map_q, 0, row0 * kHi + q * 128, &sm.qfull);
      }
      __syncwarp();
      int pages = 0, batch_run = -1, batch = 0;
      int64_t most = 0;
      uint32_t i = g;
      for (; i < g + n_tiles; ++i, cur.next(sm)) {
        if (cur.run != batch_run || cur.tile - batch >= 16) {
          if (cur.run != batch_run) {
            most = 0;
            for (int r = sm.run_r0[cur.run]; r < sm.run_r1[cur.run]; ++r) most = max64(most, sm.nvis[r]);
          }
          batch_run = cur.run;
          batch = cur.tile;
          pages = lookup_pages(a.rows, sm.seq[sm.run_r0[cur.run]], most, 2 * (int64_t)batch, lane);
        }
        const int in_batch = cur.tile - batch;
        const int p0 = __shfl_sync(0xffffffffu, pages, 2 * in_batch), p1 = __shfl_sync(0xffffffffu, pages, 2 * in_batch + 1);
        const int s = i % kBStages;
        if (i >= kBStages && !mbar_wait_fast(&sm.empty[s], ((i / kBStages) - 1) & 1, abort_flag)) break;
        __syncwarp();
        if (lane == 0)
          load_tile(&map, a.key_pages, p0, p1, sm.a[s], &sm.sc[i % kScaleRing], &sm.full[s], &sm.full[s]);
        __syncwarp();
      }
      if (*abort_flag) {
        drain_copies<kBStages>(sm.full, nullptr, i);
        const long long t_out = global_ns();
        while (!mbar_try_wait(&sm.qfull, seg & 1) && global_ns() - t_out < kWaitLimitNs) {
        }
      }
    } else if (warp >= kMma) {
      // ---------------- MMA ----------------
      const uint32_t leader = elect_one();
      bool ok = mbar_wait_fast(&sm.qfull, seg & 1, abort_flag);
      const int q_first = (warp - kMma) * 2;  // its accumulators: this and the next
      // The accumulator's last use, if any, has been read.
      auto released = [&](int k) { return mbar_wait_fast(&sm.tempty[q_first + k], (turns >> k & 1) ^ 1, abort_flag); };
      const uint64_t bd = sw128_desc(smem_u32(sm.b[q_first]));
      int run = -1;
      bool live[2] = {false, false};  // which of the two have rows of the run
      for (uint32_t i = g; ok && i < g + n_tiles; ++i, cur.next(sm)) {
        if (cur.run != run) {
          // Both have been read, and with them the last run's scales (one without rows in
          // this run holds nothing up from here on).
          ok = released(0) && released(1);
          if (!ok) break;
          run = cur.run;
#pragma unroll
          for (int k = 0; k < 2; ++k) live[k] = sm.run_r0[run] / 4 <= q_first + k && q_first + k <= (sm.run_r1[run] - 1) / 4;
        }
        const int s = i % kBStages;
        if (!mbar_wait_fast(&sm.full[s], (i / kBStages) & 1, abort_flag)) break;
        const uint64_t ad = sw128_desc(smem_u32(sm.a[s]));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (!live[k]) continue;
          if (!released(k)) {
            ok = false;
            break;
          }
          __syncwarp();
          tc_fence_after();
          const int q = q_first + k;
#pragma unroll
          for (int c = 0; c < kDi / 32; ++c)
            umma_f8(tmem + q * 128, ad + (c * 32 >> 4), bd + ((k * kGroupBytes + c * 32) >> 4), f8_idesc(128, false),
                    c > 0 ? 1u : 0u, leader);
          if (leader) {
            umma_commit(&sm.tfull[q]);
            mbar_arrive(&sm.tfull[q]);
          }
          turns ^= 1u << k;
          __syncwarp();
        }
        if (!ok) break;
        if (leader) {
          if (live[0] || live[1]) umma_commit(&sm.empty[s]);
          else mbar_arrive(&sm.empty[s]);
        }
        __syncwarp();
      }
    } else {
      // ---------------- epilogue ----------------
      const int quarter = warp & 3, group = warp >> 2, row_in = (warp >> 2) * 4;  // its four rows
      const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + row_in * 32;
      const int lane_j = quarter * 32 + lane;
      const float(*wrow)[kHi] = sm.w + row_in;
      float* o = nullptr;
      // Of a run: its tiles to come, the warp's rows in it, and the tiles [plain_lo,
      // plain_hi) whose keys are visible to all of the four and forced for none.
      int tiles_left = 0, mine = 0, plain_lo = 0, plain_hi = 0;
      for (uint32_t i = g; i < g + n_tiles; ++i) {
        if (tiles_left == 0) {
          const int r0 = sm.run_r0[cur.run], r1 = sm.run_r1[cur.run];
          tiles_left = sm.run_tiles[cur.run] - cur.tile;
          mine = 0;
          int64_t most = INT64_MAX;
          for (int u = 0; u < 4; ++u) {
            if (row_in + u >= r0 && row_in + u < r1) {
              mine |= 1 << u;
              most = min64(most, sm.nvis[row_in + u] - a.n_loc);
            }
          }
          if (mine == 0) {  // no work in this run: on to the next
            i += tiles_left - 1;
            tiles_left = 0;
            cur.tile = sm.run_tiles[cur.run] - 1;
            cur.next(sm);
            continue;
          }
          plain_lo = (a.n_init + kTile - 1) / kTile;
          plain_hi = mine == 15 ? (int)(max64(most, 0) / kTile) : 0;
          o = a.scores + (int64_t)(row0 + row_in) * a.ld + (int64_t)cur.tile * kTile + lane_j;
        }
        // What the MMA warp saw (the tile's scales in place) holds here too: it arrives on tfull as its commit does.
        if (!mbar_wait_fast(&sm.tfull[group], turns & 1, abort_flag)) break;
        turns ^= 1;
        __syncwarp();
        tc_fence_after();
        // A row at a time, its weights on the way with its products.
        uint32_t v[32];
        ulonglong2 w[8];
        tmem_ld32_request(at, v);
        load_weights(w, wrow[0]);
        const TileScales& sc = sm.sc[i % kScaleRing];
        const bool there = sc.ok[quarter >> 1] != 0;
        const float sk = score_value(1.f, sc.s[lane_j]);
        const bool plain = there && cur.tile >= plain_lo && cur.tile < plain_hi;
        auto put = [&](int u, float x) {
          if (plain) {
            o[u * a.ld] = x;
          } else if (mine >> u & 1) {
            const int64_t j = (int64_t)cur.tile * kTile + lane_j, n = sm.nvis[row_in + u];
            if (j < n) o[u * a.ld] = j < a.n_init || j >= n - a.n_loc ? INFINITY : there ? x : -INFINITY;
          }
        };
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          tmem_ld32_wait(v);
          if (u == 3) {  // the accumulator's last row is in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.tempty[group]);
          }
          const float x = weighted_sum(v, w) * sk;
          if (u < 3) {
            tmem_ld32_request(at + (u + 1) * 32, v);
            load_weights(w, wrow[u + 1]);
          }
          put(u, x);
        }
        ++cur.tile;
        o += kTile;
        if (--tiles_left == 0) {
          --cur.tile;
          cur.next(sm);
        }
      }
    }
    __syncwarp();
    __syncthreads();
    if (*abort_flag) break;
    ++seg;
    g += n_tiles;
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm.abort_flag) flag_error(a.rows.err, LSA_DEVERR_TIMEOUT);
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The most runs of rows of one sequence that the blocks can have.
int64_t most_runs(int64_t n_rows, int64_t n_seq) { return (n_rows + kRows - 1) / kRows + min64(n_seq, n_rows) - 1; }

// The form that these rows take, by what the two cost here (ns; measured over 1 to
// 1024 rows, 1 to 64 sequences, 1K to 128K keys), the rows taken to be spread evenly
// over the sequences: the streaming form 5 us and 1.75 for each row and tile of its
// keys, the block form 13 us and, for each tile of a run of rows, 3.5 and 1.3 for each
// of its groups of four. Streaming against blocks (us): 64 rows of one sequence x
// 128K 115, 48; 8 rows x 128K 19, 18; 64 rows x 2K 8, 16; 64 sequences x 32K of 2 rows
// each 93, 110; of 4 rows 180, 98; of 8 rows 328, 115.
bool use_blocks(int64_t n_rows, int64_t n_seq, int64_t max_len) {
  const int64_t tiles = (max_len + kTile - 1) / kTile, seqs = max64(1, min64(n_seq, n_rows));
  const int64_t each = (n_rows + seqs - 1) / seqs, runs = seqs * ((each + kRows - 1) / kRows), groups = seqs * ((each + 3) / 4);
  return 20 * 8000 + (70 * runs + 26 * groups) * tiles < 35 * n_rows * tiles;
}

template <typename K>
cudaError_t set_smem(K kernel, int bytes, bool (&done)[64]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || done[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

// Key pages: 64 rows of 128 codes, pages kKeyPage bytes apart; a box is one page.
bool page_map(CUtensorMap* m, const void* base, int n_pages) {
  const auto fn = tensor_map_encode();
  if (!fn) return false;
  const cuuint64_t dims[3] = {kDi, kPage, (cuuint64_t)n_pages};
  const cuuint64_t strides[2] = {kDi, kKeyPage};
  const cuuint32_t box[3] = {kDi, kPage, 1}, step[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Query codes: n rows of 128, a box is 128 of them.
bool query_map(CUtensorMap* m, const void* base, int64_t n) {
  const auto fn = tensor_map_encode();
  if (!fn) return false;
  const cuuint64_t dims[2] = {kDi, (cuuint64_t)n};
  const cuuint64_t strides[1] = {kDi};
  const cuuint32_t box[2] = {kDi, 128}, step[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_rows(const Fp8IndexArgs& a, const CUtensorMap& map, cudaStream_t st) {
  static bool done[2][64];
  const int64_t most = (int64_t)a.rows.n_rows * ((a.rows.max_len + kTile - 1) / kTile);
  const dim3 grid((unsigned)max64(1, min64(most, 2LL * sm_count())));
  const int smem = (int)sizeof(DecodeSmem);
  cudaError_t e;
  if (a.hist) {
    e = launch_zero_words(a.hist, (size_t)a.rows.n_rows * kTopkHistStride, st);
    if (e == cudaSuccess) e = set_smem(fp8_index_rows_kernel<true>, smem, done[0]);
    if (e == cudaSuccess) e = launch_pdl(fp8_index_rows_kernel<true>, grid, dim3(kDecThreads), smem, st, map, a);
  } else {
    e = set_smem(fp8_index_rows_kernel<false>, smem, done[1]);
    if (e == cudaSuccess) e = launch_pdl(fp8_index_rows_kernel<false>, grid, dim3(kDecThreads), smem, st, map, a);
  }
  count_launches(1);
  return e;
}

cudaError_t launch_blocks(Fp8IndexArgs a, const CUtensorMap& map, cudaStream_t st) {
  static bool done[64];
  const int n_rows = a.rows.n_rows;
  uint8_t* codes = static_cast<uint8_t*>(a.ws);
  float* wq = reinterpret_cast<float*>(codes + (size_t)n_rows * kHi * kDi);
  int* block_cost = reinterpret_cast<int*>(wq + (size_t)n_rows * kHi);
  // the histograms count what a row sees, which its position alone does not say
  if (a.hist && !a.top_pos) a.top_pos = block_cost + (n_rows + kRows - 1) / kRows;
  CUtensorMap map_q;
  if (!query_map(&map_q, codes, (int64_t)n_rows * kHi)) return cudaErrorInvalidValue;
  cudaError_t e = launch_pdl(fp8_index_query_kernel, dim3((unsigned)(((int64_t)n_rows * kHi * 16 + 255) / 256)), dim3(256), 0,
                             st, a, codes, wq, block_cost);
  count_launches(1);
  if (e != cudaSuccess) return e;
  e = set_smem(fp8_index_block_kernel, (int)sizeof(BlockSmem), done);
  if (e != cudaSuccess) return e;
  // A CTA's start costs about four tiles: a share is no smaller.
  const int64_t tiles = most_runs(n_rows, a.rows.n_seq) * ((a.rows.max_len + kTile - 1) / kTile);
  const unsigned ctas = (unsigned)max64(1, min64(sm_count(), tiles / 4));
  e = launch_pdl(fp8_index_block_kernel, dim3(ctas), dim3(kBlkThreads), sizeof(BlockSmem), st, map, map_q, a,
                 (const float*)wq, (const int*)block_cost);
  count_launches(1);
  if (e != cudaSuccess) return e;
  if (!a.hist) return cudaSuccess;
  // The epilogue has no room for histograms: one pass over the fresh scores builds them.
  e = launch_zero_words(a.hist, (size_t)n_rows * kTopkHistStride, st);
  if (e != cudaSuccess) return e;
  TopkArgs t;
  t.scores = a.scores;
  t.ld = a.ld;
  t.pos = a.top_pos;
  t.n_rows = n_rows;
  t.max_len = a.rows.max_len;
  t.topk = a.topk;
  t.n_init = a.n_init;
  t.n_loc = a.n_loc;
  t.idx = nullptr;
  t.count = nullptr;
  t.ws = nullptr;
  t.ws_bytes = 0;
  return launch_topk_hist_only(t, a.hist, st);
}

}  // namespace

// the block form's quantised queries, costs and last visible keys; asked for whichever form the rows take
size_t fp8_index_ws_bytes(int n_rows) {
  return (size_t)n_rows * (kHi * (kDi + sizeof(float)) + sizeof(int)) + (size_t)((n_rows + kRows - 1) / kRows) * sizeof(int);
}

bool fp8_index_streams(int n_rows, int n_seq, int64_t max_len) { return !use_blocks(n_rows, n_seq, max_len); }

cudaError_t launch_fp8_index(const Fp8IndexArgs& a, cudaStream_t st) {
  CUtensorMap map;
  if (!page_map(&map, a.key_pages, a.rows.n_pages)) return cudaErrorInvalidValue;
  return use_blocks(a.rows.n_rows, a.rows.n_seq, a.rows.max_len) ? launch_blocks(a, map, st) : launch_rows(a, map, st);
}

}  // namespace lsa
