// Sparse absorbed-latent MLA over paged 8-bit latent rows.
//
//   x_i = scale * s_i * (q . c_i),   out = sum_i softmax(x)_i s_i c_i[:512]
//
// for the keys of a row's list, c_i the e4m3 codes and s_i the power-of-two scale
// of the key's 592-byte cache row.
//
// Mathematics. The codes go to the tensor cores as they lie in the cache
// (tcgen05 kind::f8f6f4, fp32 accumulators): a key's scale is a factor of its
// logit and of its softmax weight, so no code is ever converted or rescaled.
// The other operand is carried by two e4m3 numbers, value = hi + lo / k, which
// stand side by side in the N dimension (32 heads hi, 32 heads lo; N = 64 runs
// at the rate of N = 32, 48 against 45 cycles an instruction, both held by the
// 4 KB A operand):
//   - the query, scaled by a power of two to at most 448, k = 16: bf16 has 8
//     significant bits, two e4m3 of 4 bits hold them exactly down to 2^-22 of the
//     row's largest element;
//   - the weight u = p * s_i * 2^(2 - A), at most 128, k = 64: 8 significant
//     bits, the precision of a bf16 weight, in steps of at least 2^-15 (2^-16 of
//     the largest u of its frame: what is below is lost).
// The frame A of each head follows the running maximum of log2(p s). It is kept as
// its distance from m, the largest logit where it was set: an integer, so that the
// heaviest key's u is a power of two (a row of one key comes out exact), no lower
// than -124, and changed with m also where no key of a tile adds to O. It is set
// from the first tile, raised when a u would pass 128, and set anew every 16 tiles
// (also downwards, to 2^-60 of the highest: O is then scaled up, fp32 has the
// range), so that the loss stays relative to the 2048 keys around a key however long
// the list is. The sum of the softmax is kept apart, in fp32, of the unrounded
// weights, in its own frame m (a key's scale, which is no part of its weight, cannot
// disturb it). Where a |m| passes 2^10 logits are rounded to fp32 before m is taken
// from them, and the frame is set in two steps, m first.
//
// What the weights' steps cost: a key whose weight lies 2^-14 or more below the
// largest keeps 3 bits or fewer. On rows of 2048 keys that a sink dominates (0.9 and
// 0.99 of the weight) the output's error is that of its own bf16 rounding (1.7e-3);
// relative to the other keys' part alone 0.144 where the rounding of the output
// makes 0.137, and 1.86 where it makes 1.87. Steps finer by 1, 2 or 3 bits, at the
// cost of the room to 128, take 3, 9 or 16 % more time (more frames set).
//
// Layout. One tile is 128 keys: S^T [128 keys x 64] = C Q^T (K = 576: 18
// instructions), then O^T [512 dims x 64] += C^T P (4 x 4 instructions of 128
// dims and 32 keys). Both read the same 80 KB of shared memory: a key is 128
// bytes in each of five chunks with the 128-byte swizzle, which is K-major for S
// (rows = keys) and MN-major for O (rows = the contraction). Tensor memory: S
// twice 64 columns, O 4 x 64.
//
// Roles (16 warps, one CTA per SM, persistent over (row, sub-block, split)
// items): 8 softmax warps (a thread = a key of the tile and 16 heads; between
// items the next query's codes), 7 gather warps (16-byte cp.async into the
// swizzled layout, a ring of two tiles that is refilled chunk by chunk; the first
// four also write an item's O when its last product is complete), and one MMA warp
// that issues what is ready, so that the softmax of a tile runs under the
// products of its neighbours. Every wait is bounded.
//
// What bounds it. A tile's chain (copies ~2700 cycles, S ~1400, softmax ~1400, O
// ~1200) over the ring of two; the products alone are 1650 (34 instructions at 48
// cycles, held by the 6 KB of shared memory that each reads). Measured: 2048 rows of
// 2048 keys, 2 sub-blocks: 1.02 ms, 572 TFLOP/s, ~4300 cycles a tile (the bf16
// kernel's rate for these products: ~2.4 ms); 130 rows of 1855 keys, one sub-block:
// 46 us; 16 rows of 2048, 2 sub-blocks: 25 us and one row 14 us, of which 10 to 12
// are the chain of one item (lookup, query, the first frame, output) and the join of
// the splits.
#include "fp8.cuh"
#include "launch.h"
#include "tc.cuh"

namespace lsa {
namespace {

constexpr int kTile = 128;
constexpr int kChunks = 5;                       // 128-byte chunks of a key (the fifth: rope, scale)
constexpr uint32_t kChunkBytes = kTile * 128;    // 16 KB
constexpr uint32_t kStageBytes = kChunks * kChunkBytes;
constexpr uint32_t kQChunkBytes = 64 * 128;
constexpr uint32_t kPBytes = kTile * 64;
constexpr int kSoftWarps = 8;                    // two groups of four: heads 0..15 and 16..31
constexpr int kGatherWarps = 7;                  // the first four also write O
constexpr int kMmaWarp = kSoftWarps + kGatherWarps;
constexpr int kThreads = (kMmaWarp + 1) * 32;    // 16 warps, 128 registers a thread
constexpr int kHG = kH / 2;                      // heads of a softmax group
constexpr int kFrameTiles = 16;                  // tiles after which the frame is set anew
constexpr int kMaxSplits = 32;
constexpr uint32_t kTmemO = 128;                 // S: columns 0..127, O: 128..383
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kUnset = -3.0e38f;               // no frame yet

struct __align__(1024) Fp8MlaSmem {
  uint8_t k[2][kStageBytes];
  uint8_t q[kChunks * kQChunkBytes];   // [chunk][32 hi rows, 32 lo rows][128 B]
  uint8_t p[2][kPBytes];               // [key][32 hi, 32 lo codes]
  float4 frame[kSoftWarps][kHG];       // per softmax warp, new frames: -m, 2^(2 - A + m), factors of L and O
  float2 tmax[kSoftWarps][kHG];        // each warp's maxima of a tile
  float lsum[kSoftWarps][kHG];
  uint32_t qmax[kSoftWarps];           // each softmax warp's largest magnitude of the query
  float2 fin[4][kH];                   // ring over items: 2^(A - m - 2), the sum of the softmax
  float fin_m[4][kH];
  // per stage and chunk: gathered; read by its products (chunk 4, which has none: s_empty)
  uint64_t full[2][kChunks], pv_done[2][4];
  uint64_t s_full[2], s_empty[2], p_full[2], q_full[4], fin_full[4], o_full, o_empty, drain;
  int item_tiles[4];                   // ring over items, of the MMA warp
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Fp8MlaSmem) <= 232448, "shared memory of one CTA");

struct Split {
  int n_split;
  int n_items;
};

// One (row, sub-block, split): its list and its tiles [t0, t1).
struct Item {
  int r, z, t0, t1;
  uint32_t n, nvis;  // list length, visible keys
  int seq;           // -1: no keys
  bool pad;          // a padding row: nothing of it is written
};

__device__ __forceinline__ int item_row(const Fp8MlaArgs& a, const Split& sp, int i) { return i / (sp.n_split * a.n_sub); }
__device__ __forceinline__ int item_sub(const Fp8MlaArgs& a, const Split& sp, int i) { return (i / sp.n_split) % a.n_sub; }

__device__ __forceinline__ Item load_item(const Fp8MlaArgs& a, const Split& sp, int i, bool report) {
  Item it = {0, 0, 0, 0, 0u, 0u, -1, true};
  if (i >= sp.n_items) return it;
  const int s = i % sp.n_split;
  it.z = item_sub(a, sp, i);
  it.r = item_row(a, sp, i);
  report = report && s == 0 && it.z == 0;
  const int32_t cnt = a.idx ? a.count[it.r] : 0;
  const PagedGeom g = paged_geom(a.rows, it.r, report);
  it.pad = g.pad;
  it.seq = g.seq;
  it.nvis = (uint32_t)g.nvis;
  it.n = it.nvis;
  if (g.seq < 0) return it;
  if (a.idx) {
    it.n = cnt;
    if (cnt < 0 || cnt > a.topk) {
      if (report) flag_error(a.rows.err, LSA_DEVERR_COUNT);
      it.n = cnt < 0 ? 0 : a.topk;
    }
  }
  const uint64_t tiles = ((uint64_t)it.n + kTile - 1) / kTile;
  it.t0 = (int)(tiles * s / sp.n_split);
  it.t1 = (int)(tiles * (s + 1) / sp.n_split);
  return it;
}

// The item's place among the partial outputs.
__device__ __forceinline__ int64_t item_base(const Fp8MlaArgs& a, const Split& sp, int i) {
  return ((int64_t)item_sub(a, sp, i) * a.rows.n_rows + item_row(a, sp, i)) * sp.n_split + i % sp.n_split;
}

// Lanes h and h + 16 get the maximum (or sum) over the warp of v[h]: a butterfly that halves the array.
template <bool MAX>
__device__ __forceinline__ float fold16(float (&v)[kHG], int lane) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = (lane & o) ? v[i] : v[i + o], keep = (lane & o) ? v[i + o] : v[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, o);
      v[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  const float got = __shfl_xor_sync(0xffffffffu, v[0], 16);
  return MAX ? fmaxf(v[0], got) : v[0] + got;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// 2^d for integer-valued d, 0 below the normal range.
__device__ __forceinline__ float pow2f(float d) { return d < -126.f ? 0.f : pow2i((int)fminf(fmaxf(d, -126.f), 126.f)); }

// A softmax group's barrier (1 or 2) with an OR over its threads.
__device__ __forceinline__ bool softmax_any(int group, bool v) {
  uint32_t r;
  __syncwarp();
  if (group == 0)
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 q, %1, 0;\n bar.red.or.pred p, 1, 128, q;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 q, %1, 0;\n bar.red.or.pred p, 2, 128, q;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
  return r != 0;
}

// The same for both groups.
__device__ __forceinline__ bool all_softmax_any(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %1, 0;\n bar.red.or.pred p, 3, 256, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// ---------------------------------------------------------------- query codes

// Softmax warp w quantises heads 4 w .. 4 w + 3 of an item's query, when the
// previous item's last S is complete (the warp has read it). All loads first.
constexpr int kQHeads = kH / kSoftWarps;

__device__ __forceinline__ const uint4* query_of(const Fp8MlaArgs& a, const Split& sp, int item, int warp) {
  return reinterpret_cast<const uint4*>(a.q[item_sub(a, sp, item)] + (int64_t)item_row(a, sp, item) * kH * kDLat) +
         warp * kQHeads * 72;
}
// Brings the warp's heads of a query to the L2 cache: 36 lines.
__device__ __forceinline__ void prefetch_q(const uint4* src, int lane) {
  asm volatile("prefetch.global.L2 [%0];\n" ::"l"(src + lane * 8));
  if (lane < 4) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(src + (32 + lane) * 8));
}

struct Query {
  uint4 v[kQHeads][3];  // of the warp's heads, 8 elements a lane and third
};
__device__ __forceinline__ void load_q(Query& q, const uint4* src, int lane) {
#pragma unroll
  for (int j = 0; j < kQHeads; ++j)
#pragma unroll
    for (int c = 0; c < 3; ++c)
      q.v[j][c] = lane + 32 * c < 72 ? __ldg(src + j * 72 + lane + 32 * c) : make_uint4(0, 0, 0, 0);
}

// Returns the factor of the codes' products: one power of two for all heads of
// the row (a logit's error counts absolutely) times the softmax's; NaN for a
// query with an infinity or NaN.
__device__ __forceinline__ float prepare_q(const Fp8MlaArgs& a, Fp8MlaSmem& sm, const Query& q, uint32_t nk, int warp,
                                           int lane) {
  const auto& v = q.v;
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kQHeads; ++j)
#pragma unroll
    for (int c = 0; c < 3; ++c)
      m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(m, v[j][c].x), v[j][c].y), v[j][c].z), v[j][c].w);
  m = fold_max(m);
  if (lane == 0) sm.qmax[warp] = m;
  all_softmax_any(false);
#pragma unroll
  for (int w = 0; w < kSoftWarps; ++w) m = max(m, sm.qmax[w]);
  const bool fin = bf16_finite(m);
  const int e = fin ? scale_exponent(m) : 0;
  const float inv = pow2i(-e);
#pragma unroll
  for (int j = 0; j < kQHeads; ++j) {
    const int h = warp * kQHeads + j;
#pragma unroll
    for (int c = 0; c < 3; ++c) {
      const int u = lane + 32 * c;  // eight elements
      const uint32_t w[4] = {v[j][c].x, v[j][c].y, v[j][c].z, v[j][c].w};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)  // 8 significant bits fit fp16; what is below 2^-24 of the largest goes
        split_e4m3<16>(fin ? f16x2_rn(bf16_lo(w[k]) * inv, bf16_hi(w[k]) * inv) : 0u, hi[k], lo[k]);
      const int chunk = u >> 4, unit = (u >> 1) & 7, half = (u & 1) * 8;
      uint8_t* base = sm.q + chunk * kQChunkBytes + h * 128 + ((unit ^ (h & 7)) << 4) + half;
      if (u < 72) {
        *reinterpret_cast<uint2*>(base) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2*>(base + 32 * 128) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      }
    }
  }
  fence_proxy_async();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm.q_full[nk & 3]);
  return fin ? pow2i(e) * (a.scale * kLog2e) : __uint_as_float(0x7fc00000u);
}

// ---------------------------------------------------------------- output

// An item whose tiles are all gathered: its last product is tile last_g of the CTA.
struct Done {
  int item;  // -1: none
  uint32_t nk, last_g;
};

// Writes an item's O once its last product is complete: warp w holds dims w * 32
// + lane of each 128 (the tensor-memory lanes it may read).
__device__ __forceinline__ bool write_out(const Fp8MlaArgs& a, const Split& sp, Fp8MlaSmem& sm, uint32_t tmem,
                                          const Done& done, int warp, int lane, float* part_o, float2* part_ml,
                                          volatile int* abort_flag) {
  if (!mbar_wait_fast(&sm.fin_full[done.nk & 3], (done.nk >> 2) & 1, abort_flag)) return false;
  if (!mbar_wait_fast(&sm.o_full, done.nk & 1, abort_flag)) return false;
  __syncwarp();
  tc_fence_after();
  const int z = item_sub(a, sp, done.item), r = item_row(a, sp, done.item);
  const int64_t base = item_base(a, sp, done.item);
  const uint32_t o_addr = tmem + ((uint32_t)(warp * 32) << 16) + kTmemO;
  const float2 fin = sm.fin[done.nk & 3][lane];  // lane h: head h's factor of O and sum
  const bool one = sp.n_split == 1;
  if (warp == 0) {
    const float m = sm.fin_m[done.nk & 3][lane];
    if (!one) part_ml[base * kH + lane] = make_float2(m, fin.y);
    else if (a.lse[z]) a.lse[z][(int64_t)r * kH + lane] = fin.y == 0.f ? -INFINITY : (m + log2f(fin.y)) * kLn2;
  }
  const float mine = fin.y == 0.f ? 0.f : fin.x / fin.y;  // a split's share too: its sum alone could leave fp32's range
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {  // 128 dims, 16 heads at a time (the gather's registers hold a tile)
    const int h0 = (c & 1) * 16;
    float o[16], lo[16];
    tmem_ld16_x2(o_addr + (c >> 1) * 64 + h0, o_addr + (c >> 1) * 64 + 32 + h0, o, lo);
    if (c == 7) {  // O is read: the next item may start its products
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_empty);
    }
#pragma unroll
    for (int h = 0; h < 16; ++h) o[h] = fmaf(lo[h], 0.015625f, o[h]) * __shfl_sync(0xffffffffu, mine, h0 + h);
    const int d = (c >> 1) * 128 + warp * 32 + lane;
    if (one) {
      // neighbouring lanes swap heads, so that each stores two dims of one head
      uint16_t* og = a.out[z] + ((int64_t)r * kH + h0 + (lane & 1)) * kDV + (d & ~1);
#pragma unroll
      for (int h = 0; h < 16; h += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? o[h] : o[h + 1], 1);
        *reinterpret_cast<uint32_t*>(og + h * kDV) = (lane & 1) ? bf16x2_rn(got, o[h + 1]) : bf16x2_rn(o[h], got);
      }
    } else {
      float* po = part_o + (base * kH + h0) * kDV + d;
#pragma unroll
      for (int h = 0; h < 16; ++h) po[h * kDV] = o[h];
    }
  }
  return true;
}

// ---------------------------------------------------------------- gather warps

// The tiles of a CTA's items, one after the other.
struct TileCursor {
  Item it;
  int i, t;  // item, tile in it
  __device__ __forceinline__ void start(const Fp8MlaArgs& a, const Split& sp, int item, bool report) {
    for (i = item; i < sp.n_items; i += gridDim.x) {
      it = load_item(a, sp, i, report);
      t = it.t0;
      if (it.t0 < it.t1) return;
    }
  }
  __device__ __forceinline__ void next(const Fp8MlaArgs& a, const Split& sp, bool report) {
    if (++t >= it.t1) start(a, sp, i + gridDim.x, report);
  }
};

// The arrival of this thread's copies so far (it happens when they have landed).
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}

// A warp takes groups of four keys (eight lanes a key, 16 bytes a lane and
// copy): groups warp, warp + 7, .. of the tile's 32. The chunks of a tile go one
// after the other, each into the place that the tile two before has left: the
// rope and scale chunk when its softmax has read the scales, a value chunk when
// its own products are complete. The lookups run ahead: the list entries of tile
// g + 2 and the pages of tile g + 1 are requested while tile g is copied.
__device__ __forceinline__ void gather_role(const Fp8MlaArgs& a, const Split& sp, Fp8MlaSmem& sm, uint32_t tmem,
                                            int warp, int lane, float* part_o, float2* part_ml,
                                            volatile int* abort_flag) {
  constexpr int kGroups = (kTile / 4 + kGatherWarps - 1) / kGatherWarps;
  const bool report = warp == 0 && lane == 0;
  const int unit = lane & 7;
  // lanes 0 .. 4 kGroups - 1 look up one key each: key lane & 3 of group lane >> 2
  const int key_t = 4 * (warp + kGatherWarps * (lane >> 2)) + (lane & 3);
  const bool looks = key_t < kTile && lane < 4 * kGroups;
  struct Entry {  // this lane's list entry of a tile
    uint32_t key, nvis;
    int seq;
    bool there;
  };
  struct Row {  // the page it asks for
    uint32_t key;
    int page;
    bool there;
  };
  struct Tag {  // a tile's item (-1: none), whether it is its last
    int item;
    bool last;
  };
  auto entry_of = [&](const TileCursor& c) {
    Entry e = {(uint32_t)c.t * kTile + key_t, c.it.nvis, c.it.seq, false};
    e.there = c.i < sp.n_items && looks && e.key < c.it.n;
    if (e.there && a.idx) e.key = (uint32_t)a.idx[(int64_t)c.it.r * a.topk + e.key];
    return e;
  };
  auto row_of = [&](const Entry& e) {
    Row r = {e.key, 0, e.there};
    if (e.there && e.key >= e.nvis) {  // a negative index too
      flag_error(a.rows.err, LSA_DEVERR_INDEX);
      r.there = false;
    }
    if (r.there) r.page = a.rows.block_table[(int64_t)e.seq * a.rows.max_pages + e.key / kPage];
    return r;
  };
  auto tag_of = [&](const TileCursor& c) {
    return c.i < sp.n_items ? Tag{c.i, c.t + 1 == c.it.t1} : Tag{-1, false};
  };
  TileCursor ahead;
  ahead.start(a, sp, blockIdx.x, report);
  Tag cur = tag_of(ahead);
  const Entry e0 = entry_of(ahead);
  if (ahead.i < sp.n_items) ahead.next(a, sp, report);
  Tag after = tag_of(ahead);
  Entry entry = entry_of(ahead);  // of the tile after the current one
  Row row = row_of(e0);
  Done older = {-1, 0, 0}, newer = {-1, 0, 0};  // items gathered whose O is not written yet
  uint32_t nk = 0;
  for (uint32_t g = 0; cur.item >= 0; ++g) {
    const int b = g & 1;
    int slot = -1;
    if (row.there) {
      if (page_ok(row.page, a.rows.n_pages)) slot = row.page * kPage + (int)(row.key % kPage);
      else flag_error(a.rows.err, LSA_DEVERR_PAGE);
    }
    row = row_of(entry);
    if (ahead.i < sp.n_items) ahead.next(a, sp, report);
    entry = entry_of(ahead);
    int at[kGroups];  // slots of the keys this lane copies 16 bytes of; a masked key is all zeros, its scale too
#pragma unroll
    for (int j = 0; j < kGroups; ++j) at[j] = __shfl_sync(0xffffffffu, slot, 4 * j + (lane >> 3));
    const uint8_t* lat = a.lat[item_sub(a, sp, cur.item)] + unit * 16;
    const uint32_t stage = smem_u32(sm.k[b]);
#pragma unroll
    for (int cc = 0; cc < kChunks; ++cc) {
      const int c = cc == 0 ? 4 : cc - 1;
      if (g >= 2 && !mbar_wait_fast(c == 4 ? &sm.s_empty[b] : &sm.pv_done[b][c & 3], ((g >> 1) - 1) & 1, abort_flag)) return;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const int k = 4 * (warp + kGatherWarps * j) + (lane >> 3);
        if (k < kTile && (c < 4 || unit < 5))
          cp_async16(stage + c * kChunkBytes + k * 128 + ((unit ^ (k & 7)) << 4),
                     lat + (int64_t)max(at[j], 0) * kLatRow + c * 128, at[j] >= 0 ? 16 : 0);
      }
      cp_async_arrive(&sm.full[b][c]);
    }
    // The item that ended two tiles ago is complete (this tile is in its places): its O.
    if (warp < 4 && older.item >= 0 && older.last_g + 2 == g) {
      if (!write_out(a, sp, sm, tmem, older, warp, lane, part_o, part_ml, abort_flag)) return;
      older = newer;
      newer.item = -1;
    }
    if (cur.last) {
      const Done now = {cur.item, nk++, g};
      if (older.item < 0) older = now;
      else newer = now;
    }
    cur = after;
    after = tag_of(ahead);
  }
  if (warp >= 4) return;
#pragma unroll 1
  while (older.item >= 0) {
    if (!write_out(a, sp, sm, tmem, older, warp, lane, part_o, part_ml, abort_flag)) return;
    older = newer;
    newer.item = -1;
  }
}

// ---------------------------------------------------------------- MMA warp

// Output of an item without keys (a split's empty share: its l = 0).
__device__ __forceinline__ void write_empty(const Fp8MlaArgs& a, const Split& sp, const Item& it, int item, int lane,
                                            float2* part_ml) {
  if (sp.n_split > 1) {
    part_ml[item_base(a, sp, item) * kH + lane] = make_float2(0.f, 0.f);
    return;
  }
  uint4* o = reinterpret_cast<uint4*>(a.out[it.z] + (int64_t)it.r * kH * kDV);
  for (int j = lane; j < kH * kDV / 8; j += 32) o[j] = make_uint4(0, 0, 0, 0);
  if (a.lse[it.z]) a.lse[it.z][(int64_t)it.r * kH + lane] = -INFINITY;
}

// The warp runs together; one lane issues. The two kinds of work, the next S and
// the products of the last P, are taken as they become ready, O first: it frees the places that the gather waits for.
__device__ __forceinline__ void mma_role(const Fp8MlaArgs& a, const Split& sp, Fp8MlaSmem& sm, uint32_t tmem,
                                         int lane, float2* part_ml, volatile int* abort_flag) {
  const uint32_t k_addr = smem_u32(sm.k[0]), q_addr = smem_u32(sm.q), p_addr = smem_u32(sm.p[0]);
  const uint32_t leader = elect_one();
  auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test(bar, parity)) != 0; };
  // S: tile gs of the CTA, tile ts of ts1 of item ks
  uint32_t gs = 0, ks = 0;
  int ts = 0, ts1 = 0, i = blockIdx.x;
  Item nxt = load_item(a, sp, i, false);
  // Takes the next item that has tiles; the one after it is requested ahead.
  auto next_item = [&]() {
    while (i < sp.n_items) {
      const Item it = nxt;
      const int item = i;
      i += gridDim.x;
      nxt = load_item(a, sp, i, false);
      if (it.t0 < it.t1) {
        ts = 0;
        ts1 = it.t1 - it.t0;
        if (lane == 0) sm.item_tiles[ks & 3] = ts1;
        __syncwarp();
        return true;
      }
      if (!it.pad) write_empty(a, sp, it, item, lane, part_ml);
    }
    return false;
  };
  bool s_live = next_item();
  // O: tile gp, tile tp of item kp
  uint32_t gp = 0, kp = 0;
  int tp = 0;
  uint32_t idle = 0;    // polls in a row that found nothing to issue
  long long t0 = 0;     // when a long idle stretch began (the timer's read takes as long as a product)
  while (s_live || gp < gs) {
    if (gp < gs) {
      const int b = gp & 1;
      if (ready(&sm.p_full[b], (gp >> 1) & 1) && (tp > 0 || kp == 0 || ready(&sm.o_empty, (kp - 1) & 1))) {
        tc_fence_after();
        const bool last = tp + 1 == sm.item_tiles[kp & 3];
        const uint64_t ad = sw128_mn_desc(k_addr + b * kStageBytes, 1024), bd = sw64_mn_desc(p_addr + b * kPBytes);
        constexpr uint32_t id = f8_idesc(64, true);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_f8(tmem + kTmemO + c * 64, ad + ((c * kChunkBytes + k * 4096) >> 4), bd + ((k * 2048) >> 4), id,
                    tp > 0 || k > 0 ? 1u : 0u, leader);
          if (leader) umma_commit(&sm.pv_done[b][c]);
          __syncwarp();
        }
        if (last && leader) umma_commit(&sm.o_full);
        __syncwarp();
        ++gp;
        if (last) {
          tp = 0;
          ++kp;
        } else {
          ++tp;
        }
        idle = 0;
        continue;
      }
    }
    if (s_live) {
      const int b = gs & 1;
      // The last chunk's arrivals come after those of the tile's others, and after the
      // products of tile gs - 2, so after its softmax: S's columns are free too.
      if (ready(&sm.full[b][3], (gs >> 1) & 1) && (ts > 0 || ready(&sm.q_full[ks & 3], (ks >> 2) & 1))) {
        fence_proxy_async();  // the tile came through cp.async (generic proxy)
        tc_fence_after();
        const uint64_t ad = sw128_desc(k_addr + b * kStageBytes), bd = sw128_desc(q_addr);
        constexpr uint32_t id = f8_idesc(64, false);
#pragma unroll 1
        for (int k = 0; k < 18; k += 2) {  // (a short loop: straight code waits for its instructions)
          const uint32_t c = k >> 2, o = (k & 3) * 32;
          const uint64_t a0 = ad + ((c * kChunkBytes + o) >> 4), b0 = bd + ((c * kQChunkBytes + o) >> 4);
          umma_f8(tmem + b * 64, a0, b0, id, k > 0 ? 1u : 0u, leader);
          umma_f8(tmem + b * 64, a0 + 2, b0 + 2, id, 1u, leader);
        }
        if (leader) umma_commit(&sm.s_full[b]);
        __syncwarp();
        ++gs;
        if (++ts == ts1) {
          ++ks;
          s_live = next_item();
        }
        idle = 0;
        continue;
      }
    }
    if ((++idle & 1023) == 0) {
      if (*abort_flag) return;
      const long long t = global_ns();
      if (idle == 1024) t0 = t;
      if (t - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        return;
      }
    }
  }
}

// ---------------------------------------------------------------- softmax warps

// The weights of one key (a thread) for the group's 16 heads in the given
// frames (in registers: a shared load waits behind the gather's copies): p for
// the sum, u = p s 2^(2 - A + m) for the product; S from tensor memory. `sq`: the
// key's scale times the query's factor; `su`: the scale, or 0 for a key that adds
// nothing to O. The product of a large scale and a low frame's factor would
// overflow beside a p of zero, so a scale above 1 goes to p and one below to the
// factor: u is exact wherever it counts, and infinite or NaN only where p is (or
// where u is above 128 and the frame is raised). ROUNDED: each logit is rounded
// before m is taken from it, as m was. Unrounded it can lie half a step of fp32 above
// m, which is whole binades where logits are in the thousands and beyond.
struct Frames {
  float m[kHG], w[kHG];  // -m, 2^(2 - A + m)
};
template <bool ROUNDED>
__device__ __forceinline__ void weights(uint32_t s_addr, const Frames& f, bool valid, float sq, float su,
                                        float (&p)[kHG], float (&u)[kHG], float& top_p, float& top_u) {
  tmem_ld16_x2(s_addr, s_addr + kH, p, u);  // hi and lo
  top_p = top_u = 0.f;
  const float s_up = fmaxf(su, 1.f), s_down = fminf(su, 1.f);
#pragma unroll
  for (int h = 0; h < kHG; ++h) {
    const float x = fmaf(u[h], 0.0625f, p[h]);
    p[h] = ex2(ROUNDED ? __fadd_rn(__fmul_rn(x, sq), f.m[h]) : fmaf(x, sq, f.m[h]));
    u[h] = (p[h] * s_up) * (s_down * f.w[h]);
    top_p = fmaxf(top_p, p[h]);
    top_u = fmaxf(top_u, u[h]);
  }
  if (!valid) {
#pragma unroll
    for (int h = 0; h < kHG; ++h) p[h] = u[h] = 0.f;
    top_p = top_u = 0.f;
  }
}

__device__ __forceinline__ void softmax_role(const Fp8MlaArgs& a, const Split& sp, Fp8MlaSmem& sm, uint32_t tmem,
                                             int warp, int lane, volatile int* abort_flag) {
  const int group = warp >> 2, quarter = warp & 3, w0 = group * 4;
  const int key = quarter * 32 + lane, h = lane & 15;  // this lane keeps the frames of the group's head h
  const uint32_t lanes = ((uint32_t)(quarter * 32) << 16) + group * kHG;
  float4* frame = sm.frame[warp];
  Frames f;
  uint32_t g = 0, nk = 0;
  // The first item from `from` on that has tiles.
  struct Work {
    int i, t0, t1;
  };
  auto find = [&](int from) {
    Work w = {from, 0, 0};
    for (; w.i < sp.n_items; w.i += gridDim.x) {
      const Item it = load_item(a, sp, w.i, false);
      w.t0 = it.t0;
      w.t1 = it.t1;
      if (w.t0 < w.t1) break;
    }
    return w;
  };
  if ((int)blockIdx.x < sp.n_items) prefetch_q(query_of(a, sp, blockIdx.x, warp), lane);
  Work cur = find(blockIdx.x);
  while (cur.i < sp.n_items) {
    Query q;
    load_q(q, query_of(a, sp, cur.i, warp), lane);
    const float qf = prepare_q(a, sm, q, nk, warp, lane);  // the query's factor
    const Work next = find(cur.i + gridDim.x);             // looked up while the first tile's products run
    if (next.i < sp.n_items) prefetch_q(query_of(a, sp, next.i, warp), lane);
    const int t0 = cur.t0, t1 = cur.t1;
    float L[kHG];
#pragma unroll
    for (int j = 0; j < kHG; ++j) L[j] = f.m[j] = f.w[j] = 0.f;
    float m_h = 0.f, d_h = kUnset, d_top = kUnset;  // head h's frames, m and A - m (the same in every warp of the group)
    bool framed = false, dead = false, huge = false;
    for (int t = t0; t < t1; ++t, ++g) {
      const int b = g & 1;
      // The tile is here (this thread reads its scale), so the products of tile g - 2
      // are complete: P's buffer is free.
      bool ok = mbar_wait_fast(&sm.full[b][3], (g >> 1) & 1, abort_flag);
      uint2 tail;
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n"
                   : "=r"(tail.x), "=r"(tail.y)
                   : "r"(smem_u32(sm.k[b] + 4 * kChunkBytes + key * 128 + ((4 ^ (key & 7)) << 4))));
      ok = ok && mbar_wait_fast(&sm.s_full[b], (g >> 1) & 1, abort_flag);
      __syncwarp();
      tc_fence_after();
      const uint32_t s_addr = tmem + lanes + b * 64;
      const float s = __uint_as_float(tail.x);
      const bool valid = s != 0.f;                    // a masked key's row is zeros
      const bool silent = !valid || tail.y != 0;      // adds nothing to O
      const float su = silent ? 0.f : s, sq = s * qf;
      const bool anew = (t - t0) % kFrameTiles == 0;
      float p[kHG], u[kHG], top_p = 0.f, top_u = 0.f;
      bool force = anew || !framed || !ok, moved = false, again = false;
      while (true) {
        if (!force) {
          if (huge) weights<true>(s_addr, f, valid, sq, su, p, u, top_p, top_u);
          else weights<false>(s_addr, f, valid, sq, su, p, u, top_p, top_u);
        }
        if (moved || !softmax_any(group, force || top_u > 128.f || top_p > 0x1p60f)) break;
        // Set the frames from this tile's maxima (the group's four warps, the same values).
        __syncwarp();
        tmem_ld16_x2(s_addr, s_addr + kH, p, u);
        const float e = (float)((int)(tail.x >> 23) - 127);
#pragma unroll
        for (int j = 0; j < kHG; ++j) {
          const float x = __fmul_rn(fmaf(u[j], 0.0625f, p[j]), sq);
          p[j] = valid ? x : -INFINITY;
          u[j] = silent ? -INFINITY : (huge ? __fadd_rn(x, f.m[j]) : x) + e;
        }
        const float tl_w = fold16<true>(p, lane), ta_w = fold16<true>(u, lane);
        sm.tmax[warp][h] = make_float2(tl_w, ta_w);
        dead = softmax_any(group, !ok || *abort_flag);
        if (dead) break;
        float tl = -INFINITY, ta = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          tl = fmaxf(tl, sm.tmax[w0 + w][h].x);
          ta = fmaxf(ta, sm.tmax[w0 + w][h].y);
        }
        const float m_old = m_h, d_old = d_h;
        if (tl > -INFINITY) m_h = framed ? fmaxf(m_old, tl) : tl;
        const float dm = m_h - m_old;
        // Logits of whose fp32 steps an exponent would be lost: m first, and A by what lies beside it.
        huge = huge || __any_sync(0xffffffffu, fabsf(m_h) > 1024.f);
        force = huge && !again && __any_sync(0xffffffffu, fabsf(dm) > 0.f);
        again = force;
        moved = !force;
        // A goes by its distance from m: where no key of the tile adds to O it stays, and the distance changes
        // all the same. Down by at most 2^60 from the item's highest: O, scaled up by as much, stays far from
        // overflow. No less than 2^-124 of m: the weights' factor and O's are then powers of two in range.
        const bool loud = ta > -INFINITY && !force;
        float to = d_old == kUnset ? kUnset : (loud && anew ? d_top - 60.f : d_old) - dm;
        if (loud) to = fmaxf(to, huge ? ta : ta - m_h);
        float of = 1.f;
        if (to > kUnset) {
          d_h = fmaxf(ceilf(to), -124.f);
          d_top = fmaxf(d_top - dm, d_h);
          of = ex2(fminf(d_old - dm - d_h, 126.f));
        }
        framed = framed || __any_sync(0xffffffffu, tl > -INFINITY);
        __syncwarp();
        frame[h] = make_float4(-m_h, pow2f(fminf(2.f - d_h, 126.f)), ex2(fminf(-dm, 126.f)), of);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kHG; ++j) {
          const float4 fr = frame[j];
          f.m[j] = fr.x;
          f.w[j] = fr.y;
          L[j] *= fr.z;
          u[j] = fr.w;
        }
        // O so far moves to the new frames, once its last product is complete.
        if (t > t0 && __any_sync(0xffffffffu, of != 1.f)) {
          mbar_wait_fast(&sm.pv_done[b ^ 1][3], ((g - 1) >> 1) & 1, abort_flag);
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const uint32_t o = tmem + lanes + kTmemO + c * 64;
            float lo[kHG];
            tmem_ld16_x2(o, o + kH, p, lo);
#pragma unroll
            for (int j = 0; j < kHG; ++j) {
              p[j] *= u[j];
              lo[j] *= u[j];
            }
            tmem_st16_x2(o, o + kH, p, lo);
          }
        }
      }
      if (dead) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.s_empty[b]);  // S and the scales are read
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h0, h1, l0, l1;
        split_e4m3<64>(f16x2_rn(u[4 * j], u[4 * j + 1]), h0, l0);
        split_e4m3<64>(f16x2_rn(u[4 * j + 2], u[4 * j + 3]), h1, l1);
        hi[j] = h0 | h1 << 16;
        lo[j] = l0 | l1 << 16;
      }
      uint8_t* prow = sm.p[b] + key * 64;
      const int sw = (key >> 1) & 3;
      *reinterpret_cast<uint4*>(prow + ((group ^ sw) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(prow + (((2 + group) ^ sw) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[b]);
#pragma unroll
      for (int j = 0; j < kHG; ++j) L[j] += p[j];
    }
    // The item's sums, for the output.
    sm.lsum[warp][h] = fold16<false>(L, lane);
    if (all_softmax_any(dead || *abort_flag)) return;  // both groups or neither: they meet at the next query
    if (quarter == 0) {
      const float l = (sm.lsum[w0][h] + sm.lsum[w0 + 1][h]) + (sm.lsum[w0 + 2][h] + sm.lsum[w0 + 3][h]);
      const int f = nk & 3;
      sm.fin[f][group * kHG + h] = make_float2(d_h == kUnset ? 0.f : pow2f(d_h - 2.f), l);
      sm.fin_m[f][group * kHG + h] = m_h;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.fin_full[f]);
    }
    ++nk;
    cur = next;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    fp8_mla_kernel(const __grid_constant__ Fp8MlaArgs a, const __grid_constant__ Split sp, float* part_o,
                   float2* part_ml) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {  // the swizzled tiles need it; checked, never assumed
    if (threadIdx.x == 0) flag_error(a.rows.err, LSA_DEVERR_TIMEOUT);
    return;
  }
  Fp8MlaSmem& sm = *reinterpret_cast<Fp8MlaSmem*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      for (int c = 0; c < kChunks; ++c) mbar_init(&sm.full[b][c], kGatherWarps * 32);
      for (int c = 0; c < 4; ++c) mbar_init(&sm.pv_done[b][c], 1);
      mbar_init(&sm.s_full[b], 1);
      mbar_init(&sm.s_empty[b], kSoftWarps);
      mbar_init(&sm.p_full[b], kSoftWarps);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&sm.q_full[b], kSoftWarps);
      mbar_init(&sm.fin_full[b], 2);
    }
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_empty, 4);
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::);
  }
  if (warp == kMmaWarp) tmem_alloc(&sm.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;
  // Registers: 512 threads x 128 at launch; the softmax's two warpgroups take 48 a
  // thread from the other two (2 x 176 + 2 x 80 = 4 x 128).
  if (warp < kSoftWarps) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;\n" ::);
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n" ::);
  if (warp < kSoftWarps) {
    softmax_role(a, sp, sm, tmem, warp, lane, abort_flag);
  } else if (warp < kMmaWarp) {
    gather_role(a, sp, sm, tmem, warp - kSoftWarps, lane, part_o, part_ml, abort_flag);
    asm volatile("cp.async.wait_all;\n" ::: "memory");  // none in flight when the CTA retires
  } else {
    mma_role(a, sp, sm, tmem, lane, part_ml, abort_flag);
    __syncwarp();
    if (elect_one()) umma_commit(&sm.drain);  // every product is complete before the tensor memory is freed
    const long long t0 = global_ns();
    while (!mbar_try_wait(&sm.drain, 0))
      if (global_ns() - t0 > kWaitLimitNs) break;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && sm.abort_flag) flag_error(a.rows.err, LSA_DEVERR_TIMEOUT);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// One CTA per (head, row, sub-block) joins the splits: 128 threads x 4 value dims.
__global__ void __launch_bounds__(128)
    fp8_mla_merge_kernel(const __grid_constant__ Fp8MlaArgs a, int n_split, const float* part_o, const float2* part_ml, int row0) {
  __shared__ float wgt[kMaxSplits];
  pdl_wait();
  const int h = blockIdx.x, r = row0 + blockIdx.y, z = blockIdx.z, tid = threadIdx.x;
  const int seq = a.rows.seq_of_row ? a.rows.seq_of_row[r] : r;
  if (seq == -1) return;  // a padding row
  const int64_t base = ((int64_t)z * a.rows.n_rows + r) * n_split;
  if (tid < 32) {
    // an unknown sequence has no partials; a split without keys has l = 0
    const bool there = tid < n_split;
    const float2 ml = there ? part_ml[(base + tid) * kH + h] : make_float2(0.f, 0.f);
    const bool live = there && ml.y != 0.f;
    float M = live ? ml.x : -INFINITY;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    const float wv = live ? exp2f(ml.x - M) : 0.f;
    float L = live ? wv * ml.y : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    if (there) wgt[tid] = live ? wv * ml.y / L : -1.f;  // of outputs that are divided by their own sums
    if (tid == 0) {
      if (a.lse[z]) a.lse[z][(int64_t)r * kH + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* po = part_o + (base * kH + h) * kDV + tid * 4;
#pragma unroll 8
  for (int s = 0; s < n_split; ++s) {
    const float wv = wgt[s];
    if (wv == -1.f) continue;  // an empty split wrote no output
    const float4 x = *reinterpret_cast<const float4*>(po + (int64_t)s * kH * kDV);
    acc.x = fmaf(wv, x.x, acc.x);
    acc.y = fmaf(wv, x.y, acc.y);
    acc.z = fmaf(wv, x.z, acc.z);
    acc.w = fmaf(wv, x.w, acc.w);
  }
  const uint2 pk = make_uint2(bf16x2_rn(acc.x, acc.y), bf16x2_rn(acc.z, acc.w));
  *reinterpret_cast<uint2*>(a.out[z] + ((int64_t)r * kH + h) * kDV + tid * 4) = pk;
}

// Splits of each row's list: the count with the shortest longest CTA, an item
// costing its tiles plus about two tiles' time of its own (query, output) and
// the join of the splits about one more. Measured with 1, 2, 4, 8 and 16 splits
// (us): one row of 2048 keys and 2 sub-blocks 40, 26, 19, 15, 14; 16 such rows 44,
// 31, 25, 30, 40; 130 rows of one sub-block 45, 56, 66, 84, 131: this takes 16, 4
// and 1.
int choose_splits(int n_rows, int n_sub, int64_t max_list) {
  const int sms = sm_count();
  const int64_t items = max64((int64_t)n_rows * n_sub, 1), tiles = max64((max_list + kTile - 1) / kTile, 1);
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int s = 1; s <= kMaxSplits && s <= tiles; ++s) {
    const int64_t waves = (items * s + sms - 1) / sms;
    const int64_t cost = waves * ((tiles + s - 1) / s + 2) + (s > 1 ? 1 : 0);
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

size_t ws_bytes_of(int n_rows, int n_sub, int n_split) {
  if (n_split <= 1) return 0;
  const size_t per = (size_t)kH * kDV * sizeof(float) + (size_t)kH * sizeof(float2);
  return (size_t)n_rows * n_sub * n_split * per + kH * sizeof(float2);
}

}  // namespace

size_t fp8_mla_ws_bytes(int n_rows, int n_sub, int64_t max_list) {
  // either sub-block count the call may come with (one, or all of the layer's),
  // with lists or dense
  size_t most = 0;
  for (int z = 1; z <= n_sub; ++z) {
    most = max(most, ws_bytes_of(n_rows, z, choose_splits(n_rows, z, max_list)));
    most = max(most, ws_bytes_of(n_rows, z, choose_splits(n_rows, z, min64(max_list, kMaxTopk))));
  }
  return most;
}

cudaError_t launch_fp8_mla(const Fp8MlaArgs& a, cudaStream_t st) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(fp8_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Fp8MlaSmem));
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int n_rows = a.rows.n_rows;
  const int64_t list = a.idx ? min64(a.topk, a.rows.max_len) : a.rows.max_len;
  Split sp;
  sp.n_split = choose_splits(n_rows, a.n_sub, list);
  while (sp.n_split > 1 && ws_bytes_of(n_rows, a.n_sub, sp.n_split) > a.ws_bytes) --sp.n_split;
  const int64_t items = (int64_t)n_rows * a.n_sub * sp.n_split;
  if (items > INT32_MAX - 65536) return cudaErrorInvalidValue;
  sp.n_items = (int)items;
  float* part_o = nullptr;
  float2* part_ml = nullptr;
  if (sp.n_split > 1) {
    part_o = static_cast<float*>(a.ws);
    part_ml = reinterpret_cast<float2*>(part_o + items * kH * kDV);
  }
  cudaError_t e = launch_pdl(fp8_mla_kernel, dim3((unsigned)min64(items, sm_count())), dim3(kThreads),
                             sizeof(Fp8MlaSmem), st, a, sp, part_o, part_ml);
  count_launches(1);
  if (e != cudaSuccess || sp.n_split == 1) return e;
  for (int row0 = 0; row0 < n_rows; row0 += 65535) {
    e = launch_pdl(fp8_mla_merge_kernel, dim3(kH, (unsigned)min(65535, n_rows - row0), (unsigned)a.n_sub), dim3(128),
                   0, st, a, sp.n_split, (const float*)part_o, (const float2*)part_ml, row0);
    count_launches(1);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace lsa
