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
//   - the query, scaled per head by a power of two to at most 448, k = 16: bf16
//     has 8 significant bits, two e4m3 of 4 bits hold them exactly down to 2^-22
//     of the head's largest element;
//   - the weight u = p * s_i * 2^(4 - A), at most 128, k = 64: 8 significant
//     bits, the precision of a bf16 weight; what lies below 2^-20 of the largest
//     u of its frame is lost.
// The frame A of each head (an integer, so that rescaling is exact) follows the
// running maximum of log2(p s): it is set from the first tile, raised when a u
// would pass 128, and set anew every 16 tiles (also downwards: O is then scaled
// up, fp32 has the range), so that the loss stays relative to the 2048 keys
// around a key however long the list is. The sum of the softmax is kept apart,
// in fp32, of the unrounded weights, in its own frame m (a key's scale, which is
// no part of its weight, cannot disturb it).
//
// Layout. One tile is 128 keys: S^T [128 keys x 64] = C Q^T (K = 576: 18
// instructions), then O^T [512 dims x 64] += C^T P (4 x 4 instructions of 128
// dims and 32 keys). Both read the same 80 KB of shared memory: a key is 128
// bytes in each of five chunks with the 128-byte swizzle, which is K-major for S
// (rows = keys) and MN-major for O (rows = the contraction). Tensor memory: S
// twice 64 columns, O 4 x 64.
//
// Roles (11 warps, one CTA per SM, persistent over (row, sub-block, split)
// items): 4 softmax warps (a thread = a key of the tile), 4 epilogue warps (Q
// codes of the next item, then O of this one), 2 gather warps (16-byte cp.async
// into the swizzled layout, a ring of two tiles), one MMA thread that issues
// S(t + 1) before O(t), so that the softmax of a tile runs under the products of
// its neighbours. Every wait is bounded.
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
constexpr int kGatherWarps = 2;
constexpr int kMmaWarp = 8 + kGatherWarps;
constexpr int kThreads = (kMmaWarp + 1) * 32;     // 11 warps: 168 registers a thread (12 would be allocated alike)
constexpr int kFrameTiles = 16;                  // tiles after which the frame is set anew
constexpr int kMaxSplits = 32;
constexpr uint32_t kTmemO = 128;                 // S: columns 0..127, O: 128..383
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kUnset = -1.0e9f;                // no frame yet

struct __align__(1024) Fp8MlaSmem {
  uint8_t k[2][kStageBytes];
  uint8_t q[kChunks * kQChunkBytes];   // [chunk][32 hi rows, 32 lo rows][128 B]
  uint8_t p[2][kPBytes];               // [key][32 hi, 32 lo codes]
  float4 frame[4][kH];                 // per softmax warp: q factor, m, 2^(4 - A + m), A - m + 3
  float4 move[4][kH];                  // per softmax warp: factors of L and O, shift of x
  float2 tmax[4][kH];                  // event: each warp's maxima
  float lsum[4][kH];
  float qf[4][kH];                     // ring over items: the heads' query factors
  float2 fin[4][kH];                   // ring over items: factor of O, lse (one split) ; 2^(A-m-4), L
  float fin_m[4][kH];
  uint64_t full[2], pv_done[2], s_full[2], s_empty[2], p_full[2], q_full[4], fin_full[4], q_empty, o_full, o_empty, drain;
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
  int r, z, s, t0, t1;
  int64_t n, nvis;       // list length, visible keys
  const int32_t* table;  // the sequence's block-table row
  bool pad;
};

__device__ __forceinline__ Item load_item(const Fp8MlaArgs& a, const Split& sp, int i, bool report) {
  Item it;
  it.pad = true;
  it.t0 = it.t1 = 0;
  it.r = it.z = it.s = 0;
  it.n = it.nvis = 0;
  it.table = nullptr;
  if (i >= sp.n_items) return it;
  it.s = i % sp.n_split;
  it.z = (i / sp.n_split) % a.n_sub;
  it.r = i / (sp.n_split * a.n_sub);
  report = report && it.s == 0 && it.z == 0;
  const int32_t cnt = a.idx ? a.count[it.r] : 0;
  const PagedGeom g = paged_geom(a.rows, it.r, report);
  it.pad = g.pad;
  it.nvis = g.nvis;
  it.n = g.nvis;
  if (g.seq < 0) return it;
  it.table = a.rows.block_table + (int64_t)g.seq * a.rows.max_pages;
  if (a.idx) {
    it.n = cnt;
    if (cnt < 0 || cnt > a.topk) {
      if (report) flag_error(a.rows.err, LSA_DEVERR_COUNT);
      it.n = cnt < 0 ? 0 : a.topk;
    }
  }
  const int64_t tiles = (it.n + kTile - 1) / kTile;
  it.t0 = (int)(tiles * it.s / sp.n_split);
  it.t1 = (int)(tiles * (it.s + 1) / sp.n_split);
  return it;
}

// Lane h gets the maximum (or sum) over the warp of v[h]: a butterfly that halves the array.
template <bool MAX>
__device__ __forceinline__ float fold32(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = (lane & o) ? v[i] : v[i + o], keep = (lane & o) ? v[i + o] : v[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, o);
      v[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  return v[0];
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// 2^d for integer-valued d, 0 below the normal range.
__device__ __forceinline__ float pow2f(float d) { return d < -126.f ? 0.f : pow2i((int)fminf(fmaxf(d, -126.f), 126.f)); }

// The softmax warps' barrier with an OR over all of them.
__device__ __forceinline__ bool softmax_any(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %1, 0;\n bar.red.or.pred p, 1, 128, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}

// ---------------------------------------------------------------- gather warps

__device__ __forceinline__ void gather_role(const Fp8MlaArgs& a, const Split& sp, Fp8MlaSmem& sm, int warp, int lane,
                                            volatile int* abort_flag) {
  const int key_t = warp * 64 + lane;  // this lane looks up the rows of tile keys key_t and key_t + 32
  uint32_t g = 0;
  for (int i = blockIdx.x; i < sp.n_items; i += gridDim.x) {
    const Item it = load_item(a, sp, i, warp == 0 && lane == 0);
    const int32_t* list = a.idx ? a.idx + (int64_t)it.r * a.topk : nullptr;
    const uint8_t* lat = a.lat[it.z];
    // Row of list entry e: its address, or null when it is masked.
    auto lookup = [&](int64_t e) -> const uint8_t* {
      if (e >= it.n) return nullptr;
      const int64_t key = list ? list[e] : e;
      if (key < 0 || key >= it.nvis) {
        flag_error(a.rows.err, LSA_DEVERR_INDEX);
        return nullptr;
      }
      const int page = it.table[key / kPage];
      if (!page_ok(page, a.rows.n_pages)) {
        flag_error(a.rows.err, LSA_DEVERR_PAGE);
        return nullptr;
      }
      return lat + ((int64_t)page * kPage + key % kPage) * kLatRow;
    };
    const uint8_t *row0 = nullptr, *row1 = nullptr;
    if (it.t0 < it.t1) {
      row0 = lookup((int64_t)it.t0 * kTile + key_t);
      row1 = lookup((int64_t)it.t0 * kTile + key_t + 32);
    }
    for (int t = it.t0; t < it.t1; ++t, ++g) {
      const int b = g & 1;
      const uint8_t *next0 = nullptr, *next1 = nullptr;
      if (t + 1 < it.t1) {
        next0 = lookup((int64_t)(t + 1) * kTile + key_t);
        next1 = lookup((int64_t)(t + 1) * kTile + key_t + 32);
      }
      if (g >= 2 && !mbar_wait(&sm.pv_done[b], ((g >> 1) - 1) & 1, abort_flag)) return;
      __syncwarp();
      const uint32_t stage = smem_u32(sm.k[b]);
      const int unit = lane & 7;
#pragma unroll
      for (int q = 0; q < 16; ++q) {  // four keys at a time, eight lanes a key
        const int k = 4 * q + (lane >> 3);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(q < 8 ? row0 : row1), k & 31));
        const int bytes = src ? 16 : 0;  // a masked key is all zeros, its scale too
        const uint8_t* from = (src ? src : lat) + unit * 16;
        const uint32_t dst = stage + (warp * 64 + k) * 128 + ((unit ^ (k & 7)) << 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) cp_async16(dst + c * kChunkBytes, from + c * 128, bytes);
        if (unit < 5) cp_async16(dst + 4 * kChunkBytes, from + 4 * 128, bytes);
      }
      cp_async_arrive(&sm.full[b]);
      row0 = next0;
      row1 = next1;
    }
  }
}

// ---------------------------------------------------------------- MMA thread

struct MmaRole {
  Fp8MlaSmem& sm;
  uint32_t tmem;
  volatile int* abort_flag;
  uint32_t k_addr, q_addr, p_addr;

  __device__ __forceinline__ bool s_tile(uint32_t g, bool last) {
    const int b = g & 1;
    if (!mbar_wait(&sm.full[b], (g >> 1) & 1, abort_flag)) return false;
    if (g >= 2 && !mbar_wait(&sm.s_empty[b], ((g >> 1) - 1) & 1, abort_flag)) return false;
    fence_proxy_async();  // the tile came through cp.async (generic proxy)
    tc_fence_after();
    const uint64_t ad = sw128_desc(k_addr + b * kStageBytes), bd = sw128_desc(q_addr);
    constexpr uint32_t id = f8_idesc(64, false);
#pragma unroll
    for (int ks = 0; ks < 18; ++ks) {
      const uint32_t c = ks >> 2, o = (ks & 3) * 32;
      umma_f8(tmem + b * 64, ad + ((c * kChunkBytes + o) >> 4), bd + ((c * kQChunkBytes + o) >> 4), id, ks > 0 ? 1u : 0u);
    }
    umma_commit(&sm.s_full[b]);
    if (last) umma_commit(&sm.q_empty);
    return true;
  }
  __device__ __forceinline__ bool pv_tile(uint32_t g, bool first, bool last, uint32_t nk) {
    const int b = g & 1;
    if (!mbar_wait(&sm.p_full[b], (g >> 1) & 1, abort_flag)) return false;
    if (first && nk > 0 && !mbar_wait(&sm.o_empty, (nk - 1) & 1, abort_flag)) return false;
    tc_fence_after();
    const uint64_t ad = sw128_mn_desc(k_addr + b * kStageBytes, 1024), bd = sw64_mn_desc(p_addr + b * kPBytes);
    constexpr uint32_t id = f8_idesc(64, true);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        umma_f8(tmem + kTmemO + c * 64, ad + ((c * kChunkBytes + ks * 4096) >> 4), bd + ((ks * 2048) >> 4), id,
                !first || ks > 0 ? 1u : 0u);
    umma_commit(&sm.pv_done[b]);
    if (last) umma_commit(&sm.o_full);
    return true;
  }
};

__device__ __forceinline__ void mma_role(const Fp8MlaArgs& a, const Split& sp, Fp8MlaSmem& sm, uint32_t tmem,
                                         volatile int* abort_flag) {
  MmaRole m{sm, tmem, abort_flag, smem_u32(sm.k[0]), smem_u32(sm.q), smem_u32(sm.p[0])};
  uint32_t g = 0, nk = 0;
  bool pending = false, p_first = false, p_last = false;
  uint32_t p_nk = 0;
  Item nxt = load_item(a, sp, blockIdx.x, false);
  for (int i = blockIdx.x; i < sp.n_items; i += gridDim.x) {
    const Item it = nxt;
    nxt = load_item(a, sp, i + gridDim.x, false);
    if (it.t0 >= it.t1) continue;
    for (int t = it.t0; t < it.t1; ++t, ++g) {
      const bool first = t == it.t0, last = t + 1 == it.t1;
      if (first) {  // the previous item's last product does not wait for this item's query
        if (pending && !m.pv_tile(g - 1, p_first, p_last, p_nk)) return;
        pending = false;
        if (!mbar_wait(&sm.q_full[nk & 3], (nk >> 2) & 1, abort_flag)) return;
      }
      if (!m.s_tile(g, last)) return;
      if (pending && !m.pv_tile(g - 1, p_first, p_last, p_nk)) return;
      pending = true;
      p_first = first;
      p_last = last;
      p_nk = nk;
    }
    ++nk;
  }
  if (pending) m.pv_tile(g - 1, p_first, p_last, p_nk);
}

// ---------------------------------------------------------------- softmax warps

__device__ __forceinline__ void softmax_role(const Fp8MlaArgs& a, const Split& sp, Fp8MlaSmem& sm, uint32_t tmem,
                                             int warp, int lane, volatile int* abort_flag) {
  const int key = warp * 32 + lane;
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  float4* frame = sm.frame[warp];
  float4* move = sm.move[warp];
  uint32_t g = 0, nk = 0;
  Item nxt = load_item(a, sp, blockIdx.x, false);
  for (int i = blockIdx.x; i < sp.n_items; i += gridDim.x) {
    const Item it = nxt;
    nxt = load_item(a, sp, i + gridDim.x, false);
    if (it.t0 >= it.t1) continue;
    float L[32];
#pragma unroll
    for (int h = 0; h < 32; ++h) L[h] = 0.f;
    float m_h = 0.f, a_h = kUnset, qf_h = 0.f;  // lane h: head h's frames (every warp the same)
    bool framed = false;
    for (int t = it.t0; t < it.t1; ++t, ++g) {
      const int b = g & 1;
      bool ok = true;
      if (t == it.t0) {
        ok = mbar_wait(&sm.q_full[nk & 3], (nk >> 2) & 1, abort_flag);
        qf_h = sm.qf[nk & 3][lane];
        frame[lane] = make_float4(qf_h, 0.f, 0.f, 0.f);
      }
      ok = ok && mbar_wait(&sm.s_full[b], (g >> 1) & 1, abort_flag);
      ok = ok && mbar_wait(&sm.full[b], (g >> 1) & 1, abort_flag);  // complete already: this thread reads the tile too
      if (ok && g >= 2) ok = mbar_wait(&sm.pv_done[b], ((g >> 1) - 1) & 1, abort_flag);  // P's buffer
      __syncwarp();
      tc_fence_after();
      float x[32], lo[32];
      tmem_ld32_x2(tmem + lanes + b * 64, tmem + lanes + b * 64 + 32, x, lo);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.s_empty[b]);
      const uint2 tail = *reinterpret_cast<const uint2*>(sm.k[b] + 4 * kChunkBytes + key * 128 + ((4 ^ (key & 7)) << 4));
      const float s = __uint_as_float(tail.x);
      const bool valid = s != 0.f;                    // a masked key's row is zeros
      const bool silent = !valid || tail.y != 0;      // adds nothing to O
      const float e = (float)((int)(tail.x >> 23) - 127);
      float over_u = -INFINITY, over_p = -INFINITY;
#pragma unroll
      for (int h = 0; h < 32; ++h) {
        const float4 f = frame[h];
        x[h] = fmaf(fmaf(lo[h], 0.0625f, x[h]) * f.x, s, -f.y);
        over_u = fmaxf(over_u, x[h] - f.w);
        over_p = fmaxf(over_p, x[h]);
      }
      if (!valid) {
#pragma unroll
        for (int h = 0; h < 32; ++h) x[h] = -INFINITY;
      }
      const bool anew = (t - it.t0) % kFrameTiles == 0;
      const bool need = anew || !framed || !ok || (valid && (over_p > 60.f || (!silent && over_u + e > 0.f)));
      if (softmax_any(need)) {
        // Set the frames from this tile's maxima (all four warps, the same values).
        float v[32];
#pragma unroll
        for (int h = 0; h < 32; ++h) v[h] = x[h];
        const float tl_w = fold32<true>(v, lane);
#pragma unroll
        for (int h = 0; h < 32; ++h) v[h] = silent ? -INFINITY : x[h] + e;
        const float ta_w = fold32<true>(v, lane);
        sm.tmax[warp][lane] = make_float2(tl_w, ta_w);
        if (softmax_any(!ok || *abort_flag)) return;
        float tl = -INFINITY, ta = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          tl = fmaxf(tl, sm.tmax[w][lane].x);
          ta = fmaxf(ta, sm.tmax[w][lane].y);
        }
        const float m_old = m_h, a_old = a_h;
        if (tl > -INFINITY) m_h = framed ? fmaxf(m_old, ceilf(tl + m_old)) : ceilf(tl + m_old);
        if (ta > -INFINITY) a_h = fmaxf(ceilf(ta + m_old), anew ? a_old - 60.f : a_old);
        framed = framed || __any_sync(0xffffffffu, tl > -INFINITY);
        const float d = a_h - m_h;
        const float of = pow2f(a_old - a_h);
        __syncwarp();
        frame[lane] = make_float4(qf_h, m_h, pow2f(fminf(4.f - d, 126.f)), d + 3.f);
        move[lane] = make_float4(pow2f(m_old - m_h), of, m_old - m_h, 0.f);
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 32; ++h) {
          const float4 mv = move[h];
          L[h] *= mv.x;
          x[h] += mv.z;
        }
        // O so far moves to the new frames, once its last product is complete.
        if (t > it.t0 && __any_sync(0xffffffffu, of != 1.f)) {
          mbar_wait(&sm.pv_done[b ^ 1], ((g - 1) >> 1) & 1, abort_flag);
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            float o[32];
            tmem_ld32(tmem + lanes + kTmemO + c * 32, o);
#pragma unroll
            for (int h = 0; h < 32; ++h) o[h] *= move[h].y;
            tmem_st32(tmem + lanes + kTmemO + c * 32, o);
          }
          tc_fence_before();
        }
      }
      // Weights: p for the sum, u = p s 2^(4 - A + m) in two e4m3 pieces for the product.
      const float su = silent ? 0.f : s;
      uint32_t hi[8], lw[8];
#pragma unroll
      for (int h4 = 0; h4 < 8; ++h4) {
        float u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = ex2(x[4 * h4 + j]);
          L[4 * h4 + j] += p;
          u[j] = p * su * frame[4 * h4 + j].z;
        }
        uint32_t h0, h1, l0, l1;
        split_e4m3<64>(f16x2_rn(u[0], u[1]), h0, l0);
        split_e4m3<64>(f16x2_rn(u[2], u[3]), h1, l1);
        hi[h4] = h0 | h1 << 16;
        lw[h4] = l0 | l1 << 16;
      }
      uint8_t* prow = sm.p[b] + key * 64;
      const int sw = (key >> 1) & 3;
      *reinterpret_cast<uint4*>(prow + ((0 ^ sw) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(prow + ((1 ^ sw) << 4)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
      *reinterpret_cast<uint4*>(prow + ((2 ^ sw) << 4)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
      *reinterpret_cast<uint4*>(prow + ((3 ^ sw) << 4)) = make_uint4(lw[4], lw[5], lw[6], lw[7]);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[b]);
    }
    // The item's sums, for the epilogue.
    sm.lsum[warp][lane] = fold32<false>(L, lane);
    if (softmax_any(*abort_flag != 0)) return;
    if (warp == 0) {
      const float l = (sm.lsum[0][lane] + sm.lsum[1][lane]) + (sm.lsum[2][lane] + sm.lsum[3][lane]);
      const int f = nk & 3;
      const float back = a_h == kUnset ? 0.f : pow2f(a_h - m_h - 4.f);
      sm.fin[f][lane] = make_float2(back, l);
      sm.fin_m[f][lane] = m_h;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.fin_full[f]);
    }
    ++nk;
  }
}

// ---------------------------------------------------------------- epilogue warps

// Quantises heads 8 warp .. 8 warp + 7 of the item's query into the hi and lo rows.
__device__ __forceinline__ void load_q(const Fp8MlaArgs& a, const Item& it, int warp, int lane, uint4 (&v)[8][3]) {
  const uint4* src = reinterpret_cast<const uint4*>(a.q[it.z] + (int64_t)it.r * kH * kDLat) + warp * 8 * 72;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int c = 0; c < 3; ++c)
      v[j][c] = lane + 32 * c < 72 ? __ldg(src + j * 72 + lane + 32 * c) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void store_q(const Fp8MlaArgs& a, Fp8MlaSmem& sm, uint32_t nk, int warp, int lane,
                                        const uint4 (&v)[8][3]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int h = warp * 8 + j;
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < 3; ++c)
      m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(m, v[j][c].x), v[j][c].y), v[j][c].z), v[j][c].w);
    m = fold_max(m);
    const bool fin = bf16_finite(m);
    const int e = fin ? scale_exponent(m) : 0;
    const float inv = fin ? pow2i(-e) : 0.f;
#pragma unroll
    for (int c = 0; c < 3; ++c) {
      const int u = lane + 32 * c;  // eight elements
      if (u >= 72) break;
      const uint32_t w[4] = {v[j][c].x, v[j][c].y, v[j][c].z, v[j][c].w};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x0 = fin ? bf16_lo(w[k]) * inv : 0.f, x1 = fin ? bf16_hi(w[k]) * inv : 0.f;
        hi[k] = e4m3x2(x0, x1);
        const uint32_t b = f16_e4m3x2(hi[k]);
        float b0, b1;
        asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n" : "=f"(b0), "=f"(b1) : "r"(b));
        lo[k] = e4m3x2((x0 - b0) * 16.f, (x1 - b1) * 16.f);
      }
      const int chunk = u >> 4, unit = (u >> 1) & 7, half = (u & 1) * 8;
      uint8_t* base = sm.q + chunk * kQChunkBytes + h * 128 + ((unit ^ (h & 7)) << 4) + half;
      *reinterpret_cast<uint2*>(base) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      *reinterpret_cast<uint2*>(base + 32 * 128) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
    }
    if (lane == 0) sm.qf[nk & 3][h] = fin ? pow2i(e) * (a.scale * kLog2e) : __uint_as_float(0x7fc00000u);
  }
  fence_proxy_async();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm.q_full[nk & 3]);
}

__device__ __forceinline__ void epilogue_role(const Fp8MlaArgs& a, const Split& sp, Fp8MlaSmem& sm, uint32_t tmem,
                                              int warp, int lane, float* part_o, float2* part_ml,
                                              volatile int* abort_flag) {
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  uint32_t nk = 0, nq = 0;  // items drained, queries prepared
  uint4 v[8][3];
  // The next item with tiles after `i`.
  auto next_live = [&](int i, Item& it) {
    for (; i < sp.n_items; i += gridDim.x) {
      it = load_item(a, sp, i, false);
      if (it.t0 < it.t1) break;
    }
    return i;
  };
  Item qi;
  int qat = next_live(blockIdx.x, qi);
  if (qat < sp.n_items) {
    load_q(a, qi, warp, lane, v);
    store_q(a, sm, nq++, warp, lane, v);
  }
  for (int i = blockIdx.x; i < sp.n_items; i += gridDim.x) {
    const Item it = load_item(a, sp, i, false);
    const int64_t base = ((int64_t)it.z * a.rows.n_rows + it.r) * sp.n_split + it.s;
    if (it.t0 >= it.t1) {  // nothing to attend to
      if (it.pad) continue;
      if (sp.n_split > 1) {
        if (warp == 0) part_ml[base * kH + lane] = make_float2(0.f, 0.f);
      } else {
        uint4* o = reinterpret_cast<uint4*>(a.out[it.z] + (int64_t)it.r * kH * kDV) + warp * 512;
        for (int j = lane; j < 512; j += 32) o[j] = make_uint4(0, 0, 0, 0);
        if (a.lse[it.z] && warp == 0) a.lse[it.z][(int64_t)it.r * kH + lane] = -INFINITY;
      }
      continue;
    }
    // the next item's query, as soon as this one's last S is done
    qat = next_live(i + gridDim.x, qi);
    if (qat < sp.n_items) load_q(a, qi, warp, lane, v);
    if (qat < sp.n_items) {
      if (!mbar_wait(&sm.q_empty, nk & 1, abort_flag)) return;
      store_q(a, sm, nq++, warp, lane, v);
    }
    if (!mbar_wait(&sm.fin_full[nk & 3], (nk >> 2) & 1, abort_flag)) return;
    if (!mbar_wait(&sm.o_full, nk & 1, abort_flag)) return;
    __syncwarp();
    tc_fence_after();
    const float2* fin = sm.fin[nk & 3];
    const bool one = sp.n_split == 1;
    if (warp == 0) {
      const float l = fin[lane].y, m = sm.fin_m[nk & 3][lane];
      if (!one) part_ml[base * kH + lane] = make_float2(m, l);
      else if (a.lse[it.z]) a.lse[it.z][(int64_t)it.r * kH + lane] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
    float mine = fin[lane].x;  // lane h: the factor of head h
    if (one) mine = fin[lane].y == 0.f ? 0.f : mine / fin[lane].y;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float o[32], lo[32];
      tmem_ld32_x2(tmem + lanes + kTmemO + c * 64, tmem + lanes + kTmemO + c * 64 + 32, o, lo);
      if (c == 3) {  // O is read: the next item may start its products
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_empty);
      }
#pragma unroll
      for (int h = 0; h < 32; ++h) o[h] = fmaf(lo[h], 0.015625f, o[h]) * __shfl_sync(0xffffffffu, mine, h);
      const int d = c * 128 + warp * 32 + lane;
      if (one) {
        // neighbouring lanes swap heads, so that each stores two dims of one head
        uint16_t* og = a.out[it.z] + (int64_t)it.r * kH * kDV + (d & ~1);
#pragma unroll
        for (int h = 0; h < 32; h += 2) {
          const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? o[h] : o[h + 1], 1);
          const uint32_t two = (lane & 1) ? bf16x2_rn(got, o[h + 1]) : bf16x2_rn(o[h], got);
          *reinterpret_cast<uint32_t*>(og + (h + (lane & 1)) * kDV) = two;
        }
      } else {
        float* po = part_o + base * kH * kDV + d;
#pragma unroll
        for (int h = 0; h < 32; ++h) po[h * kDV] = o[h];
      }
    }
    ++nk;
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
      mbar_init(&sm.full[b], kGatherWarps * 32);
      mbar_init(&sm.pv_done[b], 1);
      mbar_init(&sm.s_full[b], 1);
      mbar_init(&sm.s_empty[b], 4);
      mbar_init(&sm.p_full[b], 4);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&sm.q_full[b], 4);
      mbar_init(&sm.fin_full[b], 1);
    }
    mbar_init(&sm.q_empty, 1);
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
  if (warp < 4) {
    softmax_role(a, sp, sm, tmem, warp, lane, abort_flag);
  } else if (warp < 8) {
    epilogue_role(a, sp, sm, tmem, warp - 4, lane, part_o, part_ml, abort_flag);
  } else if (warp < kMmaWarp) {
    gather_role(a, sp, sm, warp - 8, lane, abort_flag);
    asm volatile("cp.async.wait_all;\n" ::: "memory");  // none in flight when the CTA retires
  } else if (lane == 0) {
    mma_role(a, sp, sm, tmem, abort_flag);
    umma_commit(&sm.drain);  // every product is complete before the tensor memory is freed
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
  __shared__ float inv_l;
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
    if (there) wgt[tid] = live ? wv : -1.f;
    if (tid == 0) {
      inv_l = L == 0.f ? 0.f : 1.f / L;
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
  const float il = inv_l;
  const uint2 pk = make_uint2(bf16x2_rn(acc.x * il, acc.y * il), bf16x2_rn(acc.z * il, acc.w * il));
  *reinterpret_cast<uint2*>(a.out[z] + ((int64_t)r * kH + h) * kDV + tid * 4) = pk;
}

int sm_count() {
  static int cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  if (cache[dev] == 0) {
    int s = 148;
    if (cudaDeviceGetAttribute(&s, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || s < 1) s = 148;
    cache[dev] = s;
  }
  return cache[dev];
}

// Splits of each row's list: the count with the shortest longest CTA, an item
// costing its tiles plus about two tiles' time of its own (query, output) and
// the join of the splits about one more.
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
