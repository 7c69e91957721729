// Lightning indexer over paged 8-bit keys.
//   score[r, j] = sk[j] * sum_h (w[r,h] * sq[r,h]) * max(0, q8[r,h] . k8[j])
// (scales are positive, so they leave the ReLU; a scale that is NaN counts as a
// product of zero, as max(0, NaN) does in the bf16 indexer).
#include "fp8.cuh"
#include "launch.h"

namespace lsa {
namespace {

constexpr int kThreads = 256;
constexpr int kKeysPerCta = 256;

// e4m3 code -> fp32
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)two));
  float lo, hi;
  asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n" : "=f"(lo), "=f"(hi) : "r"(h));
  return make_float2(lo, hi);
}

// One CTA: one row, 256 keys; a warp per key in turn, a lane per head.
__global__ void __launch_bounds__(kThreads) fp8_index_simple_kernel(Fp8IndexArgs a, int row0) {
  __shared__ float q[kHi][kDi + 1];
  __shared__ float wq[kHi];
  pdl_wait();
  const int r = row0 + blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PagedGeom g = paged_geom(a.rows, r, blockIdx.x == 0 && threadIdx.x == 0);
  const int64_t j0 = (int64_t)blockIdx.x * kKeysPerCta, j1 = min64(j0 + kKeysPerCta, g.nvis);
  if (j0 >= j1) return;
  for (int h = warp; h < kHi; h += kThreads / 32) {
    const uint2 v = reinterpret_cast<const uint2*>(a.q_idx + ((int64_t)r * kHi + h) * kDi)[lane];
    const uint32_t m = fold_max(absmax_bf16x2(absmax_bf16x2(0, v.x), v.y));
    const bool fin = bf16_finite(m);
    const int e = fin ? scale_exponent(m) : 0;
    const float inv = fin ? pow2i(-e) : 0.f;
    const float2 x = from_e4m3x2(fin ? e4m3x2(bf16_lo(v.x) * inv, bf16_hi(v.x) * inv) : 0);
    const float2 y = from_e4m3x2(fin ? e4m3x2(bf16_lo(v.y) * inv, bf16_hi(v.y) * inv) : 0);
    q[h][4 * lane] = x.x;
    q[h][4 * lane + 1] = x.y;
    q[h][4 * lane + 2] = y.x;
    q[h][4 * lane + 3] = y.y;
    if (lane == 0) wq[h] = fin ? a.w[(int64_t)r * kHi + h] * pow2i(e) : 0.f;
  }
  __syncthreads();
  for (int64_t j = j0 + warp; j < j1; j += kThreads / 32) {
    const int page = a.rows.block_table[(int64_t)g.seq * a.rows.max_pages + j / kPage];
    const bool ok = page_ok(page, a.rows.n_pages);
    float s = 0.f, sk = 0.f;
    if (ok) {
      const uint8_t* pg = a.key_pages + (int64_t)page * kKeyPage;
      sk = reinterpret_cast<const float*>(pg + kPage * kDi)[j % kPage];
      const uint32_t mine = reinterpret_cast<const uint32_t*>(pg + (j % kPage) * kDi)[lane];
      float d = 0.f;
      for (int c = 0; c < kDi / 4; ++c) {
        const uint32_t k4 = __shfl_sync(0xffffffffu, mine, c);
        const float2 x = from_e4m3x2(k4 & 0xffffu), y = from_e4m3x2(k4 >> 16);
        d = fmaf(q[lane][4 * c], x.x, d);
        d = fmaf(q[lane][4 * c + 1], x.y, d);
        d = fmaf(q[lane][4 * c + 2], y.x, d);
        d = fmaf(q[lane][4 * c + 3], y.y, d);
      }
      s = wq[lane] * fmaxf(d, 0.f);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s = sk == sk ? s * sk : 0.f;
    } else if (lane == 0) {
      flag_error(a.rows.err, LSA_DEVERR_PAGE);
    }
    const bool forced = j < a.n_init || j >= g.nvis - a.n_loc;
    if (lane == 0) a.scores[(int64_t)r * a.ld + j] = forced ? INFINITY : ok ? s : -INFINITY;
  }
}

}  // namespace

size_t fp8_index_ws_bytes(int n_rows, int n_seq) { return 0; }

cudaError_t launch_fp8_index(const Fp8IndexArgs& a, cudaStream_t st) {
  if (a.hist) {
    const cudaError_t e = launch_zero_words(a.hist, (size_t)a.rows.n_rows * kTopkHistStride, st);
    if (e != cudaSuccess) return e;
  }
  const unsigned nx = (unsigned)((a.rows.max_len + kKeysPerCta - 1) / kKeysPerCta);
  for (int row0 = 0; row0 < a.rows.n_rows; row0 += 65535) {
    const cudaError_t e = launch_pdl(fp8_index_simple_kernel, dim3(nx, (unsigned)min(65535, a.rows.n_rows - row0)),
                                     dim3(kThreads), 0, st, a, row0);
    if (e != cudaSuccess) return e;
    count_launches(1);
  }
  if (!a.hist) return cudaSuccess;
  TopkArgs t;
  t.scores = a.scores;
  t.ld = a.ld;
  t.pos = a.rows.pos;
  t.n_rows = a.rows.n_rows;
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

}  // namespace lsa
