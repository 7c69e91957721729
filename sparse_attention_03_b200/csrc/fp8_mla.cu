// Sparse absorbed-latent MLA over paged 8-bit latent rows.
//   x_i = scale * s_i * (q . c_i),  out = sum_i softmax(x)_i s_i c_i[:512]
#include "fp8.cuh"
#include "launch.h"

namespace lsa {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 16;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)two));
  float lo, hi;
  asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n" : "=f"(lo), "=f"(hi) : "r"(h));
  return make_float2(lo, hi);
}

struct Smem {
  float q[kH][kDLat + 1];
  float c[kTile][kDLat + 1];  // key rows times their scale
  float p[kTile][kH];
  float m[kH], l[kH], alpha[kH];
  int there[kTile];
};

// One CTA per (row, sub-block): tiles of 16 keys as fp32 in shared memory, online softmax.
__global__ void __launch_bounds__(kThreads) fp8_mla_simple_kernel(Fp8MlaArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  pdl_wait();
  const int z = blockIdx.y, tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  const PagedGeom g = paged_geom(a.rows, (int)r, z == 0 && tid == 0);
  if (g.pad) return;
  int64_t n = g.nvis;
  if (a.idx && g.seq >= 0) {
    n = a.count[r];
    if (n < 0 || n > a.topk) {
      if (z == 0 && tid == 0) flag_error(a.rows.err, LSA_DEVERR_COUNT);
      n = max64(0, min64(n, a.topk));
    }
  }
  for (int i = tid; i < kH * kDLat; i += kThreads)
    sm.q[i / kDLat][i % kDLat] = __uint_as_float((uint32_t)a.q[z][r * kH * kDLat + i] << 16);
  if (tid < kH) {
    sm.m[tid] = -INFINITY;
    sm.l[tid] = 0.f;
  }
  float o[kH * 2];  // dims tid, tid + 256 of every head
#pragma unroll
  for (int i = 0; i < kH * 2; ++i) o[i] = 0.f;
  for (int64_t t0 = 0; t0 < n; t0 += kTile) {
    __syncthreads();
    for (int i = tid; i < kTile * 18; i += kThreads) {
      const int k = i / 18, part = i % 18;  // 32 codes of a key
      int64_t key = -1;
      if (t0 + k < n) {
        key = a.idx ? a.idx[r * a.topk + t0 + k] : t0 + k;
        if (key < 0 || key >= g.nvis) {
          if (part == 0) flag_error(a.rows.err, LSA_DEVERR_INDEX);
          key = -1;
        }
      }
      if (key >= 0) {
        const int page = a.rows.block_table[(int64_t)g.seq * a.rows.max_pages + key / kPage];
        if (page_ok(page, a.rows.n_pages)) {
          const uint8_t* row = a.lat[z] + ((int64_t)page * kPage + key % kPage) * kLatRow;
          const float s = *reinterpret_cast<const float*>(row + kDLat);
          for (int c = 0; c < 8; ++c) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(row + part * 32 + 4 * c);
            const float2 x = from_e4m3x2(w & 0xffffu), y = from_e4m3x2(w >> 16);
            float* d = &sm.c[k][part * 32 + 4 * c];
            d[0] = x.x * s;
            d[1] = x.y * s;
            d[2] = y.x * s;
            d[3] = y.y * s;
          }
        } else {
          if (part == 0) flag_error(a.rows.err, LSA_DEVERR_PAGE);
          key = -1;
        }
      }
      if (part == 0) sm.there[k] = key >= 0;
    }
    __syncthreads();
    for (int i = tid; i < kTile * kH; i += kThreads) {
      const int k = i / kH, h = i % kH;
      float d = -INFINITY;
      if (sm.there[k]) {
        d = 0.f;
        for (int e = 0; e < kDLat; ++e) d = fmaf(sm.q[h][e], sm.c[k][e], d);
        d *= a.scale * kLog2e;
      }
      sm.p[k][h] = d;
    }
    __syncthreads();
    if (tid < kH) {
      float m = sm.m[tid];
      for (int k = 0; k < kTile; ++k)
        if (sm.there[k]) m = sm.p[k][tid] > m || !(sm.p[k][tid] == sm.p[k][tid]) ? sm.p[k][tid] : m;
      const float al = sm.m[tid] == -INFINITY ? 0.f : exp2f(sm.m[tid] - m);
      float l = sm.l[tid] * al;
      for (int k = 0; k < kTile; ++k) {
        const float p = sm.there[k] ? exp2f(sm.p[k][tid] - m) : 0.f;
        sm.p[k][tid] = p;
        l += p;
      }
      sm.m[tid] = m;
      sm.l[tid] = l;
      sm.alpha[tid] = al;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      o[2 * h] *= sm.alpha[h];
      o[2 * h + 1] *= sm.alpha[h];
    }
    for (int k = 0; k < kTile; ++k) {
      if (!sm.there[k]) continue;
      const float v0 = sm.c[k][tid], v1 = sm.c[k][tid + 256];
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        o[2 * h] = fmaf(sm.p[k][h], v0, o[2 * h]);
        o[2 * h + 1] = fmaf(sm.p[k][h], v1, o[2 * h + 1]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < kH; ++h) {
    const float il = n > 0 && sm.l[h] != 0.f ? 1.f / sm.l[h] : 0.f;
    uint16_t* og = a.out[z] + (r * kH + h) * kDV;
    og[tid] = (uint16_t)bf16x2_rn(o[2 * h] * il, 0.f);
    og[tid + 256] = (uint16_t)bf16x2_rn(o[2 * h + 1] * il, 0.f);
  }
  if (a.lse[z] && tid < kH) a.lse[z][r * kH + tid] = sm.l[tid] != 0.f ? (sm.m[tid] + log2f(sm.l[tid])) * kLn2 : -INFINITY;
}

}  // namespace

size_t fp8_mla_ws_bytes(int n_rows, int n_sub, int64_t max_list) { return 0; }

cudaError_t launch_fp8_mla(const Fp8MlaArgs& a, cudaStream_t st) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(fp8_mla_simple_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const cudaError_t e = launch_pdl(fp8_mla_simple_kernel, dim3((unsigned)a.rows.n_rows, (unsigned)a.n_sub), dim3(kThreads), sizeof(Smem), st, a);
  count_launches(1);
  return e;
}

}  // namespace lsa
