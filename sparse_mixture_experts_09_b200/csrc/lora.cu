// Low-rank adapters of many requests beside a shared projection:
//   out[r] = base[r] + scale_g (x[r] a_g^T) b_g^T,  g = adapter[r].
// Contract: include/moe.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ float dot8(uint4 a, uint4 b, float s) {
  s = fmaf(lo(a.x), lo(b.x), s);
  s = fmaf(hi(a.x), hi(b.x), s);
  s = fmaf(lo(a.y), lo(b.y), s);
  s = fmaf(hi(a.y), hi(b.y), s);
  s = fmaf(lo(a.z), lo(b.z), s);
  s = fmaf(hi(a.z), hi(b.z), s);
  s = fmaf(lo(a.w), lo(b.w), s);
  return fmaf(hi(a.w), hi(b.w), s);
}

// The row's adapter, or -1.
__device__ __forceinline__ int adapter_of(const Lora& l, int64_t r) {
  const int g = l.adapter[r];
  return g >= 0 && g < l.G ? g : -1;
}

// t[r][j] = scale_g <x[r], a_g[j]> for J neighbouring j: one block per (row, J ranks), its
// threads along the features.
template <int J>
__global__ void __launch_bounds__(kThreads) k_shrink_rows(const Lora l, float* __restrict__ t) {
  pdl_trigger();
  pdl_wait();
  __shared__ float s_sum[J][kThreads / 32];
  const int per_row = l.rank / J;
  const int64_t r = blockIdx.x / per_row;
  const int j0 = (int)(blockIdx.x - r * per_row) * J;
  const int g = adapter_of(l, r);
  if (g < 0) return;
  const uint4* x = reinterpret_cast<const uint4*>(l.x + r * l.x_stride);
  const uint4* a = reinterpret_cast<const uint4*>(l.a + ((int64_t)g * l.rank + j0) * l.H);
  const int vecs = l.H >> 3;
  float sum[J];
#pragma unroll
  for (int j = 0; j < J; ++j) sum[j] = 0.f;
#pragma unroll 4
  for (int i = threadIdx.x; i < vecs; i += kThreads) {
    const uint4 xv = __ldg(x + i);
#pragma unroll
    for (int j = 0; j < J; ++j) sum[j] = dot8(xv, __ldg(a + (int64_t)j * vecs + i), sum[j]);
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
    if ((threadIdx.x & 31) == 0) s_sum[j][threadIdx.x >> 5] = sum[j];
  }
  __syncthreads();
  if (threadIdx.x < J) {
    float all = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) all += s_sum[threadIdx.x][w];
    t[r * l.rank + j0 + threadIdx.x] = all * (l.scale ? l.scale[g] : 1.f);
  }
}

template <typename T>
__device__ __forceinline__ float load_out(const T* p) {
  return (float)*p;
}
__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// out[r][n] = base[r][n] + <t[r], b_g[n]>. P lanes share an output column (P the power of two
// from rank / 8 up), each 8 ranks of it in one 16-byte load; a warp takes 32 columns at a
// time, P of them per lane group, and adds with a butterfly that leaves one column in
// every lane.
template <typename T, int P>
__global__ void __launch_bounds__(kThreads) k_expand_rows(const Lora l, const float* __restrict__ t,
                                                          int blocks_per_row) {
  pdl_trigger();
  pdl_wait();
  const int64_t r = blockIdx.x / blocks_per_row;
  const int first = (int)(blockIdx.x - r * blocks_per_row) * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int part = lane % P, col = lane / P;
  const T* base = static_cast<const T*>(l.base) + r * l.base_stride;
  T* out = static_cast<T*>(l.out) + r * l.out_stride;
  const int g = adapter_of(l, r);
  const int step = blocks_per_row * (kThreads / 32) * 32;
  if (g < 0) {
    if (static_cast<const void*>(base) != static_cast<const void*>(out))
      for (int n = first * 32 + lane; n < l.N; n += step) out[n] = base[n];
    return;
  }
  const bool in = part * 8 < l.rank;
  float tv[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) tv[q] = in ? t[r * l.rank + part * 8 + q] : 0.f;
  const __nv_bfloat16* b0 = reinterpret_cast<const __nv_bfloat16*>(l.b) + (int64_t)g * l.N * l.rank;
  for (int n0 = first * 32; n0 < l.N; n0 += step) {
    uint4 bv[P];
#pragma unroll
    for (int u = 0; u < P; ++u) {
      const int n = n0 + u * (32 / P) + col;
      bv[u] = make_uint4(0, 0, 0, 0);
      if (in && n < l.N)
        bv[u] = __ldg(reinterpret_cast<const uint4*>(b0 + (int64_t)n * l.rank + part * 8));
    }
    const int mine = n0 + part * (32 / P) + col;
    const float was = mine < l.N ? load_out(base + mine) : 0.f;
    float sum[P];
#pragma unroll
    for (int u = 0; u < P; ++u) {
      const uint32_t q[4] = {bv[u].x, bv[u].y, bv[u].z, bv[u].w};
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s = fmaf(tv[2 * i], lo(q[i]), s);
        s = fmaf(tv[2 * i + 1], hi(q[i]), s);
      }
      sum[u] = s;
    }
    // lane `part` ends with column u = part: halve the columns held at each step
#pragma unroll
    for (int o = P / 2; o > 0; o >>= 1) {
      const bool upper = part & o;
#pragma unroll
      for (int u = 0; u < o; ++u) {
        const float give = upper ? sum[u] : sum[u + o];
        const float keep = upper ? sum[u + o] : sum[u];
        sum[u] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
    if (mine < l.N) store_out(out + mine, was + sum[0]);
  }
}

template <typename T>
cudaError_t expand_rows(const Lora& l, const float* t, cudaStream_t st) {
  const int blocks_per_row = (l.N + 32 * (kThreads / 32) - 1) / (32 * (kThreads / 32));
  const dim3 grid((unsigned)(l.R * blocks_per_row)), block(kThreads);
  if (l.rank <= 8) return launch_pdl(k_expand_rows<T, 1>, grid, block, 0, st, l, t, blocks_per_row);
  if (l.rank <= 16) return launch_pdl(k_expand_rows<T, 2>, grid, block, 0, st, l, t, blocks_per_row);
  if (l.rank <= 32) return launch_pdl(k_expand_rows<T, 4>, grid, block, 0, st, l, t, blocks_per_row);
  if (l.rank <= 64) return launch_pdl(k_expand_rows<T, 8>, grid, block, 0, st, l, t, blocks_per_row);
  return launch_pdl(k_expand_rows<T, 16>, grid, block, 0, st, l, t, blocks_per_row);
}

}  // namespace

size_t lora_workspace(const Lora& l) { return ((size_t)l.R * l.rank * 4 + 255) / 256 * 256 + 256; }

cudaError_t launch_lora(const Lora& l, void* ws, cudaStream_t st) {
  float* t = static_cast<float*>(ws);
  // ranks per block: more blocks for few rows, fewer passes over x for many
  const int64_t pairs = l.R * l.rank;
  const int64_t want = (int64_t)num_sms() * 2;
  const dim3 block(kThreads);
  cudaError_t e;
  if (pairs <= want)
    e = launch_pdl(k_shrink_rows<1>, dim3((unsigned)pairs), block, 0, st, l, t);
  else if (pairs <= 4 * want)
    e = launch_pdl(k_shrink_rows<2>, dim3((unsigned)(pairs / 2)), block, 0, st, l, t);
  else
    e = launch_pdl(k_shrink_rows<8>, dim3((unsigned)(pairs / 8)), block, 0, st, l, t);
  if (e != cudaSuccess) return e;
  return l.fp32 ? expand_rows<float>(l, t, st) : expand_rows<__nv_bfloat16>(l, t, st);
}

}  // namespace moe
