// The experts' activation on its own, and the adapter of every routed row.
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_internal.h"

namespace moe {
namespace {

__device__ __forceinline__ uint32_t pack(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.f + expf(-g)) * u; }

// One thread per 8 neighbouring values: 64 bytes in, 16 out, bound by HBM.
__global__ void __launch_bounds__(256) k_swiglu_rows(const float4* __restrict__ gate,
                                                     const float4* __restrict__ up,
                                                     const int32_t* __restrict__ offsets, int E,
                                                     int64_t rows, int vecs, uint4* __restrict__ h) {
  pdl_trigger();
  pdl_wait();
  const int64_t used = offsets[E] < rows ? offsets[E] : rows;
  const int64_t n = used * vecs;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    const float4 g0 = __ldcs(gate + 2 * i), g1 = __ldcs(gate + 2 * i + 1);
    const float4 u0 = __ldcs(up + 2 * i), u1 = __ldcs(up + 2 * i + 1);
    h[i] = make_uint4(pack(swiglu(g0.x, u0.x), swiglu(g0.y, u0.y)),
                      pack(swiglu(g0.z, u0.z), swiglu(g0.w, u0.w)),
                      pack(swiglu(g1.x, u1.x), swiglu(g1.y, u1.y)),
                      pack(swiglu(g1.z, u1.z), swiglu(g1.w, u1.w)));
  }
}

__global__ void __launch_bounds__(256) k_lora_row_ids(const int32_t* __restrict__ token_of_row,
                                                      const int32_t* __restrict__ offsets,
                                                      const int32_t* __restrict__ adapter, int64_t T,
                                                      int64_t rows, int E, int G,
                                                      int32_t* __restrict__ row_adapter) {
  pdl_trigger();
  pdl_wait();
  const int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= rows) return;
  int id = -1;
  if (r < offsets[E]) {
    const int t = token_of_row[r];
    if (t >= 0 && t < T) {
      int lo = 0, hi = E;  // the group that holds r: the last whose offset is at most r
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        (offsets[mid] <= r ? lo : hi) = mid;
      }
      const int a = adapter[t];
      if (a >= 0 && a < G) id = a * E + lo;
    }
  }
  row_adapter[r] = id;
}

}  // namespace

cudaError_t launch_swiglu_rows(const float* gate, const float* up, const int32_t* offsets, int E,
                               int64_t rows, int I, uint16_t* h, cudaStream_t st) {
  const int64_t n = rows * (I / 8);
  int64_t blocks = (n + 255) / 256;
  const int64_t cap = (int64_t)num_sms() * 16;
  if (blocks > cap) blocks = cap;
  return launch_pdl(k_swiglu_rows, dim3((unsigned)blocks), dim3(256), 0, st,
                    reinterpret_cast<const float4*>(gate), reinterpret_cast<const float4*>(up),
                    offsets, E, rows, I / 8, reinterpret_cast<uint4*>(h));
}

cudaError_t launch_lora_rows(const int32_t* token_of_row, const int32_t* offsets,
                             const int32_t* adapter, int64_t T, int64_t rows, int E, int G,
                             int32_t* row_adapter, cudaStream_t st) {
  return launch_pdl(k_lora_row_ids, dim3((unsigned)((rows + 255) / 256)), dim3(256), 0, st,
                    token_of_row, offsets, adapter, T, rows, E, G, row_adapter);
}

}  // namespace moe
