// Gradient of the weighted combine in the expert rows and the routing weights.
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxExperts = 512;

// Rows that no slot names where none was taken out: group e's pads are [offsets[e] + counts[e],
// offsets[e + 1]), the rows past the last group [offsets[E], rows). The starts and lengths
// of these E + 1 segments.
__device__ void segments(const CombineBwd& c, int32_t* start, int32_t* count) {
  for (int e = threadIdx.x; e <= c.E; e += kThreads) {
    const int64_t lo = e < c.E ? (int64_t)c.offsets[e] + c.counts[e] : c.offsets[c.E];
    const int64_t hi = e < c.E ? (int64_t)c.offsets[e + 1] : c.rows;
    const int64_t a = lo < 0 ? 0 : lo, b = hi > c.rows ? c.rows : hi;
    start[e] = (int32_t)a;
    count[e] = b > a ? (int32_t)(b - a) : 0;
  }
  __syncthreads();
}

// The block's threads zero every `stride`-th row of the segments, counting from `first`.
__device__ void zero_pads(const CombineBwd& c, int32_t* start, int32_t* count, int64_t first, int64_t stride) {
  segments(c, start, count);
  int64_t before = 0;  // rows of the segments before e
  int64_t next = first;
  const int vecs = c.H >> 2;
  for (int e = 0; e <= c.E; ++e) {
    for (; next < before + count[e]; next += stride) {
      float4* row = reinterpret_cast<float4*>(c.dy + (start[e] + (next - before)) * (int64_t)c.H);
      for (int i = threadIdx.x; i < vecs; i += kThreads) row[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    before += count[e];
  }
}

// A routed row whose slot was taken out (its row_of set outside the buffer) is in no segment, and
// no token block writes it. Owner `owner` of 2^shift finds those among the rows r with r % 2^shift =
// owner: it reads all of row_of (4 bytes a slot from L2, beside 12 H or so of HBM for its row), marks
// the rows that are named or in a segment, and zeroes the others, a warp to a row. 128 owners, or 16
// of up to 256 slots, where all blocks start at once and 128 more do not fit beside them: 16 tokens of
// 4096 features 5.8 us (6.7 with 128 owners, 6.1 with no search), 4096 tokens 52.5 (53.3 with none),
// 16384 tokens of 256 features with 8 slots 187 (178).
constexpr int kWindow = 1 << 15;  // rows of an owner that are marked at a time

__device__ void zero_dropped(const CombineBwd& c, int32_t* start, int32_t* count, int owner, int shift) {
  __shared__ uint32_t s_marked[kWindow / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vecs = c.H >> 2;
  const int64_t slots = c.T * c.k;
  const int owners = 1 << shift;
  int32_t r[8];
  const auto fetch = [&](int64_t i0) {
#pragma unroll
    for (int n = 0; n < 8; ++n) r[n] = i0 + n * kThreads < slots ? __ldg(c.row_of + i0 + n * kThreads) : -1;
  };
  fetch(threadIdx.x);  // on their way beside the segments' loads
  segments(c, start, count);
  for (int64_t q0 = 0; q0 * owners + owner < c.rows; q0 += kWindow) {
    const int64_t left = ((c.rows - owner + owners - 1) >> shift) - q0;
    const int here = left < kWindow ? (int)left : kWindow;
    const int words = (here + 31) / 32;
    for (int i = threadIdx.x; i < words; i += kThreads) s_marked[i] = 0;
    __syncthreads();
    const auto mark = [&](int64_t q) {
      if (q >= 0 && q < here) atomicOr(&s_marked[q >> 5], 1u << (q & 31));
    };
    for (int64_t i0 = threadIdx.x; i0 < slots; i0 += 8 * kThreads) {
      if (i0 != threadIdx.x || q0 > 0) fetch(i0);
#pragma unroll
      for (int n = 0; n < 8; ++n)
        if (r[n] >= 0 && (r[n] & (owners - 1)) == owner) mark((r[n] >> shift) - q0);
    }
    for (int e = warp; e <= c.E; e += kThreads / 32) {
      const int64_t lo = start[e], hi = lo + count[e];
      const int64_t first = (lo - owner + owners - 1) >> shift;  // the owner's first row from lo on
      for (int64_t q = (first > q0 ? first : q0) + lane; q < q0 + here && q * owners + owner < hi; q += 32) mark(q - q0);
    }
    __syncthreads();
    for (int i = warp; i < words; i += kThreads / 32) {
      uint32_t open = ~s_marked[i];
      if (here - i * 32 < 32) open &= (1u << (here - i * 32)) - 1;
      for (; open; open &= open - 1) {
        const int64_t r = (q0 + i * 32 + __ffs(open) - 1) * owners + owner;
        float4* row = reinterpret_cast<float4*>(c.dy + r * c.H);
        for (int v = lane; v < vecs; v += 32) row[v] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    __syncthreads();
  }
}

// The first `owners` blocks look for rows whose slot was taken out, the next token_blocks take a
// token each (striding), the others zero the pad rows. A token's d_out is read once for its k rows;
// a thread adds its products in fp32, then the warp and the block add in a fixed order. Bound by
// HBM: 2 H bytes of d_out and 8 H of every routed row. 4096 tokens, H 4096, 2 slots: 52 us, 6.1
// TB/s (94% of a plain copy's rate); 16 tokens 5.6 us, nearly all of it zeroing the 1120 pad rows.
template <int K>
__global__ void __launch_bounds__(kThreads) k_combine_bwd(const CombineBwd c, int shift, int token_blocks) {
  pdl_trigger();
  pdl_wait();
  const int owners = c.dy ? 1 << shift : 0;
  const int block = (int)blockIdx.x - owners;
  if (block < 0 || block >= token_blocks) {
    __shared__ int32_t s_start[kMaxExperts + 1], s_count[kMaxExperts + 1];
    if (block < 0)
      zero_dropped(c, s_start, s_count, blockIdx.x, shift);
    else
      zero_pads(c, s_start, s_count, block - token_blocks, (int64_t)gridDim.x - owners - token_blocks);
    return;
  }
  __shared__ float s_sum[K][kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int vecs = c.H >> 3;
  for (int64_t t = block; t < c.T; t += token_blocks) {
    int64_t row[K];
    float w[K], sum[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      row[j] = j < c.k ? c.row_of[t * c.k + j] : -1;
      if (row[j] >= c.rows) row[j] = -1;
      w[j] = c.dy && row[j] >= 0 ? c.w[t * c.k + j] : 0.f;
      sum[j] = 0.f;
    }
    for (int i = threadIdx.x; i < vecs; i += kThreads) {
      const uint4 d = __ldg(reinterpret_cast<const uint4*>(c.d_out + t * c.H) + i);
      float4 y[K][2];
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (c.d_w && row[j] >= 0) {
          const float4* p = reinterpret_cast<const float4*>(c.y + row[j] * c.H) + 2 * i;
          y[j][0] = __ldcs(p);
          y[j][1] = __ldcs(p + 1);
        }
      }
      const uint32_t q[4] = {d.x, d.y, d.z, d.w};
      float g[8];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        g[2 * n] = __uint_as_float(q[n] << 16);
        g[2 * n + 1] = __uint_as_float(q[n] & 0xFFFF0000u);
      }
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (row[j] < 0) continue;
        if (c.d_w) {
          const float v[8] = {y[j][0].x, y[j][0].y, y[j][0].z, y[j][0].w,
                              y[j][1].x, y[j][1].y, y[j][1].z, y[j][1].w};
#pragma unroll
          for (int n = 0; n < 8; ++n) sum[j] = fmaf(g[n], v[n], sum[j]);
        }
        if (c.dy) {
          float4* p = reinterpret_cast<float4*>(c.dy + row[j] * c.H) + 2 * i;
          __stcs(p, make_float4(w[j] * g[0], w[j] * g[1], w[j] * g[2], w[j] * g[3]));
          __stcs(p + 1, make_float4(w[j] * g[4], w[j] * g[5], w[j] * g[6], w[j] * g[7]));
        }
      }
    }
    if (!c.d_w) continue;
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
      if (lane == 0) s_sum[j][warp] = sum[j];
    }
    __syncthreads();
    if ((int)threadIdx.x < c.k) {
      float all = 0.f;
#pragma unroll
      for (int v = 0; v < kThreads / 32; ++v) all += s_sum[threadIdx.x][v];
      c.d_w[t * c.k + threadIdx.x] = all;
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_combine_bwd(const CombineBwd& c, cudaStream_t st) {
  const int64_t cap = (int64_t)num_sms() * 8;
  const int token_blocks = (int)(c.T < 4 * cap ? c.T : 4 * cap);
  // T * k of `rows` rows are named, or fewer where slots name no row; the rest bounds the zeroing blocks
  int64_t zero_blocks = 0;
  if (c.dy && c.rows > 0) {
    const int64_t unnamed = c.rows - c.T * c.k;
    zero_blocks = unnamed > cap ? cap : unnamed > 1 ? unnamed : 1;
  }
  const int shift = c.T * c.k <= 256 ? 4 : 7;
  const int owners = c.dy ? 1 << shift : 0;
  const int64_t blocks = owners + token_blocks + zero_blocks;
  if (blocks == 0) return cudaSuccess;
  const dim3 grid((unsigned)blocks), block(kThreads);
  if (c.k <= 2) return launch_pdl(k_combine_bwd<2>, grid, block, 0, st, c, shift, token_blocks);
  if (c.k <= 4) return launch_pdl(k_combine_bwd<4>, grid, block, 0, st, c, shift, token_blocks);
  return launch_pdl(k_combine_bwd<8>, grid, block, 0, st, c, shift, token_blocks);
}

}  // namespace moe
