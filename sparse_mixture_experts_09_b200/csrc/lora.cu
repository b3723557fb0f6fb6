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

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

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

// ---- few rows: one cluster of 8 blocks per row, one launch ----

constexpr int kCluster = 8;

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ float load_out(float v) { return v; }
__device__ __forceinline__ float load_out(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Block c of a row's cluster takes the c-th eighth of the features for all ranks (a warp
// per rank), leaves its sums in every block's shared memory, and after the cluster's barrier
// each block adds the eighths in order and takes every eighth run of 256 columns. Both
// products stream the row's adapter once; a second launch, its gap and a workspace between them
// would cost more than the work of few rows. The first columns' b and base are
// loaded before the barrier.
//
// Columns: P lanes share one (P the power of two from rank / 8 up), each 8 ranks of it in one
// 16-byte load; a warp takes 32 columns at a time, P of them per lane group, and adds with a
// butterfly that leaves one column in every lane.
//
// Bound by latency, then by the adapters' bytes: 2 rows, rank 16, 14336 -> 4096 features 6.1 us;
// 61 rows of 128 adapters, 4096 -> 14336 11.8 us, 32.7 MB, 2.8 TB/s.
template <typename T, int P>
__global__ void __launch_bounds__(kThreads) k_lora_rows(const Lora l) {
  pdl_trigger();
  pdl_wait();
  __shared__ float s_part[kCluster][128];
  constexpr int kWarps = kThreads / 32;
  const int64_t r = blockIdx.x / kCluster;
  const int c = (int)(blockIdx.x % kCluster);  // the block's rank in its cluster
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* base = static_cast<const T*>(l.base) + r * l.base_stride;
  T* out = static_cast<T*>(l.out) + r * l.out_stride;
  const int step = kCluster * kWarps * 32;
  int n0 = (c * kWarps + warp) * 32;
  const int g = adapter_of(l, r);
  if (g < 0) {  // the whole cluster
    if (l.base != l.out)
      for (int n = n0 + lane; n < l.N; n += step) out[n] = base[n];
    return;
  }
  // every block of the cluster runs before any writes to its shared memory
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int vecs = l.H >> 3, per = (vecs + kCluster - 1) / kCluster;
  const int v0 = c * per, v1 = v0 + per < vecs ? v0 + per : vecs;
  const uint4* x = reinterpret_cast<const uint4*>(l.x + r * l.x_stride);
  const uint4* a = reinterpret_cast<const uint4*>(l.a + (int64_t)g * l.rank * l.H);
  float sums[128 / kWarps];
#pragma unroll
  for (int q = 0; q < 128 / kWarps; q += 2) {
    const int j = warp + q * kWarps;
    sums[q] = sums[q + 1] = 0.f;
    if (j < l.rank) {  // rank is a multiple of 8: the pair's second is j + 8
      const bool two = j + kWarps < l.rank;
      const uint4* a0 = a + (int64_t)j * vecs;
      const uint4* a1 = two ? a0 + (int64_t)kWarps * vecs : a0;
      float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
      for (int i = v0 + lane; i < v1; i += 32) {
        const uint4 xv = __ldg(x + i), q0 = __ldg(a0 + i), q1 = __ldg(a1 + i);
        s0 = dot8(xv, q0, s0);
        s1 = dot8(xv, q1, s1);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s0 += __shfl_xor_sync(0xffffffffu, s0, o);
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      }
      sums[q] = s0;
      sums[q + 1] = s1;
    }
  }
  const int part = lane % P, col = lane / P;
  const bool in = part * 8 < l.rank;
  const uint16_t* b0 = l.b + (int64_t)g * l.N * l.rank;
  uint4 bv[P];
  const auto load_b = [&](int n0) {
#pragma unroll
    for (int u = 0; u < P; ++u) {
      const int n = n0 + u * (32 / P) + col;
      bv[u] = make_uint4(0, 0, 0, 0);
      if (in && n < l.N)
        bv[u] = __ldg(reinterpret_cast<const uint4*>(b0 + (int64_t)n * l.rank + part * 8));
    }
  };
  load_b(n0);
  int mine = n0 + part * (32 / P) + col;
  float was = mine < l.N ? load_out(base[mine]) : 0.f;
  const float scale = l.scale ? l.scale[g] : 1.f;
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  // lane q < 8 hands the warp's sums to block q
  if (lane < kCluster) {
    uint32_t there;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_addr(&s_part[c][warp])), "r"(lane));
#pragma unroll
    for (int q = 0; q < 128 / kWarps; ++q)
      if (warp + q * kWarps < l.rank)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there + q * kWarps * 4), "f"(sums[q]) : "memory");
  }
  cluster_sync();
  float tv[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float s = 0.f;
    if (in) {
#pragma unroll
      for (int w = 0; w < kCluster; ++w) s += s_part[w][part * 8 + q];
    }
    tv[q] = s * scale;
  }
  while (n0 < l.N) {
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
    const float before = was;
    const int here = mine;
    n0 += step;
    if (n0 < l.N) {  // the next columns, while these are added up
      load_b(n0);
      mine = n0 + part * (32 / P) + col;
      was = mine < l.N ? load_out(base[mine]) : 0.f;
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
    if (here < l.N) store_out(out + here, before + sum[0]);
  }
}

template <typename T, int P>
cudaError_t run_rows(const Lora& l, cudaStream_t st) {
  return launch_cluster(k_lora_rows<T, P>, (unsigned)(l.R * kCluster), kThreads, 0, kCluster, st, l);
}

template <typename T>
cudaError_t few_rows(const Lora& l, cudaStream_t st) {
  if (l.rank <= 8) return run_rows<T, 1>(l, st);
  if (l.rank <= 16) return run_rows<T, 2>(l, st);
  if (l.rank <= 32) return run_rows<T, 4>(l, st);
  if (l.rank <= 64) return run_rows<T, 8>(l, st);
  return run_rows<T, 16>(l, st);
}

// ---- many rows: tiles of up to 64 rows of one adapter on the matrix pipe ----
//
// Three launches. k_plan sorts the rows by adapter and cuts each adapter's rows into
// tiles. k_shrink_tiles forms x a^T per tile and slice of the features (slices keep the
// GPU busy when there are few tiles). k_expand_tiles adds the slices up, and streams base
// to out with t b^T on the way. Rows are independent in a matrix product and every sum's
// order is fixed by the sizes, so the order within a tile does not show in the result.
//
// The work is bound by HBM: out and base at 2 or 4 bytes an element against 2 * rank
// operations (times the parts of t, below), so mma.sync, whose fragments feed straight
// from shared memory and whose sums lie in registers beside base, is fast enough:
// with two thirds of the products left out the expand takes the same time.
// 4096 rows of 16 adapters, rank 64, 4096 -> 14336 features, fp32: 120 us (plan 6, shrink 18,
// expand 96, which moves 470 MB at 4.9 TB/s; the floor of all is 82 us).

constexpr int kTileRows = 64;
constexpr int kChunkK = 64;    // features per stage of the shrink
constexpr int kStages = 4;     // of the shrink
constexpr int kGroupN = 32;    // columns per step of a group of 4 warps of the expand
// Of the expand, by the output's bytes and RP: groups of a block, steps in flight beside the one
// at work, blocks an SM. As the shared memory has room for, at 16 warps an SM.
struct Expand {
  int groups, ahead, blocks;
};
__host__ __device__ constexpr Expand expand_of(int out_bytes, int RP) {
  return RP == 128 ? (out_bytes == 4 ? Expand{4, 1, 1} : Expand{2, 2, 2})
                   : (out_bytes == 4 ? Expand{2, 2, 2} : Expand{2, 3, 2});
}
constexpr int kMaxSlices = 8;  // of the features

// In the workspace: the tiles {adapter or -1, first sorted row, rows, 0}, their count, the
// sorted row numbers, and t = scale x a^T in bf16 parts [part][R + 64][RP], rows as sorted (a
// tile's copy of 64 rows runs into the next tile's and, for the last, past R).
struct Plan {
  int4* tiles;
  int32_t* count;
  int32_t* order;
  uint16_t* t;
};

__host__ __device__ inline int64_t max_tiles(int64_t R, int G) {
  const int64_t groups = G + 1 < R ? G + 1 : R;
  return (R + kTileRows - 1) / kTileRows + groups;
}

// Counting sort of the rows by adapter, one block: rows without an adapter form group G.
// A warp of one adapter adds once (runs of a request are the common case). A row's place in its
// group is known from the counting; later rounds leave it where t will be. 4096 rows 6 us, 7 where
// 64 adapters alternate (12 with the lanes matched, and the places found by a second count).
__global__ void __launch_bounds__(1024, 1) k_plan(const Lora l, Plan p) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ int32_t s_cursor[];  // [G + 1] counts, then each group's start
  __shared__ int32_t s_rows[32], s_tiles[32];
  const int groups = l.G + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int g = threadIdx.x; g < groups; g += 1024) s_cursor[g] = 0;
  __syncthreads();
  constexpr int kKept = 4;  // rounds whose groups and places stay in registers
  int kept[kKept], place[kKept];
  int32_t* places = reinterpret_cast<int32_t*>(p.t);  // [R]: t has 64 bytes a row or more
  const auto group_of = [&](int r) {  // R is at most 2^24
    if (r >= l.R) return -1;
    const int g = l.adapter[r];
    return g >= 0 && g < l.G ? g : l.G;
  };
#pragma unroll
  for (int i = 0; i < kKept; ++i) kept[i] = group_of(i * 1024 + threadIdx.x);
  const int rounds = (int)((l.R + 1023) / 1024);
  const auto count = [&](int g) {
    if (!__all_sync(0xffffffffu, g == __shfl_sync(0xffffffffu, g, 0)))
      return g >= 0 ? atomicAdd(&s_cursor[g], 1) : 0;
    int at = 0;
    if (g >= 0 && lane == 0) at = atomicAdd(&s_cursor[g], 32);
    return __shfl_sync(0xffffffffu, at, 0) + lane;
  };
#pragma unroll
  for (int i = 0; i < kKept; ++i)
    if (i < rounds) place[i] = count(kept[i]);
  for (int i = kKept; i < rounds; ++i) {
    const int r = i * 1024 + threadIdx.x;
    const int at = count(group_of(r));
    if (r < l.R) places[r] = at;
  }
  __syncthreads();
  // exclusive prefixes of rows and tiles over the groups: `per` neighbouring groups a thread
  const int per = (groups + 1023) / 1024;
  const int g0 = threadIdx.x * per, g1 = g0 + per < groups ? g0 + per : groups;
  int rows = 0, tiles = 0;
  for (int g = g0; g < g1; ++g) {
    rows += s_cursor[g];
    tiles += (s_cursor[g] + kTileRows - 1) / kTileRows;
  }
  int row_at = rows, tile_at = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, row_at, o);
    const int b = __shfl_up_sync(0xffffffffu, tile_at, o);
    if (lane >= o) {
      row_at += a;
      tile_at += b;
    }
  }
  if (lane == 31) {
    s_rows[warp] = row_at;
    s_tiles[warp] = tile_at;
  }
  __syncthreads();
  int row_base = 0, tile_base = 0;
  for (int w = 0; w < warp; ++w) {
    row_base += s_rows[w];
    tile_base += s_tiles[w];
  }
  row_at += row_base - rows;
  tile_at += tile_base - tiles;
  if (threadIdx.x == 1023) *p.count = tile_at + tiles;
  for (int g = g0; g < g1; ++g) {
    const int n = s_cursor[g];
    s_cursor[g] = row_at;  // where the group starts
    for (int i = 0; i < n; i += kTileRows)
      p.tiles[tile_at++] = make_int4(g < l.G ? g : -1, row_at + i, n - i < kTileRows ? n - i : kTileRows, 0);
    row_at += n;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kKept; ++i)
    if (kept[i] >= 0) p.order[s_cursor[kept[i]] + place[i]] = i * 1024 + threadIdx.x;
  for (int i = kKept; i < rounds; ++i) {
    const int r = i * 1024 + threadIdx.x;
    if (r < l.R) p.order[s_cursor[group_of(r)] + places[r]] = r;
  }
}

// 16 bytes from global to shared memory; zeros when !in (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One tile and slice of the features: 4 warps of 16 rows each by RP ranks (RP: rank rounded up
// to 16, 32, 64 or 128). x and a come in stages of 64 features by 16-byte asynchronous
// copies, their 16-byte pieces swizzled by the row. The matrix pipe's own sums are
// truncated, not rounded, at each step, so they run over one stage only (4 steps) and are
// added to the running sums by ordinary additions. The slices of a tile are a cluster: its
// blocks add them up through distributed shared memory and cut t = scale x a^T into bf16 parts whose sum holds it to 2^-24 (3 parts, fp32 out) or
// 2^-16 (2 parts, bf16 out: far below its one rounding).
template <int RP>
__global__ void __launch_bounds__(128) k_shrink_tiles(const Lora l, const Plan p, int slices) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kStageBytes = (kTileRows + RP) * kChunkK * 2;
  const int tile = blockIdx.x / slices, slice = blockIdx.x - tile * slices;
  if (tile >= *p.count) return;
  const int4 tl = p.tiles[tile];
  if (tl.x < 0) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunks = (l.H + kChunkK - 1) / kChunkK, per = (chunks + slices - 1) / slices;
  const int c0 = slice * per, c1 = c0 + per < chunks ? c0 + per : chunks;
  // this thread's pieces: column piece tid % 8 of rows tid / 8 + 16 i
  const int piece = tid & 7, row0 = tid >> 3;
  const uint16_t* xs[kTileRows / 16];
  bool x_in[kTileRows / 16];
#pragma unroll
  for (int i = 0; i < kTileRows / 16; ++i) {
    const int r = row0 + 16 * i;
    x_in[i] = r < tl.z;
    xs[i] = l.x + (x_in[i] ? (int64_t)p.order[tl.y + r] * l.x_stride : 0);
  }
  const uint16_t* as = l.a + (int64_t)tl.x * l.rank * l.H;
  const uint32_t base = smem_addr(smem);
  auto load = [&](int c, int stage) {
    const int col = c * kChunkK + piece * 8;
    const bool in = c < c1 && col < l.H;
    const uint32_t st = base + stage * kStageBytes;
#pragma unroll
    for (int i = 0; i < kTileRows / 16; ++i) {
      const int r = row0 + 16 * i;
      const bool ok = in && x_in[i];
      copy16(st + r * 128 + ((piece ^ (r & 7)) << 4), ok ? xs[i] + col : l.x, ok);
    }
#pragma unroll
    for (int i = 0; i < RP / 16; ++i) {
      const int r = row0 + 16 * i;
      const bool ok = in && r < l.rank;
      copy16(st + (kTileRows + r) * 128 + ((piece ^ (r & 7)) << 4),
             ok ? as + (int64_t)r * l.H + col : l.a, ok);
    }
    copies_end();
  };
  float sum[RP / 8][4];
#pragma unroll
  for (int n = 0; n < RP / 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[n][i] = 0.f;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load(c0 + s, s);
  for (int c = c0; c < c1; ++c) {
    copies_wait<kStages - 2>();
    __syncthreads();
    load(c + kStages - 1, (c - c0 + kStages - 1) % kStages);
    if (warp * 16 >= tl.z) continue;  // none of the tile's rows
    const uint32_t xt = base + ((c - c0) % kStages) * kStageBytes, at = xt + kTileRows * 128;
    float acc[RP / 8][4];
#pragma unroll
    for (int n = 0; n < RP / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
#pragma unroll
    for (int kk = 0; kk < kChunkK / 16; ++kk) {
      uint32_t xf[4];
      const int xr = warp * 16 + (lane & 15);
      ldsm4(xf, xt + xr * 128 + (((kk * 2 + (lane >> 4)) ^ (xr & 7)) << 4));
#pragma unroll
      for (int n = 0; n < RP / 16; ++n) {
        uint32_t bf[4];
        const int ar = n * 16 + (lane & 7) + ((lane >> 4) << 3);
        ldsm4(bf, at + ar * 128 + (((kk * 2 + ((lane >> 3) & 1)) ^ (ar & 7)) << 4));
        mma(acc[2 * n], xf, bf[0], bf[1]);
        mma(acc[2 * n + 1], xf, bf[2], bf[3]);
      }
    }
#pragma unroll
    for (int n = 0; n < RP / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[n][i] += acc[n][i];
  }
  copies_wait<0>();
  // the slices, in their order: each block of the cluster adds up a share of the tile
  __syncthreads();
  float* mine = reinterpret_cast<float*>(smem);  // [64][RP]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = warp * 16 + (lane >> 2) + 8 * h;
    float2* o = reinterpret_cast<float2*>(mine + r * RP + (lane & 3) * 2);
#pragma unroll
    for (int n = 0; n < RP / 8; ++n) o[n * 4] = make_float2(sum[n][2 * h], sum[n][2 * h + 1]);
  }
  cluster_sync();
  const float scale = l.scale ? l.scale[tl.x] : 1.f;
  const int parts = l.fp32 ? 3 : 2;
  for (int i = slice * 128 + tid; i < kTileRows * RP / 4; i += 128 * slices) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kMaxSlices; ++s) {
      if (s >= slices) break;
      uint32_t at;
      float4 q;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(base + i * 16), "r"(s));
      asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(q.x), "=f"(q.y), "=f"(q.z), "=f"(q.w) : "r"(at) : "memory");
      v[0] += q.x;
      v[1] += q.y;
      v[2] += q.z;
      v[3] += q.w;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) v[n] *= scale;
    if (i / (RP / 4) >= tl.z) continue;
    uint16_t* t = p.t + (int64_t)tl.y * RP + i * 4;
    for (int part = 0; part < parts; ++part, t += (l.R + kTileRows) * RP) {
      const uint2 both = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
      *reinterpret_cast<uint2*>(t) = both;
      v[0] -= lo(both.x);
      v[1] -= hi(both.x);
      v[2] -= lo(both.y);
      v[3] -= hi(both.y);
    }
  }
  cluster_sync();  // no block leaves while another reads its sums
}

// Sixteen bytes of the output in floats, and back (one rounding for bf16).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ void get(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  static __device__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ void get(const uint4& v, float (&f)[8]) {
    f[0] = lo(v.x), f[1] = hi(v.x), f[2] = lo(v.y), f[3] = hi(v.y);
    f[4] = lo(v.z), f[5] = hi(v.z), f[6] = lo(v.w), f[7] = hi(v.w);
  }
  static __device__ uint4 put(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
};

// out = base + t b^T. The tiles' steps of 32 columns a group, in a row, are cut evenly among as
// many blocks as run at once; a block takes its steps tile by tile. A group of 4 warps (16 rows
// each) has its own columns, copies and barrier, so that one group's products run beside
// another's copies and stores (with one barrier for all 8 warps: 125 us instead of 120 on the
// case above; with 8 warps an SM at rank 128, 4096 -> 4096 features, bf16 80 instead of 64).
// t's parts times b are exact in fp32; t's fragments stay in registers up to rank 64.
// base and b come by 16-byte asynchronous copies one to three steps ahead: what has to be in flight
// to keep HBM busy (some 50 KB an SM) would not fit the registers beside the sums. b's rows
// go to shared memory in the order in which a thread's columns of neighbouring 8-wide
// products are neighbours in out, so that out is written 16 bytes at a time.
template <typename T, int RP>
__global__ void __launch_bounds__(128 * expand_of(sizeof(T), RP).groups, expand_of(sizeof(T), RP).blocks)
    k_expand_tiles(const Lora l, const Plan p) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kParts = sizeof(T) == 4 ? 3 : 2;
  constexpr int kPitch = RP * 2 + 16;  // odd in 16-byte units: ldmatrix rows fall on distinct banks
  constexpr int kVec = Vec<T>::kN;     // columns of one 16-byte access
  constexpr int kWide = kVec / 2;      // 8-wide products that share it
  constexpr Expand kE = expand_of(sizeof(T), RP);
  constexpr int kThr = 128 * kE.groups, kChunkN = kGroupN * kE.groups;
  constexpr int kRowBytes = kGroupN * (int)sizeof(T);
  constexpr int kBaseBytes = kTileRows * kRowBytes;
  constexpr int kStepBytes = kBaseBytes + kGroupN * kPitch;
  constexpr int kPieces = RP / 8, kAhead = kE.ahead;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = warp >> 2, gtid = tid & 127;
  const T* base = static_cast<const T*>(l.base);
  T* out = static_cast<T*>(l.out);
  const int steps = (l.N + kChunkN - 1) / kChunkN;
  const int64_t units = (int64_t)*p.count * steps;
  int64_t unit = units * blockIdx.x / gridDim.x;
  const int64_t end = units * (blockIdx.x + 1) / gridDim.x;
  const uint32_t t_at = smem_addr(smem);
  const uint32_t ring = t_at + kParts * kTileRows * kPitch + group * (kAhead + 1) * kStepBytes;
  // this thread's pieces of its group's step: of base, rows `brow` + kRowStep i at one 16-byte
  // column; of b, columns (rows of b) q / kPieces at one 16-byte piece
  constexpr int kRowPieces = kRowBytes / 16, kRowStep = 128 / kRowPieces, kBase = kTileRows / kRowStep;
  const int brow = gtid / kRowPieces, bpiece = gtid % kRowPieces;
  // a quarter of a warp reads 64 bytes of two rows: where a row takes all banks, rows of odd
  // number have their halves swapped
  constexpr int kSwap = kRowBytes == 128 ? 4 : 0;
  const uint32_t base_dst = ring + brow * kRowBytes + ((bpiece ^ (brow & 1) * kSwap) << 4);
  constexpr int kB = (kGroupN * kPieces + 127) / 128;
  const int b_piece = gtid % kPieces * 8;
  const int wr = (warp & 3) * 16, wc = group * kGroupN;
  const int r0 = wr + (lane >> 2), r1 = r0 + 8;
  constexpr bool kKeep = RP <= 64;  // t's fragments stay in registers
  uint32_t kept[kKeep ? RP / 16 : 1][kParts][4];
  const uint32_t t_row = t_at + (wr + (lane & 15)) * kPitch + (lane >> 4) * 16;
  const uint32_t b_row = kBaseBytes + ((lane & 7) + ((lane >> 4) << 3)) * kPitch + ((lane >> 3) & 1) * 16;
  constexpr int kGroups = 32 / (8 * kWide);
  while (unit < end) {
    const int tile = (int)(unit / steps), first = (int)(unit - (int64_t)tile * steps);
    const int last = end - unit < steps - first ? first + (int)(end - unit) : steps;
    unit += last - first;
    const int4 tl = p.tiles[tile];
    if (tl.x < 0) {  // rows without an adapter
      if (l.base == l.out) continue;
      const int n0 = first * kChunkN, n1 = last * kChunkN < l.N ? last * kChunkN : l.N;
      const int vecs = (n1 - n0) / kVec, all = vecs * tl.z;
      for (int i0 = tid; i0 < all; i0 += kThr * 4) {  // four pieces of a thread in flight
        uint4 v[4];
        int64_t at[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int i = i0 + kThr * q;
          if (i >= all) continue;
          const int64_t r = p.order[tl.y + i / vecs];
          const int n = n0 + i % vecs * kVec;
          at[q] = r * l.out_stride + n;
          v[q] = *reinterpret_cast<const uint4*>(base + r * l.base_stride + n);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (i0 + kThr * q < all) *reinterpret_cast<uint4*>(out + at[q]) = v[q];
      }
      continue;
    }
    const T* from[kBase];
    bool row_in[kBase];
#pragma unroll
    for (int i = 0; i < kBase; ++i) {
      const int r = brow + kRowStep * i;
      row_in[i] = r < tl.z;
      from[i] = base + (row_in[i] ? (int64_t)p.order[tl.y + r] * l.base_stride : 0) + wc + bpiece * kVec;
    }
    const bool in_row[2] = {r0 < tl.z, r1 < tl.z};
    T* to[2] = {out + (in_row[0] ? (int64_t)p.order[tl.y + r0] * l.out_stride : 0),
                out + (in_row[1] ? (int64_t)p.order[tl.y + r1] * l.out_stride : 0)};
    const uint16_t* bg = l.b + (int64_t)tl.x * l.N * l.rank + b_piece;
    auto load = [&](int s, int stage) {
      const bool in = s < last;
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        const int n = (gtid + 128 * i) / kPieces;
        if (kGroupN * kPieces % 128 && n >= kGroupN) break;
        // column n = 8 kWide G + 2 kWide c + 2 w + e sits at row 8 kWide G + 8 w + 2 c + e
        const int row = n / (8 * kWide) * (8 * kWide) + (n % (2 * kWide)) / 2 * 8 +
                        (n % (8 * kWide)) / (2 * kWide) * 2 + (n & 1);
        const int col = s * kChunkN + wc + n;
        const bool ok = in && b_piece < l.rank && col < l.N;
        copy16(ring + stage * kStepBytes + kBaseBytes + row * kPitch + b_piece * 2,
               ok ? bg + (int64_t)col * l.rank : l.b, ok);
      }
      const int col = s * kChunkN + wc + bpiece * kVec;
#pragma unroll
      for (int i = 0; i < kBase; ++i) {
        const bool ok = in && row_in[i] && col < l.N;
        copy16(base_dst + stage * kStepBytes + i * kRowStep * kRowBytes,
               ok ? static_cast<const void*>(from[i] + s * kChunkN) : l.b, ok);
      }
      copies_end();
    };
    __syncthreads();  // the tile before is done with the shared memory
    const uint16_t* t = p.t + (int64_t)tl.y * RP;
#pragma unroll
    for (int i = 0; i < (kParts * kTileRows * kPieces + kThr - 1) / kThr; ++i) {
      const int q = tid + kThr * i, row = q / kPieces;  // rows of all parts, one after another
      if (q < kParts * kTileRows * kPieces)
        copy16(t_at + row * kPitch + q % kPieces * 16,
               t + ((int64_t)(row / kTileRows) * (l.R + kTileRows) + row % kTileRows) * RP + q % kPieces * 8, true);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(first + i, i);
    int stage = 0, col0 = first * kChunkN + wc + (lane & 3) * kVec;
    for (int s = first; s < last; ++s, col0 += kChunkN) {
      copies_wait<kAhead - 1>();
      if (s == first)
        __syncthreads();  // t, which all groups copied
      else
        asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
      load(s + kAhead, stage == 0 ? kAhead : stage - 1);
      if constexpr (kKeep) {
        if (s == first) {
#pragma unroll
          for (int kk = 0; kk < RP / 16; ++kk)
#pragma unroll
            for (int part = 0; part < kParts; ++part)
              ldsm4(kept[kk][part], t_row + part * kTileRows * kPitch + kk * 32);
        }
      }
      const uint32_t at = ring + stage * kStepBytes;
      // one 16-byte access's columns at a time
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        float acc[kWide][4];
#pragma unroll
        for (int w = 0; w < kWide; ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[w][i] = 0.f;
#pragma unroll
        for (int kk = 0; kk < RP / 16; ++kk) {
          uint32_t tf[kParts][4];
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            if constexpr (kKeep) {
#pragma unroll
              for (int i = 0; i < 4; ++i) tf[part][i] = kept[kk][part][i];
            } else {
              ldsm4(tf[part], t_row + part * kTileRows * kPitch + kk * 32);
            }
          }
#pragma unroll
          for (int w = 0; w < kWide; w += 2) {
            uint32_t bf[4];
            ldsm4(bf, at + b_row + (g * kWide + w) * 8 * kPitch + kk * 32);
#pragma unroll
            for (int part = kParts - 1; part >= 0; --part) {
              mma(acc[w], tf[part], bf[0], bf[1]);
              mma(acc[w + 1], tf[part], bf[2], bf[3]);
            }
          }
        }
        const int col = col0 + g * 8 * kWide;
        if (col >= l.N) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!in_row[h]) continue;
          const int row = h ? r1 : r0, piece = g * 8 * kWide / kVec + (lane & 3);
          const uint4 was = *reinterpret_cast<const uint4*>(
              smem + (at - t_at) + row * kRowBytes + ((piece ^ (row & 1) * kSwap) << 4));
          float f[kVec];
          Vec<T>::get(was, f);
#pragma unroll
          for (int w = 0; w < kWide; ++w) {
            f[2 * w] += acc[w][2 * h];
            f[2 * w + 1] += acc[w][2 * h + 1];
          }
          *reinterpret_cast<uint4*>(to[h] + col) = Vec<T>::put(f);
        }
      }
      stage = stage == kAhead ? 0 : stage + 1;
    }
    copies_wait<0>();
  }
}

int rank_pad(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// Whether the rows go by tiles. A row on its own streams its adapter again for every row; a
// tile costs as much for one row as for 64, and the sorting and two more launches some 8 us.
// Device times, rows / tiles, where the rows fall on all of the adapters: 64 rows of 4 adapters,
// rank 64, 4096 -> 14336 features 27 / 20 us, of 64 38 / 60. 4096 -> 4096 features, rank 16: 128 rows
// of 2 adapters 11.5 / 12, of 16 11.5 / 15; 256 rows of 16 20 / 16, of 64 20 / 22, of 256 23 / 39, of 1024
// 25 / 51; 512 rows of 64 36 / 23, of 256 44 / 53; rank 64: 128 rows of 16 34 / 22, of 256 45 / 52.
// How many adapters a batch uses is not known here, only how many there are: where the better
// form depends on that, the one whose worst case loses less is taken.
bool use_tiles(const Lora& l) {
  const bool light = l.R * (int64_t)l.rank * (l.H + l.N) * 2 < (int64_t)64 << 20;
  if (l.R < 128) return !light && l.R >= 12 * (int64_t)l.G;
  if (l.R < 160) return !light;
  if (l.R < 256) return !light || l.R >= 8 * (int64_t)l.G;
  if (l.R < 512 && l.rank <= 16) return l.R >= 4 * (int64_t)l.G;
  return true;
}

// Slices of the features: as many blocks as the SMs hold at once (three each; a second
// round for a few blocks would double the time), at least two stages each, and a power of
// two, as clusters of 5 to 7 blocks leave SMs empty: 4096 rows, rank 64, 4096 features
// 31 / 20 / 19 / 19 / 28 us at 1 / 2 / 4 / 6 / 8 slices, rank 128 51 / 31 / 27 / 40 / 44 us. How
// many tiles the adapters leave partly filled is not known here; twice the full ones is
// the most allowed for.
int feature_slices(const Lora& l) {
  const int64_t full = (l.R + kTileRows - 1) / kTileRows, most = max_tiles(l.R, l.G);
  const int64_t tiles = most < 2 * full ? most : 2 * full;
  const int64_t chunks = (l.H + kChunkK - 1) / kChunkK;
  int64_t s = (int64_t)num_sms() * 3 / tiles;
  if (s > chunks / 2) s = chunks / 2;
  return s >= 8 ? 8 : s >= 4 ? 4 : s >= 2 ? 2 : 1;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

Plan plan_at(const Lora& l, void* ws, size_t* end) {
  char* at = static_cast<char*>(ws);
  Plan p;
  p.count = reinterpret_cast<int32_t*>(at);
  at += 256;
  p.tiles = reinterpret_cast<int4*>(at);
  at += up256((size_t)max_tiles(l.R, l.G) * 16);
  p.order = reinterpret_cast<int32_t*>(at);
  at += up256((size_t)l.R * 4);
  p.t = reinterpret_cast<uint16_t*>(at);
  at += up256((size_t)(l.fp32 ? 3 : 2) * (l.R + kTileRows) * rank_pad(l.rank) * 2);
  *end = (size_t)(at - static_cast<char*>(ws));
  return p;
}

// A block's shared memory above 48 KB has to be asked for (1 KB is left to static arrays). The limit
// belongs to the kernel, not to the call, so calls of one kernel all ask for `most`, the most that it
// ever takes: no host thread lowers it between another's request and its launch.
template <typename F>
cudaError_t allow_smem(F* kernel, size_t bytes, size_t most) {
  if (bytes <= 47 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

template <int RP>
cudaError_t run_tiles(const Lora& l, const Plan& p, cudaStream_t st) {
  const int slices = feature_slices(l);
  const int64_t tiles = max_tiles(l.R, l.G);
  const size_t shrink_smem = (size_t)kStages * (kTileRows + RP) * kChunkK * 2;
  cudaError_t e = allow_smem(k_shrink_tiles<RP>, shrink_smem, shrink_smem);
  if (e != cudaSuccess) return e;
  e = launch_cluster(k_shrink_tiles<RP>, (unsigned)(tiles * slices), 128, shrink_smem,
                     (unsigned)slices, st, l, p, slices);
  if (e != cudaSuccess) return e;
  const int parts = l.fp32 ? 3 : 2, size = l.fp32 ? 4 : 2;
  const Expand x = expand_of(size, RP);
  const size_t smem = (size_t)parts * kTileRows * (RP * 2 + 16) +
                      (size_t)(x.ahead + 1) * x.groups * kGroupN * (kTileRows * size + RP * 2 + 16);
  const dim3 grid((unsigned)(num_sms() * x.blocks)), block(128 * x.groups);
  if (l.fp32) {
    e = allow_smem(k_expand_tiles<float, RP>, smem, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_expand_tiles<float, RP>, grid, block, smem, st, l, p);
  }
  e = allow_smem(k_expand_tiles<__nv_bfloat16, RP>, smem, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_expand_tiles<__nv_bfloat16, RP>, grid, block, smem, st, l, p);
}

}  // namespace

size_t lora_workspace(const Lora& l) {
  if (!use_tiles(l)) return 0;
  size_t end = 0;
  plan_at(l, nullptr, &end);
  return end;
}

cudaError_t launch_lora(const Lora& l, void* ws, cudaStream_t st) {
  if (use_tiles(l)) {
    size_t end = 0;
    const Plan p = plan_at(l, ws, &end);
    const size_t smem = (size_t)(l.G + 1) * 4;
    cudaError_t e = allow_smem(k_plan, smem, (size_t)(kLoraMaxAdapters + 1) * 4);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_plan, dim3(1), dim3(1024), smem, st, l, p);
    if (e != cudaSuccess) return e;
    switch (rank_pad(l.rank)) {
      case 16: return run_tiles<16>(l, p, st);
      case 32: return run_tiles<32>(l, p, st);
      case 64: return run_tiles<64>(l, p, st);
      default: return run_tiles<128>(l, p, st);
    }
  }
  return l.fp32 ? few_rows<float>(l, st) : few_rows<__nv_bfloat16>(l, st);
}

}  // namespace moe
