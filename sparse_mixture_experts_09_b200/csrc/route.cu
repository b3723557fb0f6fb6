// General routing from router logits, the two router losses, and the gradient of both
// in the logits. Formulas and conventions: include/moe.h.
//
// All three kernels give a token L lanes of a warp (L = 8, 16 or 32) and each lane V
// neighbouring experts, L * V >= E: a token's logits stay in registers, and L is the
// least that holds a slot per lane with V at most 8 (16 above 256 experts), so that one
// instruction serves several tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;  // per block

__device__ __forceinline__ float logit_at(const float* p) { return __ldg(p); }
__device__ __forceinline__ float logit_at(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// NaN -> -inf, +inf -> the largest float: exp(l - max) is then 0 or finite everywhere.
__device__ __forceinline__ float clean(float l) { return l == l ? fminf(l, FLT_MAX) : -INFINITY; }

// The lanes of one token, and butterfly reductions over them.
template <int L>
struct Team {
  unsigned mask;
  int rank;  // lane within the token
  int base;  // the token's first lane
  __device__ Team() {
    const int lane = threadIdx.x & 31;
    rank = lane % L;
    base = lane - rank;
    mask = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1u) << base;
  }
  template <typename T>
  __device__ T sum(T v) const {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    return v;
  }
  __device__ float max(float v) const {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(mask, v, o));
    return v;
  }
  __device__ uint32_t max(uint32_t v) const {
    if constexpr (L == 32) {
      return __reduce_max_sync(0xffffffffu, v);
    } else {
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) {
        const uint32_t w = __shfl_xor_sync(mask, v, o);
        v = w > v ? w : v;
      }
      return v;
    }
  }
  // the largest key; among equal keys the lowest index
  __device__ void best(double& key, int& at) const {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      const double k2 = __shfl_xor_sync(mask, key, o);
      const int a2 = __shfl_xor_sync(mask, at, o);
      if (k2 > key || (k2 == key && a2 < at)) {
        key = k2;
        at = a2;
      }
    }
  }
  template <typename T>
  __device__ T from(T v, int r) const {
    return __shfl_sync(mask, v, base + r);
  }
};

// This lane's logits, cleaned; experts past E count as -inf. vec: rows start on a boundary
// of the lane's V logits (16 bytes at most) and E is a multiple of V.
template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, int rank, int E, bool vec, float (&l)[V]) {
  constexpr int kBytes = V * (int)sizeof(T);
  const int e0 = rank * V;
  if (vec && kBytes >= 4) {
    uint32_t q[(kBytes + 3) / 4];
    if (e0 < E) {
      const char* p = reinterpret_cast<const char*>(row + e0);
      if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
          q[4 * i] = v.x, q[4 * i + 1] = v.y, q[4 * i + 2] = v.z, q[4 * i + 3] = v.w;
        }
      } else if constexpr (kBytes == 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        q[0] = v.x, q[1] = v.y;
      } else {
        q[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f;
      if constexpr (sizeof(T) == 4)
        f = __uint_as_float(q[v]);
      else
        f = __uint_as_float(v & 1 ? q[v / 2] & 0xFFFF0000u : q[v / 2] << 16);
      l[v] = e0 < E ? clean(f) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = e0 + v < E ? clean(logit_at(row + e0 + v)) : -INFINITY;
  }
}

constexpr int kNone = 0x7fffffff;

// Floats as unsigned numbers of the same order (-0 as +0); every float is above 0.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((uint32_t)((int32_t)~u >> 31) | 0x80000000u));
}

// The choice in double, for tokens whose fp32 values are too close to call and for group
// values of more than two experts: one arg-max over the lanes at a time. Returns the expert
// of slot `rank`. Apart from the kernel so that its registers are not the fast path's.
template <typename T, int L, int V>
__device__ __noinline__ int choose_in_double(const Routing r, const T* row, const float* bias) {
  const Team<L> team;
  const int gs = r.E / r.groups;
  float l[V];
  double key[V];
  load_logits<T, V>(row, team.rank, r.E, false, l);
  float mx = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) mx = fmaxf(mx, l[v]);
  mx = team.max(mx);
  double total = 1.0;
  if (!r.sigmoid) {
    total = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (l[v] > -INFINITY) total += exp((double)l[v] - (double)mx);
    total = team.sum(total);
    if (total == 0.0) total = 1.0;  // no expert has a score
  }
  unsigned open = 0;  // experts of this lane that may still be chosen
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = team.rank * V + v;
    if (e >= r.E) continue;
    open |= 1u << v;
    key[v] = l[v] == -INFINITY ? 0.0
             : r.sigmoid       ? 1.0 / (1.0 + exp(-(double)l[v]))
                               : exp((double)l[v] - (double)mx) / total;
    if (bias) key[v] += (double)__ldg(bias + e);
    if (!(key[v] == key[v])) key[v] = -INFINITY;
  }
  if (r.groups > 1) {
    constexpr int kSlots = (32 + L - 1) / L;
    double value[kSlots];  // group g's value in lane g % L, slot g / L
#pragma unroll
    for (int q = 0; q < kSlots; ++q) value[q] = -INFINITY;
    for (int g = 0; g < r.groups; ++g) {
      unsigned left = open;
      double sum = 0.0;
      for (int m = 0; m < r.group_top; ++m) {
        double k1 = -INFINITY;
        int at = kNone;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int e = team.rank * V + v;
          if ((left >> v & 1u) && e / gs == g && (at == kNone || key[v] > k1)) {
            k1 = key[v];
            at = e;
          }
        }
        team.best(k1, at);
        sum += k1;
        if (at / V == team.rank) left &= ~(1u << (at % V));
      }
#pragma unroll
      for (int q = 0; q < kSlots; ++q)
        if (g == q * L + team.rank) value[q] = sum;
    }
    unsigned stay = 0;  // groups, the same in every lane
    for (int m = 0; m < r.topk_groups; ++m) {
      double k1 = -INFINITY;
      int at = kNone;
#pragma unroll
      for (int q = 0; q < kSlots; ++q) {
        const int g = q * L + team.rank;
        if (g < r.groups && !(stay >> g & 1u) && (at == kNone || value[q] > k1)) {
          k1 = value[q];
          at = g;
        }
      }
      team.best(k1, at);
      stay |= 1u << at;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if ((open >> v & 1u) && !(stay >> ((team.rank * V + v) / gs) & 1u)) open &= ~(1u << v);
  }
  if (!bias) {  // the logits order the experts
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = l[v];
  }
  int mine = -1;
  for (int j = 0; j < r.k; ++j) {
    double k1 = -INFINITY;
    int at = kNone;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if ((open >> v & 1u) && (at == kNone || key[v] > k1)) {
        k1 = key[v];
        at = team.rank * V + v;
      }
    team.best(k1, at);
    if (at / V == team.rank) open &= ~(1u << (at % V));
    if (j == team.rank) mine = at;
  }
  return mine;
}

// Routing, one team of L lanes per token. The logits alone decide where nothing else is
// asked for (both scores rise with the logit, so fp32 is exact); else the values s + bias
// and the groups' sums are formed in fp32, and a token two of whose compared values lie
// within the sums of their error bounds is chosen again in double (about one token in
// a thousand): fp32 work, decisions as in double. Bounds, u = 2^-24: a sigmoid is off by
// 4u (exponential, two ulp) + 2u, a softmax by at most 32u of the largest probability
// (exponential 4u, its argument's rounding, a sum of up to 512 terms in a tree, a
// division), and the sum with the bias by u of its value.
//
// The k largest are taken one by one: each lane keeps the largest of its own values, the
// team finds the largest of those, the lowest lane that has it gives its lowest expert.
// Bound by instructions, not bytes: a team is as narrow as 8 values per lane allow, so
// that a warp's instruction serves up to four tokens.
template <typename T, int L, int V>
__global__ void __launch_bounds__(32 * kWarps) k_route(const Routing r, const T* __restrict__ logits,
                                                       const float* __restrict__ bias, int vec,
                                                       int32_t* __restrict__ idx_out,
                                                       float* __restrict__ w_out) {
  pdl_trigger();
  pdl_wait();
  __shared__ float s_value[kWarps * 32 / L][L * V + 1];
  const Team<L> team;
  constexpr int kPer = 32 / L * kWarps;  // tokens per block
  float* value_of = s_value[threadIdx.x / L];
  const int gs = r.E / r.groups;
  const bool grouped = r.groups > 1;
  const bool scores = bias || r.group_top > 1;
  // lanes of a group: a power of two, so that they can reduce among themselves
  int lanes = L;
  while (lanes * r.groups > L) lanes >>= 1;
  const bool narrow = lanes > 0 && r.group_top <= 2;
  int bit[V];  // of each of the lane's experts' groups in `stay`
#pragma unroll
  for (int v = 0; v < V; ++v) bit[v] = grouped ? team.base + (team.rank * V + v) / gs * lanes : 0;
  for (int64_t t0 = (int64_t)blockIdx.x * kPer; t0 < r.T; t0 += (int64_t)gridDim.x * kPer) {
    const int64_t t = t0 + threadIdx.x / L;
    if (t >= r.T) continue;  // a token's lanes leave together
    const T* row = logits + t * r.stride;
    float l[V], c[V];
    load_logits<T, V>(row, team.rank, r.E, vec, l);
    float mx = -INFINITY, tol = 0.f, sum = 1.f;
    if (!r.sigmoid && (scores || !r.renorm)) {
#pragma unroll
      for (int v = 0; v < V; ++v) mx = fmaxf(mx, l[v]);
      mx = team.max(mx);
    }
    if (scores) {
      if (r.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = l[v] > -INFINITY ? 1.f / (1.f + expf(-l[v])) : 0.f;
        tol = 0x1p-20f;
      } else {
        sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          c[v] = l[v] > -INFINITY ? expf(l[v] - mx) : 0.f;
          sum += c[v];
        }
        sum = team.sum(sum);
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] *= inv;
        tol = 0x1p-18f * inv;  // the largest probability is 1 / sum
      }
      if (bias) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int e = team.rank * V + v;
          if (e < r.E) c[v] += __ldg(bias + e);
          if (!(c[v] == c[v])) c[v] = -INFINITY;
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = l[v];
    }
    bool close = false;
    unsigned stay = 0xffffffffu;  // bit base + g * lanes: group g stays
    if (grouped) {
      close = !narrow;
      if (narrow) {
        __syncwarp(team.mask);
#pragma unroll
        for (int v = 0; v < V; ++v) value_of[team.rank * V + v] = c[v];
        __syncwarp(team.mask);
        const int g = team.rank / lanes;
        float m1 = -INFINITY, m2 = -INFINITY;
        if (g < r.groups) {
          for (int i = team.rank - g * lanes; i < gs; i += lanes) {
            const float v = value_of[g * gs + i];
            m2 = fmaxf(m2, fminf(v, m1));
            m1 = fmaxf(m1, v);
          }
        }
        for (int o = lanes >> 1; o > 0; o >>= 1) {
          const float o1 = __shfl_xor_sync(team.mask, m1, o), o2 = __shfl_xor_sync(team.mask, m2, o);
          m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
          m1 = fmaxf(m1, o1);
        }
        const float value = r.group_top == 2 ? m1 + m2 : m1;
        // what the group's value may be off by: its terms' bounds and their sum's rounding
        const float off = 2.f * tol + 0x1p-21f * (fabsf(m1) + (r.group_top == 2 ? fabsf(m2) : 0.f));
        int above = 0;
        for (int j = 0; j < r.groups; ++j) {
          const float other = team.from(value, j * lanes);
          above += other > value || (other == value && j < g);
          if (scores) {
            const float reach = off + team.from(off, j * lanes);
            if (j != g && g < r.groups && !(fabsf(other - value) > reach)) close = true;
          }
        }
        stay = __ballot_sync(team.mask, above < r.topk_groups);
        close = __any_sync(team.mask, close);
      }
    }
    int mine = -1;
    if (!close) {
      uint32_t key[V], top = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = team.rank * V + v;
        const bool open = e < r.E && (!grouped || (stay >> bit[v] & 1u));
        key[v] = open ? ordered(bias ? c[v] : l[v]) : 0u;
        top = key[v] > top ? key[v] : top;
      }
      float before = 0.f;
      const int passes = bias ? r.k + 1 : r.k;  // one more to see how far the next one is
      for (int j = 0; j < passes; ++j) {
        const uint32_t m = team.max(top);
        if (bias) {
          const float now = unordered(m);
          if (j > 0 && m != 0 && !(before - now > 2.f * tol + 0x1p-21f * fabsf(before))) close = true;
          before = now;
          if (j == r.k) break;
        }
        const int src = __ffs(__ballot_sync(team.mask, top == m)) - 1;
        int e = 0;
        if ((int)(threadIdx.x & 31) == src) {
          int at = 0;
#pragma unroll
          for (int v = V - 1; v >= 0; --v)
            if (key[v] == m) at = v;
          top = 0;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            if (v == at) key[v] = 0;
            top = key[v] > top ? key[v] : top;
          }
          e = team.rank * V + at;
        }
        e = __shfl_sync(team.mask, e, src);
        if (j == team.rank) mine = e;
      }
    }
    if (close) mine = choose_in_double<T, L, V>(r, row, bias);
    // weights: one lane per slot, in double, rounded once
    const bool slot = team.rank < r.k;
    const float ls = slot ? clean(logit_at(row + mine)) : -INFINITY;
    double s = 0.0;
    if (r.sigmoid) {
      if (ls > -INFINITY) s = 1.0 / (1.0 + exp(-(double)ls));
    } else if (r.renorm) {  // the sum over all experts cancels
      const float most = team.max(ls);
      if (ls > -INFINITY) s = exp((double)ls - (double)most);
    } else {
      double total = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (l[v] > -INFINITY) total += exp((double)l[v] - (double)mx);
      total = team.sum(total);
      if (ls > -INFINITY) s = exp((double)ls - (double)mx) / total;
    }
    if (r.renorm) {
      const double all = team.sum(s);
      s = all > 0.0 ? s / all : 0.0;
    }
    if (slot) {
      idx_out[t * r.k + team.rank] = mine;
      w_out[t * r.k + team.rank] = (float)(s * (double)r.scale);
    }
  }
}

// First pass of the losses: a block's sums of p and of logsumexp^2 and its counts. A lane
// adds its experts' p over the block's tokens in fp32 (at most a few dozen), the block
// adds its warps' sums in warp order in double.
template <typename T, int L, int V>
__global__ void __launch_bounds__(32 * kWarps) k_losses(const Routing r, const T* __restrict__ logits,
                                                        const int32_t* __restrict__ idx,
                                                        const uint8_t* __restrict__ mask, int vec,
                                                        double* __restrict__ part_sum,
                                                        int32_t* __restrict__ part_count) {
  pdl_trigger();
  pdl_wait();
  __shared__ int32_t s_count[513];
  __shared__ float s_sum[kWarps * 32 / L][L * V];
  __shared__ double s_z[kWarps * 32 / L];
  const Team<L> team;
  constexpr int kPer = 32 / L * kWarps;
  for (int e = threadIdx.x; e <= r.E; e += blockDim.x) s_count[e] = 0;
  __syncthreads();
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  double z = 0.0;
  for (int64_t t0 = (int64_t)blockIdx.x * kPer; t0 < r.T; t0 += (int64_t)gridDim.x * kPer) {
    const int64_t t = t0 + threadIdx.x / L;
    if (t >= r.T || (mask && !mask[t])) continue;
    const T* row = logits + t * r.stride;
    float l[V], mx = -INFINITY;
    load_logits<T, V>(row, team.rank, r.E, vec, l);
#pragma unroll
    for (int v = 0; v < V; ++v) mx = fmaxf(mx, l[v]);
    mx = team.max(mx);
    float x[V], sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = l[v] > -INFINITY ? expf(l[v] - mx) : 0.f;
      sum += x[v];
    }
    sum = team.sum(sum);
    const float lse = sum > 0.f ? mx + logf(sum) : 0.f;  // no expert has a score: no z term
    if (r.sigmoid) {
      sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[v] = l[v] > -INFINITY ? 1.f / (1.f + expf(-l[v])) : 0.f;
        sum += x[v];
      }
      sum = team.sum(sum);
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] += x[v] * inv;
    if (team.rank == 0) {
      z += (double)lse * (double)lse;
      atomicAdd(&s_count[r.E], 1);
    }
    if (team.rank < r.k) {
      const int e = idx[t * r.k + team.rank];
      if (e >= 0 && e < r.E) atomicAdd(&s_count[e], 1);
    }
  }
  const int who = threadIdx.x / L;
#pragma unroll
  for (int v = 0; v < V; ++v) s_sum[who][team.rank * V + v] = acc[v];
  if (team.rank == 0) s_z[who] = z;
  __syncthreads();
  const int64_t out = (int64_t)blockIdx.x * (r.E + 1);
  for (int e = threadIdx.x; e <= r.E; e += blockDim.x) {
    double sum = 0.0;
    for (int w = 0; w < kPer; ++w) sum += e < r.E ? (double)s_sum[w][e] : s_z[w];
    part_sum[out + e] = sum;
    part_count[out + e] = s_count[e];
  }
}

// Second pass, one block: thread (e, part) adds every nparts-th block's partials, then
// the parts are added in order, and one warp's worth of threads the experts.
__global__ void __launch_bounds__(1024) k_losses_end(const Routing r, int blocks,
                                                     const double* __restrict__ part_sum,
                                                     const int32_t* __restrict__ part_count,
                                                     float* __restrict__ losses,
                                                     int32_t* __restrict__ counts,
                                                     float* __restrict__ prob_mean) {
  pdl_trigger();
  pdl_wait();
  __shared__ double s_sum[1024];
  __shared__ int32_t s_count[1024];
  __shared__ double s_bal[32];
  const int n = r.E + 1;
  const int nparts = 1024 / n;
  const int part = threadIdx.x / n, e = threadIdx.x - part * n;
  double sum = 0.0;
  int32_t count = 0;
  if (part < nparts) {
    for (int b = part; b < blocks; b += nparts) {
      sum += part_sum[(int64_t)b * n + e];
      count += part_count[(int64_t)b * n + e];
    }
  }
  s_sum[threadIdx.x] = sum;
  s_count[threadIdx.x] = count;
  __syncthreads();
  if (threadIdx.x < n) {
    for (int p = 1; p < nparts; ++p) {
      sum += s_sum[p * n + threadIdx.x];
      count += s_count[p * n + threadIdx.x];
    }
    counts[threadIdx.x] = count;
  }
  __syncthreads();
  if (threadIdx.x < n) {
    s_sum[threadIdx.x] = sum;
    s_count[threadIdx.x] = count;
  }
  __syncthreads();
  const double tokens = s_count[r.E] > 0 ? (double)s_count[r.E] : 1.0;
  double bal = 0.0;
  if (threadIdx.x < r.E) {
    const double mean = sum / tokens;
    prob_mean[threadIdx.x] = (float)mean;
    bal = (double)count / tokens * mean;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) bal += __shfl_xor_sync(0xffffffffu, bal, o);
  if ((threadIdx.x & 31) == 0) s_bal[threadIdx.x >> 5] = bal;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0.0;
    for (int w = 0; w < 32; ++w) all += s_bal[w];
    losses[0] = (float)(all * r.E);
    losses[1] = (float)(s_sum[r.E] / tokens);
  }
}

// Gradient in the logits. With g_j = weight_scale * d_topk_w[j], and for the losses
// c_e = d0 E count_e / N^2 (the counts are constants):
//   softmax, renormalised: u = softmax over the chosen logits; dl_j = u_j (g_j - sum g u)
//     (the sum over all experts cancels, and with it the loss of digits in it);
//   softmax: dl_e = p_e ([chosen] g_e - sum g p);
//   sigmoid, renormalised: dl_j = (1 - s_j) u_j (g_j - sum g u), u = s / sum of chosen s;
//   sigmoid: dl_j = s_j (1 - s_j) g_j;
//   balance: softmax p_e (c_e - sum c p); sigmoid s_e (1 - s_e) (c_e - sum c p) / sum s;
//   z: 2 d1 / N * logsumexp * softmax_e.
template <typename T, int L, int V>
__global__ void __launch_bounds__(32 * kWarps)
    k_route_bwd(const Routing r, const T* __restrict__ logits, const int32_t* __restrict__ idx,
                const float* __restrict__ d_w, const int32_t* __restrict__ counts,
                const float* __restrict__ d_losses, const uint8_t* __restrict__ mask, int vec,
                T* __restrict__ d_logits) {
  pdl_trigger();
  pdl_wait();
  const Team<L> team;
  constexpr int kPer = 32 / L * kWarps;
  float c[V], zc = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = 0.f;
  if (d_losses) {
    const double n = counts[r.E] > 0 ? (double)counts[r.E] : 1.0;
    const double d0 = (double)d_losses[0] * r.E / (n * n);
    zc = (float)(2.0 * (double)d_losses[1] / n);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = team.rank * V + v;
      if (e < r.E) c[v] = (float)(d0 * (double)counts[e]);
    }
  }
  for (int64_t t0 = (int64_t)blockIdx.x * kPer; t0 < r.T; t0 += (int64_t)gridDim.x * kPer) {
    const int64_t t = t0 + threadIdx.x / L;
    if (t >= r.T) continue;
    const T* row = logits + t * r.stride;
    const bool losses = d_losses && (!mask || mask[t]);
    float l[V], mx = -INFINITY;
    load_logits<T, V>(row, team.rank, r.E, vec, l);
#pragma unroll
    for (int v = 0; v < V; ++v) mx = fmaxf(mx, l[v]);
    // the chosen experts, one per lane: what arrives at their scores
    int my_e = -1;
    float g = 0.f, ls = -INFINITY;
    if (d_w && team.rank < r.k) {
      my_e = idx[t * r.k + team.rank];
      if (my_e < 0 || my_e >= r.E) my_e = -1;
      if (my_e >= 0) {
        g = d_w[t * r.k + team.rank] * r.scale;
        ls = clean(logit_at(row + my_e));
      }
    }
    float p[V], dl[V], lse = 0.f;
    const bool need_p = losses || (d_w && !r.sigmoid && !r.renorm);
    if (need_p) {
      mx = team.max(mx);
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        p[v] = l[v] > -INFINITY ? expf(l[v] - mx) : 0.f;
        sum += p[v];
      }
      sum = team.sum(sum);
      lse = sum > 0.f ? mx + logf(sum) : 0.f;
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] *= inv;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) dl[v] = 0.f;
    if (losses) {
      float cs = 0.f;
      if (r.sigmoid) {
        float s[V], sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          s[v] = l[v] > -INFINITY ? 1.f / (1.f + expf(-l[v])) : 0.f;
          sum += s[v];
          cs += c[v] * s[v];
        }
        sum = team.sum(sum);
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        cs = team.sum(cs) * inv;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float rest = l[v] > -INFINITY ? 1.f / (1.f + expf(l[v])) : 0.f;  // 1 - s
          dl[v] = s[v] * rest * (c[v] - cs) * inv + zc * lse * p[v];
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) cs += c[v] * p[v];
        cs = team.sum(cs);
#pragma unroll
        for (int v = 0; v < V; ++v) dl[v] = p[v] * (c[v] - cs + zc * lse);
      }
    }
    if (d_w) {
      float u = 0.f, rest = 1.f;
      if (r.sigmoid) {
        if (my_e >= 0 && ls > -INFINITY) {
          u = 1.f / (1.f + expf(-ls));
          rest = 1.f / (1.f + expf(ls));
        }
      } else if (r.renorm) {
        const float top = team.max(ls);
        if (ls > -INFINITY) u = expf(ls - top);
      }
      float term = 0.f;  // what slot `rank` adds to its expert
      if (r.renorm) {
        const float sum = team.sum(u);
        u = sum > 0.f ? u / sum : 0.f;
        term = u * (g - team.sum(g * u)) * rest;
      } else if (r.sigmoid) {
        term = u * rest * g;
      } else {
        float gp = 0.f;
        if (my_e >= 0 && ls > -INFINITY) u = expf(ls - lse);
        gp = team.sum(g * u);
        term = u * g;
#pragma unroll
        for (int v = 0; v < V; ++v) dl[v] -= p[v] * gp;
      }
      for (int j = 0; j < r.k; ++j) {
        const int e = team.from(my_e, j);
        const float add = team.from(term, j);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (e == team.rank * V + v) dl[v] += add;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = team.rank * V + v;
      if (e < r.E) store(d_logits + t * r.E + e, dl[v]);
    }
  }
}

// Blocks: all tokens at once, at most `waves` blocks per SM (the kernels stride).
template <int L>
unsigned token_blocks(const Routing& r, int waves) {
  const int64_t per = 32 / L * kWarps;
  const int64_t want = (r.T + per - 1) / per, cap = (int64_t)num_sms() * waves;
  return (unsigned)(want < cap ? want : cap);
}

template <int L, int V, typename F>
cudaError_t with(F f) {
  return f(std::integral_constant<int, L>(), std::integral_constant<int, V>());
}

template <typename F>
cudaError_t by_sizes(const Routing& r, F f) {
  if (r.k <= 8 && r.groups <= 8) {  // a lane per slot, and one per group at least
    if (r.E <= 8) return with<8, 1>(f);
    if (r.E <= 16) return with<8, 2>(f);
    if (r.E <= 32) return with<8, 4>(f);
    if (r.E <= 64) return with<8, 8>(f);
    if (r.E <= 128) return with<16, 8>(f);
  } else {
    if (r.E <= 64) return with<32, 2>(f);
    if (r.E <= 128) return with<32, 4>(f);
  }
  if (r.E <= 256) return with<32, 8>(f);
  return with<32, 16>(f);
}

// Whether every lane's V logits start on a boundary of their size (16 bytes at most).
template <typename T, int V>
int vectors(const Routing& r, const T* logits) {
  constexpr size_t kBytes = V * sizeof(T) < 16 ? V * sizeof(T) : 16;
  return r.E % V == 0 && reinterpret_cast<uintptr_t>(logits) % kBytes == 0 &&
         (r.T == 1 || r.stride * (int64_t)sizeof(T) % (int64_t)kBytes == 0);
}

}  // namespace

cudaError_t launch_route(const Routing& r, const void* logits, const float* bias, int32_t* idx,
                         float* w, cudaStream_t st) {
  return by_sizes(r, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value;
    const dim3 grid(token_blocks<L>(r, 8)), block(32 * kWarps);
    if (r.bf16) {
      const auto* p = static_cast<const __nv_bfloat16*>(logits);
      return launch_pdl(k_route<__nv_bfloat16, L, V>, grid, block, 0, st, r, p, bias,
                        vectors<__nv_bfloat16, V>(r, p), idx, w);
    }
    const auto* p = static_cast<const float*>(logits);
    return launch_pdl(k_route<float, L, V>, grid, block, 0, st, r, p, bias,
                      vectors<float, V>(r, p), idx, w);
  });
}

int router_loss_blocks(const Routing& r) {
  int n = 0;
  by_sizes(r, [&](auto l, auto) {
    n = (int)token_blocks<decltype(l)::value>(r, 2);
    return cudaSuccess;
  });
  return n;
}

cudaError_t launch_router_losses(const Routing& r, const void* logits, const int32_t* idx,
                                 const uint8_t* mask, float* losses, int32_t* counts,
                                 float* prob_mean, double* part_sum, int32_t* part_count,
                                 cudaStream_t st) {
  const int blocks = router_loss_blocks(r);
  if (blocks > 0) {
    const cudaError_t e = by_sizes(r, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, V = decltype(v)::value;
      const dim3 grid((unsigned)blocks), block(32 * kWarps);
      if (r.bf16) {
        const auto* p = static_cast<const __nv_bfloat16*>(logits);
        return launch_pdl(k_losses<__nv_bfloat16, L, V>, grid, block, 0, st, r, p, idx, mask,
                          vectors<__nv_bfloat16, V>(r, p), part_sum, part_count);
      }
      const auto* p = static_cast<const float*>(logits);
      return launch_pdl(k_losses<float, L, V>, grid, block, 0, st, r, p, idx, mask,
                        vectors<float, V>(r, p), part_sum, part_count);
    });
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k_losses_end, dim3(1), dim3(1024), 0, st, r, blocks, part_sum, part_count,
                    losses, counts, prob_mean);
}

cudaError_t launch_route_backward(const Routing& r, const void* logits, const int32_t* idx,
                                  const float* d_w, const int32_t* counts, const float* d_losses,
                                  const uint8_t* mask, void* d_logits, cudaStream_t st) {
  return by_sizes(r, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value;
    const dim3 grid(token_blocks<L>(r, 8)), block(32 * kWarps);
    if (r.bf16) {
      const auto* p = static_cast<const __nv_bfloat16*>(logits);
      return launch_pdl(k_route_bwd<__nv_bfloat16, L, V>, grid, block, 0, st, r, p, idx, d_w, counts,
                        d_losses, mask, vectors<__nv_bfloat16, V>(r, p),
                        static_cast<__nv_bfloat16*>(d_logits));
    }
    const auto* p = static_cast<const float*>(logits);
    return launch_pdl(k_route_bwd<float, L, V>, grid, block, 0, st, r, p, idx, d_w, counts, d_losses,
                      mask, vectors<float, V>(r, p), static_cast<float*>(d_logits));
  });
}

}  // namespace moe
