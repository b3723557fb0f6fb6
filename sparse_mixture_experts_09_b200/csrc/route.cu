// General routing from router logits, the two router losses, and the gradient of both
// in the logits. Formulas and conventions: include/moe.h.
//
// All three kernels give a token L lanes of a warp (L = 8, 16 or 32) and each lane V
// neighbouring experts, L * V >= E: a token's logits stay in registers, and L is small,
// so that one instruction serves several tokens, but holds a lane per slot.
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

// 2^x to within 2^-22 of the value, and 1 / x to within one ulp (subnormals as 0).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// sigmoid(l) and 1 - sigmoid(l), each to within (8 + 1.5 |l|) 2^-24 of itself.
__device__ __forceinline__ void sigmoid_pair(float l, float& s, float& rest) {
  const float x = fast_exp2(-kLog2e * fabsf(l)), big = fast_rcp(1.f + x), small = x * big;
  s = l >= 0.f ? big : small;
  rest = l >= 0.f ? small : big;
}

// Below -32 a sigmoid is an exponential to 2^-46, and the shares s / sum s do not change with a common
// offset of the logits: where the largest logit `top` is below, it is moved to -32 for them, so
// that none is lost to the subnormals. Below kNoScore the routing's own sigmoids (in double) are 0.
constexpr float kNoScore = -709.f;
__device__ __forceinline__ float share_shift(float top) {
  return top < -32.f && top > kNoScore ? top + 32.f : 0.f;
}

// NaN -> -inf, +inf -> the largest float: exp(l - max) is then 0 or finite everywhere.
__device__ __forceinline__ float clean(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX); }

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

// The reverse of load_logits, one rounding for bf16.
template <typename T, int V>
__device__ __forceinline__ void store_row(T* row, int rank, int E, bool vec, const float (&f)[V]) {
  constexpr int kBytes = V * (int)sizeof(T);
  const int e0 = rank * V;
  if (vec && kBytes >= 4) {
    if (e0 >= E) return;
    uint32_t q[(kBytes + 3) / 4];
#pragma unroll
    for (int i = 0; i < (kBytes + 3) / 4; ++i) {
      if constexpr (sizeof(T) == 4)
        q[i] = __float_as_uint(f[i]);
      else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(q[i]) : "f"(f[(2 * i + 1) % V]), "f"(f[2 * i % V]));
    }
    char* p = reinterpret_cast<char*>(row + e0);
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
    } else {
      *reinterpret_cast<uint32_t*>(p) = q[0];
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e0 + v < E) store(row + e0 + v, f[v]);
  }
}


// Descending, by Batcher's odd-even merge (all indices are known at compile time).
template <int V>
__device__ __forceinline__ void sort_down(float (&a)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i >= k % p && (i - k % p) % (2 * k) < k && i + k < V && i / (2 * p) == (i + k) / (2 * p)) {
          const float hi = fmaxf(a[i], a[i + k]);
          a[i + k] = fminf(a[i], a[i + k]);
          a[i] = hi;
        }
}

// How a team's lanes share the groups: `lanes` of them (a power of two) to a group.
template <int L, int V>
struct Groups {
  int lanes, size;
  unsigned bits[(V + 3) / 4];  // the lane's experts' groups in a ballot of the warp, a byte each
  __device__ Groups(const Routing& r, const Team<L>& team) {
    size = r.E / r.groups;
    lanes = L;
    while (lanes * r.groups > L) lanes >>= 1;
    int g = 0, in = 0;
    if (r.groups > 1) {
      g = team.rank * V / size;
      in = team.rank * V - g * size;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const unsigned b = r.groups > 1 ? team.base + g * lanes : 0;
      bits[v / 4] = (v % 4 ? bits[v / 4] : 0u) | (b & 31u) << (8 * (v % 4));
      if (++in == size) {
        in = 0;
        ++g;
      }
    }
  }
  __device__ bool stays(unsigned stay, int v) const {
    return stay >> (bits[v / 4] >> (8 * (v % 4)) & 31u) & 1u;
  }
};

__device__ __forceinline__ double sigmoid_in_double(float l) {
  return l > -INFINITY ? 1.0 / (1.0 + exp(-(double)l)) : 0.0;
}

// The groups that stay, as a ballot (bit base + g * lanes for group g). A value may be off by
// tol + 2 u |value|; `close` is set where the last group that stays and the first that goes
// are not further apart than that allows. With no bias and one expert a group the values are the
// logits themselves, which fp32 compares exactly; they are not judged again by scores, which are equal
// for different logits where a sigmoid saturates. A group's one or two best: its lanes take their own
// values, or every lanes-th from shared memory, and merge their pairs. Close groups of
// sigmoid scores are judged again by the values in double of those experts that can be
// among their best.
template <typename T, int L, int V>
__device__ __forceinline__ unsigned open_groups(const Routing& r, const Team<L>& team,
                                                const Groups<L, V>& groups, const T* row,
                                                const float* bias, const float (&value)[V],
                                                float tol, float* shared, bool& close) {
  const int lanes = groups.lanes, g = team.rank / lanes;
  const auto at_expert = [](int e) { return e + (e >> 5); };  // groups of 32 on distinct banks
  const bool own = groups.size == V * lanes;  // the lanes hold their group's values
  if (!own) {
    __syncwarp(team.mask);
#pragma unroll
    for (int v = 0; v < V; ++v) shared[at_expert(team.rank * V + v)] = value[v];
    __syncwarp(team.mask);
  }
  float m1 = -INFINITY, m2 = -INFINITY;
  const auto add = [&](float x) {
    m2 = fmaxf(m2, fminf(x, m1));
    m1 = fmaxf(m1, x);
  };
  if (own) {
#pragma unroll
    for (int v = 0; v < V; ++v) add(value[v]);
  } else if (g < r.groups) {
    for (int i = team.rank - g * lanes; i < groups.size; i += lanes)
      add(shared[at_expert(g * groups.size + i)]);
  }
  for (int o = lanes >> 1; o > 0; o >>= 1) {
    const float o1 = __shfl_xor_sync(team.mask, m1, o), o2 = __shfl_xor_sync(team.mask, m2, o);
    m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
    m1 = fmaxf(m1, o1);
  }
  const float mine = r.group_top == 2 ? m1 + m2 : m1;
  int above = 0;
  for (int j = 0; j < r.groups; ++j) {
    const float other = team.from(mine, j * lanes);
    above += other > mine || (other == mine && j < g);
  }
  const bool in = above < r.topk_groups;
  close = false;
  if (!bias && r.group_top == 1) return __ballot_sync(team.mask, in);  // logits: exact
  const bool real = g < r.groups;
  // what a group's value may be off by: its terms' bounds and their sum's rounding
  const float off = real ? 2 * tol + 0x1p-22f * (fabsf(m1) + (r.group_top == 2 ? fabsf(m2) : 0.f)) : 0.f;
  const float least = -team.max(real && in ? -mine : -INFINITY), most = team.max(real && !in ? mine : -INFINITY);
  const float reach = 2 * team.max(off);
  close = r.topk_groups < r.groups && !(least - most > reach);
  if (!close || !r.sigmoid) return __ballot_sync(team.mask, in);
  close = false;
  if (own) {
    __syncwarp(team.mask);
#pragma unroll
    for (int v = 0; v < V; ++v) shared[at_expert(team.rank * V + v)] = value[v];
    __syncwarp(team.mask);
  }
  double d1 = -INFINITY, d2 = -INFINITY;
  const float least_of_two = reach < INFINITY ? (r.group_top == 2 ? m2 : m1) - reach : -INFINITY;
  if (g < r.groups) {
#pragma unroll 1
    for (int i = team.rank - g * lanes; i < groups.size; i += lanes) {
      const int e = g * groups.size + i;
      if (!(shared[at_expert(e)] >= least_of_two)) continue;
      double c = sigmoid_in_double(clean(logit_at(row + e)));
      if (bias) c += (double)__ldg(bias + e);
      if (!(c == c)) c = -INFINITY;
      d2 = fmax(d2, fmin(c, d1));
      d1 = fmax(d1, c);
    }
  }
#pragma unroll 1
  for (int o = lanes >> 1; o > 0; o >>= 1) {
    const double o1 = __shfl_xor_sync(team.mask, d1, o), o2 = __shfl_xor_sync(team.mask, d2, o);
    d2 = fmax(fmax(d2, o2), fmin(d1, o1));
    d1 = fmax(d1, o1);
  }
  // a group with a value of +infinity has that, whatever the other is
  const double exact = r.group_top == 2 && d1 < INFINITY ? d1 + d2 : d1;
  above = 0;
#pragma unroll 1
  for (int j = 0; j < r.groups; ++j) {
    const double other = team.from(exact, j * lanes);
    above += other > exact || (other == exact && j < g);
  }
  return __ballot_sync(team.mask, above < r.topk_groups);
}

// The best experts in order, one to a lane; order[v] compares them, -inf is none. Returns
// the expert of lane `rank` below n. Each lane sorts its own and lays them out in shared memory;
// then the team finds the largest head, and the lowest lane that has it gives it up; which
// expert it was is looked up for all at the end. n = k where the order is exact (tol < 0). Else an
// order may be off by tol + 2 u |order|: n is the first place from k on at which all that
// follow are certainly less, and `close` is set where neighbours among the n may stand in
// the wrong order. n = 0: not to be had this way (fewer than k finite values, or a run of
// near ties longer than the team).
template <int L, int V>
__device__ __forceinline__ int best_experts(const Routing& r, const Team<L>& team, const float (&order)[V],
                                            float tol, float* shared, int& n, bool& close) {
  float sorted[V];
#pragma unroll
  for (int v = 0; v < V; ++v) sorted[v] = order[v];
  sort_down(sorted);
  __syncwarp(team.mask);
#pragma unroll
  for (int v = 1; v < V; ++v) shared[v * L + team.rank] = sorted[v];
  float head = sorted[0], my_key = 0.f, last_key = INFINITY;
  int next = 1, my_src = team.base, my_nth = 0, last_src = -1, nth = 0, j = 0;
  const float reach = 2.f * tol;
  for (;; ++j) {
    if (tol < 0.f && j == r.k) break;
    const float m = team.max(head);
    if (m == -INFINITY) {
      if (j < r.k) j = 0;
      break;
    }
    if (tol >= 0.f && j > 0) {
      const bool far = last_key - m > reach + 0x1p-22f * fabsf(last_key);
      if (j >= r.k && far) break;
      if (!far) close = true;
      if (j == L) {
        j = 0;
        break;
      }
    }
    const int src = __ffs(__ballot_sync(team.mask, head == m)) - 1;
    nth = m == last_key && src == last_src ? nth + 1 : 0;  // of equal values in one lane
    last_key = m;
    last_src = src;
    if (j == team.rank) {
      my_key = m;
      my_src = src;
      my_nth = nth;
    }
    if ((int)(threadIdx.x & 31) == src) {
      head = next < V ? shared[next * L + team.rank] : -INFINITY;
      ++next;
    }
  }
  n = j;
  int at = 0;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (__shfl_sync(team.mask, order[v], my_src) == my_key && my_nth-- == 0) at = v;
  return (my_src - team.base) * V + at;
}

// As best_experts for k <= 8, without its k rounds in a row: the lanes' sorted lists, cut to 8,
// are merged in log2 L steps (of two descending lists the larger of each pair a[i], b[7 - i] is
// the best 8, and three exchange stages sort them), the k-th value marks the candidates, and a
// prefix sum gives each a lane: n of them, in the order of their indices. Returns the lane's
// candidate and its `value` (-inf from lane n on). `unsure` (a team's lanes agree): not to be
// had this way (fewer than k finite values, or more candidates than lanes).
template <int L, int V>
__device__ __forceinline__ int few_candidates(const Routing& r, const Team<L>& team,
                                              const float (&order)[V], float tol, float2* shared,
                                              float& value, int& n, bool& unsure) {
  int mine = team.rank;
  value = order[0];
  n = L;
  if constexpr (V > 1) {
    float sorted[V], top[8];
#pragma unroll
    for (int v = 0; v < V; ++v) sorted[v] = order[v];
    sort_down(sorted);
#pragma unroll
    for (int i = 0; i < 8; ++i) top[i] = i < V ? sorted[i < V ? i : 0] : -INFINITY;
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
      float other[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(team.mask, top[i], o);
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = fmaxf(top[i], other[7 - i]);
#pragma unroll
      for (int d = 4; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!(i & d)) {
            const float hi = fmaxf(top[i], top[i + d]);
            top[i + d] = fminf(top[i], top[i + d]);
            top[i] = hi;
          }
    }
    float last = top[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) last = i < r.k ? top[i] : last;
    if (last == -INFINITY) {  // fewer than k finite values
      unsure = true;
      return 0;
    }
    const float low = tol < 0.f ? last : last - (2.f * tol + 0x1p-22f * fabsf(last));
    int count = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) count += order[v] >= low;
    int upto = count;
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
      const int before = __shfl_up_sync(team.mask, upto, o, L);
      if (team.rank >= o) upto += before;
    }
    n = team.from(upto, L - 1);
    if (n > L || n < r.k) {  // less than k: an infinite bound
      unsure = true;
      return 0;
    }
    __syncwarp(team.mask);
    int at = upto - count;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (order[v] >= low) shared[at++] = make_float2(order[v], __int_as_float(team.rank * V + v));
    __syncwarp(team.mask);
    value = -INFINITY;
    if (team.rank < n) {
      const float2 got = shared[team.rank];
      value = got.x;
      mine = __float_as_int(got.y);
    }
  }
  return mine;
}

// The softmax's denominator in double: the sum of exp(l - mx) over the experts.
template <int L, int V>
__device__ __forceinline__ double sum_in_double(const Team<L>& team, const float (&l)[V], float mx) {
  double total = 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (l[v] > -INFINITY) total += exp((double)l[v] - (double)mx);
  return team.sum(total);
}

// Slot `slot` < k of each lane (expert `mine`, logit `ls`; the slots' lanes are below `reduce`, a
// power of two) to the outputs: weights in double, one lane per slot, rounded once. s: the
// lane's sigmoid.
template <typename T, int L, int V>
__device__ __forceinline__ void write_slots(const Routing& r, const Team<L>& team, const T* row,
                                            int64_t t, int mine, float ls, double s, int slot,
                                            int reduce, int vec, int32_t* idx_out, float* w_out) {
  const bool chosen = slot < r.k;
  if (!chosen) {
    ls = -INFINITY;
    s = 0.0;
  }
  if (!r.sigmoid) {
    s = 0.0;
    if (r.renorm) {  // the sum over all experts cancels
      float most = ls;
      for (int o = reduce >> 1; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(team.mask, most, o));
      if (ls > -INFINITY) s = exp((double)ls - (double)most);
    } else {
      float l[V], mx = -INFINITY;
      load_logits<T, V>(row, team.rank, r.E, vec, l);
#pragma unroll
      for (int v = 0; v < V; ++v) mx = fmaxf(mx, l[v]);
      mx = team.max(mx);
      const double total = sum_in_double(team, l, mx);
      if (ls > -INFINITY) s = exp((double)ls - (double)mx) / total;
    }
  }
  if (r.renorm) {
    double all = s;
    for (int o = reduce >> 1; o > 0; o >>= 1) all += __shfl_xor_sync(team.mask, all, o);
    s = all > 0.0 ? s / all : 0.0;
  }
  if (chosen) {
    idx_out[t * r.k + slot] = mine;
    w_out[t * r.k + slot] = (float)(s * (double)r.scale);
  }
}

// A token with every comparison in double, by a whole warp. Few tokens come here, but the
// kernel ends with the last of them, and what they wait for is this code itself, which is in
// no cache: so it is short, loops over shared memory (E doubles) and is not unrolled.
template <typename T, int V>
__device__ __noinline__ void route_in_double(const Routing r, const T* row, const float* bias, int64_t t,
                                             double* shared, int32_t* idx_out, float* w_out) {
  const Team<32> team;
  const auto at_expert = [](int e) { return e + (e >> 5); };
  const int gs = r.E / r.groups;
  float mx = -INFINITY;
  for (int e = team.rank; e < r.E; e += 32) mx = fmaxf(mx, clean(logit_at(row + e)));
  mx = team.max(mx);
  double total = 0.0;
  __syncwarp();
#pragma unroll 1
  for (int e = team.rank; e < r.E; e += 32) {
    const float l = clean(logit_at(row + e));
    const double x = l > -INFINITY ? exp(r.sigmoid ? -(double)l : (double)l - (double)mx) : 0.0;
    shared[at_expert(e)] = x;
    total += x;
  }
  total = team.sum(total);
#pragma unroll 1
  for (int e = team.rank; e < r.E; e += 32) {
    const float l = clean(logit_at(row + e));
    double c = 0.0;
    if (l > -INFINITY)
      c = r.sigmoid ? 1.0 / (1.0 + shared[at_expert(e)]) : shared[at_expert(e)] / total;
    if (bias) c += (double)__ldg(bias + e);
    if (!bias && r.group_top == 1) c = l;
    shared[at_expert(e)] = c == c ? c : -INFINITY;
  }
  __syncwarp();
  unsigned stay = 0xffffffffu;
  if (r.groups > 1) {  // lane g has group g's value: the largest left, group_top times
    double value = -INFINITY;
    if (team.rank < r.groups) {
      value = 0.0;
      unsigned taken[16] = {};
#pragma unroll 1
      for (int m = 0; m < r.group_top; ++m) {
        double best = -INFINITY;
        int at = -1;
#pragma unroll 1
        for (int i = 0; i < gs; ++i) {
          const double c = shared[at_expert(team.rank * gs + i)];
          if (!(taken[i >> 5] >> (i & 31) & 1u) && (at < 0 || c > best)) {
            best = c;
            at = i;
          }
        }
        if (value < INFINITY) value += best;  // +infinity (the first, if any) stays, whatever follows
        taken[at >> 5] |= 1u << (at & 31);
      }
    }
    int above = 0;
#pragma unroll 1
    for (int j = 0; j < r.groups; ++j) {
      const double other = team.from(value, j);
      above += other > value || (other == value && j < team.rank);
    }
    stay = __ballot_sync(team.mask, above < r.topk_groups);
  }
  __syncwarp();
  // with no bias the logits order the experts; a closed or taken one is a NaN
#pragma unroll 1
  for (int e = team.rank; e < r.E; e += 32) {
    if (!bias) shared[at_expert(e)] = clean(logit_at(row + e));
    if (r.groups > 1 && !(stay >> (e / gs) & 1u)) shared[at_expert(e)] = __longlong_as_double(-1ll);
  }
  int mine = 0;
#pragma unroll 1
  for (int j = 0; j < r.k; ++j) {
    double best = 0.0;
    int at = 0x7fffffff;
#pragma unroll 1
    for (int e = team.rank; e < r.E; e += 32) {
      const double c = shared[at_expert(e)];
      if (c == c && (at == 0x7fffffff || c > best)) {
        best = c;
        at = e;
      }
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) {
      const double b2 = __shfl_xor_sync(team.mask, best, o);
      const int a2 = __shfl_xor_sync(team.mask, at, o);
      if (a2 != 0x7fffffff && (at == 0x7fffffff || b2 > best || (b2 == best && a2 < at))) {
        best = b2;
        at = a2;
      }
    }
    if (at % 32 == team.rank) shared[at_expert(at)] = __longlong_as_double(-1ll);
    if (j == team.rank) mine = at;
  }
  const float ls = team.rank < r.k ? clean(logit_at(row + mine)) : -INFINITY;
  write_slots<T, 32, V>(r, team, row, t, mine, ls, sigmoid_in_double(ls), team.rank, 32, 0, idx_out, w_out);
  __syncwarp();
}

// Routing, one team of L lanes per token. The logits alone decide where nothing else is
// asked for (both scores rise with the logit, so fp32 is exact); else the values s + bias
// and the groups' sums are formed in fp32 with the approximate exponential and reciprocal: they
// give the groups and the candidates, which under sigmoid scores are then ordered by their own
// s + bias in double. A token with another decision within its error bounds, with more candidates
// than the team has lanes, or with a group_top above 2 is put aside and routed in double after up to
// 32 others of the team. Of fp32 logits that is a few tokens in ten thousand, but of bf16 ones, whose
// values repeat, 2 to 5 in a hundred where 8 slots meet 8 lanes (by logits alone, or with a bias of
// zeros): 65536 x 64, 8 slots 53 us instead of 25; 6 slots 26. group_top 3: all tokens, 16384 x 256
// 164 us. Bounds, with
// u = 2^-24: the exponential is off by 4 u and by 1.5 u |x| for its argument, the reciprocal by
// 2 u; s (1 - s) is at most 1/4 and |x| s (1 - s) at most 0.23, so a sigmoid is off by less than 5 u
// (6 u are allowed); |x| e^x is at most 0.37 below 0, so a softmax is off by less than 32 u of the
// largest probability (its sum of up to 512 terms is a tree of 20 levels); the sum with the bias
// by u of its value.
//
// Bound by instructions and their latency, not bytes (some 760 a token at 256 experts with groups and
// a bias, 56% of the issue slots at 24% of the warps): a team is as narrow as 16 values per lane allow, so that a warp's
// instruction serves up to four tokens. Device times: 16384 tokens, 256 experts, 8 slots, sigmoid
// scores, bias, 4 of 8 groups 24.3 us (17.8 MB: 2.7 us at HBM's rate), groups by their logits 22.5,
// without groups 18.9, by logits alone 20.0; 65536 x 64 25 us; one token 3.3 us.
template <typename T, int L, int V, bool FEW>
__global__ void __launch_bounds__(32 * kWarps, V <= 4 ? 4 : V <= 8 ? 3 : 2)
    k_route(const Routing r, const T* __restrict__ logits, const float* __restrict__ bias, int vec,
            int32_t* __restrict__ idx_out, float* __restrict__ w_out) {
  pdl_trigger();
  pdl_wait();
  __shared__ double s_value[kWarps * 32 / L][L * V + L * V / 32 + 1];
  __shared__ __align__(16) float s_bias[L * V];
  const Team<L> team;
  const Groups<L, V> groups(r, team);
  constexpr int kPer = 32 / L * kWarps;  // tokens per block
  double* shared = s_value[threadIdx.x / L];
  const bool scores = bias || r.group_top > 1;
  int pairs = 1;  // lanes up to the next power of two of k: the slots' reductions
  while (pairs < r.k) pairs *= 2;
  if (bias) {
    for (int e = threadIdx.x; e < L * V; e += 32 * kWarps) {
      const float b = e < r.E ? __ldg(bias + e) : -INFINITY;
      s_bias[e] = b == b ? b : -INFINITY;
    }
    __syncthreads();
  }
  // true where the token is done
  const auto route = [&](const T* row, int64_t t) {
    float l[V], c[V];
    load_logits<T, V>(row, team.rank, r.E, vec, l);
    float tol = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = l[v];
    if (scores) {
      if (r.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = fast_rcp(1.f + fast_exp2(-kLog2e * l[v]));
        tol = 0x1.8p-22f;
      } else {
        float mx = -INFINITY, sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) mx = fmaxf(mx, l[v]);
        mx = team.max(mx);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          c[v] = l[v] > -INFINITY ? fast_exp2(kLog2e * (l[v] - mx)) : 0.f;
          sum += c[v];
        }
        sum = team.sum(sum);
        const float inv = sum > 0.f ? fast_rcp(sum) : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] *= inv;
        tol = 0x1p-19f * inv;  // the largest probability is 1 / sum
      }
      if (bias) {
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] += s_bias[team.rank * V + v];
      }
    }
    unsigned stay = 0xffffffffu;
    if (r.groups > 1) {
      bool near = false;
      stay = open_groups(r, team, groups, row, bias, c, tol, reinterpret_cast<float*>(shared), near);
      if (near) return false;
    }
    if (bias) {
#pragma unroll
      for (int v = 0; v < V; ++v) l[v] = c[v];
    }
    if (r.groups > 1) {
      if (groups.size == V * groups.lanes) {  // one group's all
        const bool open = groups.stays(stay, 0);
#pragma unroll
        for (int v = 0; v < V; ++v) l[v] = open ? l[v] : -INFINITY;
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) l[v] = groups.stays(stay, v) ? l[v] : -INFINITY;
      }
    }
    int mine, n = 0, slot = team.rank;
    bool unsure = false;
    if constexpr (FEW) {
      float value;
      mine = few_candidates(r, team, l, bias ? tol : -1.f, reinterpret_cast<float2*>(shared), value, n, unsure);
      if (unsure) return false;
      if (!bias || !r.sigmoid) {  // by value: exact, or with no two of the chosen too close
        const float reach = bias ? 2.f * tol + 0x1p-22f * fabsf(value) : -1.f;
        bool near = false;
        slot = 0;
        for (int j = 0; j < n; ++j) {
          const float other = team.from(value, j);
          slot += other > value || (other == value && j < team.rank);
          near |= j != team.rank && !(fabsf(other - value) > reach);
        }
        unsure = __any_sync(team.mask, slot < r.k && (value == -INFINITY || (bias && near)));
      } else if (V == 1) {  // all experts are candidates
        const int finite = __popc(__ballot_sync(team.mask, value > -INFINITY));
        unsure = finite < r.k;
      }
    } else {
      bool near = false;
      mine = best_experts(r, team, l, bias ? tol : -1.f, reinterpret_cast<float*>(shared), n, near);
      unsure = n == 0 || (near && !r.sigmoid);
    }
    if (unsure) return false;
    // the chosen are among the first n lanes
    const bool real = team.rank < n && mine < r.E;
    const float ls = real ? clean(logit_at(row + mine)) : -INFINITY;
    const double sg = r.sigmoid ? sigmoid_in_double(ls) : 0.0;
    if (bias && r.sigmoid) {  // the candidates' own values, which the weights need anyhow
      const bool open = real && (V > 1 || !FEW || l[0] > -INFINITY);
      const double c = open ? sg + (double)s_bias[mine] : -INFINITY;
      slot = 0;
      for (int j = 0; j < n; ++j) {
        const double other = team.from(c, j);
        const int e = team.from(mine, j);
        slot += other > c || (other == c && e < mine);
      }
      if (!real) slot = r.k;
    }
    write_slots<T, L, V>(r, team, row, t, mine, ls, sg, slot, n > pairs ? L : pairs, vec, idx_out, w_out);
    return true;
  };
  const int64_t stride = (int64_t)gridDim.x * kPer;
  constexpr int kTeams = 32 / L;
  // of the warp's first team; its lanes stay together for the tokens put aside
  for (int64_t t0 = (int64_t)blockIdx.x * kPer + threadIdx.x / 32 * kTeams; t0 < r.T; t0 += 32 * stride) {
    unsigned aside = 0;
    if (r.group_top > 2) {
      aside = 0xffffffffu;
    } else {
      for (int i = 0; i < 32; ++i) {
        const int64_t t = t0 + team.base / L + i * stride;
        if (t >= r.T) break;  // a token's lanes leave together
        if (!route(logits + t * r.stride, t)) aside |= 1u << i;
      }
    }
    __syncwarp();
    if (__ballot_sync(0xffffffffu, aside != 0) == 0) continue;
#pragma unroll
    for (int q = 0; q < kTeams; ++q) {
      unsigned left = __shfl_sync(0xffffffffu, aside, q * L);
      for (; left; left &= left - 1) {
        const int64_t t = t0 + q + (__ffs(left) - 1) * stride;
        if (t < r.T)
          route_in_double<T, (L * V + 31) / 32>(r, logits + t * r.stride, bias, t, s_value[threadIdx.x / 32 * kTeams],
                                                idx_out, w_out);
      }
    }
  }
}

// First pass of the losses: a block's sums of p and of logsumexp^2 and its counts. A lane
// adds its experts' p over its tokens in fp32 (every 3552nd at 256 experts, 14208th at 64), the block
// adds its teams' sums in order in double: E + 1 sums and counts. Bound by latency: few bytes
// and few steps per token, so the next token's loads go out before this one's sums (65521
// tokens, 64 experts, 6 slots: 13.0 us with the second pass, 14.0 with sigmoid scores; 18.4 MB, 2.8 us at
// HBM's rate).
template <typename T, int L, int V, int WARPS>
__device__ __forceinline__ void block_losses(const Routing& r, const T* __restrict__ logits,
                                             const int32_t* __restrict__ idx,
                                             const uint8_t* __restrict__ mask, int vec,
                                             double* part_sum, int32_t* part_count) {
  __shared__ int32_t s_count[513];
  __shared__ float s_sum[WARPS * 32 / L][L * V];
  __shared__ double s_z[WARPS * 32 / L];
  const Team<L> team;
  constexpr int kPer = 32 / L * WARPS;
  for (int e = threadIdx.x; e <= r.E; e += blockDim.x) s_count[e] = 0;
  __syncthreads();
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  double z = 0.0;
  int tokens = 0;
  float ahead[V];
  int slot = -1;
  bool keep = false;
  const auto fetch = [&](int64_t t) {
    keep = t < r.T;
    slot = -1;
    if (!keep) return;
    load_logits<T, V>(logits + t * r.stride, team.rank, r.E, vec, ahead);
    if (team.rank < r.k) slot = idx[t * r.k + team.rank];
    if (mask) keep = mask[t];
  };
  int64_t t = (int64_t)blockIdx.x * kPer + threadIdx.x / L;
  fetch(t);
  while (t < r.T) {
    float l[V], mx = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      l[v] = ahead[v];
      mx = fmaxf(mx, l[v]);
    }
    const bool counts = keep;
    const int e = slot;
    t += (int64_t)gridDim.x * kPer;
    fetch(t);
    if (!counts) continue;
    mx = team.max(mx);
    const float top = mx > -INFINITY ? mx : 0.f;  // exp(l - top) is 0 where no expert has a score
    float x[V], sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = fast_exp2(kLog2e * (l[v] - top));
      sum += x[v];
    }
    sum = team.sum(sum);
    const float lse = sum > 0.f ? top + logf(sum) : 0.f;  // no expert has a score: no z term
    if (r.sigmoid) {
      const float shift = share_shift(top);
      sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float rest;
        sigmoid_pair(l[v] - shift, x[v], rest);
        sum += x[v];
      }
      sum = team.sum(sum);
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = fmaf(x[v], inv, acc[v]);
    z += (double)lse * (double)lse;
    ++tokens;
    if (e >= 0 && e < r.E) atomicAdd(&s_count[e], 1);
  }
  const int who = threadIdx.x / L;
#pragma unroll
  for (int v = 0; v < V; ++v) s_sum[who][team.rank * V + v] = acc[v];
  if (team.rank == 0) {
    s_z[who] = z;
    atomicAdd(&s_count[r.E], tokens);
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= r.E; e += blockDim.x) {
    double sum = 0.0;
#pragma unroll 8
    for (int w = 0; w < kPer; ++w) sum += e < r.E ? (double)s_sum[w][e] : s_z[w];
    part_sum[e] = sum;
    part_count[e] = s_count[e];
  }
}

template <typename T, int L, int V>
__global__ void __launch_bounds__(32 * kWarps, V <= 8 ? 3 : 2)
    k_losses(const Routing r, const T* __restrict__ logits, const int32_t* __restrict__ idx,
             const uint8_t* __restrict__ mask, int vec, double* __restrict__ part_sum,
             int32_t* __restrict__ part_count) {
  pdl_trigger();
  pdl_wait();
  const int64_t out = (int64_t)blockIdx.x * (r.E + 1);
  block_losses<T, L, V, kWarps>(r, logits, idx, mask, vec, part_sum + out, part_count + out);
}

// The losses from the sums over all tokens, by one block of 1024 threads: thread e <= E holds
// expert e's sum of p (e = E: the sum of logsumexp^2) and count (e = E: the tokens).
__device__ __forceinline__ void finish_losses(const Routing& r, double sum, int32_t count,
                                              float* __restrict__ losses, int32_t* __restrict__ counts,
                                              float* __restrict__ prob_mean) {
  __shared__ double s_bal[32], s_z;
  __shared__ int32_t s_tokens;
  const int e = threadIdx.x;
  if (e == r.E) {
    s_z = sum;
    s_tokens = count;
  }
  __syncthreads();
  const double tokens = s_tokens > 0 ? (double)s_tokens : 1.0;
  double bal = 0.0;
  if (e <= r.E) counts[e] = count;
  if (e < r.E) {
    const double mean = sum / tokens;
    prob_mean[e] = (float)mean;
    bal = (double)count / tokens * mean;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) bal += __shfl_xor_sync(0xffffffffu, bal, o);
  if ((e & 31) == 0) s_bal[e >> 5] = bal;
  __syncthreads();
  if (e == 0) {
    double all = 0.0;
    for (int w = 0; w < (r.E + 31) / 32; ++w) all += s_bal[w];
    losses[0] = (float)(all * r.E);
    losses[1] = (float)(s_z / tokens);
  }
}

// The blocks of the grid are one cluster of 8, each with its E + 1 sums and counts in shared
// memory: the first adds them up in order.
constexpr int kLossCluster = 8;

__device__ __forceinline__ void finish_cluster(const Routing& r, const double* s_sum, const int32_t* s_count,
                                               float* __restrict__ losses, int32_t* __restrict__ counts,
                                               float* __restrict__ prob_mean) {
  cluster_sync();
  if (blockIdx.x == 0) {
    double sum = 0.0;
    int32_t count = 0;
    if ((int)threadIdx.x <= r.E) {
      const uint32_t a = (uint32_t)__cvta_generic_to_shared(&s_sum[threadIdx.x]);
      const uint32_t b = (uint32_t)__cvta_generic_to_shared(&s_count[threadIdx.x]);
#pragma unroll
      for (int w = 0; w < kLossCluster; ++w) {
        uint32_t there;
        double s;
        int32_t c;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(a), "r"(w));
        asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(s) : "r"(there) : "memory");
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(b), "r"(w));
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c) : "r"(there) : "memory");
        sum += s;
        count += c;
      }
    }
    finish_losses(r, sum, count, losses, counts, prob_mean);
  }
  cluster_sync();  // no block leaves while the first reads its sums
}

// Little work: one launch, a cluster of 8 blocks of 1024 threads whose first block adds the sums
// up from their shared memory; no workspace. It saves a launch and an allocation of the caller's
// (some 4 us), but has 8 SMs only: it is the quicker form for single calls, the slower one in a captured
// graph. Device and whole call with no mask, one launch / two passes: 4096 x 8 8.2 / 6.7 and 13.0 / 17.1 us, 8192 x 8 11.9 / 7.3 and 13.0 / 17.1, 4096 x 64 10.7 / 7.6 and
// 13.2 / 17.3, 8192 x 64 16.5 / 8.1 and 16.8 / 17.3, 1024 x 256 10.2 / 8.1 and 13.0 / 17.1, 4096 x 256
// 28.1 / 11.4 and 28.7 / 17.1.
constexpr int64_t kLossTokens = 8192, kLossLogits = 1 << 18;

template <typename T, int L, int V>
__global__ void __launch_bounds__(1024)
    k_losses_few(const Routing r, const T* __restrict__ logits, const int32_t* __restrict__ idx,
                 const uint8_t* __restrict__ mask, int vec, float* __restrict__ losses,
                 int32_t* __restrict__ counts, float* __restrict__ prob_mean) {
  pdl_trigger();
  pdl_wait();
  __shared__ double s_part[L * V + 1];
  __shared__ int32_t s_parts[L * V + 1];
  block_losses<T, L, V, 32>(r, logits, idx, mask, vec, s_part, s_parts);
  finish_cluster(r, s_part, s_parts, losses, counts, prob_mean);
}

// Second pass, a cluster of 8 blocks: thread (e, part) adds every (8 nparts)-th block's partials,
// four loads at a time, then a block's parts are added in pairs, and the blocks and the experts in
// order. One block alone reads some 60 bytes a cycle: 65521 x 64 17.1 us for both passes instead of
// 13.2, 16384 x 256 34.9 instead of 15.8; only up to 16 experts is it quicker, by 0.3 us.
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
  const int n = r.E + 1;
  const int nparts = 1024 / n;
  const int part = threadIdx.x / n, e = threadIdx.x - part * n;
  const int step = kLossCluster * nparts;
  double sum = 0.0;
  int32_t count = 0;
  if (part < nparts) {
    for (int b = (int)blockIdx.x * nparts + part; b < blocks; b += 4 * step) {
      double s[4];
      int32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = b + i * step;
        s[i] = at < blocks ? part_sum[(int64_t)at * n + e] : 0.0;
        c[i] = at < blocks ? part_count[(int64_t)at * n + e] : 0;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum += s[i];
        count += c[i];
      }
    }
  }
  s_sum[threadIdx.x] = sum;
  s_count[threadIdx.x] = count;
  __syncthreads();
  // the parts in pairs, log2 steps
  int live = nparts;
  while (live > 1) {
    const int half = (live + 1) / 2;
    if (part < live - half) {
      s_sum[threadIdx.x] += s_sum[threadIdx.x + half * n];
      s_count[threadIdx.x] += s_count[threadIdx.x + half * n];
    }
    live = half;
    __syncthreads();
  }
  finish_cluster(r, s_sum, s_count, losses, counts, prob_mean);
}

// Gradient in the logits. With g_j = weight_scale * d_topk_w[j], and for the losses
// c_e = d0 E count_e / N^2 (the counts are constants):
//   softmax, renormalised: u = softmax over the chosen logits; dl_j = u_j (g_j - sum g u)
//     (the sum over all experts cancels, and with it the loss of digits in it);
//   softmax: dl_e = p_e ([chosen] g_e - sum g p);
//   sigmoid, renormalised: dl_j = (1 - s_j) u_j (g_j - sum g u), u = s / sum of chosen s
//     (u and the balance's s / sum s of very negative logits from logits moved up);
//   sigmoid: dl_j = s_j (1 - s_j) g_j;
//   balance: softmax p_e (c_e - sum c p); sigmoid s_e (1 - s_e) (c_e - sum c p) / sum s;
//   z: 2 d1 / N * logsumexp * softmax_e.
// A slot's term crosses from its lane to its expert's through shared memory. Bound by
// instructions (600 a token at 256 experts, 57% of the issue slots): 16384 x 256 with sigmoid scores
// and losses 16.9 us (34.6 MB: 5.3 us at HBM's rate), 4096 x 8 4.4 us. The exponentials are 2^x (see
// fast_exp2) and the divisions of sums __fdividef (2 units in the last place): some 2 and 1 u more
// than expf and a rounded division, of the 128 u that a gradient's terms are held to.
template <typename T, int L, int V>
__global__ void __launch_bounds__(32 * kWarps, V <= 4 ? 6 : V <= 8 ? 4 : 2)
    k_route_bwd(const Routing r, const T* __restrict__ logits, const int32_t* __restrict__ idx,
                const float* __restrict__ d_w, const int32_t* __restrict__ counts,
                const float* __restrict__ d_losses, const uint8_t* __restrict__ mask, int vec,
                int vec_out, T* __restrict__ d_logits) {
  pdl_trigger();
  pdl_wait();
  const Team<L> team;
  constexpr int kPer = 32 / L * kWarps;
  __shared__ __align__(16) float s_slots[kWarps * 32 / L][L * V];
  float* slots = s_slots[threadIdx.x / L];
  int pairs = 1;  // lanes up to the next power of two of k
  while (pairs < r.k) pairs *= 2;
  const unsigned slot_mask = (pairs == 32 ? 0xffffffffu : (1u << pairs) - 1u) << team.base;
  // over the slots' lanes (the others get what theirs amount to)
  const auto slots_sum = [&](float v) {
    for (int o = pairs >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(team.mask, v, o);
    return v;
  };
  const auto slots_max = [&](float v) {
    for (int o = pairs >> 1; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(team.mask, v, o));
    return v;
  };
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
    float p[V], dl[V], lse = 0.f, top = 0.f, inv = 0.f;
    const bool need_p = losses || (d_w && !r.sigmoid && !r.renorm);
    if (need_p) {
      mx = team.max(mx);
      top = mx > -INFINITY ? mx : 0.f;  // exp(l - top) is 0 where no expert has a score
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        p[v] = fast_exp2(kLog2e * (l[v] - top));
        sum += p[v];
      }
      sum = team.sum(sum);
      lse = sum > 0.f ? top + logf(sum) : 0.f;
      inv = sum > 0.f ? __fdividef(1.f, sum) : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] *= inv;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) dl[v] = 0.f;
    if (losses) {
      float cs = 0.f;
      if (r.sigmoid) {
        const float shift = share_shift(top);
        float s[V], sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float rest;
          sigmoid_pair(l[v] - shift, s[v], rest);
          sum += s[v];
          cs += c[v] * s[v];
          dl[v] = s[v] * rest;
        }
        sum = team.sum(sum);
        const float over = sum > 0.f ? __fdividef(1.f, sum) : 0.f;
        cs = team.sum(cs) * over;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          dl[v] = dl[v] * ((c[v] - cs) * over) + zc * lse * p[v];
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
        if (my_e >= 0) sigmoid_pair(ls, u, rest);
      } else if (r.renorm) {
        const float top = slots_max(ls);
        if (ls > -INFINITY) u = fast_exp2(kLog2e * (ls - top));
      }
      float term = 0.f;  // what slot `rank` adds to its expert
      if (r.renorm) {
        float sum = slots_sum(u);
        if (r.sigmoid && sum < 0x1p-46f && team.rank < pairs) {  // all of the slots' lanes, or none
          float most = ls;
          for (int o = pairs >> 1; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(slot_mask, most, o));
          u = most > kNoScore ? fast_exp2(kLog2e * (ls - most)) : 0.f;
          sum = u;
          for (int o = pairs >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(slot_mask, sum, o);
        }
        u = sum > 0.f ? __fdividef(u, sum) : 0.f;
        term = u * (g - slots_sum(g * u)) * rest;
      } else if (r.sigmoid) {
        term = u * rest * g;
      } else {
        float gp = 0.f;
        // as p is formed: lse, once rounded, would bring in an error of |lse| 2^-24
        if (my_e >= 0) u = fast_exp2(kLog2e * (ls - top)) * inv;
        gp = team.sum(g * u);  // every lane needs it
        term = u * g;
#pragma unroll
        for (int v = 0; v < V; ++v) dl[v] -= p[v] * gp;
      }
      // From the slots' lanes to their experts': plain stores, and where a list names an expert
      // more than once (a slot does not find its own rank again) additions in the slots' order.
      float* own = slots + team.rank * V;
      __syncwarp(team.mask);
      if constexpr (V % 4 == 0) {
#pragma unroll
        for (int v = 0; v < V; v += 4) *reinterpret_cast<float4*>(own + v) = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) own[v] = 0.f;
      }
      __syncwarp(team.mask);
      if (my_e >= 0) slots[my_e] = (float)team.rank;
      __syncwarp(team.mask);
      const bool shared = my_e >= 0 && slots[my_e] != (float)team.rank;
      const bool any = __any_sync(team.mask, shared);  // every lane has read by then
      if (my_e >= 0) slots[my_e] = any ? 0.f : term;
      __syncwarp(team.mask);
      if (any) {
        for (int s = 0; s < r.k; ++s) {
          if (my_e >= 0 && team.rank == s) slots[my_e] += term;
          __syncwarp(team.mask);
        }
      }
      if constexpr (V % 4 == 0) {
#pragma unroll
        for (int v = 0; v < V; v += 4) {
          const float4 f = *reinterpret_cast<const float4*>(own + v);
          dl[v] += f.x, dl[v + 1] += f.y, dl[v + 2] += f.z, dl[v + 3] += f.w;
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) dl[v] += own[v];
      }
    }
    store_row<T, V>(d_logits + t * r.E, team.rank, r.E, vec_out, dl);
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

// Routing: a lane per slot, and one per group at least; up to 8 slots by the merge. Few tokens
// leave the SMs idle, so up to 128 experts their teams are wider: shorter chains, and lanes
// for near ties beside 8 slots (250 x 64: sigmoid scores with a bias 10.4 -> 3.9 us, softmax
// without renormalising 5.3 -> 4.5; but 65536 x 64 24 -> 40, and 1024 x 256 5.5 -> 6.0).
template <typename F>
cudaError_t by_choice(const Routing& r, F f) {
  const auto few = [&](auto l, auto v) { return f(l, v, std::true_type()); };
  const auto many = [&](auto l, auto v) { return f(l, v, std::false_type()); };
  if (r.k <= 8 && r.groups <= 8) {
    if (r.E <= 8) return with<8, 1>(few);
    if (r.E <= 16) return with<8, 2>(few);
    if (r.E <= 32) return with<8, 4>(few);
    const bool wide = r.T <= 4096;
    if (r.E <= 64) return wide ? with<16, 4>(few) : with<8, 8>(few);
    if (r.E <= 128) return wide ? with<16, 8>(few) : with<8, 16>(few);
    if (r.E <= 256) return with<16, 16>(few);
    return with<32, 16>(few);
  }
  if (r.E <= 64) return with<32, 2>(many);
  if (r.E <= 128) return with<32, 4>(many);
  if (r.E <= 256) return with<32, 8>(many);
  return with<32, 16>(many);
}

// Losses and gradient: a lane per slot.
template <typename F>
cudaError_t by_sizes(const Routing& r, F f) {
  if (r.k <= 8) {
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

// Whether every lane's V values start on a boundary of their size (16 bytes at most).
template <typename T, int V>
int vectors(const Routing& r, const T* p, int64_t stride) {
  constexpr size_t kBytes = V * sizeof(T) < 16 ? V * sizeof(T) : 16;
  return r.E % V == 0 && reinterpret_cast<uintptr_t>(p) % kBytes == 0 &&
         (r.T == 1 || stride * (int64_t)sizeof(T) % (int64_t)kBytes == 0);
}

}  // namespace

cudaError_t launch_route(const Routing& r, const void* logits, const float* bias, int32_t* idx,
                         float* w, cudaStream_t st) {
  return by_choice(r, [&](auto l, auto v, auto few) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value;
    constexpr bool FEW = decltype(few)::value;
    const dim3 grid(token_blocks<L>(r, V <= 4 ? 4 : V <= 8 ? 3 : 2)), block(32 * kWarps);
    if (r.bf16) {
      const auto* p = static_cast<const __nv_bfloat16*>(logits);
      return launch_pdl(k_route<__nv_bfloat16, L, V, FEW>, grid, block, 0, st, r, p, bias,
                        vectors<__nv_bfloat16, V>(r, p, r.stride), idx, w);
    }
    const auto* p = static_cast<const float*>(logits);
    return launch_pdl(k_route<float, L, V, FEW>, grid, block, 0, st, r, p, bias,
                      vectors<float, V>(r, p, r.stride), idx, w);
  });
}

namespace {
bool few_for_losses(const Routing& r) {
  return r.E <= 256 && r.T <= kLossTokens && r.T * r.E <= kLossLogits;
}
}  // namespace

int router_loss_blocks(const Routing& r) {
  if (few_for_losses(r)) return 0;
  int n = 0;
  by_sizes(r, [&](auto l, auto v) {
    n = (int)token_blocks<decltype(l)::value>(r, decltype(v)::value <= 8 ? 3 : 2);
    return cudaSuccess;
  });
  return n;
}

cudaError_t launch_router_losses(const Routing& r, const void* logits, const int32_t* idx,
                                 const uint8_t* mask, float* losses, int32_t* counts,
                                 float* prob_mean, double* part_sum, int32_t* part_count,
                                 cudaStream_t st) {
  if (few_for_losses(r))
    return by_sizes(r, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, V = decltype(v)::value;
      if constexpr (V > 8) {
        return cudaErrorInvalidValue;  // not reached: E <= 256
      } else {
        if (r.bf16) {
          const auto* p = static_cast<const __nv_bfloat16*>(logits);
          return launch_cluster(k_losses_few<__nv_bfloat16, L, V>, kLossCluster, 1024, 0, kLossCluster,
                                st, r, p, idx, mask, vectors<__nv_bfloat16, V>(r, p, r.stride), losses,
                                counts, prob_mean);
        }
        const auto* p = static_cast<const float*>(logits);
        return launch_cluster(k_losses_few<float, L, V>, kLossCluster, 1024, 0, kLossCluster, st, r, p,
                              idx, mask, vectors<float, V>(r, p, r.stride), losses, counts, prob_mean);
      }
    });
  const int blocks = router_loss_blocks(r);
  if (blocks > 0) {
    const cudaError_t e = by_sizes(r, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, V = decltype(v)::value;
      const dim3 grid((unsigned)blocks), block(32 * kWarps);
      if (r.bf16) {
        const auto* p = static_cast<const __nv_bfloat16*>(logits);
        return launch_pdl(k_losses<__nv_bfloat16, L, V>, grid, block, 0, st, r, p, idx, mask,
                          vectors<__nv_bfloat16, V>(r, p, r.stride), part_sum, part_count);
      }
      const auto* p = static_cast<const float*>(logits);
      return launch_pdl(k_losses<float, L, V>, grid, block, 0, st, r, p, idx, mask,
                        vectors<float, V>(r, p, r.stride), part_sum, part_count);
    });
    if (e != cudaSuccess) return e;
  }
  return launch_cluster(k_losses_end, kLossCluster, 1024, 0, kLossCluster, st, r, blocks, part_sum,
                        part_count, losses, counts, prob_mean);
}

cudaError_t launch_route_backward(const Routing& r, const void* logits, const int32_t* idx,
                                  const float* d_w, const int32_t* counts, const float* d_losses,
                                  const uint8_t* mask, void* d_logits, cudaStream_t st) {
  return by_sizes(r, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value;
    const dim3 grid(token_blocks<L>(r, V <= 4 ? 6 : V <= 8 ? 4 : 2)), block(32 * kWarps);
    if (r.bf16) {
      const auto* p = static_cast<const __nv_bfloat16*>(logits);
      return launch_pdl(k_route_bwd<__nv_bfloat16, L, V>, grid, block, 0, st, r, p, idx, d_w, counts,
                        d_losses, mask, vectors<__nv_bfloat16, V>(r, p, r.stride),
                        vectors<__nv_bfloat16, V>(r, static_cast<__nv_bfloat16*>(d_logits), r.E),
                        static_cast<__nv_bfloat16*>(d_logits));
    }
    const auto* p = static_cast<const float*>(logits);
    return launch_pdl(k_route_bwd<float, L, V>, grid, block, 0, st, r, p, idx, d_w, counts, d_losses,
                      mask, vectors<float, V>(r, p, r.stride),
                      vectors<float, V>(r, static_cast<float*>(d_logits), r.E),
                      static_cast<float*>(d_logits));
  });
}

}  // namespace moe
