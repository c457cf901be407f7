// Gate with expert groups (moe_gate) and its backward.
//
//   s = softmax or logistic function of the logits, c = s + bias; the best
//   topk_groups of the expert groups stay, ranked by their two largest c; the K
//   largest c of those groups are chosen; the gates are the chosen s, rescaled.
//
// A row of at most 1024 logits is a few instructions for each score and a
// selection, so a warp takes a token and keeps the row in registers: the lanes
// are dealt out to the groups, neighbours of a group to neighbouring lanes, and
// a group's two largest scores meet in a segmented shuffle.  The selection goes
// through a threshold: the K-th largest of the lanes' maxima is a lower bound of
// the K-th largest score, and the few scores at or above it (K plus about a
// quarter) are collected into one lane each and ranked by counting.
//
// The choice is that of 64-bit scores.  fp32 scores carry a bound on their error;
// where two scores that decide something (a rank among the first K, a group in or
// out) are closer than their bounds, the few scores in question are computed
// again in fp64 (GB300 does 1/64 of its fp32 rate there: a whole row in fp64, the
// simplest form of this kernel, took 1628 us for 32768 x 384 logits).  Without a
// bias the logits are compared, which order as the scores do.
#include <limits.h>
#include <math.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int WARPS = 4;

// how the lanes of a warp are dealt out
struct GateShape {
  int T, E, K;
  int G, KG;       // groups and how many stay; 1 and 1 without a limit
  int gs, lpg, vpl;  // experts of a group, lanes of a group, experts of a lane
  int mode;
  float scale;
};

__device__ __forceinline__ int order_key(float x) {  // integers that order as the floats do
  const int k = __float_as_int(x);
  return k ^ ((k >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_key(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

struct Row64 {  // what a row's 64-bit scores need
  const float* row;
  const float* bias;
  double m, z;
  bool sigmoid;
  __device__ double score(float l) const {
    if (l == -INFINITY) return 0.0;
    return sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - m) / z;
  }
  __device__ double value(int e) const {  // c, -inf where it takes no part
    const float l = row[e];
    const double v = bias ? score(l) + (double)bias[e] : score(l);
    return l == -INFINITY || v != v ? -INFINITY : v;
  }
};

__device__ __noinline__ Row64 row64(const float* row, const float* bias, int E, bool sigmoid, float m) {
  Row64 r{row, bias, (double)m, 1.0, sigmoid};
  if (!sigmoid) {
    double z = 0;
    for (int e = threadIdx.x & 31; e < E; e += 32) z += m == -INFINITY ? 0.0 : exp((double)row[e] - r.m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(FULL, z, o);
    r.z = z;
  }
  return r;
}

// groups ranked by 64-bit scores: lane g of a group's first lane returns whether its group stays
__device__ __noinline__ bool keep_groups64(const Row64& r, const GateShape& p, int g, int lig, float second,
                                           float margin) {
  const int lane = threadIdx.x & 31;
  const bool group_max = p.mode & MOE_GATE_GROUP_MAX;
  double a = -INFINITY, b = -INFINITY;
  if (g < p.G)
    for (int j = 0; j < p.vpl; ++j) {
      const int pos = lig * p.vpl + j;
      if (pos >= p.gs) break;
      const int e = g * p.gs + pos;
      // only what may be among the group's two largest: `second` is the second largest in fp32
      float c = r.row[e];
      if (r.bias) c = (r.sigmoid ? 1.f / (1.f + expf(-c)) : expf(c - (float)r.m) / (float)r.z) + r.bias[e];
      if (c < second - margin) continue;
      const double v = r.value(e);
      if (v > a) { b = a; a = v; } else if (v > b) b = v;
    }
  for (int o = 1; o < p.lpg; o <<= 1) {
    const double c = __shfl_down_sync(FULL, a, o), d = __shfl_down_sync(FULL, b, o);
    if (lig + o < p.lpg) {
      b = fmax(fmin(a, c), fmax(b, d));
      a = fmax(a, c);
    }
  }
  double rank = group_max || b == -INFINITY ? a : a + b;
  rank = __shfl_sync(FULL, rank, lane - lig);
  int ahead = 0;
  for (int o = 0; o < p.G; ++o) {
    const double w = __shfl_sync(FULL, rank, o * p.lpg);
    ahead += w > rank || (w == rank && o < g);
  }
  return ahead < p.KG;
}

// the K best of the kept groups in 64 bits, K rounds over the row: rows with fewer than K
// experts in service, or with more equal scores than a warp holds.  keep: bit g set where
// group g stays.  Lane k returns the k-th chosen expert.
__device__ __noinline__ int choose64(const Row64& r, const GateShape& p, unsigned keep) {
  const int lane = threadIdx.x & 31;
  int mine = 0;
  double last = INFINITY;
  int last_e = -1;
  for (int k = 0; k < p.K; ++k) {
    // the best behind the one taken last, in the order (value desc, expert asc)
    double v = -INFINITY;
    int e = 0x7fffffff;
    for (int i = lane; i < p.E; i += 32) {
      if (!((keep >> (i / p.gs)) & 1u)) continue;
      const float l = r.row[i];
      double w = r.bias ? r.value(i) : (l != l ? -INFINITY : (double)l);
      if (w > last || (w == last && i <= last_e)) continue;
      if (e == 0x7fffffff || w > v) {
        v = w;
        e = i;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double w = __shfl_xor_sync(FULL, v, o);
      const int f = __shfl_xor_sync(FULL, e, o);
      if (f != 0x7fffffff && (e == 0x7fffffff || w > v || (w == v && f < e))) {
        v = w;
        e = f;
      }
    }
    if (lane == k) mine = e;
    last = v;
    last_e = e;
  }
  return mine;
}

// the gates of the chosen experts from their logits; lanes with on = false take no part
__device__ __forceinline__ float gate_value(float l, bool on, bool sigmoid, bool renorm, float m, float z) {
  float base = 0.f;
  if (renorm) {  // a common factor of the row: its largest chosen score becomes about 1
    base = warp_max(on ? l : -INFINITY);
    if (sigmoid) base = fminf(base, 0.f);
  }
  float s = 0.f;
  if (on && l != -INFINITY)
    s = sigmoid ? expf(fminf(l, 0.f) - base) / (1.f + expf(-fabsf(l))) : expf(l - (renorm ? base : m));
  if (renorm) {
    const float sum = warp_sum(s);
    return sum > 0.f || sum != sum ? s / sum : 0.f;
  }
  return sigmoid || s == 0.f ? s : s / z;
}

template <int VMAX>
__global__ void __launch_bounds__(32 * WARPS)
gate_kernel(float* __restrict__ logits, const float* __restrict__ part, int S, const float* __restrict__ bias,
            GateShape p, int32_t* __restrict__ idx, float* __restrict__ gate) {
  __shared__ float cand_c[WARPS][32], cand_l[WARPS][32];
  __shared__ int cand_e[WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned below = (1u << lane) - 1;
  const bool sigmoid = (p.mode & 0xf) == MOE_GATE_SIGMOID, renorm = p.mode & MOE_GATE_RENORM;
  const bool group_max = p.mode & MOE_GATE_GROUP_MAX;
  const int g = lane / p.lpg, lig = lane - g * p.lpg;
  const int pos0 = lig * p.vpl;
  // experts of this lane: e0 .. e0 + count - 1
  const int count = g < p.G ? max(0, min(p.vpl, p.gs - pos0)) : 0;
  const int e0 = g * p.gs + pos0;
  const bool vec = ((p.vpl | p.gs) & 3) == 0;  // whole 16-byte pieces, aligned in every row

  auto load = [&](const float* a, float fill, float (&v)[VMAX]) {
    if (vec) {
#pragma unroll
      for (int q = 0; q < (VMAX + 3) / 4; ++q) {
        float4 f = make_float4(fill, fill, fill, fill);
        if (4 * q < count) f = *reinterpret_cast<const float4*>(a + e0 + 4 * q);
        const float w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * q + j < VMAX) v[4 * q + j] = w[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < VMAX; ++j) v[j] = j < count ? a[e0 + j] : fill;
    }
  };

  float b[VMAX], margin = 0.f;
  if (bias) {
    load(bias, 0.f, b);
    float mb = 0.f;
#pragma unroll
    for (int j = 0; j < VMAX; ++j) mb = fmaxf(mb, fabsf(b[j]) < INFINITY ? fabsf(b[j]) : 0.f);
    mb = warp_max(mb);
    // twice the error of a score (u = 2^-24): expf 4u, the sum and quotient 4u; softmax: the
    // sum over vpl values and 5 shuffles; then the rounding of s + b
    const float u = 5.9604645e-8f;
    margin = 2.f * u * ((sigmoid ? 12.f : 20.f + p.vpl) + mb);
  }

  for (long long t = (long long)blockIdx.x * WARPS + warp; t < p.T; t += (long long)gridDim.x * WARPS) {
    float* row = logits + t * p.E;
    float l[VMAX];
    if (part) {
      load(part + t * p.E, -INFINITY, l);
      for (int i = 1; i < S; ++i) {
        float w[VMAX];
        load(part + ((long long)i * p.T + t) * p.E, 0.f, w);
#pragma unroll
        for (int j = 0; j < VMAX; ++j) l[j] += w[j];
      }
#pragma unroll
      for (int j = 0; j < VMAX; ++j)
        if (j < count) row[e0 + j] = l[j];
      __syncwarp();
    } else {
      load(row, -INFINITY, l);
    }
    bool bad = false;
#pragma unroll
    for (int j = 0; j < VMAX; ++j) bad |= l[j] != l[j];
    bad = __any_sync(FULL, bad);

    // softmax: the row's maximum and sum, where something needs them
    float m = 0.f, z = 1.f;
    const bool by_sum = p.KG < p.G && !group_max;
    if (!sigmoid && (bias || !renorm || by_sum)) {
      m = -INFINITY;
#pragma unroll
      for (int j = 0; j < VMAX; ++j) m = fmaxf(m, l[j]);
      m = from_key(__reduce_max_sync(FULL, order_key(m)));
    }
    // the selection values: scores plus bias, or the logits
    float c[VMAX];
    if (bias) {
      if (sigmoid) {
#pragma unroll
        for (int j = 0; j < VMAX; ++j) c[j] = __fdividef(1.f, 1.f + expf(-l[j]));
      } else {
        z = 0.f;
#pragma unroll
        for (int j = 0; j < VMAX; ++j) {
          c[j] = l[j] == -INFINITY ? 0.f : expf(l[j] - m);
          z += c[j];
        }
        z = warp_sum(z);
        const float r = 1.f / z;
#pragma unroll
        for (int j = 0; j < VMAX; ++j) c[j] *= r;
      }
#pragma unroll
      for (int j = 0; j < VMAX; ++j) {
        c[j] += b[j];
        if (l[j] == -INFINITY || c[j] != c[j]) c[j] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int j = 0; j < VMAX; ++j) c[j] = l[j] != l[j] ? -INFINITY : l[j];
      if (!sigmoid && !renorm) {
        z = 0.f;
#pragma unroll
        for (int j = 0; j < VMAX; ++j) z += l[j] == -INFINITY ? 0.f : expf(l[j] - m);
        z = warp_sum(z);
      }
    }

    bool stay = g < p.G;
    if (p.KG < p.G) {
      float a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
      for (int j = 0; j < VMAX; ++j) {
        a2 = fmaxf(a2, fminf(a1, c[j]));
        a1 = fmaxf(a1, c[j]);
      }
      for (int o = 1; o < p.lpg; o <<= 1) {
        const float d1 = __shfl_down_sync(FULL, a1, o), d2 = __shfl_down_sync(FULL, a2, o);
        if (lig + o < p.lpg) {
          a2 = fmaxf(fminf(a1, d1), fmaxf(a2, d2));
          a1 = fmaxf(a1, d1);
        }
      }
      // a group's rank and how far it may be off
      float rank, off = 0.f;
      if (group_max) {
        rank = a1;
        off = margin;
      } else if (bias) {
        rank = a2 == -INFINITY ? a1 : a1 + a2;
        off = 2.f * margin + fabsf(rank) * 1.2e-7f;
      } else {
        const float base = sigmoid ? 0.f : m;
        auto score = [&](float x) {
          return x == -INFINITY ? 0.f : sigmoid ? 1.f / (1.f + expf(-x)) : expf(x - base);
        };
        rank = a1 == -INFINITY ? a1 : score(a1) + score(a2);
        // u = 2^-24: expf 4u, the rounding of its argument |a1 - m| u, sum and quotient 4u, on
        // both sides; and what numbers below 2^-126 lose
        off = rank * 1.2e-7f * (12.f + (sigmoid || a1 == -INFINITY ? 0.f : fabsf(a1 - m))) + 4e-45f;
      }
      const int first = lane - lig;
      rank = __shfl_sync(FULL, rank, first);
      off = __shfl_sync(FULL, off, first);
      a2 = __shfl_sync(FULL, a2, first);
      int ahead = 0, surely = 0, maybe = 0;
      for (int o = 0; o < p.G; ++o) {
        const float w = __shfl_sync(FULL, rank, o * p.lpg);
        ahead += w > rank || (w == rank && o < g);
        surely += w > rank + off;
        maybe += w >= rank - off;
      }
      stay = stay && ahead < p.KG;
      // the comparison of logits, or of groups that are out altogether, is exact
      const bool exact = (group_max && !bias) || rank == -INFINITY;
      const bool open = g < p.G && !exact && maybe > p.KG && surely < p.KG;  // `maybe` counts the group itself
      if (__any_sync(FULL, open))
        stay = keep_groups64(row64(row, bias, p.E, sigmoid, m), p, g, lig, group_max ? a1 : a2, margin) && g < p.G;
      if (!stay) {
#pragma unroll
        for (int j = 0; j < VMAX; ++j) c[j] = -INFINITY;
      }
    }

    // a bound of the K-th largest from the lanes' maxima
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < VMAX; ++j) top = fmaxf(top, c[j]);
    int key = order_key(top), kth = key;
    for (int k = 0; k < p.K; ++k) {
      kth = __reduce_max_sync(FULL, key);
      if (key == kth) key = INT_MIN;
    }
    float limit = kth == INT_MIN ? -INFINITY : from_key(kth);
    auto collect = [&]() {
      unsigned n = 0;
      const float lim = limit - margin;
#pragma unroll
      for (int j = 0; j < VMAX; ++j) {
        const bool in = c[j] >= lim && c[j] > -INFINITY;
        const unsigned who = __ballot_sync(FULL, in);
        const unsigned at = n + __popc(who & below);
        if (in && at < 32) {
          cand_c[warp][at] = c[j];
          cand_l[warp][at] = l[j];
          cand_e[warp][at] = e0 + j;
        }
        n += __popc(who);
      }
      return (int)n;
    };
    int n = collect();
    if (n > 32) {
      // few lanes hold the kept groups: the K-th largest itself, K rounds over the registers
      float lower = INFINITY;
      int taken = 0;
      while (taken < p.K) {
        float best = -INFINITY;
#pragma unroll
        for (int j = 0; j < VMAX; ++j)
          if (c[j] < lower) best = fmaxf(best, c[j]);
        best = from_key(__reduce_max_sync(FULL, order_key(best)));
        int same = 0;
#pragma unroll
        for (int j = 0; j < VMAX; ++j) same += c[j] == best;
        if (lower == INFINITY) {  // values of +inf come first and are never below `lower`
          int inf = 0;
#pragma unroll
          for (int j = 0; j < VMAX; ++j) inf += c[j] == INFINITY;
          taken += __reduce_add_sync(FULL, inf);
          if (taken >= p.K) best = INFINITY;
        }
        if (best != INFINITY) taken += __reduce_add_sync(FULL, same);
        lower = best;
        if (best == INFINITY) break;
      }
      limit = lower;
      __syncwarp();
      n = collect();
    }
    __syncwarp();

    int e = 0, place = 32;
    float mine = -INFINITY;
    if (n >= p.K && n <= 32) {
      float v = -INFINITY;
      if (lane < n) {
        v = cand_c[warp][lane];
        mine = cand_l[warp][lane];
        e = cand_e[warp][lane];
      }
      int ahead = 0, near = 0;
      for (int i = 0; i < n; ++i) {
        const float w = cand_c[warp][i];
        ahead += w > v || (w == v && cand_e[warp][i] < e);
        near += fabsf(w - v) <= margin;
      }
      place = lane < n ? ahead : 32;
      // `near` counts the lane itself; without a bias values compare exactly
      if (bias && __any_sync(FULL, lane < n && near > 1)) {
        const Row64 r = row64(row, bias, p.E, sigmoid, m);
        const double x = lane < n ? r.value(e) : 0.0;
        place = 0;
        for (int i = 0; i < n; ++i) {
          const double w = __shfl_sync(FULL, x, i);
          const int f = __shfl_sync(FULL, e, i);
          place += w > x || (w == x && f < e);
        }
        if (lane >= n) place = 32;
      }
    } else {
      const unsigned who = __ballot_sync(FULL, stay && lig == 0);
      unsigned keep = 0;
      for (int o = 0; o < p.G; ++o) keep |= ((who >> (o * p.lpg)) & 1u) << o;
      e = choose64(row64(row, bias, p.E, sigmoid, m), p, keep);
      if (lane < p.K) {
        place = lane;
        mine = row[e];
      }
    }
    const bool on = place < p.K;
    const float s = gate_value(mine, on, sigmoid, renorm, m, z);
    if (on) {
      idx[t * p.K + place] = e;
      gate[t * p.K + place] = bad ? __int_as_float(0x7fffffff) : s * p.scale;
    }
    __syncwarp();
  }
}

__global__ void __launch_bounds__(32 * WARPS)
gate_bwd_kernel(const float* __restrict__ d_gate, const float* __restrict__ logits, const int32_t* __restrict__ idx,
                int T, int E, int K, int mode, float scale, float* __restrict__ d_logits, unsigned* err) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool sigmoid = (mode & 0xf) == MOE_GATE_SIGMOID, renorm = mode & MOE_GATE_RENORM;
  for (long long t = (long long)blockIdx.x * WARPS + warp; t < T; t += (long long)gridDim.x * WARPS) {
    const float* row = logits + t * E;
    int e = -1;
    float dg = 0.f, l = -INFINITY;
    if (lane < K) {
      e = idx[t * K + lane];
      if (e < 0 || e >= E) {
        set_error(err, DEV_BOUNDS);
        e = -1;
      } else {
        dg = d_gate[t * K + lane];
        l = row[e];
      }
    }
    float m = l, z = 0.f;
    if (!sigmoid && !renorm)
      for (int i = lane; i < E; i += 32) m = fmaxf(m, row[i]);
    m = warp_max(m);
    if (sigmoid) m = fminf(m, 0.f);
    if (!sigmoid && !renorm) {
      for (int i = lane; i < E; i += 32) z += m == -INFINITY ? 0.f : expf(row[i] - m);
      z = warp_sum(z);
    }
    // a chosen score, up to the factor exp(m) (a common factor of the row, or 1 without RENORM)
    float s = 0.f, rest = 1.f;
    if (l != -INFINITY) {
      if (sigmoid) {
        const float base = renorm ? m : 0.f;
        s = expf(fminf(l, 0.f) - base) / (1.f + expf(-fabsf(l)));
        rest = 1.f / (1.f + expf(l));
      } else {
        s = expf(l - m);
      }
    }
    const float sum = renorm ? warp_sum(s) : z;
    const float q = sigmoid && !renorm ? s : sum > 0.f ? s / sum : 0.f;
    const float inner = warp_sum(dg * q);
    float d;
    if (sigmoid) d = renorm ? q * rest * (dg - inner) : q * rest * dg;
    else d = q * (renorm ? dg - inner : dg);
    // an expert listed more than once: its first place takes the sum
    float all = 0.f;
    int first = K;
    for (int k = 0; k < K; ++k) {
      const int f = __shfl_sync(FULL, e, k);
      const float o = __shfl_sync(FULL, d, k);
      if (f == e) {
        all += o;
        first = min(first, k);
      }
    }
    float* out = d_logits + t * E;
    for (int i = lane; i < E; i += 32) {
      float v = 0.f;
      if (!sigmoid && !renorm) v = row[i] == -INFINITY ? 0.f : -scale * inner * (expf(row[i] - m) / z);
      out[i] = v;
    }
    __syncwarp();
    if (e >= 0 && first == lane) out[e] = scale * (sigmoid || renorm ? all : all - q * inner);
    __syncwarp();
  }
}

int warp_grid(long long T) {
  const long long ctas = (T + WARPS - 1) / WARPS, cap = (long long)sm_count() * 16;
  return (int)(ctas < cap ? ctas : cap);
}

}  // namespace

int launch_gate(float* logits, const float* part, int S, const float* bias, int T, int E, int K, int G, int KG,
                int mode, float scale, int32_t* idx, float* gate, cudaStream_t s) {
  if (T == 0) return MOE_OK;
  if (KG == G) G = KG = 1;  // every group stays: nothing to rank
  GateShape p{T, E, K, G, KG, E / G, 32 / G, 0, mode, scale};
  p.vpl = (p.gs + p.lpg - 1) / p.lpg;
  if (p.gs % 4 == 0 && p.vpl > 2) p.vpl = (p.vpl + 3) / 4 * 4;  // 16-byte loads
  const int grid = warp_grid(T);
#define MOE_GATE(V) gate_kernel<V><<<grid, 32 * WARPS, 0, s>>>(logits, part, S, bias, p, idx, gate)
  if (p.vpl <= 2) MOE_GATE(2);
  else if (p.vpl <= 4) MOE_GATE(4);
  else if (p.vpl <= 8) MOE_GATE(8);
  else if (p.vpl <= 12) MOE_GATE(12);
  else if (p.vpl <= 16) MOE_GATE(16);
  else if (p.vpl <= 32) MOE_GATE(32);
  else MOE_GATE(64);
#undef MOE_GATE
  return launch_status();
}

int launch_gate_bwd(const float* d_gate, const float* logits, const int32_t* idx, int T, int E, int K, int mode,
                    float scale, float* d_logits, cudaStream_t s) {
  if (T == 0) return MOE_OK;
  gate_bwd_kernel<<<warp_grid(T), 32 * WARPS, 0, s>>>(d_gate, logits, idx, T, E, K, mode, scale, d_logits,
                                                      device_error_word());
  return launch_status();
}

}  // namespace moe
