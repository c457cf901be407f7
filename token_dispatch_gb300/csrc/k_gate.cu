// Gate with expert groups (moe_gate) and its backward.
//
//   s = softmax or logistic function of the logits, c = s + bias; the best
//   topk_groups of the expert groups stay, ranked by their two largest c; the K
//   largest c of those groups are chosen; the gates are the chosen s, rescaled.
//
// A row of at most 1024 logits is a few instructions for each score and a
// selection, so a warp takes a token and keeps the row in registers: the lanes
// are dealt out to the groups, neighbours of a group to neighbouring lanes, and
// a group's two largest scores meet in shuffles.  Each lane keeps its three largest
// scores, and K + 1 rounds of a warp-wide integer maximum take the largest one by one.
//
// The choice is that of 64-bit scores.  fp32 scores carry a bound on their error;
// where two scores that decide something (a rank among the first K, a group in or
// out) are closer than their bounds, the few scores in question are computed
// again in fp64 (GB300 does 1/64 of its fp32 rate there: a whole row in fp64, the
// simplest form of this kernel, took 1628 us for 32768 x 384 logits).  Without a
// bias the logits are compared, which order as the scores do.
//
// What bounds it is instructions, not the 50 MB that 32768 x 384 logits are (7.8 us at the
// rate of a copy): 677 a token there, 63% of the issue slots, 35 us with 8 groups, K = 8 (31 with
// logits that L2 holds; without groups 29.5, 559 a token).  16384 x 64 take 12.3 us (489 a token;
// without groups 10.4), one token 7.2 us, of which a launch is 5-6.  A row
// that needs fp64 takes 2-6 us more of its warp, which shows in calls of one round.
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

// 2^x, 1/x: relative errors of 4u and 2u (u = 2^-24), numbers below 2^-126 as zero.  The
// selection's scores alone are made with them; the gates are not.
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
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
constexpr float LOG2E = 1.4426950408889634f;
constexpr float U = 5.9604645e-8f;  // half a step of fp32

// exp(x), x <= 0, within 6u: x log2(e) in two parts, the second one (the first's rounding and
// the constant's, at most 2^-15) by 1 + d ln 2; below -200, where nothing is left, as -200
__device__ __forceinline__ float exp_neg(float x) {
  x = x < -200.f ? -200.f : x;
  const float t = x * LOG2E;
  const float d = fmaf(x, LOG2E, -t) + x * 1.9259630e-8f;  // log2(e) - LOG2E
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(t));
  return fmaf(y, d * 0.69314718f, y);
}

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
  // what orders the experts: c, without a bias the logits
  __device__ double order(int e) const {
    const float l = row[e];
    return bias ? value(e) : l != l ? -INFINITY : (double)l;
  }
};

// `scored`: scores are asked for, not the logits' order alone (then m is the row's maximum in every lane,
// and a softmax needs its sum)
__device__ __noinline__ Row64 row64(const float* row, const float* bias, int E, bool sigmoid, float m, bool scored) {
  Row64 r{row, bias, (double)m, 1.0, sigmoid};
  if (!sigmoid && scored) {
    double z = 0;
#pragma unroll 4
    for (int e = threadIdx.x & 31; e < E; e += 32) z += m == -INFINITY ? 0.0 : exp((double)row[e] - r.m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(FULL, z, o);
    r.z = z;
  }
  return r;
}

// groups ranked by 64-bit scores: whether the lane's group stays
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
      const double v = group_max ? r.order(e) : r.value(e);
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

// The groups at the border in 64 bits, from the values that the lanes have at hand: f1 >= f2 >= f3
// with their places in the lowest bits, of which those from `bound` on may be among their
// group's two largest.  `open`: the lane's group is at the border; `in`: it surely stays.
// Returns whether the lane's group stays.
__device__ __noinline__ bool settle_groups64(const Row64& r, const GateShape& p, int g, int lig, int e0, const float3& f,
                                             unsigned places, float bound, bool open, bool in) {
  const int lane = threadIdx.x & 31;
  const bool group_max = p.mode & MOE_GATE_GROUP_MAX;
  double a = -INFINITY, b = -INFINITY;
  const float at[3] = {f.x, f.y, f.z};
  for (int i = 0; i < 3; ++i) {
    const bool need = open && at[i] >= bound && at[i] > -INFINITY;
    if (!__any_sync(FULL, need)) break;
    if (need) {
      const int e = e0 + (__float_as_uint(at[i]) & places);
      const double v = group_max ? r.order(e) : r.value(e);
      if (v > a) { b = a; a = v; } else if (v > b) b = v;
    }
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
  const unsigned ins = __ballot_sync(FULL, in && lig == 0), opens = __ballot_sync(FULL, open && lig == 0);
  int ahead = __popc(ins);
  for (unsigned left = opens; left; left &= left - 1) {
    const int from = __ffs(left) - 1;
    const double w = __shfl_sync(FULL, rank, from);
    ahead += w > rank || (w == rank && from < lane - lig);
  }
  return in || (open && ahead < p.KG);
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
      const double w = r.order(i);
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
    if (lane == k) mine = e < p.E ? e : 0;  // KG gs >= K: there always is a next one
    last = v;
    last_e = e;
  }
  return mine;
}

// the gates of the chosen experts from their logits; lanes with on = false take no part
__device__ __forceinline__ float gate_value(float l, bool on, bool sigmoid, bool renorm, float m, float rz) {
  float base = sigmoid ? 0.f : m;
  if (renorm) {  // a common factor of the row: its largest chosen score becomes about 1
    base = from_key(__reduce_max_sync(FULL, on ? order_key(l) : INT_MIN));
    if (sigmoid) base = fminf(base, 0.f);
  }
  float s = 0.f;
  if (on && l != -INFINITY) {
    s = exp_neg((sigmoid ? fminf(l, 0.f) : l) - base);
    if (sigmoid) s *= fast_rcp(1.f + exp_neg(-fabsf(l)));  // a divisor of 1 to 2
  }
  if (renorm) {
    const float sum = warp_sum(s);  // 1/2 to K, or 0
    return sum > 0.f || sum != sum ? s * fast_rcp(sum) : 0.f;
  }
  return sigmoid || s == 0.f ? s : s * rz;
}

// SIGMOID_BIAS: logistic scores with a bias (one set of logits, held by L2: 32768 x 384 32.9 us with both
// as arguments, 30.9 so; 16384 x 384 20.6 and 18.9).  Six CTAs to an SM: 80 registers (131072 x 384 with five 120 us,
// with six 115; 131072 x 64 with eight 80 us, with six 78).
template <int VMAX, bool SIGMOID_BIAS>
__global__ void __launch_bounds__(32 * WARPS, VMAX <= 12 ? 6 : 1)
gate_kernel(float* __restrict__ logits, const float* __restrict__ part, int S, const float* __restrict__ bias,
            GateShape p, int32_t* __restrict__ idx, float* __restrict__ gate) {
  __shared__ __align__(16) float cand_c[WARPS][32];
  __shared__ int cand_e[WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool sigmoid = SIGMOID_BIAS || (p.mode & 0xf) == MOE_GATE_SIGMOID, renorm = p.mode & MOE_GATE_RENORM;
  const bool biased = SIGMOID_BIAS || bias;
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

  float b[VMAX], mb = 0.f;
  // `odd`: a bias of +inf, or one that the logistic scores' upper bound of 1e30 below would cut; one of
  // -inf or NaN takes its expert out of the choice
  bool odd = false;
  if (biased) {
    load(bias, 0.f, b);
#pragma unroll
    for (int j = 0; j < VMAX; ++j) {
      const bool number = fabsf(b[j]) < INFINITY;
      mb = fmaxf(mb, number ? fabsf(b[j]) : 0.f);
      odd = odd || b[j] >= (SIGMOID_BIAS ? 1e29f : INFINITY);
      if (b[j] != b[j]) b[j] = -INFINITY;
    }
    mb = warp_max(mb);
    odd = __any_sync(FULL, odd);
  }

  for (long long t = (long long)blockIdx.x * WARPS + warp; t < p.T; t += (long long)gridDim.x * WARPS) {
    float* row = logits + t * p.E;
    float c[VMAX];  // the logits, then the selection values
    if (part) {
      load(part + t * p.E, -INFINITY, c);
      for (int i = 1; i < S; ++i) {
        float w[VMAX];
        load(part + ((long long)i * p.T + t) * p.E, 0.f, w);
#pragma unroll
        for (int j = 0; j < VMAX; ++j) c[j] += w[j];
      }
#pragma unroll
      for (int j = 0; j < VMAX; ++j)
        if (j < count) row[e0 + j] = c[j];
      __syncwarp();
    } else {
      load(row, -INFINITY, c);
    }
    // `bad`: a NaN in the row; `usual`: no NaN, nor a +inf where the logits are compared
    bool bad, usual;
    float m = -INFINITY, rz = 1.f;
    // the score of a logit, fast
    auto score = [&](float l) { return sigmoid ? fast_rcp(1.f + fast_exp2(l * -LOG2E)) : fast_exp2((l - m) * LOG2E) * rz; };
    // How far two scores must be apart to be surely in order: the errors of both.  A logistic
    // score s is off by 4u of its exponential and |l| u of that one's argument, both times
    // s (1 - s), and by 3u of the sum and reciprocal: under 6u; then s + b rounds.
    float margin = biased ? 2.f * U * (8.f + mb) : 0.f;
    const bool by_sum = p.KG < p.G && !group_max;
    if (SIGMOID_BIAS) {
      float zero = 0.f;  // NaN where a score is
#pragma unroll
      for (int j = 0; j < VMAX; ++j) {
        const float x = score(c[j]);
        zero = fmaf(x, 0.f, zero);
        // -inf for a logit of -inf, whatever the score
        c[j] = fminf(x + b[j], fmaf(c[j], 5.4210109e-20f, 1e30f));
      }
      bad = __any_sync(FULL, zero != zero);
      usual = !bad && !odd;
    } else {
#pragma unroll
      for (int j = 0; j < VMAX; ++j) m = max_nan(m, c[j]);
      usual = !__any_sync(FULL, !(m < INFINITY)) && !odd;
      bad = !usual && __any_sync(FULL, m != m);
      // softmax: the row's maximum and sum, where something needs them
      if (!sigmoid && (biased || !renorm || by_sum)) {
        m = bad ? __int_as_float(0x7fffffff) : from_key(__reduce_max_sync(FULL, order_key(m)));
        if (biased || !renorm) {
          float z = 0.f;
          if (m > -INFINITY) {
#pragma unroll
            for (int j = 0; j < VMAX; ++j) z += fast_exp2((c[j] - m) * LOG2E);
          } else if (m != m) {
            z = m;
          }
          z = warp_sum(z);
          rz = fast_rcp(z);
        }
      }
      if (biased) {
        // a softmax score, at most 1/z, by the same of its exponential and quotient and by its sum
        // over vpl values and 5 shuffles
        margin = 2.f * U * ((22.f + p.vpl) * rz + 1.f + mb);
#pragma unroll
        for (int j = 0; j < VMAX; ++j) c[j] = c[j] > -INFINITY && usual ? score(c[j]) + b[j] : -INFINITY;
      } else {
#pragma unroll
        for (int j = 0; j < VMAX; ++j) c[j] += 0.f;  // -0 as 0; NaN is never larger than anything
      }
    }

    // Each lane's three largest, in order.  The place of a value in its lane rides in its lowest
    // bits (which makes NaN of -inf, and that is passed over): Q is what that moves a value by.
    constexpr int BITS = VMAX <= 2 ? 1 : VMAX <= 4 ? 2 : VMAX <= 8 ? 3 : VMAX <= 16 ? 4 : VMAX <= 32 ? 5 : 6;
    constexpr float Q = 2.f * U * (1 << BITS), LEAST = 2e-43f;  // relative; and of numbers near zero
    float f1 = -INFINITY, f2 = -INFINITY, f3 = -INFINITY;
#pragma unroll
    for (int j = 0; j < VMAX; ++j) {
      const float f = __uint_as_float((__float_as_uint(c[j]) & ~((1u << BITS) - 1)) | j);
      const float lo = min_nan(f1, f), lo2 = min_nan(f2, lo);
      f1 = fmaxf(f1, f);
      f2 = fmaxf(f2, lo);
      f3 = fmaxf(f3, lo2);
    }

    bool stay = g < p.G;
    if (p.KG < p.G) {
      float a1 = f1, a2 = f2;
      if ((p.lpg & (p.lpg - 1)) == 0) {
        for (int o = 1; o < p.lpg; o <<= 1) {
          const float d1 = __shfl_xor_sync(FULL, a1, o), d2 = __shfl_xor_sync(FULL, a2, o);
          a2 = fmaxf(fminf(a1, d1), fmaxf(a2, d2));
          a1 = fmaxf(a1, d1);
        }
      } else {
        for (int o = 1; o < p.lpg; o <<= 1) {
          const float d1 = __shfl_down_sync(FULL, a1, o), d2 = __shfl_down_sync(FULL, a2, o);
          if (lig + o < p.lpg) {
            a2 = fmaxf(fminf(a1, d1), fmaxf(a2, d2));
            a1 = fmaxf(a1, d1);
          }
        }
        a1 = __shfl_sync(FULL, a1, lane - lig);
        a2 = __shfl_sync(FULL, a2, lane - lig);
      }
      // a group's rank, and how far two ranks must be apart to be surely in order
      float rank = a1, off = margin + 2.f * Q * fabsf(a1) + LEAST;
      if (!group_max && biased) {
        if (a2 > -INFINITY) {
          rank += a2;
          off += off + 2.f * Q * fabsf(a2) + 4.f * U * fabsf(rank);
        }
      } else if (!group_max && a1 > -INFINITY) {
        // relative: 12u of each score and the sum, twice |a - base| u of its exponential's argument,
        // |a| Q of the logit's lowest bits; each bounded, so that it is a number times a score of 0
        auto one = [&](float x) { return sigmoid ? score(x) : fast_exp2((x - m) * LOG2E); };
        auto off_of = [&](float x) {
          return 2.f * U * (12.f + 2.f * fminf(fabsf(sigmoid ? x : x - m), 1e30f)) + 2.f * Q * fminf(fabsf(x), 1e30f);
        };
        rank = one(a1);
        off = rank * off_of(a1) + 4e-38f;
        if (a2 > -INFINITY) {
          const float s2 = one(a2);
          rank += s2;
          off += s2 * off_of(a2);
        }
      }
      // the KG-th largest rank and the next; equal ones go together
      const int mine = g < p.G ? order_key(rank) : INT_MIN;
      int key = mine, kth = INT_MIN;
      for (int i = 0; i < p.KG; ++i) {
        kth = __reduce_max_sync(FULL, key);
        if (key == kth) key = INT_MIN;
      }
      int after = __reduce_max_sync(FULL, key);
      stay = mine >= kth && g < p.G;
      int kept = __popc(__ballot_sync(FULL, stay && lig == 0));
      if (kept != p.KG && __popc(__ballot_sync(FULL, mine > kth && lig == 0)) >= p.KG) {
        // equal ranks above put that too low: again, counting them
        key = mine;
        for (int n = 0;;) {
          kth = __reduce_max_sync(FULL, key);
          n += __popc(__ballot_sync(FULL, key == kth && lig == 0));
          if (key == kth) key = INT_MIN;
          if (n >= p.KG || kth == INT_MIN) break;
        }
        after = __reduce_max_sync(FULL, key);
        stay = mine >= kth && g < p.G;
        kept = __popc(__ballot_sync(FULL, stay && lig == 0));
      }
      // Every group tells whether it is as far beyond the border as its own error asks: then each pair
      // of a kept and a left group is further apart than the larger of its two errors.  Ranks of
      // -inf, of groups with no expert in service, have none.
      const float border = from_key(kth);
      const bool near = g < p.G && rank != -INFINITY && !(fabsf(rank - (stay ? from_key(after) : border)) > off);
      if (kept != p.KG || !usual || __any_sync(FULL, near)) {
        const float bound = (group_max ? a1 : a2) - 2.f * Q * fabsf(group_max ? a1 : a2) - LEAST - margin;
        // Sure with any group's error: those further above the KG + 1st rank (at most KG can be ahead of
        // or level with them, themselves among these) and those further below the KG-th (KG are ahead).
        // Ranks that overflowed have no distance: they are open.
        const float next = kept > p.KG ? border : from_key(after);
        const float slack =
            from_key(__reduce_max_sync(FULL, g < p.G && rank != -INFINITY ? order_key(off) : INT_MIN));
        const bool in = g < p.G && rank - next > slack;
        const bool open = g < p.G && !in && !(border - rank > slack);
        // from the values at hand, unless a lane may have more of them
        const bool plain = border > -INFINITY && usual &&
                           !__any_sync(FULL, open && f3 >= bound && f3 > -INFINITY && count > 3);
        const Row64 r = row64(row, bias, p.E, sigmoid, m, biased || !group_max);
        stay = plain ? settle_groups64(r, p, g, lig, e0, make_float3(f1, f2, f3), (1u << BITS) - 1, bound, open,
                                       in)
                     : keep_groups64(r, p, g, lig, bound + margin, margin) && g < p.G;
      }
    }

    // K + 1 rounds take the warp's largest one by one
    int e = 0, place = 32;
    float mine = -INFINITY;
    bool sure = usual;
    float limit = -INFINITY;
    if (sure) {
      const int none = order_key(-INFINITY);  // what a lane with no more values offers
      int k1 = none, k2 = none, k3 = none;
      if (stay) {
        k1 = order_key(f1);
        k2 = order_key(f2);
        k3 = order_key(f3);
      }
      int best = none;
      unsigned from = 0;
#pragma unroll 3
      for (int k = 0; k <= p.K; ++k) {
        const int top = __reduce_max_sync(FULL, k1);
        const bool gives = k1 == top;
        const unsigned who = __ballot_sync(FULL, gives);
        if (lane == k) {
          best = top;
          from = who;
        }
        k1 = gives ? k2 : k1;
        k2 = gives ? k3 : k2;
        k3 = gives ? none : k3;
      }
      // The values in order: lane k holds the k-th, and looks at the next one.  The rounds are
      // what they seem where each took one value, the values are clear of each other and K
      // experts were in service.
      const float v = from_key(best), after = __shfl_down_sync(FULL, v, 1);
      const bool clear = best != none && (from & (from - 1)) == 0 &&
                         (v - after > margin + 2.f * Q * fabsf(v) + LEAST || after == -INFINITY);
      sure = __all_sync(FULL, lane >= p.K || clear);
      const bool gave_all = stay && f3 > -INFINITY && k1 == none;
      if (VMAX > 3 && sure && __any_sync(FULL, gave_all)) {
        // a lane gave all three: none of its others may come before the last one taken
        const float last = __shfl_sync(FULL, v, p.K);
        const float lim = last > -INFINITY ? last - (margin + 2.f * Q * fabsf(last) + LEAST) : -3.4028235e38f;
        int above = 0;
#pragma unroll
        for (int j = 0; j < VMAX; ++j) above += c[j] >= lim;
        sure = !__any_sync(FULL, gave_all && above > 3);
      }
      e = __shfl_sync(FULL, e0, __ffs(from) - 1 & 31) + (__float_as_uint(v) & ((1u << BITS) - 1));
      // where that does not hold, the K-th value (or one below it) bounds the candidates
      limit = __shfl_sync(FULL, v, p.K - 1);
      limit -= Q * fabsf(limit) + LEAST;
      if (sure && lane < p.K) {
        mine = row[e];
        place = lane;
      }
    }
    if (!sure) {
      if (!stay) {
#pragma unroll
        for (int j = 0; j < VMAX; ++j) c[j] = -INFINITY;
      }
      // the scores at or above it, one to a lane
      auto collect = [&]() {
        const float lim = fmaxf(limit - margin, -3.4028235e38f);
        unsigned in[(VMAX + 31) / 32];
        int mine = 0;
#pragma unroll
        for (int w = 0; w < (VMAX + 31) / 32; ++w) {
          in[w] = 0;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (32 * w + j < VMAX && c[32 * w + j] >= lim) in[w] |= 1u << j;
          mine += __popc(in[w]);
        }
        int at = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(FULL, at, o);
          if (lane >= o) at += up;
        }
        const int n = __shfl_sync(FULL, at, 31);
        at -= mine;
#pragma unroll
        for (int w = 0; w < (VMAX + 31) / 32; ++w)
          for (; in[w] && at < 32; ++at) {
            cand_e[warp][at] = e0 + 32 * w + __ffs(in[w]) - 1;
            in[w] &= in[w] - 1;
          }
        return n;
      };
      int n = collect();
      if (n > 32) {
        // a bound too low: the K-th largest itself, K rounds over the registers
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
      if (n >= p.K && n <= 32) {
        const bool in = lane < n;
        float v = -INFINITY;
        if (in) {
          e = cand_e[warp][lane];
          mine = row[e];
          v = biased ? score(mine) + __ldg(bias + e) : mine;
        }
        cand_c[warp][lane] = v;
        __syncwarp();
        int ahead = 0, close = 0;  // how many are larger; how many are not surely smaller
        const float lim = v - margin;
        for (int i = 0; i < n; i += 4) {
          const float4 w = *reinterpret_cast<const float4*>(&cand_c[warp][i]);
          ahead += (w.x > v) + (w.y > v) + (w.z > v) + (w.w > v);
          close += (w.x >= lim) + (w.y >= lim) + (w.z >= lim) + (w.w >= lim);
        }
        place = in ? ahead : 32;
        // `close` counts the lane itself and those ahead
        if (__any_sync(FULL, in && ahead < p.K && close > ahead + 1)) {
          double x = mine;
          if (biased) {
            const Row64 r = row64(row, bias, p.E, sigmoid, m, true);
            x = in ? r.value(e) : 0.0;
          }
          place = 0;
          for (int i = 0; i < n; ++i) {
            const double w = __shfl_sync(FULL, x, i);
            const int f = __shfl_sync(FULL, e, i);
            place += w > x || (w == x && f < e);
          }
          if (!in) place = 32;
        }
      } else {
        const unsigned who = __ballot_sync(FULL, stay && lig == 0);
        unsigned keep = 0;
        for (int o = 0; o < p.G; ++o) keep |= ((who >> (o * p.lpg)) & 1u) << o;
        e = choose64(row64(row, bias, p.E, sigmoid, m, biased), p, keep);
        if (lane < p.K) {
          place = lane;
          mine = row[e];
        }
      }
    }
    const bool on = place < p.K;
    const float s = gate_value(mine, on, sigmoid, renorm, m, rz);
    if (on) {
      idx[t * p.K + place] = e;
      gate[t * p.K + place] = bad ? __int_as_float(0x7fffffff) : s * p.scale;
    }
    __syncwarp();
  }
}

// Backward: a warp to a token.  All but the softmax without RENORM have a gradient at the
// chosen experts alone: the row is filled with zeros while the chosen logits are on their
// way, then their lanes overwrite K of them.  The softmax's row goes through registers in VQ
// 16-byte pieces a lane (VQ = 0: rows of any length, one value at a time, read twice; 16384
// x 256 take 10.7 us in pieces and 14.6 so).  The launch bounds it: 8192 x 384, logistic, 7.1 us
// (2.0 at the rate of a copy); 16384 x 64, softmax, 8.2 us (1.4).
template <int VQ>
__global__ void __launch_bounds__(32 * WARPS)
gate_bwd_kernel(const float* __restrict__ d_gate, const float* __restrict__ logits, const int32_t* __restrict__ idx,
                int T, int E, int K, int mode, float scale, float* __restrict__ d_logits, unsigned* err) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool sigmoid = (mode & 0xf) == MOE_GATE_SIGMOID, renorm = mode & MOE_GATE_RENORM;
  const bool whole = !sigmoid && !renorm;
  for (long long t = (long long)blockIdx.x * WARPS + warp; t < T; t += (long long)gridDim.x * WARPS) {
    const float* row = logits + t * E;
    float* out = d_logits + t * E;
    int e = -1;
    float dg = 0.f, l = -INFINITY;
    if (lane < K) {
      e = __ldg(idx + t * K + lane);
      dg = __ldg(d_gate + t * K + lane);
    }
    float4 v[VQ > 0 ? VQ : 1];
    float m = -INFINITY, z = 0.f;
    if (whole) {
      if (VQ > 0) {
#pragma unroll
        for (int q = 0; q < VQ; ++q) {
          const int i = (q * 32 + lane) * 4;
          v[q] = i < E ? __ldg(reinterpret_cast<const float4*>(row + i)) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          m = fmaxf(m, fmaxf(fmaxf(v[q].x, v[q].y), fmaxf(v[q].z, v[q].w)));
        }
      } else {
        for (int i = lane; i < E; i += 32) m = fmaxf(m, row[i]);
      }
      m = warp_max(m);
    } else if (VQ > 0) {
#pragma unroll
      for (int q = 0; q < VQ; ++q) {
        const int i = (q * 32 + lane) * 4;
        if (i < E) *reinterpret_cast<float4*>(out + i) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    } else {
      for (int i = lane; i < E; i += 32) out[i] = 0.f;
    }
    if (lane < K) {
      if (e < 0 || e >= E) {
        set_error(err, DEV_BOUNDS);
        e = -1;
        dg = 0.f;
      } else {
        l = row[e];
      }
    }
    if (whole) {
      auto power = [&](float x) { return x == -INFINITY ? 0.f : expf(x - m); };  // a row of -inf has m = -inf
      if (VQ > 0) {
#pragma unroll
        for (int q = 0; q < VQ; ++q) {
          v[q] = make_float4(power(v[q].x), power(v[q].y), power(v[q].z), power(v[q].w));
          z += (v[q].x + v[q].y) + (v[q].z + v[q].w);
        }
      } else {
        for (int i = lane; i < E; i += 32) z += power(row[i]);
      }
      z = warp_sum(z);
    } else if (renorm) {  // a common factor of the chosen scores: the largest becomes about 1
      m = warp_max(l);
      if (sigmoid) m = fminf(m, 0.f);
    } else {
      m = 0.f;
    }
    float s = 0.f, rest = 1.f;
    if (l != -INFINITY) {
      if (sigmoid) {
        s = expf(fminf(l, 0.f) - m) / (1.f + expf(-fabsf(l)));
        rest = 1.f / (1.f + expf(l));
      } else {
        s = expf(l - m);
      }
    }
    const float sum = renorm ? warp_sum(s) : z;
    // a sum of 0, where nothing is in service, has no shares; a NaN stays one
    const float q = sigmoid && !renorm ? s : sum == 0.f ? 0.f : s / sum;
    const float inner = sigmoid && !renorm ? 0.f : warp_sum(dg * q);
    float d = q * (whole ? dg : rest * (dg - inner));
    // an expert listed more than once: its first place takes the sum
    const unsigned same = __match_any_sync(FULL, e) & ((1u << K) - 1);
    bool first = e >= 0;
    if (__any_sync(FULL, lane < K && e >= 0 && __popc(same) > 1)) {
      float all = 0.f;
      for (int k = 0; k < K; ++k) {
        const float o = __shfl_sync(FULL, d, k);
        if ((same >> k) & 1u) all += o;
      }
      d = all;
      first = first && __ffs(same) - 1 == lane;
    }
    if (whole) {
      const float f = z == 0.f ? 0.f : -scale * inner / z;
      if (VQ > 0) {
#pragma unroll
        for (int q4 = 0; q4 < VQ; ++q4) {
          const int i = (q4 * 32 + lane) * 4;
          if (i < E)
            *reinterpret_cast<float4*>(out + i) = make_float4(f * v[q4].x, f * v[q4].y, f * v[q4].z, f * v[q4].w);
        }
      } else {
        for (int i = lane; i < E; i += 32) out[i] = f * (row[i] == -INFINITY ? 0.f : expf(row[i] - m));
      }
      d -= q * inner;
    }
    __syncwarp();
    if (first) out[e] = scale * d;
    __syncwarp();
  }
}

// one CTA for WARPS tokens, at most as many as the GPU holds at once: each then walks its
// even share (more would run as a second, partly filled round)
template <auto KERNEL> int resident_grid(long long T) {
  static const int per_sm = [] {
    int n = 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERNEL, 32 * WARPS, 0) == cudaSuccess && n > 0 ? n : 1;
  }();
  const long long ctas = (T + WARPS - 1) / WARPS, cap = (long long)sm_count() * per_sm;
  return (int)(ctas < cap ? ctas : cap);
}

template <int VMAX, bool SIGMOID_BIAS>
void gate_v(float* logits, const float* part, int S, const float* bias, const GateShape& p, int32_t* idx, float* gate,
            cudaStream_t s) {
  gate_kernel<VMAX, SIGMOID_BIAS><<<resident_grid<gate_kernel<VMAX, SIGMOID_BIAS>>(p.T), 32 * WARPS, 0, s>>>(
      logits, part, S, bias, p, idx, gate);
}

template <int VQ>
void gate_bwd_v(const float* d_gate, const float* logits, const int32_t* idx, int T, int E, int K, int mode,
                float scale, float* d_logits, cudaStream_t s) {
  gate_bwd_kernel<VQ><<<resident_grid<gate_bwd_kernel<VQ>>(T), 32 * WARPS, 0, s>>>(
      d_gate, logits, idx, T, E, K, mode, scale, d_logits, device_error_word());
}

}  // namespace

int launch_gate(float* logits, const float* part, int S, const float* bias, int T, int E, int K, int G, int KG,
                int mode, float scale, int32_t* idx, float* gate, cudaStream_t s) {
  if (T == 0) return MOE_OK;
  if (KG == G) G = KG = 1;  // every group stays: nothing to rank
  GateShape p{T, E, K, G, KG, E / G, 32 / G, 0, mode, scale};
  p.vpl = (p.gs + p.lpg - 1) / p.lpg;
  if (p.gs % 4 == 0 && p.vpl > 2) p.vpl = (p.vpl + 3) / 4 * 4;  // 16-byte loads
  // the least instance that holds a lane's experts (32768 x 384 in the one of 12: 33 us, of 16: 44).  Lanes
  // of 17 to 32 share one: 16384 x 640 in 8 groups (20 of a lane) 33 us, x 1024 (32) 36
  const bool sigmoid_bias = bias && (mode & 0xf) == MOE_GATE_SIGMOID;
#define MOE_GATE(V)                                                           \
  (sigmoid_bias ? gate_v<V, true>(logits, part, S, bias, p, idx, gate, s) : \
                  gate_v<V, false>(logits, part, S, bias, p, idx, gate, s))
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
  const int pieces = E % 4 == 0 ? (E + 127) / 128 : 0;
#define MOE_GATE_BWD(V) gate_bwd_v<V>(d_gate, logits, idx, T, E, K, mode, scale, d_logits, s)
  if (pieces == 0) MOE_GATE_BWD(0);
  else if (pieces <= 1) MOE_GATE_BWD(1);
  else if (pieces <= 2) MOE_GATE_BWD(2);
  else if (pieces <= 4) MOE_GATE_BWD(4);
  else MOE_GATE_BWD(8);
#undef MOE_GATE_BWD
  return launch_status();
}

}  // namespace moe
