// Gate with expert groups (moe_gate) and its backward.
//
//   s = softmax or logistic function of the logits, c = s + bias; the best
//   topk_groups of the expert groups stay, ranked by their two largest c; the K
//   largest c of those groups are chosen; the gates are the chosen s, rescaled.
//
// One warp per token.  Scores are held in 64 bits in shared memory, the choice
// is made by K rounds of a warp-wide (value desc, expert asc) arg-max.
#include <math.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int WARPS = 4;

__device__ __forceinline__ double nan64() { return __longlong_as_double(0x7ff8000000000000ll); }

// the larger (value, lower index) of the warp; NaN values never win, e < 0 = none
__device__ __forceinline__ void warp_best(double& v, int& e) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(0xffffffffu, v, o);
    const int f = __shfl_xor_sync(0xffffffffu, e, o);
    if (f >= 0 && (e < 0 || w > v || (w == v && f < e))) {
      v = w;
      e = f;
    }
  }
}

__global__ void __launch_bounds__(32 * WARPS)
gate_kernel(float* logits, const float* __restrict__ part, int S, const float* __restrict__ bias, int T, int E, int K, int G, int KG,
            int mode, float scale, int32_t* __restrict__ idx, float* __restrict__ gate) {
  extern __shared__ double smem[];
  __shared__ int chosen[WARPS][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double* c = smem + (size_t)warp * E;
  const bool sigmoid = (mode & 0xf) == MOE_GATE_SIGMOID;
  const int gs = E / G;
  for (long long t = (long long)blockIdx.x * WARPS + warp; t < T; t += (long long)gridDim.x * WARPS) {
    float* row = logits + t * E;
    if (part) {
      for (int e = lane; e < E; e += 32) {
        float l = part[t * E + e];
        for (int i = 1; i < S; ++i) l += part[((long long)i * T + t) * E + e];
        row[e] = l;
      }
      __syncwarp();
    }
    float m = -INFINITY;
    bool bad = false;
    for (int e = lane; e < E; e += 32) {
      const float l = row[e];
      bad |= l != l;
      m = fmaxf(m, l);
    }
    m = warp_max(m);
    bad = __any_sync(0xffffffffu, bad);
    double z = 0;
    if (!sigmoid) {
      for (int e = lane; e < E; e += 32) z += m == -INFINITY ? 0.0 : exp((double)row[e] - (double)m);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    auto score = [&](float l) -> double {
      if (l == -INFINITY) return 0.0;
      return sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)m) / z;
    };
    for (int e = lane; e < E; e += 32) {
      const float l = row[e];
      double v = bias ? score(l) + (double)bias[e] : (double)l;
      if (l == -INFINITY || v != v) v = -INFINITY;
      c[e] = v;
    }
    __syncwarp();
    if (KG < G) {
      // lane g ranks group g, then counts the groups ahead of it
      double rank = -INFINITY;
      if (lane < G) {
        double a = -INFINITY, b = -INFINITY;
        for (int e = lane * gs; e < (lane + 1) * gs; ++e) {
          double v = c[e];
          if (!bias && !(mode & MOE_GATE_GROUP_MAX)) v = v == -INFINITY ? v : score(row[e]);
          if (v > a) { b = a; a = v; } else if (v > b) b = v;
        }
        rank = (mode & MOE_GATE_GROUP_MAX) || b == -INFINITY ? a : a + b;
      }
      int ahead = 0;
      for (int g = 0; g < G; ++g) {
        const double o = __shfl_sync(0xffffffffu, rank, g);
        ahead += o > rank || (o == rank && g < lane);
      }
      __syncwarp();
      if (lane < G && ahead >= KG)
        for (int e = lane * gs; e < (lane + 1) * gs; ++e) c[e] = nan64();
      __syncwarp();
    }
    for (int k = 0; k < K; ++k) {
      double best = -INFINITY;
      int be = -1;
      for (int e = lane; e < E; e += 32) {
        const double v = c[e];
        if (v > best || (be < 0 && v == v)) {
          best = v;
          be = e;
        }
      }
      warp_best(best, be);
      if (lane == 0) {
        chosen[warp][k] = be;
        c[be] = nan64();
      }
      __syncwarp();
    }
    double s = 0, sum = 0;
    if (lane < K) s = score(row[chosen[warp][lane]]);
    if (mode & MOE_GATE_RENORM) {
      for (int k = 0; k < K; ++k) sum += __shfl_sync(0xffffffffu, s, k);
      s = sum > 0 ? s / sum : s;
    }
    if (lane < K) {
      idx[t * K + lane] = chosen[warp][lane];
      gate[t * K + lane] = bad ? __int_as_float(0x7fffffff) : (float)(s * (double)scale);
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
      const int f = __shfl_sync(0xffffffffu, e, k);
      const float o = __shfl_sync(0xffffffffu, d, k);
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
  gate_kernel<<<warp_grid(T), 32 * WARPS, WARPS * E * sizeof(double), s>>>(logits, part, S, bias, T, E, K, G, KG, mode,
                                                                         scale, idx, gate);
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
