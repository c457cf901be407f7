// Activation checkpoint in 8 bits: runs of 32 neighbours of a row share a power
// of two, the least that holds the run's largest magnitude in 127 steps.  Powers
// of two keep every division exact, so the only rounding is the one to integers,
// and the restored values have at most 8 significant bits: exact in bf16 too.
#include <math.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int RUN = 32;

// the least e >= -126 with a <= 127 * 2^e, for finite a >= 0
__device__ __forceinline__ int run_exponent(float a) {
  const unsigned bits = __float_as_uint(a);
  // a = 1.f * 2^k: 127 = 1.984375 * 2^6, so e = k - 6 where 1.f <= 1.984375
  const int e = (int)(bits >> 23) - 127 - 6 + ((bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return e < -126 ? -126 : e;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }

// a warp per run, a lane per value
template <typename T>
__global__ void __launch_bounds__(256) ckpt_pack_kernel(const T* __restrict__ x, long long rows, int N, int runs,
                                                        int8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  const int lane = threadIdx.x & 31;
  const long long total = rows * runs;
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (long long)gridDim.x * 8) {
    const long long row = i / runs;
    const int c = (int)(i - row * runs) * RUN + lane;
    const float v = c < N ? to_f32(x[row * N + c]) : 0.f;
    const bool bad = __any_sync(0xffffffffu, !(fabsf(v) < INFINITY));
    const float a = warp_max(fabsf(v));
    const int e = bad ? 128 : run_exponent(a);
    if (c < N) q[row * N + c] = bad ? 0 : (int8_t)__float2int_rn(v * pow2(-e));
    if (lane == 0) scale[i] = (uint8_t)(e + 127);
  }
}

__device__ __forceinline__ float restore(int8_t q, uint8_t scale) {
  // scale 0 is 2^-127 and never written; 255 marks a run with an infinity or a NaN
  const float s = scale == 255 ? __int_as_float(0x7fffffff) : scale == 0 ? 5.877471754e-39f : pow2((int)scale - 127);
  return (float)q * s;
}

template <typename T>
__global__ void __launch_bounds__(256) ckpt_unpack_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                                          long long rows, int N, int runs, T* __restrict__ x) {
  const long long n = rows * N;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long row = i / N;
    x[i] = from_f32<T>(restore(q[i], scale[row * runs + (i - row * N) / RUN]));
  }
}

// g / (1 + exp(-g)) with the exponential of -|g|, so that far negative g keep their
// small values (exp(-g) itself overflows from g = -89 on)
__device__ __forceinline__ float silu(float g) {
  const float e = expf(-fabsf(g));
  return (g < 0.f ? g * e : g) / (1.f + e);
}

template <typename T>
__global__ void __launch_bounds__(256) ckpt_swiglu_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                                          long long rows, int Hp, int runs, T* __restrict__ gu,
                                                          T* __restrict__ act) {
  const long long n = rows * Hp;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long row = i / Hp;
    const int c = (int)(i - row * Hp);
    const long long at = row * 2 * Hp + c;
    const float g = restore(q[at], scale[row * runs + c / RUN]);
    const float u = restore(q[at + Hp], scale[row * runs + (Hp + c) / RUN]);
    if (gu) {
      gu[at] = from_f32<T>(g);
      gu[at + Hp] = from_f32<T>(u);
    }
    if (act) act[i] = from_f32<T>(silu(g) * u);
  }
}

int grid_for(long long work, int per_cta) {
  const long long ctas = (work + per_cta - 1) / per_cta, cap = (long long)sm_count() * 32;
  return (int)(ctas < cap ? ctas : cap);
}

}  // namespace

int launch_ckpt_pack(const void* x, int rows, int N, int dtype, int8_t* q, uint8_t* scale, cudaStream_t s) {
  if (rows == 0) return MOE_OK;
  const int runs = (N + RUN - 1) / RUN, grid = grid_for((long long)rows * runs, 8);
  if (dtype == MOE_BF16) ckpt_pack_kernel<bf16><<<grid, 256, 0, s>>>(static_cast<const bf16*>(x), rows, N, runs, q, scale);
  else ckpt_pack_kernel<float><<<grid, 256, 0, s>>>(static_cast<const float*>(x), rows, N, runs, q, scale);
  return launch_status();
}

int launch_ckpt_unpack(const int8_t* q, const uint8_t* scale, int rows, int N, int dtype, void* x, cudaStream_t s) {
  if (rows == 0) return MOE_OK;
  const int runs = (N + RUN - 1) / RUN, grid = grid_for((long long)rows * N, 256);
  if (dtype == MOE_BF16) ckpt_unpack_kernel<bf16><<<grid, 256, 0, s>>>(q, scale, rows, N, runs, static_cast<bf16*>(x));
  else ckpt_unpack_kernel<float><<<grid, 256, 0, s>>>(q, scale, rows, N, runs, static_cast<float*>(x));
  return launch_status();
}

int launch_ckpt_swiglu(const int8_t* q, const uint8_t* scale, int rows, int Hp, int dtype, void* gu, void* act,
                       cudaStream_t s) {
  if (rows == 0 || (!gu && !act)) return MOE_OK;
  const int runs = (2 * Hp + RUN - 1) / RUN, grid = grid_for((long long)rows * Hp, 256);
  if (dtype == MOE_BF16)
    ckpt_swiglu_kernel<bf16><<<grid, 256, 0, s>>>(q, scale, rows, Hp, runs, static_cast<bf16*>(gu), static_cast<bf16*>(act));
  else
    ckpt_swiglu_kernel<float><<<grid, 256, 0, s>>>(q, scale, rows, Hp, runs, static_cast<float*>(gu), static_cast<float*>(act));
  return launch_status();
}

}  // namespace moe
