// Activation checkpoint in 8 bits: runs of 32 neighbours of a row share a power
// of two, the least that holds the run's largest magnitude in 127 steps.  Powers
// of two keep every division exact, so the only rounding is the one to integers,
// and the restored values have at most 8 significant bits: exact in bf16 too.
//
// The memory bounds all three.  16384 x 28672 bf16: pack 205 us (6.9 TB/s), unpack 221 (6.4),
// [g | u] and act 290 (6.5), where a copy runs at 6.8; 16384 x 4096 fp32: 51, 55 and 74 us (6.6,
// 6.1 and 6.4 TB/s).
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

// A thread takes VECS 16-byte vectors of neighbours, so a run is 32 / (VECS V) lanes, and whole
// rows of runs (FLAT: N % 32 == 0) move without an index division for each.  Other widths move
// the same values in pieces of one vector, the last run of a row in fewer of them (unpack of
// 16384 x 28672 bf16 that way: 244 us instead of 221).
//
// 16 values a thread, but one vector where fp32 is written: four to a thread left each sector
// to two stores (16384 x 4096 fp32, unpack 71 -> 55 us, [g | u] and act 102 -> 74).  Reading is the
// other way round, it wants the bytes in flight (pack 51 us with four, 60 with one).
constexpr int NT = 256;
template <typename T> constexpr int IN = 16 / Vec16<T>::N;           // vectors of a thread that reads them
template <typename T> constexpr int OUT = sizeof(T) == 2 ? 2 : 1;  // and of one that writes them

// where thread i's values are: value 0 at `at`, `live` of them in the row, run `run`
struct Place {
  long long at, run;
  int live;
};
template <int PER, bool FLAT>
__device__ __forceinline__ Place place_of(long long i, int N, int runs) {
  constexpr int LANES = RUN / PER;
  const long long run = i / LANES;
  if (FLAT) return {i * PER, run, PER};
  const long long row = run / runs;
  const int c = (int)(run - row * runs) * RUN + (int)(i % LANES) * PER;
  return {row * N + c, run, max(0, min(PER, N - c))};
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(NT) ckpt_pack_kernel(const T* __restrict__ x, long long threads, int N, int runs,
                                                       int8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  constexpr int V = Vec16<T>::N, VECS = IN<T>, PER = VECS * V, LANES = RUN / PER;
  // the lanes of a run are in range together; whole warps stay for the shuffles
  const long long last = (threads + 31) / 32 * 32;
  for (long long i = (long long)blockIdx.x * NT + threadIdx.x; i < last; i += (long long)gridDim.x * NT) {
    Place p = place_of<PER, FLAT>(i, N, runs);
    if (i >= threads) p.live = 0;
    uint4 raw[VECS];
#pragma unroll
    for (int k = 0; k < VECS; ++k)
      raw[k] = k * V < p.live ? __ldg(reinterpret_cast<const uint4*>(x + p.at) + k) : make_uint4(0, 0, 0, 0);
    float v[PER];
#pragma unroll
    for (int k = 0; k < VECS; ++k) Vec16<T>::load_raw_unpack(raw[k], v + k * V);
    // magnitudes as integers: they order as the numbers do, with infinity and NaN above
    unsigned top = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool bad = top >= 0x7f800000u;
    const int e = bad ? 128 : run_exponent(__uint_as_float(top));
    const float inv = bad ? 0.f : pow2(-e);
    // x / 2^e + 1.5 * 2^23 rounds to an integer, halves to even, and leaves it in the low byte
    unsigned w[PER / 4];
#pragma unroll
    for (int k = 0; k < PER / 4; ++k) {
      unsigned b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(fmaf(v[4 * k + j], inv, 12582912.f));
      w[k] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
      if (bad) w[k] = 0;
    }
    if (FLAT) {
      if (p.live) *reinterpret_cast<uint4*>(q + p.at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int k = 0; k < VECS; ++k) {
        if (k * V >= p.live) continue;
        if constexpr (V == 8) *reinterpret_cast<uint2*>(q + p.at + 8 * k) = make_uint2(w[2 * k], w[2 * k + 1]);
        else *reinterpret_cast<unsigned*>(q + p.at + 4 * k) = w[k];
      }
    }
    if (i % LANES == 0 && i < threads) scale[p.run] = (uint8_t)(e + 127);
  }
}

// the factor that a scale byte stands for; 255 marks a run with an infinity or a NaN, 0 is
// 2^-127 and never written
__device__ __forceinline__ float factor(uint8_t s) {
  return __uint_as_float(s == 255 ? 0x7fffffffu : s == 0 ? 0x00400000u : (unsigned)s << 23);
}
// four integers of a word times f: a byte under the exponent of 2^23 is the number 2^23 +
// q + 128 (its sign bit flipped), so one subtraction converts it
__device__ __forceinline__ void restore4(unsigned w, float f, float* v) {
  w ^= 0x80808080u;
  v[0] = (__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)) - 8388736.f) * f;
  v[1] = (__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441)) - 8388736.f) * f;
  v[2] = (__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7442)) - 8388736.f) * f;
  v[3] = (__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7443)) - 8388736.f) * f;
}

// a thread's restored values, `live` of them in the row
template <typename T, bool FLAT>
__device__ __forceinline__ void restore(const int8_t* q, int live, float f, float (&v)[OUT<T> * Vec16<T>::N]) {
  constexpr int V = Vec16<T>::N, VECS = OUT<T>;
  unsigned w[VECS * V / 4];
  if constexpr (V == 4) {
    w[0] = __ldg(reinterpret_cast<const unsigned*>(q));
  } else if (FLAT) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(q));
    w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
  } else {
#pragma unroll
    for (int k = 0; k < VECS; ++k) {
      const uint2 r = k * V < live ? __ldg(reinterpret_cast<const uint2*>(q) + k) : make_uint2(0, 0);
      w[2 * k] = r.x;
      w[2 * k + 1] = r.y;
    }
  }
#pragma unroll
  for (int k = 0; k < VECS * V / 4; ++k) restore4(w[k], f, v + 4 * k);
}

template <typename T>
__device__ __forceinline__ void store(T* x, int live, const float (&v)[OUT<T> * Vec16<T>::N]) {
  constexpr int V = Vec16<T>::N;
#pragma unroll
  for (int k = 0; k < OUT<T>; ++k)
    if (k * V < live) Vec16<T>::store(x + k * V, v + k * V);
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(NT) ckpt_unpack_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                                         long long threads, int N, int runs, T* __restrict__ x) {
  constexpr int PER = OUT<T> * Vec16<T>::N;
  for (long long i = (long long)blockIdx.x * NT + threadIdx.x; i < threads; i += (long long)gridDim.x * NT) {
    const Place p = place_of<PER, FLAT>(i, N, runs);
    if (p.live == 0) continue;
    float v[PER];
    restore<T, FLAT>(q + p.at, p.live, factor(__ldg(scale + p.run)), v);
    store<T>(x + p.at, p.live, v);
  }
}

// g / (1 + exp(-g)) with the exponential of -|g|, so that far negative g keep their
// small values (exp(-g) itself overflows from g = -89 on)
__device__ __forceinline__ float silu(float g) {
  const float e = expf(-fabsf(g));
  return __fdividef(g < 0.f ? g * e : g, 1.f + e);
}

// FLAT (Hp % 32 == 0): a thread's columns of g and the same of u; otherwise the columns of one 16-byte
// vector, which lie in one run of g and one of u whatever Hp is
template <typename T, bool FLAT>
__global__ void __launch_bounds__(NT) ckpt_swiglu_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                                         int rows, int Hp, int runs, int per_row, T* __restrict__ gu,
                                                         T* __restrict__ act) {
  constexpr int PER = OUT<T> * Vec16<T>::N, STEP = FLAT ? PER : Vec16<T>::N;
  for (long long i = (long long)blockIdx.x * NT + threadIdx.x; i < (long long)rows * per_row;
       i += (long long)gridDim.x * NT) {
    const long long row = i / per_row;
    const int c = (int)(i - row * per_row) * STEP;
    const long long at = row * 2 * Hp + c;
    const uint8_t* s = scale + row * runs;
    float g[PER], u[PER];
    restore<T, FLAT>(q + at, STEP, factor(__ldg(s + c / RUN)), g);
    restore<T, FLAT>(q + at + Hp, STEP, factor(__ldg(s + (Hp + c) / RUN)), u);
    if (gu) {
      store<T>(gu + at, STEP, g);
      store<T>(gu + at + Hp, STEP, u);
    }
    if (act) {
#pragma unroll
      for (int j = 0; j < PER; ++j) g[j] = silu(g[j]) * u[j];
      store<T>(act + row * Hp + c, STEP, g);
    }
  }
}

int grid_for(long long threads) {
  const long long ctas = (threads + NT - 1) / NT, cap = (long long)sm_count() * 64;
  return (int)(ctas < cap ? ctas : cap);
}

template <typename T>
void pack_t(const void* x, int rows, int N, int8_t* q, uint8_t* scale, cudaStream_t s) {
  const int runs = (N + RUN - 1) / RUN;
  const long long threads = (long long)rows * runs * (RUN / 16);
  if (N % RUN == 0)
    ckpt_pack_kernel<T, true><<<grid_for(threads), NT, 0, s>>>(static_cast<const T*>(x), threads, N, runs, q, scale);
  else
    ckpt_pack_kernel<T, false><<<grid_for(threads), NT, 0, s>>>(static_cast<const T*>(x), threads, N, runs, q, scale);
}

template <typename T>
void unpack_t(const int8_t* q, const uint8_t* scale, int rows, int N, void* x, cudaStream_t s) {
  const int runs = (N + RUN - 1) / RUN;
  const long long threads = (long long)rows * runs * (RUN / (OUT<T> * Vec16<T>::N));
  if (N % RUN == 0)
    ckpt_unpack_kernel<T, true><<<grid_for(threads), NT, 0, s>>>(q, scale, threads, N, runs, static_cast<T*>(x));
  else
    ckpt_unpack_kernel<T, false><<<grid_for(threads), NT, 0, s>>>(q, scale, threads, N, runs, static_cast<T*>(x));
}

template <typename T>
void swiglu_t(const int8_t* q, const uint8_t* scale, int rows, int Hp, void* gu, void* act, cudaStream_t s) {
  const int runs = (2 * Hp + RUN - 1) / RUN;
  const bool flat = Hp % RUN == 0;
  const int per_row = Hp / (flat ? OUT<T> * Vec16<T>::N : Vec16<T>::N);
  const int grid = grid_for((long long)rows * per_row);
  if (flat)
    ckpt_swiglu_kernel<T, true><<<grid, NT, 0, s>>>(q, scale, rows, Hp, runs, per_row, static_cast<T*>(gu), static_cast<T*>(act));
  else
    ckpt_swiglu_kernel<T, false><<<grid, NT, 0, s>>>(q, scale, rows, Hp, runs, per_row, static_cast<T*>(gu), static_cast<T*>(act));
}

}  // namespace

int launch_ckpt_pack(const void* x, int rows, int N, int dtype, int8_t* q, uint8_t* scale, cudaStream_t s) {
  if (rows == 0) return MOE_OK;
  if (dtype == MOE_BF16) pack_t<bf16>(x, rows, N, q, scale, s);
  else pack_t<float>(x, rows, N, q, scale, s);
  return launch_status();
}

int launch_ckpt_unpack(const int8_t* q, const uint8_t* scale, int rows, int N, int dtype, void* x, cudaStream_t s) {
  if (rows == 0) return MOE_OK;
  if (dtype == MOE_BF16) unpack_t<bf16>(q, scale, rows, N, x, s);
  else unpack_t<float>(q, scale, rows, N, x, s);
  return launch_status();
}

int launch_ckpt_swiglu(const int8_t* q, const uint8_t* scale, int rows, int Hp, int dtype, void* gu, void* act,
                       cudaStream_t s) {
  if (rows == 0 || (!gu && !act)) return MOE_OK;
  if (dtype == MOE_BF16) swiglu_t<bf16>(q, scale, rows, Hp, gu, act, s);
  else swiglu_t<float>(q, scale, rows, Hp, gu, act, s);
  return launch_status();
}

}  // namespace moe
