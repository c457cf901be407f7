// Expert weights in 4 bits with group scales, and the expert FFN that reads them.
//
// Packed form of a weight tensor w [E, rows, cols]: `in` is the axis that the product sums
// over (rows of gate and up, cols of down), `out` the other one.  Of each output, groups
// of G (32, 64 or 128) neighbours along `in` share a scale of 5 significant bits; a code q in
// -8..7 (pack makes -7..7) is held as q + 8, so q s has at most 8 significant bits: exact in
// bf16.  Codes lie in blocks of 128 inputs, 16 words of 8 codes (the last block is padded with
// zeros).  Word 4 j + w of a block (inputs 32 j + 8 w ..) is stored at w * 4 + j, and code i of a word in bits
// 4 (i / 2) + 16 (i % 2): a lane of a warp-level MMA then reads 16 neighbouring bytes that hold its
// inputs of four steps of 32, and every pair of neighbours comes out of a word by a shift and a mask, each in a half
// of its own.
#include <math.h>

#include "tc_ptx.cuh"

namespace moe {
namespace w4 {

constexpr int BLOCK = 128;         // inputs of a block
constexpr int WORDS = BLOCK / 8;   // its words

__host__ __device__ inline int blocks_of(int in) { return (int)(((long long)in + BLOCK - 1) / BLOCK); }

// ------------------------------------------------------------ the 4-bit form ---
// the least number of 5 significant bits >= amax * (1/7 in fp32, which is above 1/7), at least
// 2^-126; NaN for a group that holds a NaN, an infinity or a magnitude of 2^127 and more (its
// largest code might stand for an infinity)
__device__ __forceinline__ float scale_of(float amax) {
  if (!(amax < 1.7014118346046923e38f)) return __uint_as_float(0x7fc00000u);
  const float s = __uint_as_float((__float_as_uint(amax * (1.f / 7.f)) + 0x7ffffu) & ~0x7ffffu);
  return fmaxf(s, 1.1754943508222875e-38f);
}
// That product lies above the 7th part where amax is 7 times a number of 5 bits with a significand of 1.375 or more:
// the scale is then a step too large, and weights that were restored from codes would come out as others.  So a group
// that fits the number below its scale without error takes that: the number, or 0 where there is none to be tried
// (7% of the groups of 32 bf16 weights have one to be tried; 64 x 2048 x 1408 bf16, axis 1: 148 us without, 158 so).
__device__ __forceinline__ float below(float s, float amax) {
  const float lo = __uint_as_float(__float_as_uint(s) - 0x80000u);
  return lo >= 1.1754943508222875e-38f && 7.f * lo == amax ? lo : 0.f;
}
// whether v is k lo with a whole k, |v| <= 7 lo
__device__ __forceinline__ bool fits(float v, float lo) {
  const float k = v * __fdividef(1.f, lo) + 12582912.f - 12582912.f;
  return k * lo == v;
}
__device__ __forceinline__ int shift_of(int i) { return 4 * (i >> 1) + 16 * (i & 1); }
// A word of 8 codes.  w / s is the quotient rounded to fp32, and then to the nearest integer, halves to even.  It is
// formed by Markstein's theorem (IBM J. Res. Dev. 34, 1990): with y = 1 / s rounded, q = w y and r = w - q s exact,
// q + r y rounded once is w / s rounded once (but where s has a significand of ones alone; it has 5 bits).  Where r might
// fall below the least number the division itself is made.  Adding 1.5 * 2^23 + 8 rounds to an integer and leaves
// code + 8 in the low bits.  (With a division, a rounding and a conversion for each value their pipes took three
// times as long as the memory: 248 us for 64 x 2048 x 1408 bf16, axis 1.)
//
// Each sum's bits are 0x4b400000 + code + 8; shifted to their places they add up to the word and a constant.
__device__ __forceinline__ unsigned word_of_codes(const float (&v)[8], float s) {
  if (isnan(s)) return 0x88888888u;
  unsigned x = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) x -= 0x4b400000u << shift_of(k);
  if (s < 1e-28f) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x += __float_as_uint(v[k] / s + 12582920.f) << shift_of(k);
    return x;
  }
  const float y = 1.f / s;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float q = v[k] * y;
    x += __float_as_uint(fmaf(fmaf(-q, s, v[k]), y, q) + 12582920.f) * (1u << shift_of(k));
  }
  return x;
}
// magnitudes as integers: they order as the numbers do, with infinity and NaN above
__device__ __forceinline__ unsigned max_abs(unsigned a, float v) { return max(a, __float_as_uint(v) & 0x7fffffffu); }

// Measured, 64 x 2048 x 1408, group 32 (pack, unpack): bf16 axis 0 126 and 93 us (3.8 and 5.1 TB/s), axis 1 158 and 108;
// fp32 axis 0 152 and 141 (5.5 and 5.9), axis 1 152 and 176.  Of bf16 along axis 1 issue slots (78%) and the integer pipe
// (75%) bound the packing, along axis 0 that a warp's loads, conversion and barriers take turns (68% and 63%, 24 warps an
// SM).  Two words a lane unpacked at a time instead of four: 59 -> 48 registers, axis 1 of bf16 164 -> 158 us.

// w [E, out, in]: a thread takes the 8 inputs of a word, the G / 8 lanes of a group share its largest; a CTA takes
// COL_WORDS neighbours of all words.
constexpr int COL_NT = 256;
constexpr int COL_ITEMS = 4;
constexpr int COL_WORDS = COL_NT * COL_ITEMS;
struct Spot {
  long long row;
  int word;
};
// number `at` of a CTA's words: one division of 64 bits for the CTA's first, of 32 from there
__device__ __forceinline__ Spot spot_of(long long first_row, int first_word, int at, int words) {
  const unsigned off = (unsigned)(first_word + at), rows = off / (unsigned)words;
  return {first_row + rows, (int)(off - rows * (unsigned)words)};
}
template <typename T, int G>
__global__ void __launch_bounds__(COL_NT) w4_pack_cols_kernel(const T* __restrict__ w, long long rows, int in, int blocks,
                                                              unsigned* __restrict__ q, bf16* __restrict__ scale) {
  const int words = blocks * WORDS;
  const long long begin = (long long)blockIdx.x * COL_WORDS, first_row = begin / words;
  const int first_word = (int)(begin - first_row * words);
  constexpr int N = Vec16<T>::N;
  uint4 raw[COL_ITEMS][8 / N];  // unpacked one word at a time: more warps to an SM
#pragma unroll
  for (int i = 0; i < COL_ITEMS; ++i) {
    const Spot at = spot_of(first_row, first_word, i * COL_NT + threadIdx.x, words);
    const int c = at.word * 8;
#pragma unroll
    for (int k = 0; k < 8; k += N)
      raw[i][k / N] = at.row < rows && c + k < in ? __ldg(reinterpret_cast<const uint4*>(w + at.row * in + c + k))
                                                  : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < COL_ITEMS; ++i) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; k += N) Vec16<T>::load_raw_unpack(raw[i][k / N], v + k);
    unsigned top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max_abs(top, v[k]);
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    float s = scale_of(__uint_as_float(top));
    const float lo = below(s, __uint_as_float(top));
    bool all = lo > 0.f && fits(v[0], lo);
    if (__any_sync(0xffffffffu, all)) {  // of other weights the first tells it nearly always
#pragma unroll
      for (int k = 1; k < 8; ++k) all = all && fits(v[k], lo);
      // the lanes of this one's group
      const unsigned group = ((1u << (G / 8)) - 1) << (threadIdx.x & 31 & ~(G / 8 - 1));
      if ((__ballot_sync(0xffffffffu, all) & group) == group) s = lo;
    }
    const Spot at = spot_of(first_row, first_word, i * COL_NT + threadIdx.x, words);
    if (at.row >= rows) continue;
    const int word = at.word, place = word % WORDS;
    q[(at.row * blocks + word / WORDS) * WORDS + place % 4 * 4 + place / 4] = word_of_codes(v, s);
    if (word % (G / 8) == 0) scale[at.row * (blocks * BLOCK / G) + word / (G / 8)] = __float2bfloat16_rn(s);
  }
}

// w [E, in, out]: a CTA takes 64 V outputs (V in 4 bytes) of up to ROW_BLOCKS blocks; a thread V of them over a run of 32
// inputs, read down the rows in whole lines.  The runs of a group share its largest magnitude, and the words and
// scales, which lie along an output, go out through shared memory (a thread to an output's whole block: 299 us for
// 64 x 2048 x 1408 bf16, where memory allows 66).
constexpr int ROW_NT = 256;
constexpr int ROW_BLOCKS = 4;
template <typename T> constexpr int PER4 = 4 / sizeof(T);
template <typename T> __device__ __forceinline__ float of4(unsigned raw, int c);
template <> __device__ __forceinline__ float of4<float>(unsigned raw, int) { return __uint_as_float(raw); }
template <> __device__ __forceinline__ float of4<bf16>(unsigned raw, int c) {
  return __uint_as_float(c ? raw & 0xffff0000u : raw << 16);
}

template <typename T, int G>
__global__ void __launch_bounds__(ROW_NT) w4_pack_rows_kernel(const T* __restrict__ w, int in, int out, int blocks,
                                                              unsigned* __restrict__ q, bf16* __restrict__ scale) {
  constexpr int V = PER4<T>, COLS = 64 * V, SC = BLOCK / G;
  __shared__ unsigned words[COLS][WORDS + 1];
  __shared__ unsigned top[4][COLS];
  __shared__ bool fit[4][COLS];
  __shared__ bf16 scales[COLS][ROW_BLOCKS * SC];
  const int tx = threadIdx.x & 63, run = threadIdx.x >> 6, e = blockIdx.z;
  const int o0 = blockIdx.x * COLS, o = o0 + tx * V, b0 = blockIdx.y * ROW_BLOCKS;
  const int n_blocks = min(ROW_BLOCKS, blocks - b0);
  for (int bb = 0; bb < n_blocks; ++bb) {
    const int b = b0 + bb, k0 = b * BLOCK + run * 32;
    const T* src = w + ((long long)e * in + k0) * out + o;
    unsigned raw[32];
#pragma unroll
    for (int k = 0; k < 32; ++k)
      raw[k] = o < out && k0 + k < in ? __ldg(reinterpret_cast<const unsigned*>(src + (long long)k * out)) : 0u;
    {
      unsigned a = 0;  // of bf16: the two columns' magnitudes as integers, side by side
#pragma unroll
      for (int k = 0; k < 32; ++k) a = V == 2 ? __vmaxu2(a, raw[k] & 0x7fff7fffu) : max(a, raw[k] & 0x7fffffffu);
#pragma unroll
      for (int c = 0; c < V; ++c) top[run][tx * V + c] = V == 1 ? a : c ? a & 0xffff0000u : a << 16;
    }
    __syncthreads();  // and the words of the block before have been written
    constexpr int RUNS = G / 32;
    const int r0 = run / RUNS * RUNS;
    float scale_c[V], lower[V];
    bool all[V], any = false;  // whether this thread's part of the column's group fits the lower scale
#pragma unroll
    for (int c = 0; c < V; ++c) {
      unsigned a = top[r0][tx * V + c];
#pragma unroll
      for (int r = 1; r < RUNS; ++r) a = max(a, top[r0 + r][tx * V + c]);
      scale_c[c] = scale_of(__uint_as_float(a));
      lower[c] = below(scale_c[c], __uint_as_float(a));
      all[c] = lower[c] > 0.f && fits(of4<T>(raw[0], c), lower[c]);
      any |= all[c];
    }
    // Of other weights the first few tell it; a loop that reads them again keeps the registers and the code small.
#pragma unroll 1
    for (int k = 1; k < 32 && __any_sync(0xffffffffu, any); ++k) {
      const unsigned x = o < out && k0 + k < in ? __ldg(reinterpret_cast<const unsigned*>(src + (long long)k * out)) : 0u;
      any = false;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        all[c] = all[c] && fits(of4<T>(x, c), lower[c]);
        any |= all[c];
      }
    }
    if (RUNS > 1) {
#pragma unroll
      for (int c = 0; c < V; ++c) fit[run][tx * V + c] = all[c];
      __syncthreads();
#pragma unroll
      for (int c = 0; c < V; ++c)
#pragma unroll
        for (int r = 0; r < RUNS; ++r) all[c] = all[c] && fit[r0 + r][tx * V + c];
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const float s = all[c] ? lower[c] : scale_c[c];
      if (run == r0) scales[tx * V + c][bb * SC + run / RUNS] = __float2bfloat16_rn(s);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = of4<T>(raw[8 * v + k], c);
        words[tx * V + c][v * 4 + run] = word_of_codes(x, s);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < COLS * WORDS; i += ROW_NT) {
      const int col = i / WORDS, at = i % WORDS;
      if (o0 + col < out) q[(((long long)e * out + o0 + col) * blocks + b) * WORDS + at] = words[col][at];
    }
  }
  for (int i = threadIdx.x; i < COLS * n_blocks * SC; i += ROW_NT) {
    const int col = i / (n_blocks * SC), at = i - col * (n_blocks * SC);
    if (o0 + col < out) scale[((long long)e * out + o0 + col) * (blocks * SC) + b0 * SC + at] = scales[col][at];
  }
}

__device__ __forceinline__ unsigned bits_of(__nv_bfloat162 v) { return *reinterpret_cast<unsigned*>(&v); }
__device__ __forceinline__ __nv_bfloat162 pair_from(unsigned v) { return *reinterpret_cast<__nv_bfloat162*>(&v); }
__device__ __forceinline__ __nv_bfloat162 times(__nv_bfloat162 v, float by) { return __hmul2(v, __float2bfloat162_rn(by)); }

// Weights as bf16 numbers, two neighbours at a time.  The least bf16 numbers, subnormal ones and the first normal ones,
// are the multiples k 2^-133 for k < 256, with k as their bits.  So a word masked to a pair of codes is a pair of numbers
// already, of code 2^-133 or (4 bits up) code 2^-129, and  fma(code 2^-133, 2^133 s, -8 s)  is the weight q s, rounded
// once (not at all where s has 5 significant bits).  2^133 s is finite for |s| < 2^-5; for other scales 128 + code is
// made, 136 subtracted and the rest multiplied, with the same result in more operations.
struct Scaled {
  __nv_bfloat162 s, s133, s129, minus8;
  __device__ __forceinline__ explicit Scaled(__nv_bfloat162 scale)
      : s(scale), s133(times(times(scale, 0x1p100f), 0x1p33f)), s129(times(s133, 0x1p-4f)), minus8(times(scale, -8.f)) {}
};
__device__ __forceinline__ bool is_small(__nv_bfloat162 s) { return __hblt2(__habs2(s), __float2bfloat162_rn(0x1p-5f)); }
// pair t of a word; SMALL: is_small(s.s)
template <bool SMALL>
__device__ __forceinline__ unsigned weights_of(unsigned word, int t, const Scaled& s) {
  if (SMALL) {
    const unsigned x = (t < 2 ? word : word >> 8) & (t & 1 ? 0x00f000f0u : 0x000f000fu);
    return bits_of(__hfma2(pair_from(x), t & 1 ? s.s129 : s.s133, s.minus8));
  }
  const unsigned x = ((word >> (4 * t)) & 0x000f000fu) | 0x43004300u;
  return bits_of(__hmul2(__hsub2(pair_from(x), __float2bfloat162_rn(136.f)), s.s));
}

// code + 8 under the exponent of 2^23 is the number 2^23 + code + 8
__device__ __forceinline__ float value_of(unsigned word, int i, float s) {
  return (__uint_as_float(((word >> shift_of(i)) & 15u) | 0x4b000000u) - 8388616.f) * s;
}

template <typename T>
__global__ void __launch_bounds__(COL_NT)
w4_unpack_cols_kernel(const unsigned* __restrict__ q, const bf16* __restrict__ scale, long long rows, int in, int blocks,
                      int G, T* __restrict__ w) {
  const int words = blocks * WORDS;
  const long long begin = (long long)blockIdx.x * COL_WORDS, first_row = begin / words;
  const int first_word = (int)(begin - first_row * words);
  unsigned x[COL_ITEMS];
  bf16 s[COL_ITEMS];
  Spot at[COL_ITEMS];
#pragma unroll
  for (int i = 0; i < COL_ITEMS; ++i) {
    at[i] = spot_of(first_row, first_word, i * COL_NT + threadIdx.x, words);
    if (at[i].row >= rows) continue;
    const int word = at[i].word, place = word % WORDS;
    x[i] = __ldg(q + (at[i].row * blocks + word / WORDS) * WORDS + place % 4 * 4 + place / 4);
    s[i] = scale[at[i].row * (blocks * BLOCK / G) + word * 8 / G];
  }
#pragma unroll
  for (int i = 0; i < COL_ITEMS; ++i) {
    const int c = at[i].word * 8;
    if (at[i].row >= rows || c >= in) continue;
    if (sizeof(T) == 2) {
      const Scaled sc(__nv_bfloat162(s[i], s[i]));
      uint4 o;
      if (is_small(sc.s))
        o = make_uint4(weights_of<true>(x[i], 0, sc), weights_of<true>(x[i], 1, sc), weights_of<true>(x[i], 2, sc),
                       weights_of<true>(x[i], 3, sc));
      else
        o = make_uint4(weights_of<false>(x[i], 0, sc), weights_of<false>(x[i], 1, sc), weights_of<false>(x[i], 2, sc),
                       weights_of<false>(x[i], 3, sc));
      *reinterpret_cast<uint4*>(w + at[i].row * in + c) = o;
      continue;
    }
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = value_of(x[i], k, to_f32(s[i]));
#pragma unroll
    for (int k = 0; k < 8; k += Vec16<T>::N)
      if (c + k < in) Vec16<T>::store(w + at[i].row * in + c + k, v + k);
  }
}

// the same way round as w4_pack_rows_kernel
template <typename T>
__global__ void __launch_bounds__(ROW_NT)
w4_unpack_rows_kernel(const unsigned* __restrict__ q, const bf16* __restrict__ scale, int in, int out, int blocks, int G,
                      T* __restrict__ w) {
  constexpr int V = PER4<T>, COLS = 64 * V;
  __shared__ unsigned words[COLS][WORDS + 1];
  __shared__ bf16 scales[COLS][ROW_BLOCKS * 4];
  const int tx = threadIdx.x & 63, run = threadIdx.x >> 6, e = blockIdx.z, sc = BLOCK / G;
  const int o0 = blockIdx.x * COLS, o = o0 + tx * V, b0 = blockIdx.y * ROW_BLOCKS;
  const int n_blocks = min(ROW_BLOCKS, blocks - b0);
  for (int i = threadIdx.x; i < COLS * n_blocks * sc; i += ROW_NT) {
    const int col = i / (n_blocks * sc), at = i - col * (n_blocks * sc);
    if (o0 + col < out) scales[col][at] = scale[((long long)e * out + o0 + col) * (blocks * sc) + b0 * sc + at];
  }
  for (int bb = 0; bb < n_blocks; ++bb) {
    const int b = b0 + bb, k0 = b * BLOCK + run * 32;
    __syncthreads();
    for (int i = threadIdx.x; i < COLS * WORDS; i += ROW_NT) {
      const int col = i / WORDS, at = i % WORDS;
      if (o0 + col < out) words[col][at] = __ldg(q + (((long long)e * out + o0 + col) * blocks + b) * WORDS + at);
    }
    __syncthreads();
    if (o >= out) continue;
    unsigned mine[V][4];
    bf16 sv[V];
#pragma unroll
    for (int c = 0; c < V; ++c) {
#pragma unroll
      for (int v = 0; v < 4; ++v) mine[c][v] = words[tx * V + c][v * 4 + run];
      sv[c] = scales[tx * V + c][bb * sc + run * 32 / G];
    }
    T* dst = w + ((long long)e * in + k0) * out + o;
    if (V == 2) {  // two neighbours of either column, then of either row (the number of rows is even)
      const Scaled s0(__nv_bfloat162(sv[0], sv[0])), s1(__nv_bfloat162(sv[V - 1], sv[V - 1]));
      auto put = [&](auto weights) {
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          if (k0 + k >= in) break;
          const unsigned a = weights(mine[0][k / 8], k % 8 / 2, s0), b = weights(mine[V - 1][k / 8], k % 8 / 2, s1);
          *reinterpret_cast<unsigned*>(dst + (long long)k * out) = __byte_perm(a, b, 0x5410);
          *reinterpret_cast<unsigned*>(dst + (long long)(k + 1) * out) = __byte_perm(a, b, 0x7632);
        }
      };
      if (is_small(s0.s) && is_small(s1.s)) put([](unsigned x, int t, const Scaled& s) { return weights_of<true>(x, t, s); });
      else put([](unsigned x, int t, const Scaled& s) { return weights_of<false>(x, t, s); });
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        if (k0 + k >= in) break;
        dst[(long long)k * out] = from_f32<T>(value_of(mine[0][k / 8], k % 8, to_f32(sv[0])));
      }
    }
  }
}

// ------------------------------------------------------------ tiles and items ---
constexpr int MAX_E = 1024;

struct Args {
  const bf16* x = nullptr;
  const int32_t* src_tok;  // row r of x, or nullptr: row r itself
  int x_rows;
  const int32_t* cu;
  int E, R, in, out;  // out: outputs of a tensor
  int group, tile;  // tile: its rows
  const bf16 *s0, *s1;
  bf16* y;  // [R, out]
  int wk = 0;  // w4_rows_kernel: warps that share a strip of outputs
  unsigned* err;
  unsigned long long wait_limit;
};

// Tiles of N rows that R rows of E experts make at most.
inline long long most_tiles(int R, int E, int N) { return (long long)(E < R ? E : R) + R / N; }

// The tiles of N rows of all experts: before[e] = tiles of the experts before e.  Offsets that do not begin with 0 and
// end with R, or lie outside, are cut off there and reported.  Where they run downwards, experts would share rows
// and make more tiles than most_tiles: there are none then.
struct Tiles {
  int before[MAX_E + 1], row0[MAX_E], row1[MAX_E];
  int warp_sum[8];
};
template <int N>
__device__ __forceinline__ void count_tiles(Tiles& t, const int32_t* cu, int E, int R, unsigned* err) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int PER = MAX_E / 256;  // experts of a thread; the first 256 threads
  const int e0 = threadIdx.x * PER;
  int n[PER], sum = 0, incl = 0;
  bool down = false;
  if (threadIdx.x < 256) {
    int at[PER + 1];
#pragma unroll
    for (int k = 0; k <= PER; ++k) at[k] = e0 + k <= E ? __ldg(cu + e0 + k) : R;
    if (threadIdx.x == 0 && blockIdx.x == 0 && (at[0] != 0 || __ldg(cu + E) != R)) set_error(err, DEV_BOUNDS);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int a = min(max(at[k], 0), R), b = min(max(at[k + 1], a), R);
      n[k] = e0 + k < E && b > a ? (b - a - 1) / N + 1 : 0;
      down |= e0 + k < E && at[k + 1] < at[k];
      sum += n[k];
      if (e0 + k < E) t.row0[e0 + k] = a, t.row1[e0 + k] = b;
    }
    incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) t.warp_sum[warp] = incl;
  }
  const bool none = __syncthreads_or(down) != 0;
  if (none && threadIdx.x == 0 && blockIdx.x == 0) set_error(err, DEV_BOUNDS);
  if (threadIdx.x < 256) {
    int run = none ? 0 : incl - sum;
    for (int w = 0; w < warp && !none; ++w) run += t.warp_sum[w];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (e0 + k <= E) t.before[e0 + k] = run;
      if (!none) run += n[k];
    }
    if (threadIdx.x == 255) t.before[E] = run;
  }
  __syncthreads();
}

struct Item {
  int e, r0, rows, n0;  // n0: first output; rows 0: no more items
};
// Item i: experts in order, in each its strips of outputs in order, in each strip its tiles of rows.  A whole warp
// calls it, and with growing i: the experts from the last call's on are looked at 32 at a time.  (By
// bisection, with 64-bit quotients, an item cost each warp some 300 cycles, 10% of the time of T = 16.)
struct ItemSearch {
  int e = 0;
  template <int N>
  __device__ __forceinline__ Item at(const Tiles& t, int E, int i, int strips, int width) {
    Item w = {0, 0, 0, 0};
    const int tile_no = (int)((unsigned)i / (unsigned)strips);
    if (tile_no >= t.before[E]) return w;
    const int lane = threadIdx.x & 31;
    for (;;) {  // to the last expert whose tiles begin at or before this one
      const int next = e + 1 + lane;
      const int n = __popc(__ballot_sync(0xffffffffu, next <= E && t.before[next] <= tile_no));
      e += n;
      if (n < 32) break;
    }
    const int first = t.before[e], tiles = t.before[e + 1] - first, local = i - first * strips;
    const int strip = tiles == 1 ? local : (int)((unsigned)local / (unsigned)tiles), tile = local - strip * tiles;
    w.e = e;
    w.r0 = t.row0[e] + tile * N;
    w.rows = min(N, t.row1[e] - w.r0);
    w.n0 = strip * width;
    return w;
  }
};

// ------------------------------------------------------ products of few rows ---
// Weights are the MMA's A operand (16 outputs x 16 inputs), up to 8 routed rows its B operand, so a
// weight is read and turned into bf16 once for the tile's rows.  A pair of codes comes out of its word by a mask and
// an fma as two numbers q 2^-10: exact, so a code of 0 leaves no trace of its entry, and small enough that no
// sum over a group of 128 leaves fp32's range while its result is inside.  (As numbers 128 + (q + 8), with 136 sum x
// taken off by another MMA, an infinite x was NaN in every output, and an entry of 2^20 left errors of some 2^20 2^-16
// scales everywhere.  Sums below 2^-116 lose bits so, to 2^-140 or thereabouts; bf16 ends at 2^-133.)  The group's scale is applied to its fp32 sums, 2^10 to the whole ones.
//
// An item is a strip of outputs (16 of gate and the same of up, or 32 of down) for one tile of rows.  WK
// warps share its inputs, each every WK-th pair of blocks; their sums meet in shared memory in a
// fixed order.  The weights' way from memory comes first: each warp keeps a ring of STAGES pairs of blocks in
// flight by TMA, across items.  (Loads into registers met two limits before that one: the 64-byte
// pieces of 8 rows took the L1's tag stage, and too few of them were under way.)
// The rows x are read through L1, where the strips of an expert find them again.
//
// Measured, with the second product: one row to 8 of 384 experts of 7168 x 2048, groups of 128, 50 us (3.6 TB/s of
// codes and scales; 56 with the offset taken off by MMAs).  Loads under way, the integer pipe (44%, 34% in the second product)
// and the warp-level MMAs (22%, 17%) take turns in 16 warps an SM, too few to hide each other; two or four tiles of rows a weight, more warps with fewer registers (spills) and asking L2 for the
// weights ahead brought nothing.
//
// A stage holds 32 rows of 128 bytes, swizzled: 16-byte piece c of row r lies at c ^ (r & 7).  Lane
// group g reads row 4 (g & 1) + g / 2 of each eight, so that the two rows which a quarter
// of a warp reads together lie in different halves of the banks.
constexpr int NT_WARPS = 8;
constexpr int STAGES = 2;
constexpr int STAGE_BYTES = 32 * 128;
constexpr int AHEAD = 8;  // items that a warp's loads may be ahead, a power of two above STAGES + 1

// d = a b + c
__device__ __forceinline__ void mma_bf16(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1,
                                         const float (&c)[4]) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, "
      "%12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// codes of a word's pair t as bf16 numbers q 2^-10; masked they are the numbers code 2^-133 or code 2^-129 (see Scaled)
constexpr float UNIT = 1024.f;
__device__ __forceinline__ unsigned pair_of(unsigned word, int t) {
  const unsigned x = (t < 2 ? word : word >> 8) & (t & 1 ? 0x00f000f0u : 0x000f000fu);
  // times 2^119 or 2^123, minus 2^-7
  return bits_of(__hfma2(pair_from(x), pair_from(t & 1 ? 0x7b007b00u : 0x7d007d00u), pair_from(0xbc00bc00u)));
}
__device__ __forceinline__ unsigned word_of(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// The scales of a pair of blocks for one output, 2 SC bf16 numbers in SC registers (a row of scales
// is aligned to those of one block alone).  Lane r of a warp holds those of row r of a stage.
template <int SC>
__device__ __forceinline__ void load_scales(unsigned (&v)[SC], const bf16* p, bool second) {
  if (SC == 4) {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(p));
    const uint2 b = second ? __ldg(reinterpret_cast<const uint2*>(p) + 1) : make_uint2(0, 0);
    v[0] = a.x, v[1 % SC] = a.y, v[2 % SC] = b.x, v[3 % SC] = b.y;
  } else if (SC == 2) {
    v[0] = __ldg(reinterpret_cast<const unsigned*>(p));
    v[1 % SC] = second ? __ldg(reinterpret_cast<const unsigned*>(p) + 1) : 0u;
  } else {
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
    v[0] = __ldg(q) | (second ? (unsigned)__ldg(q + 1) << 16 : 0u);
  }
}

__device__ const uint4 zero_row[16] = {};  // what a lane without a row reads

constexpr int RESIDENT = 2;  // CTAs of an SM
constexpr int ROWS = 8;      // rows of a tile
constexpr int SUMS = 8 * 32;  // a warp's sums: [2 tiles of outputs][4][32 lanes]
// stages, sums (two places in turn save a barrier an item), and room to align the stages
constexpr size_t ROWS_SMEM = (size_t)NT_WARPS * STAGES * STAGE_BYTES + 2 * NT_WARPS * SUMS * 4 + 1024;

template <int G, bool GATE_UP>
__global__ void __launch_bounds__(32 * NT_WARPS, RESIDENT)
w4_rows_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1, const Args p) {
  constexpr int STRIP = GATE_UP ? 16 : 32, SC = BLOCK / G;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Tiles tiles;
  __shared__ Item coming[NT_WARPS][AHEAD];
  __shared__ uint64_t bars[NT_WARPS][STAGES];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tg = lane & 3;
  const int prow = 4 * (g & 1) + (g >> 1);  // this lane group's row of eight
  const int wk = p.wk, kw = warp % wk, sub = warp / wk;
  const int blocks = blocks_of(p.in), pairs = (blocks + 1) / 2;
  const int strips = (p.out + STRIP - 1) / STRIP;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + warp * STAGES * STAGE_BYTES;
  float* red = reinterpret_cast<float*>(smem + NT_WARPS * STAGES * STAGE_BYTES);

  if (threadIdx.x == 0) {
    abort_flag = 0;
    tc::prefetch_tmap(&tm0);
    tc::prefetch_tmap(&tm1);
  }
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) tc::mbar_init(tc::smem_u32(&bars[warp][s]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  count_tiles<ROWS>(tiles, p.cu, p.E, p.R, p.err);  // ends with a barrier of the CTA
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the warp's loads: stage `issued` of its sequence of (item, pair of blocks)
  const int stride = gridDim.x * (NT_WARPS / wk);
  int load_i = blockIdx.x * (NT_WARPS / wk) + sub;
  ItemSearch search;
  int load_items = 0, load_pair = kw, issued = 0, load_row = 0;
  bool loading;
  const bf16* load_s = nullptr;  // scales of this lane's row of the stage
  auto next_item = [&]() {
    const Item w = search.at<ROWS>(tiles, p.E, load_i, strips, STRIP);
    if (lane == 0) coming[warp][load_items % AHEAD] = w;
    load_i += stride;
    ++load_items;
    load_pair = kw;
    loading = w.rows > 0;
    load_row = w.e * p.out + w.n0;
    const long long row = (long long)w.e * p.out + min(w.n0 + (GATE_UP ? lane & 15 : lane), p.out - 1);
    load_s = (GATE_UP && lane >= 16 ? p.s1 : p.s0) + (row * blocks + 2 * kw) * SC;
  };
  next_item();
  unsigned sc_in[STAGES][SC];  // scales of the stages under way, the next one's first
  auto issue = [&](bool load) {  // without `load` only the place moves on
    if (!loading) return;
    if (load) {
      const int slot = issued % STAGES;
      if (tc::elect_one()) {
        const uint32_t bar = tc::smem_u32(&bars[warp][slot]), dst = tc::smem_u32(ring + slot * STAGE_BYTES);
        tc::mbar_expect_tx(bar, STAGE_BYTES);
        tc::tma_load_2d(dst, &tm0, bar, load_pair * 2 * WORDS, load_row);
        if (GATE_UP) tc::tma_load_2d(dst + STAGE_BYTES / 2, &tm1, bar, load_pair * 2 * WORDS, load_row);
      }
      load_scales<SC>(sc_in[STAGES - 1], load_s, 2 * load_pair + 1 < blocks);
      ++issued;
    }
    load_pair += wk;
    load_s += 2 * wk * SC;
    if (load_pair >= pairs) next_item();
  };
  auto shift_scales = [&]() {
#pragma unroll
    for (int s = 0; s + 1 < STAGES; ++s)
#pragma unroll
      for (int k = 0; k < SC; ++k) sc_in[s][k] = sc_in[s + 1][k];
  };
#pragma unroll
  for (int s = 0; s < STAGES; ++s) {
    shift_scales();
    issue(true);
  }
  __syncwarp();
  if (!GATE_UP) asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows that gate and up left

  int done = 0, landed = 0;
  bool ok = true;
  for (int round = 0;; ++round) {
    const Item it = coming[warp][round % AHEAD];
    if (it.rows <= 0) break;
    const uint4* xr = zero_row;  // this lane's row
    int step = 0;
    if (g < it.rows) {
      long long from = it.r0 + g;
      if (p.src_tok) from = __ldg(p.src_tok + from);
      if (from < 0 || from >= p.x_rows) {
        set_error(p.err, DEV_BOUNDS);
      } else {
        xr = reinterpret_cast<const uint4*>(p.x + from * p.in) + tg;
        step = BLOCK / 8;
      }
    }
    float acc[2][4] = {};
#pragma unroll 1
    for (int pair = kw; pair < pairs; pair += wk) {
      const int slot = done % STAGES;
      // the row's values of the pair, asked for before the weights are waited for; lanes past the last input
      // get zeros
      uint4 xv[2][4];
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int b = 2 * pair + half;
          xv[half][j] = b * BLOCK + 32 * j + 8 * tg < p.in ? xr[b * step + 4 * j] : make_uint4(0, 0, 0, 0);
        }
      // a wait that gives up: the warp goes on without loads, so that its barriers are met
      if (ok) ok = tc::wait_bounded(tc::smem_u32(&bars[warp][slot]), (done / STAGES) & 1, &abort_flag, p);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) ++landed;
      const uint8_t* st = ring + slot * STAGE_BYTES + prow * 128;
      auto block = [&](int half) {
        uint4 w[2][2];
        float sc[2][2][SC];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            w[t][h] = *reinterpret_cast<const uint4*>(st + (2 * t + h) * 1024 + (((4 * half + tg) ^ prow) << 4));
#pragma unroll
            for (int k = 0; k < SC; ++k) {  // number SC half + k of the pair's
              const int at = SC * half + k;
              const unsigned v = __shfl_sync(0xffffffffu, sc_in[0][at / 2], 16 * t + 8 * h + prow);
              sc[t][h][k] = __uint_as_float(at & 1 ? v & 0xffff0000u : v << 16);
            }
          }
        constexpr int RUNS = 4 / SC;  // runs of 32 inputs in a group
#pragma unroll
        for (int k = 0; k < SC; ++k) {
          float c[2][4] = {};
#pragma unroll
          for (int j = k * RUNS; j < (k + 1) * RUNS; ++j)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const unsigned u = word_of(w[t][0], j), v = word_of(w[t][1], j);
              const unsigned a0[4] = {pair_of(u, 0), pair_of(v, 0), pair_of(u, 1), pair_of(v, 1)};
              const unsigned a1[4] = {pair_of(u, 2), pair_of(v, 2), pair_of(u, 3), pair_of(v, 3)};
              mma_bf16(c[t], a0, xv[half][j].x, xv[half][j].y, c[t]);
              mma_bf16(c[t], a1, xv[half][j].z, xv[half][j].w, c[t]);
            }
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int m = 0; m < 4; ++m) acc[t][m] = fmaf(sc[t][m / 2][k], c[t][m], acc[t][m]);
        }
      };
      block(0);
      if (2 * pair + 1 < blocks) block(1);
      ++done;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the slot has been read
      __syncwarp();
      shift_scales();
      issue(ok);
    }

    // the strip's warps add up, and each finishes some of the sums
    float* buf = red + (round & 1) * (NT_WARPS * SUMS);
    float* mine = buf + warp * SUMS + lane;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int m = 0; m < 4; ++m) mine[(t * 4 + m) * 32] = acc[t][m];
    if (wk == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "r"(32 * wk) : "memory");
    const float* strip = buf + (warp - kw) * SUMS + lane;
    for (int m = kw; m < 4; m += wk) {
      float v[2] = {0.f, 0.f};
      for (int k = 0; k < wk; ++k)
#pragma unroll
        for (int t = 0; t < 2; ++t) v[t] += strip[k * SUMS + (t * 4 + m) * 32];
      v[0] *= UNIT, v[1] *= UNIT;
      const int r = 2 * tg + (m & 1), n = it.n0 + prow + 8 * (m >> 1);
      if (r >= it.rows) continue;
      bf16* dst = p.y + (long long)(it.r0 + r) * p.out;
      if (GATE_UP) {
        if (n < p.out) dst[n] = __float2bfloat16_rn(v[0] / (1.f + expf(-v[0])) * v[1]);
      } else {
        if (n < p.out) dst[n] = __float2bfloat16_rn(v[0]);
        if (n + 16 < p.out) dst[n + 16] = __float2bfloat16_rn(v[1]);
      }
    }
  }
  // a warp whose wait gave up leaves nothing under way
  for (; landed < issued; ++landed) {
    const long long t0 = clock64();
    while (!tc::mbar_try_wait(tc::smem_u32(&bars[warp][landed % STAGES]), (landed / STAGES) & 1)) {
      if ((unsigned long long)(clock64() - t0) > tc::DRAIN_LIMIT) { set_error(p.err, DEV_TIMEOUT); break; }
    }
  }
}

// codes of [rows, in] weights, `words` of a row and `box_rows` rows at a time
bool map_codes(CUtensorMap* m, const void* q, long long rows, int in, int box_words, int box_rows) {
  const long long words = (long long)blocks_of(in) * WORDS;
  cuuint64_t dims[2] = {(cuuint64_t)words, (cuuint64_t)rows};
  cuuint64_t str[1] = {(cuuint64_t)words * 4};
  cuuint32_t box[2] = {(cuuint32_t)box_words, (cuuint32_t)box_rows};
  return tc::make_map(m, q, 2, dims, str, box, CU_TENSOR_MAP_DATA_TYPE_UINT32,
                      box_words == WORDS ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int G, bool GATE_UP>
int launch_rows(const void* x, const void* q0, const void* q1, Args p, cudaStream_t s) {
  constexpr int STRIP = GATE_UP ? 16 : 32;
  CUtensorMap tm0, tm1;
  const long long outs = (long long)p.E * p.out;
  if (!map_codes(&tm0, q0, outs, p.in, 2 * WORDS, STRIP) || !map_codes(&tm1, q1, outs, p.in, 2 * WORDS, STRIP))
    return MOE_ERR_CUDA;
  p.x = static_cast<const bf16*>(x);
  const int pairs = (blocks_of(p.in) + 1) / 2, strips = (p.out + STRIP - 1) / STRIP;
  const long long slots = most_tiles(p.R, p.E, ROWS);
  const long long resident = (long long)RESIDENT * sm_count();
  if (slots * strips > 0x3fffffffll) return MOE_ERR_UNSUPPORTED;
  // Warps to a strip: more of them make the items finer, and each item costs its warps a meeting
  // (about as much as 0.7 pairs of blocks).  The least of rounds x time of an item.
  double best = 0;
  for (int wk = 1; wk <= NT_WARPS && wk <= pairs; wk *= 2) {
    const long long groups = resident * (NT_WARPS / wk), rounds = (slots * strips + groups - 1) / groups;
    const double cost = (double)rounds * ((pairs + wk - 1) / wk + 0.7);
    if (wk == 1 || cost < best) p.wk = wk, best = cost;
  }
  const long long ctas = (slots * strips * p.wk + NT_WARPS - 1) / NT_WARPS;
  auto k = w4_rows_kernel<G, GATE_UP>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ROWS_SMEM) != cudaSuccess)
    return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas < resident ? ctas : resident));
  cfg.blockDim = dim3(32 * NT_WARPS);
  cfg.dynamicSmemBytes = ROWS_SMEM;
  cfg.stream = s;
  // the second product's CTAs start, and fetch their first weights, while the first one's finish
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = GATE_UP ? 0 : 1;
  if (cudaLaunchKernelEx(&cfg, k, tm0, tm1, p) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

// ----------------------------------------------------- products of more rows ---
// A tile is 128 outputs (64 of gate and the same 64 of up, or 128 of down) for up to N routed rows of one
// expert.  The weights are the MMA's A operand and live in tensor memory: a thread takes one
// output, turns a block of its codes into 128 bf16 numbers in registers and stores them into its
// lane's columns, where tcgen05.mma reads them.  Only the codes themselves and the rows x pass
// through shared memory.  (With the bf16 weights there too, 16 KB written and read for every 4 KB of codes,
// shared memory would bound the kernel at half the memory's rate.)
//
// The conversion (weights_of) is 9 operations for 8 weights, 5 of them on the integer pipe.
//
// Roles of a CTA, one to an SM: warp 0 loads codes (TMA), warp 1 issues the MMAs, warps 2 to 5 are the
// epilogue, then SETS x 8 warps convert (a set takes every SETS-th pair of blocks, four warps a block), and the last
// warp loads the rows x.  All loops run over the same sequence of tiles and blocks, so loads and
// conversion do not stop between tiles.  Every wait is bounded.
//
// Measured, with the second product: 4 rows to each of 8 experts of 4096 x 14336, groups of 64, 166 us (4.5 TB/s of codes
// and scales); 6 to each of 64 experts of 2048 x 1408, groups of 32, 80 us (3.9); 384 to each, groups of 128, 404-420 us
// (1.03 PFLOP/s).  What bounds it for few rows are issue slots: 65 to 75% of all and 72 to 93% of the scheduler's that also
// has the MMA warp, start and end of the launches included.  (6 rows: with 16 + code and fma(., s, -24 s), three more shifts
// a word, 90 us; with a subtraction and a product 92; a set of four warps for a whole pair 82 us for 54% of the
// slots, as fewer warps wait longer.)  For 128 rows MMAs and conversion take turns: tensor memory has no room for a
// third pair of blocks.  Shifts as products on the other pipe, the scales asked for earlier or through L2,
// waits that sleep: nothing.
constexpr int TILE = 128;                     // outputs of a tile
constexpr int CODE_BYTES = TILE * BLOCK / 2;  // a block of codes of a tile
constexpr int A_COLS = BLOCK / 2;             // tensor memory columns of a block of bf16 weights
template <int N>
struct Cfg {
  // pairs of blocks that may be converted, and have their rows x loaded, ahead of the MMAs
  static constexpr int PAIRS = N <= 64 ? 3 : 2;
  static constexpr int SETS = PAIRS;
  static constexpr int THREADS = 32 * (6 + 8 * SETS + 1);
  // Pairs of blocks of codes under way: two places for each set's, so that what lay in a place before is known to have
  // been read when a set asks for its next codes by their parity.
  static constexpr int CODES = 2 * SETS;
  static constexpr int X_BYTES = N * BLOCK * 2;  // a block of the rows: two halves of 64 inputs
  static constexpr int ACC_COLS = N < 32 ? 32 : N;
  static constexpr int A_BASE = 2 * ACC_COLS;
  static constexpr int EX_BYTES = 2 * 4 * 16 * 32 * 4;  // sums of gate and up on their way to each other's warps
  static constexpr size_t SMEM = (size_t)2 * CODES * CODE_BYTES + (size_t)2 * PAIRS * X_BYTES + EX_BYTES + 1024;
  static_assert(A_BASE + 2 * PAIRS * A_COLS <= 512, "tensor memory");
};

// The 16 words of run j's weights, of which the codes are w[v]'s component j and the scale is one of `scales`.
template <bool SMALL>
__device__ __forceinline__ void convert_run(const uint4 (&w)[4], int j, unsigned scales, unsigned (&r)[16]) {
  const Scaled s(pair_from(__byte_perm(scales, scales, j & 1 ? 0x3232 : 0x1010)));
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const unsigned word = j == 0 ? w[v].x : j == 1 ? w[v].y : j == 2 ? w[v].z : w[v].w;
#pragma unroll
    for (int t = 0; t < 4; ++t) r[v * 4 + t] = weights_of<SMALL>(word, t, s);
  }
}
// 32 lanes x 16 columns of tensor memory
__device__ __forceinline__ void tmem_st16(uint32_t at, const unsigned (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
      : "memory");
}
// 32 lanes x 32 or 16 columns of sums
__device__ __forceinline__ void sums_of(uint32_t at, float (&v)[32]) { tc::tmem_ld32(at, v); }
__device__ __forceinline__ void sums_of(uint32_t at, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
}
// D (+)= A B with A in tensor memory
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// whether a phase has completed, without waiting
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// whether all 128 threads of the epilogue say yes
__device__ __forceinline__ bool all_of_epilogue(bool yes) {
  unsigned ok = yes;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %0, 0;\n\t"
      "barrier.cta.red.and.pred q, 3, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "+r"(ok)::"memory");
  return ok != 0;
}

// R rows of one output a lane, `rows` of them there: neighbouring lanes swap, so that each writes two
// neighbours of every other row.  The number of outputs is even.
template <int R>
__device__ __forceinline__ void store_rows(const float (&v)[R], bf16* dst, long long ld, int rows, bool store) {
  const int odd = threadIdx.x & 1;
#pragma unroll
  for (int k = 0; k < R / 2; ++k) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[2 * k] : v[2 * k + 1], 1);
    const __nv_bfloat162 h = odd ? __floats2bfloat162_rn(got, v[2 * k + 1]) : __floats2bfloat162_rn(v[2 * k], got);
    if (store && 2 * k + odd < rows) *reinterpret_cast<__nv_bfloat162*>(dst + (2 * k + odd) * ld - odd) = h;
  }
}

// the scales of a block: four, two or one bf16 number
template <int G>
__device__ __forceinline__ uint2 load_scales(const bf16* p) {
  if (G == 32) return __ldg(reinterpret_cast<const uint2*>(p));
  if (G == 64) return make_uint2(__ldg(reinterpret_cast<const unsigned*>(p)), 0u);
  return make_uint2(__ldg(reinterpret_cast<const unsigned short*>(p)), 0u);
}
// and one for each of its runs of 32 inputs, once they are needed
template <int G>
__device__ __forceinline__ uint2 spread_scales(uint2 v) {
  if (G == 32) return v;
  if (G == 64) return make_uint2(__byte_perm(v.x, v.x, 0x1010), __byte_perm(v.x, v.x, 0x3232));
  const unsigned two = v.x | v.x << 16;
  return make_uint2(two, two);
}

template <int N, int G, bool GATE_UP>
__global__ void __launch_bounds__(Cfg<N>::THREADS, 1)
w4_ffn_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
              const __grid_constant__ CUtensorMap tmx, const Args p) {
  using C = Cfg<N>;
  using namespace tc;
  constexpr int WIDTH = GATE_UP ? TILE / 2 : TILE, SC = BLOCK / G, SETS = C::SETS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* xs = smem + 2 * C::CODES * CODE_BYTES;
  float* ex = reinterpret_cast<float*>(xs + 2 * C::PAIRS * C::X_BYTES);
  __shared__ Tiles tiles;
  __shared__ uint64_t bars[2 * C::CODES + 3 * C::PAIRS + 5];
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;
  auto codef = [&](int s) { return smem_u32(&bars[s]); };                       // codes have landed
  auto codee = [&](int s) { return smem_u32(&bars[C::CODES + s]); };            // and been read
  auto xf = [&](int b) { return smem_u32(&bars[2 * C::CODES + b]); };           // rows have landed
  auto af = [&](int b) { return smem_u32(&bars[2 * C::CODES + C::PAIRS + b]); };  // weights are in tensor memory
  auto done = [&](int b) { return smem_u32(&bars[2 * C::CODES + 2 * C::PAIRS + b]); };  // and have been multiplied
  auto accf = [&](int a) { return smem_u32(&bars[2 * C::CODES + 3 * C::PAIRS + a]); };
  auto acce = [&](int a) { return smem_u32(&bars[2 * C::CODES + 3 * C::PAIRS + 2 + a]); };
  const uint32_t drain = smem_u32(&bars[2 * C::CODES + 3 * C::PAIRS + 4]);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = blocks_of(p.in), pairs = (blocks + 1) / 2, strips = (p.out + WIDTH - 1) / WIDTH;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < C::CODES; ++s) {
      mbar_init(codef(s), 1);
      mbar_init(codee(s), 8);  // the warps of a set
    }
    for (int b = 0; b < C::PAIRS; ++b) {
      mbar_init(xf(b), 1);
      mbar_init(af(b), 8);
      mbar_init(done(b), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf(a), 1);
      mbar_init(acce(a), 128);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tm0);
    prefetch_tmap(&tm1);
    prefetch_tmap(&tmx);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_slot)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  count_tiles<N>(tiles, p.cu, p.E, p.R, p.err);  // with barriers of the CTA
  tc_fence_after();
  // All of tensor memory, which begins at 0: known here, its addresses stay in uniform registers.
  constexpr uint32_t tmem = 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  ItemSearch search;
  auto item = [&](int i) { return search.at<N>(tiles, p.E, i, strips, WIDTH); };
  const int items = tiles.before[p.E] * strips;
  // waits for loads under way when a role stops: nothing lands after the CTA has gone
  auto drain_loads = [&](auto bar, int stages, int issued) {
    for (int k = max(0, issued - stages); k < issued; ++k) {
      const long long t0 = clock64();
      while (!mbar_try_wait(bar(k % stages), (k / stages) & 1)) {
        if ((unsigned long long)(clock64() - t0) > DRAIN_LIMIT) { set_error(p.err, DEV_TIMEOUT); break; }
      }
    }
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- codes
    int u = 0;  // pair of the whole sequence
    bool ok = true;
    for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
      const Item it = item(i);
      const int row = it.e * p.out + it.n0;
      for (int b = 0; b < blocks; b += 2, ++u) {
        const int s = u % C::CODES;
        ok = __all_sync(0xffffffffu, wait_lazily(codee(s), (u / C::CODES & 1) ^ 1, &abort_flag, p));
        if (!ok) break;
        const uint32_t dst = smem_u32(smem + 2 * s * CODE_BYTES);
        const bool two = b + 1 < blocks;
        if (elect_one()) {
          mbar_expect_tx(codef(s), two ? 2 * CODE_BYTES : CODE_BYTES);
          tma_load_2d(dst, &tm0, codef(s), b * WORDS, row);
          if (GATE_UP) tma_load_2d(dst + CODE_BYTES / 2, &tm1, codef(s), b * WORDS, row);
          if (two) {
            tma_load_2d(dst + CODE_BYTES, &tm0, codef(s), (b + 1) * WORDS, row);
            if (GATE_UP) tma_load_2d(dst + CODE_BYTES + CODE_BYTES / 2, &tm1, codef(s), (b + 1) * WORDS, row);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0) drain_loads(codef, C::CODES, u);
  } else if (warp == 6 + 8 * SETS) {
    // ---------------------------------------------------------------- rows x
    if (!GATE_UP) asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows that gate and up left
    int u = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
      const Item it = item(i);
      for (int b = 0; b < blocks; b += 2, ++u) {
        const int s = u % C::PAIRS;
        ok = __all_sync(0xffffffffu, wait_lazily(done(s), (u / C::PAIRS & 1) ^ 1, &abort_flag, p));
        if (!ok) break;
        const uint32_t dst = smem_u32(xs + 2 * s * C::X_BYTES);
        const int halves = b + 1 < blocks ? 4 : 2;
        if (elect_one()) {
          mbar_expect_tx(xf(s), halves * (N * 128));
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (h < halves) tma_load_2d(dst + h * (N * 128), &tmx, xf(s), b * BLOCK + 64 * h, it.r0);
        }
        __syncwarp();
      }
    }
    if (lane == 0) drain_loads(xf, C::PAIRS, u);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    constexpr uint32_t IDESC = instr_desc(TILE, N, false, false);
    int u = 0, n = 0;
    bool ok = true, ready = false;
    for (int i = blockIdx.x; ok && i < items; i += gridDim.x, ++n) {
      const int a = n & 1;
      ok = __all_sync(0xffffffffu, wait_bounded(acce(a), (n / 2 & 1) ^ 1, &abort_flag, p));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + a * C::ACC_COLS;
      for (int b = 0; b < blocks; b += 2, ++u) {
        const int buf = u % C::PAIRS, next = (u + 1) % C::PAIRS;
        if (!ready) {
          ok = wait_bounded(xf(buf), u / C::PAIRS & 1, &abort_flag, p) &&
               wait_bounded(af(buf), u / C::PAIRS & 1, &abort_flag, p);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        tc_fence_after();
        // asked here, the answers for the next pair are there once this one's MMAs have been issued
        const bool next_x = mbar_test_wait(xf(next), (u + 1) / C::PAIRS & 1);
        const bool next_a = mbar_test_wait(af(next), (u + 1) / C::PAIRS & 1);
        // a descriptor holds its address in units of 16 bytes, in its low bits
        const uint64_t x = smem_desc(smem_u32(xs + 2 * buf * C::X_BYTES), 16, 1024);
        const uint32_t w = tmem + C::A_BASE + 2 * buf * A_COLS;
        const bool two = b + 1 < blocks;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 2 * BLOCK / 16; ++k)
            if (k < BLOCK / 16 || two)
              mma_tmem_a(d, w + k * 8, x + (k / 4 * (N * 128) + k % 4 * 32) / 16, IDESC, b > 0 || k > 0);
          tc_commit(done(buf));
        }
        ready = __all_sync(0xffffffffu, next_x && next_a);
      }
      if (ok && elect_one()) tc_commit(accf(a));
      __syncwarp();
    }
    if (u > 0) {
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      const long long t0 = clock64();
      while (!mbar_try_wait(drain, 0)) {
        if ((unsigned long long)(clock64() - t0) > DRAIN_LIMIT) { set_error(p.err, DEV_TIMEOUT); break; }
      }
    }
  } else if (warp >= 6) {
    // ------------------------------------------------------------ conversion
    const int set = (warp - 6) >> 3, half = (warp - 6) >> 2 & 1, q = warp & 3;
    const int row = q * 32 + lane;  // of the tile, and lane of tensor memory
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    // The set's pairs of blocks are set, set + SETS, .. of the whole sequence: always in the same place of tensor
    // memory, and in one of two places of codes.  Four warps take a pair's first block, four its second one (if any).
    static_assert(SETS == C::PAIRS && C::CODES == 2 * SETS, "a set's places");
    const uint32_t at = tmem + lanes + C::A_BASE + (2 * set + half) * A_COLS;
    const uint8_t* from = smem + (2 * set + half) * CODE_BYTES + row * 64;
    // the scales of this thread's output in an item (outputs behind the last one: the last one's)
    auto scales_of = [&](const Item& it) {
      const int n = min(it.n0 + (GATE_UP ? row & 63 : row), p.out - 1);
      return (GATE_UP && row >= 64 ? p.s1 : p.s0) + ((long long)it.e * p.out + n) * blocks * SC;
    };
    const int mine = (items - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    auto scales_at = [&](int k) { return k < mine ? scales_of(item(blockIdx.x + k * gridDim.x)) : nullptr; };
    // the next pair of the set is number b of the CTA's item k
    int k = 0, b = set;
    while (b >= pairs) b -= pairs, ++k;
    const bf16* sp = scales_at(k);
    uint2 sc = make_uint2(0, 0);
    auto next_scales = [&]() {
      if (sp && 2 * b + half < blocks) sc = load_scales<G>(sp + (2 * b + half) * SC);
    };
    next_scales();
    for (int round = 0; k < mine; ++round) {
      const uint2 raw = sc;
      const bool real = 2 * b + half < blocks;
      b += SETS;
      if (b >= pairs) {
        do b -= pairs, ++k;
        while (b >= pairs);
        sp = scales_at(k);
      }
      next_scales();
      const int second = round & 1, s = set + SETS * second;
      if (!__all_sync(0xffffffffu, wait_bounded(codef(s), round >> 1 & 1, &abort_flag, p))) break;
      // 64 bytes of the row, in four pieces whose places are exchanged by the row's bits 1 and 2
      uint4 w[4];
      if (real)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          w[v] = *reinterpret_cast<const uint4*>(from + 2 * SETS * second * CODE_BYTES + ((v ^ (row >> 1 & 3)) << 4));
      // the codes have been read, not just asked for, before a TMA may write their place again
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(codee(s));
      if (!__all_sync(0xffffffffu, wait_bounded(done(set), (round & 1) ^ 1, &abort_flag, p))) break;
      tc_fence_after();
      if (real) {
        const uint2 now = spread_scales<G>(raw);
        const bool all_small = __all_sync(0xffffffffu, is_small(pair_from(now.x)) && is_small(pair_from(now.y)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          unsigned r[16];
          if (all_small) {
            convert_run<true>(w, j, j < 2 ? now.x : now.y, r);
            tmem_st16(at + j * 16, r);
          } else {
            convert_run<false>(w, j, j < 2 ? now.x : now.y, r);
            tmem_st16(at + j * 16, r);
          }
        }
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(af(set));
    }
  } else {
    // -------------------------------------------------------------- epilogue
    constexpr int R = N < 32 ? N : 32;  // rows of a round
    const int q = warp & 3;
    int n = 0;
    bool ok = true;  // after a wait that gave up the barriers between warps are still met
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++n) {
      const Item it = item(i);
      const int a = n & 1;
      // one warp looks, the others are woken by a barrier of the four
      if (ok && warp == 2) ok = __all_sync(0xffffffffu, wait_lazily(accf(a), n / 2 & 1, &abort_flag, p));
      ok = all_of_epilogue(ok);
      tc_fence_after();
      const uint32_t src = tmem + a * C::ACC_COLS + ((uint32_t)(q * 32) << 16);
      const int out = it.n0 + (GATE_UP ? q & 1 : q) * 32 + lane;
      bf16* dst = p.y + (long long)it.r0 * p.out + out;
      const bool store = ok && out < p.out;
#pragma unroll 1
      for (int r0 = 0; r0 < it.rows; r0 += R) {
        float v[R];
        sums_of(src + r0, v);
        if (GATE_UP) {
          // gate's warp and up's give each other half of the rows, and each finishes the other half; two
          // places in turn save a barrier
          constexpr int HALF = R / 2;
          float* ex_at = ex + ((r0 >> 5) & 1) * (4 * 512) + lane;
          float y[HALF];
#pragma unroll
          for (int r = 0; r < HALF; ++r) ex_at[q * 512 + r * 32] = q < 2 ? v[HALF + r] : v[r];
          asm volatile("bar.sync %0, 64;" ::"r"(1 + (q & 1)) : "memory");
#pragma unroll
          for (int r = 0; r < HALF; ++r) {
            const float other = ex_at[(q ^ 2) * 512 + r * 32];
            const float g = q < 2 ? v[r] : other, u = q < 2 ? other : v[HALF + r];
            y[r] = __fdividef(g, 1.f + __expf(-g)) * u;
          }
          const int at = r0 + (q < 2 ? 0 : HALF);
          store_rows<HALF>(y, dst + (long long)at * p.out, p.out, it.rows - at, store);
        } else {
          store_rows<R>(v, dst + (long long)r0 * p.out, p.out, it.rows - r0, store);
        }
      }
      // a tile of one round fills the first place again
      if (GATE_UP) asm volatile("bar.sync %0, 64;" ::"r"(1 + (q & 1)) : "memory");
      tc_fence_before();
      mbar_arrive(acce(a));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

bool map_rows(CUtensorMap* m, const void* x, long long rows, int in, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)in, (cuuint64_t)rows};
  cuuint64_t str[1] = {(cuuint64_t)in * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  return tc::make_map(m, x, 2, dims, str, box);
}

template <int N, int G, bool GATE_UP>
int launch_ffn(const void* x, const void* q0, const void* q1, const Args& p, cudaStream_t s) {
  using C = Cfg<N>;
  constexpr int WIDTH = GATE_UP ? TILE / 2 : TILE;
  static_assert(C::SMEM + sizeof(Tiles) + 512 <= 227 * 1024, "shared memory");
  CUtensorMap tm0, tm1, tmx;
  const long long rows = (long long)p.E * p.out;
  if (!map_codes(&tm0, q0, rows, p.in, WORDS, WIDTH) || !map_codes(&tm1, q1, rows, p.in, WORDS, WIDTH) ||
      !map_rows(&tmx, x, p.x_rows, p.in, N))
    return MOE_ERR_CUDA;
  const long long strips = (p.out + WIDTH - 1) / WIDTH;
  const long long items = most_tiles(p.R, p.E, N) * strips;
  const long long sms = sm_count();
  if (items > 0x3fffffffll) return MOE_ERR_UNSUPPORTED;
  auto k = w4_ffn_kernel<N, G, GATE_UP>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM) != cudaSuccess)
    return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < sms ? items : sms));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  // the second product's CTAs start, and convert their first weights, while the first one's finish
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = GATE_UP ? 0 : 1;
  if (cudaLaunchKernelEx(&cfg, k, tm0, tm1, tmx, p) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

// Rows of a tile, by the mean of an expert's: the conversion of a weight costs the same for any number of rows, so a
// tile should hold nearly all of an expert's, but its MMAs take the longer the wider it is.  Measured, in us, for
// routings at random to 8 experts of 2048 x 5632, by the rows of a tile:
//   mean   5   6   8  12  16  20  24  32  48  64  96
//   16    60  60  60  64  79  89  93
//   32    62  60  62  60  60  62  60  83  95
//   64    64  64  64  64  64  64  64  64  67  89 103
//   128   70  70  70  70  72  72  72  72  72  74  76
// Up to 4 rows the warp-level form (ROWS) finishes sooner what is small, as its items are finer and its start is
// shorter; the other one does more in the same time.  Measured (ROWS, the other one):
//   experts, T, K               items an SM  blocks an SM
//   8 of 2048 x 5632, 8, 2              4.7            96     41   46
//   12, 2                               5.2           106     57   52
//   8 of 4096 x 14336, 1, 2             3.0           125     58   73
//   2, 2                                5.3           223     87   87
//   8, 2                               11.6           488    126  138
//   16, 2                              13.2           556    195  173
//   64 of 2048 x 1408, 2, 6             2.7            38     30   34
//   4, 6                                5.0            69     46   44
//   16, 6                              12.4           173     83   74
//   384 of 7168 x 2048, 1, 8            4.6           140     56   63
//   2, 8                                9.0           277     99  104
//   4, 8                               17.9           552    170  168
//   48 of 1000 x 712, 64, 3             6.2            45     30   37
// (the rule costs up to 9% where it takes the slower one: 8 of 4096 x 14336 at 8 tokens).
// Routings are at random there; a crowded expert takes several tiles, each of which converts its weights again, but few
// experts do.  With one expert that has a third of all rows (rows of a tile 16, 32, 64, 128; the chosen one in brackets):
//   64 of 2048 x 1408, T 64, K 6    [93]   92  102  117   (at random [88]  90  101  118)
//   256, 6                          132   104 [110] 127   (149  94 [104] 125)
//   512, 6                          236   151 [116] 138   (233 151 [105] 129)
//   8 of 2048 x 5632, 64, 2          69  [60]  61   71   (70 [56]  60  70)
inline int tile_rows(int R, int E, int H, int Hp) {
  const int mean = R / E;
  if (mean > 4) return mean <= 8 ? 16 : mean <= 20 ? 32 : mean <= 48 ? 64 : 128;
  const double active = E * (1 - exp(-(double)R / E));  // experts with rows, for a routing at random
  const double gate_up = (Hp + TILE / 2 - 1) / (TILE / 2), down = (H + TILE - 1) / TILE;  // strips
  const double items = active * (gate_up + down), blocks = active * (gate_up * blocks_of(H) + down * blocks_of(Hp));
  return items < 4.8 * sm_count() || blocks < 64. * sm_count() ? ROWS : 16;
}
template <int G, bool GATE_UP>
int launch_ffn_n(const void* x, const void* q0, const void* q1, const Args& p, cudaStream_t s) {
  switch (p.tile) {
    case ROWS: return launch_rows<G, GATE_UP>(x, q0, q1, p, s);
    case 16: return launch_ffn<16, G, GATE_UP>(x, q0, q1, p, s);
    case 32: return launch_ffn<32, G, GATE_UP>(x, q0, q1, p, s);
    case 64: return launch_ffn<64, G, GATE_UP>(x, q0, q1, p, s);
    default: return launch_ffn<128, G, GATE_UP>(x, q0, q1, p, s);
  }
}
template <bool GATE_UP>
int launch_ffn_g(const void* x, const void* q0, const void* q1, const Args& p, cudaStream_t s) {
  return p.group == 32 ? launch_ffn_n<32, GATE_UP>(x, q0, q1, p, s)
                       : p.group == 64 ? launch_ffn_n<64, GATE_UP>(x, q0, q1, p, s)
                                       : launch_ffn_n<128, GATE_UP>(x, q0, q1, p, s);
}

// the routed rows side by side, for tiles of rows that are loaded as a whole; a row that does not exist is zeros
__global__ void __launch_bounds__(256) w4_gather_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ src_tok,
                                                        int T, int vecs, uint4* __restrict__ xs, unsigned* err) {
  const long long r = blockIdx.x;
  const int from = __ldg(src_tok + r);
  const bool ok = from >= 0 && from < T;
  if (!ok && threadIdx.x == 0) set_error(err, DEV_BOUNDS);
  for (int i = threadIdx.x; i < vecs; i += 256)
    xs[r * vecs + i] = ok ? __ldg(x + (long long)from * vecs + i) : make_uint4(0, 0, 0, 0);
}

unsigned col_grid(long long rows, int blocks) {
  return (unsigned)((rows * blocks * WORDS + COL_WORDS - 1) / COL_WORDS);
}

template <typename T, int G>
int pack(const void* w, int E, int rows, int cols, int axis, void* q, void* scale, cudaStream_t s) {
  if (axis == 1) {
    const int blocks = blocks_of(cols);
    const long long n = (long long)E * rows;
    if (n * blocks * WORDS / COL_WORDS >= 0x7fffffffll) return MOE_ERR_UNSUPPORTED;
    w4_pack_cols_kernel<T, G><<<col_grid(n, blocks), COL_NT, 0, s>>>(
        static_cast<const T*>(w), n, cols, blocks, static_cast<unsigned*>(q), static_cast<bf16*>(scale));
  } else {
    const int blocks = blocks_of(rows);
    constexpr int COLS = 64 * PER4<T>;
    w4_pack_rows_kernel<T, G>
        <<<dim3((cols + COLS - 1) / COLS, (blocks + ROW_BLOCKS - 1) / ROW_BLOCKS, E), ROW_NT, 0, s>>>(
            static_cast<const T*>(w), rows, cols, blocks, static_cast<unsigned*>(q), static_cast<bf16*>(scale));
  }
  return launch_status();
}

template <typename T>
int unpack(const void* q, const void* scale, int E, int rows, int cols, int axis, int G, void* w, cudaStream_t s) {
  if (axis == 1) {
    const int blocks = blocks_of(cols);
    const long long n = (long long)E * rows;
    if (n * blocks * WORDS / COL_WORDS >= 0x7fffffffll) return MOE_ERR_UNSUPPORTED;
    w4_unpack_cols_kernel<T><<<col_grid(n, blocks), COL_NT, 0, s>>>(
        static_cast<const unsigned*>(q), static_cast<const bf16*>(scale), n, cols, blocks, G, static_cast<T*>(w));
  } else {
    const int blocks = blocks_of(rows);
    constexpr int COLS = 64 * PER4<T>;
    w4_unpack_rows_kernel<T><<<dim3((cols + COLS - 1) / COLS, (blocks + ROW_BLOCKS - 1) / ROW_BLOCKS, E), ROW_NT, 0, s>>>(
        static_cast<const unsigned*>(q), static_cast<const bf16*>(scale), rows, cols, blocks, G, static_cast<T*>(w));
  }
  return launch_status();
}

}  // namespace w4

int launch_w4_pack(const void* w, int E, int rows, int cols, int axis, int group, int dtype, void* q, void* scale,
                   cudaStream_t s) {
  if (dtype == MOE_BF16)
    return group == 32 ? w4::pack<bf16, 32>(w, E, rows, cols, axis, q, scale, s)
                       : group == 64 ? w4::pack<bf16, 64>(w, E, rows, cols, axis, q, scale, s)
                                     : w4::pack<bf16, 128>(w, E, rows, cols, axis, q, scale, s);
  return group == 32 ? w4::pack<float, 32>(w, E, rows, cols, axis, q, scale, s)
                     : group == 64 ? w4::pack<float, 64>(w, E, rows, cols, axis, q, scale, s)
                                   : w4::pack<float, 128>(w, E, rows, cols, axis, q, scale, s);
}

int launch_w4_unpack(const void* q, const void* scale, int E, int rows, int cols, int axis, int group, int dtype,
                     void* w, cudaStream_t s) {
  return dtype == MOE_BF16 ? w4::unpack<bf16>(q, scale, E, rows, cols, axis, group, w, s)
                           : w4::unpack<float>(q, scale, E, rows, cols, axis, group, w, s);
}

size_t expert_ffn_w4_ws_bytes(int rows, int H, int E, int Hp) {
  return w4::tile_rows(rows, E, H, Hp) >= 16 ? (size_t)rows * H * sizeof(bf16) : 0;
}

int launch_expert_ffn_w4(const void* x, const int32_t* src_tok, int T, const int32_t* cu, int rows, const void* q_gate,
                         const void* s_gate, const void* q_up, const void* s_up, const void* q_down, const void* s_down,
                         int E, int H, int Hp, int group, void* act, void* h, void* ws, cudaStream_t s) {
  if (rows == 0) return MOE_OK;
  w4::Args a;
  a.tile = w4::tile_rows(rows, E, H, Hp);
  if (src_tok && a.tile >= 16) {
    w4::w4_gather_kernel<<<rows, 256, 0, s>>>(static_cast<const uint4*>(x), src_tok, T, H / 8, static_cast<uint4*>(ws),
                                              device_error_word());
    const int st = launch_status();
    if (st != MOE_OK) return st;
    x = ws;
    src_tok = nullptr;
  }
  a.src_tok = src_tok, a.x_rows = src_tok ? T : rows;
  a.cu = cu, a.E = E, a.R = rows, a.in = H, a.out = Hp, a.group = group;
  a.err = device_error_word(), a.wait_limit = tc::g_wait_limit;
  a.s0 = static_cast<const bf16*>(s_gate), a.s1 = static_cast<const bf16*>(s_up);
  a.y = static_cast<bf16*>(act);
  const int st = w4::launch_ffn_g<true>(x, q_gate, q_up, a, s);
  if (st != MOE_OK) return st;
  a.src_tok = nullptr, a.x_rows = rows;
  a.in = Hp, a.out = H;
  a.s0 = a.s1 = static_cast<const bf16*>(s_down);
  a.y = static_cast<bf16*>(h);
  return w4::launch_ffn_g<false>(act, q_down, q_down, a, s);
}

}  // namespace moe
