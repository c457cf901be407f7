// Expert weights in 4 bits with group scales, and the expert FFN that reads them.
//
// Packed form of a weight tensor w [E, rows, cols]: `in` is the axis that the product sums
// over (rows of gate and up, cols of down), `out` the other one.  Of each output, groups
// of G (32, 64 or 128) neighbours along `in` share a scale of 5 significant bits; a code q in
// -8..7 (pack makes -7..7) is held as q + 8, so q s has at most 8 significant bits: exact in
// bf16.  Codes lie in blocks of 128 inputs, 16 words of 8 codes (the last block is padded with
// zeros).  Word 4 j + w of a block (inputs 32 j + 8 w ..) is stored at w * 4 + j, and code i of a word in bits
// 4 (i / 2) + 16 (i % 2): a lane of a warp-level MMA then reads 16 neighbouring bytes that hold its
// inputs of four steps of 32, and every pair of neighbours comes out of a word by a shift and
// a mask as two bf16 numbers 128 + (q + 8).
#include <math.h>

#include "moe_internal.cuh"

namespace moe {
namespace w4 {

constexpr int BLOCK = 128;         // inputs of a block
constexpr int WORDS = BLOCK / 8;   // its words

__host__ __device__ inline int blocks_of(int in) { return (int)(((long long)in + BLOCK - 1) / BLOCK); }

// ------------------------------------------------------------ the 4-bit form ---
// the least number of 5 significant bits >= amax / 7, at least 2^-126; NaN for a group that holds
// a NaN, an infinity or a magnitude of 2^127 and more (its largest code might stand for an infinity)
__device__ __forceinline__ float scale_of(float amax) {
  if (!(amax < 1.7014118346046923e38f)) return __uint_as_float(0x7fc00000u);
  const float s = __uint_as_float((__float_as_uint(amax / 7.f) + 0x7ffffu) & ~0x7ffffu);
  return fmaxf(s, 1.1754943508222875e-38f);
}
__device__ __forceinline__ unsigned code_of(float w, float s) {
  const float q = rintf(w / s);
  return isnan(q) ? 8u : (unsigned)((int)q + 8);
}
__device__ __forceinline__ int shift_of(int i) { return 4 * (i >> 1) + 16 * (i & 1); }
__device__ __forceinline__ float max_abs(float a, float v) {  // keeps a NaN
  v = fabsf(v);
  return v > a || v != v ? v : a;
}

// w [E, out, in]: a thread takes the 8 inputs of a word, the G / 8 lanes of a group share its largest
template <typename T, int G>
__global__ void __launch_bounds__(256) w4_pack_cols_kernel(const T* __restrict__ w, long long rows, int in, int blocks,
                                                           unsigned* __restrict__ q, bf16* __restrict__ scale) {
  const long long words = rows * blocks * WORDS, last = (words + 31) / 32 * 32;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < last; i += (long long)gridDim.x * 256) {
    const long long row = i / (blocks * WORDS);
    const int word = (int)(i - row * (blocks * WORDS)), c = word * 8;
    float v[8], amax = 0.f;
#pragma unroll
    for (int k = 0; k < 8; k += Vec16<T>::N) {
      if (i < words && c + k < in) {
        Vec16<T>::load(w + row * in + c + k, v + k);
      } else {
#pragma unroll
        for (int u = 0; u < Vec16<T>::N; ++u) v[k + u] = 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = max_abs(amax, v[k]);
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1) amax = max_abs(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (i >= words) continue;
    const float s = scale_of(amax);
    unsigned x = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) x |= code_of(v[k], s) << shift_of(k);
    const int at = word % WORDS;
    q[(row * blocks + word / WORDS) * WORDS + at % 4 * 4 + at / 4] = x;
    if (c % G == 0) scale[row * (blocks * BLOCK / G) + c / G] = __float2bfloat16_rn(s);
  }
}

// w [E, in, out]: a thread takes the block of 128 inputs of one output
template <typename T, int G>
__global__ void __launch_bounds__(128) w4_pack_rows_kernel(const T* __restrict__ w, int in, int out, int blocks,
                                                           unsigned* __restrict__ q, bf16* __restrict__ scale) {
  const int o = blockIdx.x * 128 + threadIdx.x, b = blockIdx.y, e = blockIdx.z;
  if (o >= out) return;
  const T* src = w + ((long long)e * in + b * BLOCK) * out + o;
  const long long row = (long long)e * out + o;
  unsigned x[WORDS];
#pragma unroll
  for (int g = 0; g < BLOCK / G; ++g) {
    float v[G], amax = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) v[k] = b * BLOCK + g * G + k < in ? to_f32(src[(long long)(g * G + k) * out]) : 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) amax = max_abs(amax, v[k]);
    const float s = scale_of(amax);
#pragma unroll
    for (int n = 0; n < G / 8; ++n) {
      unsigned y = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) y |= code_of(v[8 * n + k], s) << shift_of(k);
      const int at = g * (G / 8) + n;
      x[at % 4 * 4 + at / 4] = y;
    }
    scale[row * (blocks * BLOCK / G) + b * (BLOCK / G) + g] = __float2bfloat16_rn(s);
  }
  uint4* dst = reinterpret_cast<uint4*>(q + (row * blocks + b) * WORDS);
#pragma unroll
  for (int k = 0; k < 4; ++k) dst[k] = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
}

__device__ __forceinline__ float value_of(unsigned word, int i, float s) {
  return (float)((int)((word >> shift_of(i)) & 15u) - 8) * s;
}

template <typename T>
__global__ void __launch_bounds__(256) w4_unpack_cols_kernel(const unsigned* __restrict__ q, const bf16* __restrict__ scale,
                                                             long long rows, int in, int blocks, int G,
                                                             T* __restrict__ w) {
  const long long words = rows * blocks * WORDS;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < words; i += (long long)gridDim.x * 256) {
    const long long row = i / (blocks * WORDS);
    const int word = (int)(i - row * (blocks * WORDS)), c = word * 8, at = word % WORDS;
    if (c >= in) continue;
    const unsigned x = q[(row * blocks + word / WORDS) * WORDS + at % 4 * 4 + at / 4];
    const float s = to_f32(scale[row * (blocks * BLOCK / G) + c / G]);
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = value_of(x, k, s);
#pragma unroll
    for (int k = 0; k < 8; k += Vec16<T>::N)
      if (c + k < in) Vec16<T>::store(w + row * in + c + k, v + k);
  }
}

template <typename T>
__global__ void __launch_bounds__(128) w4_unpack_rows_kernel(const unsigned* __restrict__ q, const bf16* __restrict__ scale,
                                                             int in, int out, int blocks, int G, T* __restrict__ w) {
  const int o = blockIdx.x * 128 + threadIdx.x, b = blockIdx.y, e = blockIdx.z;
  if (o >= out) return;
  T* dst = w + ((long long)e * in + b * BLOCK) * out + o;
  const long long row = (long long)e * out + o;
  const uint4* src = reinterpret_cast<const uint4*>(q + (row * blocks + b) * WORDS);
  unsigned x[WORDS];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint4 v = __ldg(src + k);
    x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
  }
  const bf16* sc = scale + row * (blocks * BLOCK / G) + b * (BLOCK / G);
#pragma unroll
  for (int at = 0; at < WORDS; ++at) {
    const float s = to_f32(sc[at * 8 / G]);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (b * BLOCK + at * 8 + k < in)
        dst[(long long)(at * 8 + k) * out] = from_f32<T>(value_of(x[at % 4 * 4 + at / 4], k, s));
  }
}

// ------------------------------------------------------ products of few rows ---
// Weights are the MMA's A operand (16 outputs x 16 inputs), up to 8 NT routed rows its B operand, so a
// weight is read and turned into bf16 once for all of an expert's rows in the tile.  With w' = 128 + (q + 8)
// straight out of the word,  sum q x = sum w' x - 136 sum x;  the sum of x is one more MMA with ones
// for A, and the group's scale is applied to its fp32 sums.
//
// A warp takes two tiles of 16 outputs (the same outputs of gate and up, or 32 outputs of down) over
// every WK-th block of inputs; the WK warps' sums meet in shared memory in a fixed order.
constexpr int NT_WARPS = 8;

struct Args {
  const bf16* x;
  const int32_t* src_tok;  // row r of x, or nullptr: row r itself
  int x_rows;
  const int32_t* cu;
  int E, R, in, out;       // out: rows of q0
  const unsigned *q0, *q1;
  const bf16 *s0, *s1;
  bf16* y;                 // [R, out]
  int wk;                  // warps that share a strip of outputs: 1, 2, 4 or 8
  unsigned* err;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// codes of a word's pair t as bf16 numbers 128 + (q + 8)
__device__ __forceinline__ unsigned pair_of(unsigned word, int t) {
  return ((word >> (4 * t)) & 0x000f000fu) | 0x43004300u;
}

// slot `slot` of the tiles of TT rows over all experts: expert, first row, rows (0: no such tile)
template <int TT>
__device__ __forceinline__ int3 find_tile(const int32_t* cu, int E, int R, int slot, unsigned* err) {
  __shared__ int warp_sum[NT_WARPS];
  __shared__ int3 found;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (E + 32 * NT_WARPS - 1) / (32 * NT_WARPS);
  const int e0 = min(E, (int)threadIdx.x * per), e1 = min(E, e0 + per);
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    const int a = min(max(cu[e], 0), R), b = min(max(cu[e + 1], a), R);
    sum += (b - a + TT - 1) / TT;
  }
  if (threadIdx.x == 0) {
    found = make_int3(0, 0, 0);
    if (slot == 0 && (cu[0] != 0 || cu[E] != R)) set_error(err, DEV_BOUNDS);
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int before = incl - sum;
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  if (slot >= before && slot < before + sum) {
    for (int e = e0; e < e1; ++e) {
      const int a = min(max(cu[e], 0), R), b = min(max(cu[e + 1], a), R), tiles = (b - a + TT - 1) / TT;
      if (slot < before + tiles) {
        const int r0 = a + (slot - before) * TT;
        found = make_int3(e, r0, min(TT, b - r0));
        break;
      }
      before += tiles;
    }
  }
  __syncthreads();
  return found;
}

template <int NT, int G, bool GATE_UP>
__global__ void __launch_bounds__(32 * NT_WARPS) w4_rows_kernel(const Args p) {
  extern __shared__ float red[];  // [warp][2 NT 4][32]
  const int3 tile = find_tile<8 * NT>(p.cu, p.E, p.R, blockIdx.y, p.err);
  const int e = tile.x, r0 = tile.y, rows = tile.z;
  if (rows <= 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tg = lane & 3;
  const int wk = p.wk, kw = warp % wk;
  constexpr int STRIP = GATE_UP ? 16 : 32;
  const int n0 = (blockIdx.x * (NT_WARPS / wk) + warp / wk) * STRIP;
  const int blocks = blocks_of(p.in), live = (rows + 7) / 8;
  constexpr int SC = BLOCK / G;  // scales of a block

  const uint4* q[2][2];
  const bf16* sc[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = min(n0 + (GATE_UP ? 0 : 16 * t) + 8 * h + g, p.out - 1);
      const long long row = (long long)e * p.out + n;
      q[t][h] = reinterpret_cast<const uint4*>((GATE_UP && t ? p.q1 : p.q0) + row * blocks * WORDS) + tg;
      sc[t][h] = (GATE_UP && t ? p.s1 : p.s0) + row * blocks * SC;
    }
  const bf16* xr[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    xr[i] = nullptr;
    if (i * 8 + g < rows) {
      long long r = r0 + i * 8 + g;
      if (p.src_tok) r = p.src_tok[r];
      if (r < 0 || r >= p.x_rows) set_error(p.err, DEV_BOUNDS);
      else xr[i] = p.x + r * p.in + tg * 8;
    }
  }

  float acc[2][NT][4];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[t][i][k] = 0.f;

  if (n0 < p.out) {
    for (int b = kw; b < blocks; b += wk) {
      uint4 w[2][2];
      float s[2][2][SC];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w[t][h] = __ldg(q[t][h] + b * 4);
#pragma unroll
          for (int k = 0; k < SC; ++k) s[t][h][k] = to_f32(sc[t][h][b * SC + k]);
        }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (i >= live) break;
        uint4 xv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xv[j] = make_uint4(0, 0, 0, 0);
          if (xr[i] && b * BLOCK + 32 * j + 8 * tg < p.in)
            xv[j] = __ldg(reinterpret_cast<const uint4*>(xr[i] + b * BLOCK + 32 * j));
        }
#pragma unroll
        for (int k = 0; k < SC; ++k) {
          float c[2][4] = {}, one[4] = {};
#pragma unroll
          for (int j = k * 4 / SC; j < (k + 1) * 4 / SC; ++j) {
            const unsigned ones[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
            mma_bf16(one, ones, xv[j].x, xv[j].y);
            mma_bf16(one, ones, xv[j].z, xv[j].w);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const unsigned u = j == 0 ? w[t][0].x : j == 1 ? w[t][0].y : j == 2 ? w[t][0].z : w[t][0].w;
              const unsigned v = j == 0 ? w[t][1].x : j == 1 ? w[t][1].y : j == 2 ? w[t][1].z : w[t][1].w;
              const unsigned a0[4] = {pair_of(u, 0), pair_of(v, 0), pair_of(u, 1), pair_of(v, 1)};
              const unsigned a1[4] = {pair_of(u, 2), pair_of(v, 2), pair_of(u, 3), pair_of(v, 3)};
              mma_bf16(c[t], a0, xv[j].x, xv[j].y);
              mma_bf16(c[t], a1, xv[j].z, xv[j].w);
            }
          }
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int m = 0; m < 4; ++m) acc[t][i][m] = fmaf(s[t][m / 2][k], fmaf(-136.f, one[m], c[t][m]), acc[t][i][m]);
        }
      }
    }
  }

  // the strip's warps add up, and each finishes some of the rows
  float* mine = red + warp * (8 * NT * 32) + lane;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m) mine[((t * NT + i) * 4 + m) * 32] = acc[t][i][m];
  __syncthreads();
  if (n0 >= p.out) return;
  const float* strip = red + (warp - kw) * (8 * NT * 32) + lane;
  for (int i = kw; i < live; i += wk) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      float v[2] = {0.f, 0.f};
      for (int k = 0; k < wk; ++k)
#pragma unroll
        for (int t = 0; t < 2; ++t) v[t] += strip[k * (8 * NT * 32) + ((t * NT + i) * 4 + m) * 32];
      const int r = i * 8 + 2 * tg + (m & 1), n = n0 + g + 8 * (m >> 1);
      if (r >= rows) continue;
      bf16* dst = p.y + (long long)(r0 + r) * p.out;
      if (GATE_UP) {
        if (n < p.out) dst[n] = __float2bfloat16_rn(v[0] / (1.f + expf(-v[0])) * v[1]);
      } else {
        if (n < p.out) dst[n] = __float2bfloat16_rn(v[0]);
        if (n + 16 < p.out) dst[n + 16] = __float2bfloat16_rn(v[1]);
      }
    }
  }
}

template <int NT, int G, bool GATE_UP>
int launch_rows(Args p, cudaStream_t s) {
  constexpr int STRIP = GATE_UP ? 16 : 32, TT = 8 * NT;
  constexpr size_t smem = (size_t)NT_WARPS * 8 * NT * 32 * 4;
  const int blocks = blocks_of(p.in);
  p.wk = blocks >= 8 ? 8 : blocks >= 4 ? 4 : blocks >= 2 ? 2 : 1;
  const int strips = (p.out + STRIP - 1) / STRIP, per = NT_WARPS / p.wk;
  const long long slots = (long long)(p.E < p.R ? p.E : p.R) + p.R / TT;
  if (slots > 65535) return MOE_ERR_UNSUPPORTED;
  auto k = w4_rows_kernel<NT, G, GATE_UP>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return MOE_ERR_CUDA;
  k<<<dim3((strips + per - 1) / per, (unsigned)slots), 32 * NT_WARPS, smem, s>>>(p);
  return launch_status();
}

template <int G, bool GATE_UP>
int launch_rows_nt(const Args& p, cudaStream_t s) {
  const int mean = p.R / p.E;  // rows of an expert
  if (mean <= 4) return launch_rows<1, G, GATE_UP>(p, s);
  if (mean <= 12) return launch_rows<2, G, GATE_UP>(p, s);
  if (mean <= 24) return launch_rows<4, G, GATE_UP>(p, s);
  return launch_rows<8, G, GATE_UP>(p, s);
}
template <bool GATE_UP>
int launch_rows_g(const Args& p, int G, cudaStream_t s) {
  return G == 32 ? launch_rows_nt<32, GATE_UP>(p, s)
                 : G == 64 ? launch_rows_nt<64, GATE_UP>(p, s) : launch_rows_nt<128, GATE_UP>(p, s);
}

unsigned grid_of(long long threads, int nt) {
  const long long want = (threads + nt - 1) / nt, most = 8LL * sm_count();
  return (unsigned)(want < most ? want : most);
}

template <typename T, int G>
int pack(const void* w, int E, int rows, int cols, int axis, void* q, void* scale, cudaStream_t s) {
  if (axis == 1) {
    const int blocks = blocks_of(cols);
    const long long n = (long long)E * rows;
    w4_pack_cols_kernel<T, G><<<grid_of(n * blocks * WORDS, 256), 256, 0, s>>>(
        static_cast<const T*>(w), n, cols, blocks, static_cast<unsigned*>(q), static_cast<bf16*>(scale));
  } else {
    const int blocks = blocks_of(rows);
    w4_pack_rows_kernel<T, G><<<dim3((cols + 127) / 128, blocks, E), 128, 0, s>>>(
        static_cast<const T*>(w), rows, cols, blocks, static_cast<unsigned*>(q), static_cast<bf16*>(scale));
  }
  return launch_status();
}

template <typename T>
int unpack(const void* q, const void* scale, int E, int rows, int cols, int axis, int G, void* w, cudaStream_t s) {
  if (axis == 1) {
    const int blocks = blocks_of(cols);
    const long long n = (long long)E * rows;
    w4_unpack_cols_kernel<T><<<grid_of(n * blocks * WORDS, 256), 256, 0, s>>>(
        static_cast<const unsigned*>(q), static_cast<const bf16*>(scale), n, cols, blocks, G, static_cast<T*>(w));
  } else {
    const int blocks = blocks_of(rows);
    w4_unpack_rows_kernel<T><<<dim3((cols + 127) / 128, blocks, E), 128, 0, s>>>(
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

size_t expert_ffn_w4_ws_bytes(int R, int H, int E, int Hp) { return 0; }

int launch_expert_ffn_w4(const void* x, const int32_t* src_tok, int T, const int32_t* cu, int rows, const void* q_gate,
                         const void* s_gate, const void* q_up, const void* s_up, const void* q_down, const void* s_down,
                         int E, int H, int Hp, int group, void* act, void* h, void* ws, cudaStream_t s) {
  if (rows == 0) return MOE_OK;
  w4::Args a;
  a.x = static_cast<const bf16*>(x), a.src_tok = src_tok, a.x_rows = src_tok ? T : rows;
  a.cu = cu, a.E = E, a.R = rows, a.in = H, a.out = Hp, a.wk = 0, a.err = device_error_word();
  a.q0 = static_cast<const unsigned*>(q_gate), a.q1 = static_cast<const unsigned*>(q_up);
  a.s0 = static_cast<const bf16*>(s_gate), a.s1 = static_cast<const bf16*>(s_up);
  a.y = static_cast<bf16*>(act);
  const int st = w4::launch_rows_g<true>(a, group, s);
  if (st != MOE_OK) return st;
  a.x = static_cast<const bf16*>(act), a.src_tok = nullptr, a.x_rows = rows;
  a.in = Hp, a.out = H;
  a.q0 = a.q1 = static_cast<const unsigned*>(q_down);
  a.s0 = a.s1 = static_cast<const bf16*>(s_down);
  a.y = static_cast<bf16*>(h);
  return w4::launch_rows_g<false>(a, group, s);
}

}  // namespace moe
