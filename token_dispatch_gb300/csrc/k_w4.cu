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
// weight is read and turned into bf16 once for all of an expert's rows in the tile.  A pair of codes
// comes out of its word as w' = 128 + (q + 8) by a shift, a mask and an or (bf16 holds whole numbers up to 256).
// For one tile of 8 rows  sum q x = sum w' x - 136 sum x,  the last term by an MMA whose A is -136 throughout and
// that the others add to, saves the subtraction of each weight; for more rows that MMA would cost more
// than subtracting once.  The group's scale is applied to its fp32 sums.
//
// An item is a strip of outputs (16 of gate and the same of up, or 32 of down) for one tile of rows.  WK
// warps share its inputs, each every WK-th pair of blocks; their sums meet in shared memory in a
// fixed order.  What bounds the kernel is the weights' way from memory, so each warp keeps a ring of
// STAGES pairs of blocks in flight by TMA, across items.  (Loads into registers met two limits
// before that one: the 64-byte pieces of 8 rows took the L1's tag stage, and too few of them were under way.)
// The rows x are read through L1, where the strips of an expert find them again.
//
// A stage holds 32 rows of 128 bytes, swizzled: 16-byte piece c of row r lies at c ^ (r & 7).  Lane
// group g reads row 4 (g & 1) + g / 2 of each eight, so that the two rows which a quarter
// of a warp reads together lie in different halves of the banks.
constexpr int NT_WARPS = 8;
constexpr int MAX_E = 1024;
constexpr int STAGES = 2;
constexpr int STAGE_BYTES = 32 * 128;
constexpr int AHEAD = 8;  // items that a warp's loads may be ahead, a power of two above STAGES + 1

struct Args {
  const bf16* x;
  const int32_t* src_tok;  // row r of x, or nullptr: row r itself
  int x_rows;
  const int32_t* cu;
  int E, R, in, out;       // out: rows of q0
  const bf16 *s0, *s1;
  bf16* y;                 // [R, out]
  int wk;                  // warps that share a strip of outputs: 1, 2, 4 or 8
  unsigned* err;
  unsigned long long wait_limit;
};

// d = a b + c
__device__ __forceinline__ void mma_bf16(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1,
                                         const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, "
      "%12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// codes of a word's pair t as bf16 numbers 128 + (q + 8), or with SUB as q
template <bool SUB>
__device__ __forceinline__ unsigned pair_of(unsigned word, int t) {
  unsigned v;  // (word >> 4 t) & 0x000f000f | 0x43004300
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(v) : "r"(word >> (4 * t)), "r"(0x43004300u));
  if (SUB) {
    const __nv_bfloat162 q = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __float2bfloat162_rn(136.f));
    v = *reinterpret_cast<const unsigned*>(&q);
  }
  return v;
}
__device__ __forceinline__ unsigned word_of(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// The tiles of TT rows of all experts: before[e] = tiles of the experts before e.  Offsets that
// do not run upwards from 0 to R are cut off there and reported.
struct Tiles {
  int before[MAX_E + 1], row0[MAX_E + 1];
  int warp_sum[NT_WARPS];
};
template <int TT>
__device__ __forceinline__ void count_tiles(Tiles& t, const int32_t* cu, int E, int R, unsigned* err) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int PER = MAX_E / (32 * NT_WARPS);  // experts of a thread
  const int e0 = threadIdx.x * PER;
  int at[PER + 1], sum = 0;
#pragma unroll
  for (int k = 0; k <= PER; ++k) at[k] = e0 + k <= E ? __ldg(cu + e0 + k) : R;
  if (threadIdx.x == 0 && blockIdx.x == 0 && (at[0] != 0 || __ldg(cu + E) != R)) set_error(err, DEV_BOUNDS);
  int n[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int a = min(max(at[k], 0), R), b = min(max(at[k + 1], a), R);
    n[k] = e0 + k < E ? (b - a + TT - 1) / TT : 0;
    sum += n[k];
    if (e0 + k < E) t.row0[e0 + k] = a;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) t.warp_sum[warp] = incl;
  __syncthreads();
  int run = incl - sum;
  for (int w = 0; w < warp; ++w) run += t.warp_sum[w];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    if (e0 + k <= E) t.before[e0 + k] = run;
    run += n[k];
  }
  if (threadIdx.x == 32 * NT_WARPS - 1) t.before[E] = run;
  __syncthreads();
}

struct Item {
  int e, r0, rows, n0;  // n0: first output; rows 0: no more items
};
// item i: experts in order, in each its strips in order, in each strip its tiles
template <int TT>
__device__ __forceinline__ Item item_of(const Tiles& t, const int32_t* cu, int E, int R, long long i, int strips,
                                        int width) {
  Item w = {0, 0, 0, 0};
  if (i >= (long long)t.before[E] * strips) return w;
  int lo = 0, hi = E - 1;
  while (lo < hi) {  // the last expert whose items begin at or before i
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)t.before[mid] * strips <= i) lo = mid;
    else hi = mid - 1;
  }
  const int tiles = t.before[lo + 1] - t.before[lo], local = (int)(i - (long long)t.before[lo] * strips);
  const int strip = local / tiles, tile = local - strip * tiles;
  w.e = lo;
  w.r0 = t.row0[lo] + tile * TT;
  w.rows = min(TT, min(max(__ldg(cu + lo + 1), t.row0[lo]), R) - w.r0);
  w.n0 = strip * width;
  return w;
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
// buffers where the warps' sums meet: two in turn save a barrier an item
template <int NT>
constexpr int sum_bufs() { return NT <= 2 ? 2 : 1; }
template <int NT>
constexpr size_t rows_smem() {  // stages, sums, and room to align the stages
  return (size_t)NT_WARPS * STAGES * STAGE_BYTES + (size_t)sum_bufs<NT>() * NT_WARPS * 8 * NT * 32 * 4 + 1024;
}

template <int NT, int G, bool GATE_UP>
__global__ void __launch_bounds__(32 * NT_WARPS, RESIDENT)
w4_rows_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1, const Args p) {
  constexpr int STRIP = GATE_UP ? 16 : 32, TT = 8 * NT, SC = BLOCK / G;
  constexpr int SUMS = 8 * NT * 32;  // floats of a warp: [2 NT 4][32 lanes]
  constexpr bool ONES = NT == 1;
  constexpr int XH = NT == 1 ? 2 : 1;
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

  if (threadIdx.x == 0) abort_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) tc::mbar_init(tc::smem_u32(&bars[warp][s]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  count_tiles<TT>(tiles, p.cu, p.E, p.R, p.err);  // ends with a barrier of the CTA
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the warp's loads: stage `issued` of its sequence of (item, pair of blocks)
  const long long stride = (long long)gridDim.x * (NT_WARPS / wk);
  long long load_i = (long long)blockIdx.x * (NT_WARPS / wk) + sub;
  int load_items = 0, load_pair = kw, issued = 0, load_row = 0;
  bool loading;
  const bf16* load_s = nullptr;  // scales of this lane's row of the stage
  auto next_item = [&]() {
    const Item w = item_of<TT>(tiles, p.cu, p.E, p.R, load_i, strips, STRIP);
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
      if (lane == 0) {
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
    const int rows = it.rows, live = (rows + 7) / 8;
    const uint4* xr[NT];  // of the next pair of blocks
    int step[NT];
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      xr[r] = zero_row;
      step[r] = 0;
      if (r * 8 + g < rows) {
        long long from = it.r0 + r * 8 + g;
        if (p.src_tok) from = __ldg(p.src_tok + from);
        if (from < 0 || from >= p.x_rows) {
          set_error(p.err, DEV_BOUNDS);
        } else {
          xr[r] = reinterpret_cast<const uint4*>(p.x + from * p.in) + tg;
          step[r] = BLOCK / 8;
        }
      }
    }
    float acc[2][NT][4] = {};
#pragma unroll 1
    for (int pair = kw; pair < pairs; pair += wk) {
      const int slot = done % STAGES;
      // a row's values of run j of block b for tile r; lanes past the last input get zeros
      auto load_x = [&](int r, int b, int j) {
        const uint4* xp = xr[r] + b * step[r] + 4 * j;
        return b * BLOCK + 32 * j + 8 * tg < p.in ? *xp : make_uint4(0, 0, 0, 0);
      };
      uint4 xv[XH][4];
      if (NT == 1) {  // one tile of rows: its values are asked for before the weights are waited for
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int j = 0; j < 4; ++j) xv[half % XH][j] = load_x(0, 2 * pair + half, j);
      }
      // a wait that gives up: the warp goes on without loads, so that its barriers are met
      if (ok) ok = tc::wait_bounded(tc::smem_u32(&bars[warp][slot]), (done / STAGES) & 1, &abort_flag, p);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) ++landed;
      const uint8_t* st = ring + slot * STAGE_BYTES + prow * 128;
      auto block = [&](int half) {
        const int b = 2 * pair + half;
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
          float c[NT][2][4] = {};
          if (ONES) {
            const unsigned minus136[4] = {0xc308c308u, 0xc308c308u, 0xc308c308u, 0xc308c308u};
#pragma unroll
            for (int j = k * RUNS; j < (k + 1) * RUNS; ++j) {
              mma_bf16(c[0][0], minus136, xv[half % XH][j].x, xv[half % XH][j].y, c[0][0]);
              mma_bf16(c[0][0], minus136, xv[half % XH][j].z, xv[half % XH][j].w, c[0][0]);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) c[0][1][m] = c[0][0][m];
          }
#pragma unroll
          for (int j = k * RUNS; j < (k + 1) * RUNS; ++j) {
            // the run's weights, once for all tiles of rows
            unsigned a[2][2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const unsigned u = word_of(w[t][0], j), v = word_of(w[t][1], j);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                a[t][i / 2][i % 2 * 2] = pair_of<!ONES>(u, i);
                a[t][i / 2][i % 2 * 2 + 1] = pair_of<!ONES>(v, i);
              }
            }
#pragma unroll
            for (int r = 0; r < NT; ++r) {
              if (r > 0 && r >= live) break;
              const uint4 x = NT == 1 ? xv[half % XH][j] : load_x(r, b, j);
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                mma_bf16(c[r][t], a[t][0], x.x, x.y, c[r][t]);
                mma_bf16(c[r][t], a[t][1], x.z, x.w, c[r][t]);
              }
            }
          }
#pragma unroll
          for (int r = 0; r < NT; ++r)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int m = 0; m < 4; ++m) acc[t][r][m] = fmaf(sc[t][m / 2][k], c[r][t][m], acc[t][r][m]);
        }
      };
      block(0);
      if (2 * pair + 1 < blocks) block(1);
      ++done;
      __syncwarp();  // the slot has been read
      shift_scales();
      issue(ok);
    }

    // the strip's warps add up, and each finishes some of the rows
    auto meet = [&]() {
      if (wk == 1) __syncwarp();
      else asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "r"(32 * wk) : "memory");
    };
    float* buf = red + round % sum_bufs<NT>() * (NT_WARPS * SUMS);
    float* mine = buf + warp * SUMS + lane;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < NT; ++r)
#pragma unroll
        for (int m = 0; m < 4; ++m) mine[((t * NT + r) * 4 + m) * 32] = acc[t][r][m];
    meet();
    const float* strip = buf + (warp - kw) * SUMS + lane;
    // pieces of 8 rows x 2 outputs a lane, shared out among the strip's warps
    for (int u = kw; u < live * 4; u += wk) {
      const int r8 = u >> 2, m = u & 3;
      float v[2] = {0.f, 0.f};
      for (int k = 0; k < wk; ++k)
#pragma unroll
        for (int t = 0; t < 2; ++t) v[t] += strip[k * SUMS + ((t * NT + r8) * 4 + m) * 32];
      const int r = r8 * 8 + 2 * tg + (m & 1), n = it.n0 + prow + 8 * (m >> 1);
      if (r >= rows) continue;
      bf16* dst = p.y + (long long)(it.r0 + r) * p.out;
      if (GATE_UP) {
        if (n < p.out) dst[n] = __float2bfloat16_rn(v[0] / (1.f + expf(-v[0])) * v[1]);
      } else {
        if (n < p.out) dst[n] = __float2bfloat16_rn(v[0]);
        if (n + 16 < p.out) dst[n + 16] = __float2bfloat16_rn(v[1]);
      }
    }
    if (sum_bufs<NT>() == 1) meet();
  }
  // a warp whose wait gave up leaves nothing under way
  for (; landed < issued; ++landed) {
    const long long t0 = clock64();
    while (!tc::mbar_try_wait(tc::smem_u32(&bars[warp][landed % STAGES]), (landed / STAGES) & 1)) {
      if ((unsigned long long)(clock64() - t0) > tc::DRAIN_LIMIT) { set_error(p.err, DEV_TIMEOUT); break; }
    }
  }
}

// codes of [rows, in] weights: [rows, words] by pairs of blocks
bool map_codes(CUtensorMap* m, const void* q, long long rows, int in, int box_rows) {
  const long long words = (long long)blocks_of(in) * WORDS;
  cuuint64_t dims[2] = {(cuuint64_t)words, (cuuint64_t)rows};
  cuuint64_t str[1] = {(cuuint64_t)words * 4};
  cuuint32_t box[2] = {2 * WORDS, (cuuint32_t)box_rows};
  return tc::make_map(m, q, 2, dims, str, box, CU_TENSOR_MAP_DATA_TYPE_UINT32);
}

template <int NT, int G, bool GATE_UP>
int launch_rows(Args p, const CUtensorMap& tm0, const CUtensorMap& tm1, cudaStream_t s) {
  constexpr int STRIP = GATE_UP ? 16 : 32, TT = 8 * NT;
  constexpr size_t smem = rows_smem<NT>();
  const int pairs = (blocks_of(p.in) + 1) / 2, strips = (p.out + STRIP - 1) / STRIP;
  const long long slots = (p.E < p.R ? p.E : p.R) + (long long)(p.R / TT);  // at most
  const long long resident = (long long)RESIDENT * sm_count();
  // Warps to a strip: more of them make the items finer, and each item costs its warps a meeting
  // (about as much as 0.7 pairs of blocks).  The least of rounds x time of an item.
  double best = 0;
  for (int wk = 1; wk <= NT_WARPS && wk <= pairs; wk *= 2) {
    const long long groups = resident * (NT_WARPS / wk), rounds = (slots * strips + groups - 1) / groups;
    const double cost = (double)rounds * ((pairs + wk - 1) / wk + 0.7);
    if (wk == 1 || cost < best) p.wk = wk, best = cost;
  }
  const long long ctas = (slots * strips * p.wk + NT_WARPS - 1) / NT_WARPS;
  auto k = w4_rows_kernel<NT, G, GATE_UP>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas < resident ? ctas : resident));
  cfg.blockDim = dim3(32 * NT_WARPS);
  cfg.dynamicSmemBytes = smem;
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

template <int G, bool GATE_UP>
int launch_rows_nt(const Args& p, const CUtensorMap& tm0, const CUtensorMap& tm1, cudaStream_t s) {
  const int mean = p.R / p.E;  // rows of an expert
  if (mean <= 4) return launch_rows<1, G, GATE_UP>(p, tm0, tm1, s);
  if (mean <= 12) return launch_rows<2, G, GATE_UP>(p, tm0, tm1, s);
  return launch_rows<4, G, GATE_UP>(p, tm0, tm1, s);
}
template <bool GATE_UP>
int launch_rows_g(const Args& p, int G, const void* q0, const void* q1, cudaStream_t s) {
  CUtensorMap tm0, tm1;
  const long long rows = (long long)p.E * p.out;
  if (!map_codes(&tm0, q0, rows, p.in, GATE_UP ? 16 : 32) || !map_codes(&tm1, q1, rows, p.in, GATE_UP ? 16 : 32))
    return MOE_ERR_CUDA;
  return G == 32 ? launch_rows_nt<32, GATE_UP>(p, tm0, tm1, s)
                 : G == 64 ? launch_rows_nt<64, GATE_UP>(p, tm0, tm1, s) : launch_rows_nt<128, GATE_UP>(p, tm0, tm1, s);
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
  a.cu = cu, a.E = E, a.R = rows, a.in = H, a.out = Hp, a.wk = 0;
  a.err = device_error_word(), a.wait_limit = tc::g_wait_limit;
  a.s0 = static_cast<const bf16*>(s_gate), a.s1 = static_cast<const bf16*>(s_up);
  a.y = static_cast<bf16*>(act);
  const int st = w4::launch_rows_g<true>(a, group, q_gate, q_up, s);
  if (st != MOE_OK) return st;
  a.x = static_cast<const bf16*>(act), a.src_tok = nullptr, a.x_rows = rows;
  a.in = Hp, a.out = H;
  a.s0 = a.s1 = static_cast<const bf16*>(s_down);
  a.y = static_cast<bf16*>(h);
  return w4::launch_rows_g<false>(a, group, q_down, q_down, s);
}

}  // namespace moe
