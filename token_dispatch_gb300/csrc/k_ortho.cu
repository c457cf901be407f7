// Orthogonalised updates of weight matrices by Newton-Schulz products, and the
// momentum step around them.
//
// For each matrix U [M, N] of a batch, m = min(M, N), n = max(M, N):
//   X = U / (|U|_F + eps), transposed where M > N, so that X is [m, n];
//   `steps` times  A = X X^T,  X <- a X + (b A + c A A) X.
// A step is three products of matrices on the tensor cores (ns_gemm_kernel):
//   GRAM   A = X X^T, kept as its diagonal s (fp32) and the rest D
//   POLY   D D, whose epilogue forms b A + c A A = diag(d) + P:
//            P_ij = (b + c (s_i + s_j)) D_ij + c (D D)_ij,   i != j
//            d_i  = a + b s_i + c s_i^2 + c (D D)_ii         (a X taken in)
//   APPLY  X <- diag(d) X + P X
// GRAM and POLY are symmetric: the 256 x 256 tiles on and above the diagonal are computed and kept, and
// a tile below it is read as the transposed one above (the tensor core takes either order).
//
// Operands are fp16 with fp32 sums.  Every operand is within a small factor of 1 in size,
// so fp16's range is enough (X, D and P are held times 2^10: an element of X is about
// 1 / sqrt(m n) at first) and it keeps 3 bits more than bf16 for the same rate.  What fp16 loses
// is further made small by keeping the diagonals of A and P in fp32: at the end A is near 1
// and a + b A + c A A near 0.7 while its terms are near 3.4, -4.8 and 2.0, so a rounding of
// the diagonal would come back several times larger.  Measured in simulation on noise with a few
// directions that stand out of it: relative error of the result 0.7 to 1.2e-3, against 1.7 to
// 2.5e-3 with the diagonals in fp16 and 1.3 to 2.1e-2 in bf16.  Directions of U whose singular
// value is below some 2^-11 of the root mean square are not resolved (they come out as small noise).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "tc_ptx.cuh"

namespace moe {
namespace ns {

using namespace tc;

constexpr int BM = 128;  // rows of a CTA; a pair has 256
constexpr int BN = 256;
constexpr int BK = 64;
constexpr int OPERAND_BYTES = BM * BK * 2;  // A rows of a CTA, and its half of the B columns
constexpr int STAGE_BYTES = 2 * OPERAND_BYTES;
constexpr int EPI_WARPS = 8;  // two for each quarter of tensor memory's lanes, half of the columns each
constexpr int THREADS = 32 * (2 + EPI_WARPS);
constexpr int STG = 36;       // floats between the rows of FINAL's staging tiles
constexpr float HELD = 1024.f;  // X, D and P are stored times this
constexpr float INV = 1.f / 1024.f;

// PART: GRAM's sums over a part of K
enum Mode { GRAM = 0, POLY = 1, APPLY = 2, FINAL = 3, PART = 4 };
enum Kind { ORTHO = 0, MUON_BF16 = 1, MUON_F32 = 2 };  // what FINAL writes
template <int MODE>
struct Cfg {
  static constexpr int STAGES = MODE == FINAL ? 5 : 6;
  // an epilogue warp's tile of 32 x 32 on its way between rows a lane and whole row pieces, and the
  // diagonal at its columns
  static constexpr int WARP_BYTES = (MODE == FINAL ? 32 * STG * 4 : 2048) + (MODE == POLY ? 512 : 0);
  static constexpr size_t SMEM = (size_t)STAGES * STAGE_BYTES + EPI_WARPS * WARP_BYTES + (2 * STAGES + 5) * 8 + 1024;
  static_assert(SMEM + 1024 <= 227 * 1024, "shared memory");
};

// Where the last step's result goes: `o` (bf16), or the weights' update
// w_out = keep * w - step * X (dtype of the weights; w_low: a bf16 copy).
struct Result {
  bf16* o = nullptr;
  const void* w = nullptr;
  void* w_out = nullptr;
  bf16* w_low = nullptr;
  float keep = 1.f, step = 0.f;
  bool tall = false;  // X is the transposed matrix
  bool vec = false;   // rows of the result are multiples of four elements
};

struct Params {
  int E, m, n;
  long long ldx, lda;  // elements between rows of X, and of D and P
  const __half* in;    // POLY: D, APPLY and FINAL: X
  __half* out;
  float *s, *d;  // [E][lda]
  float a, b, c;
  Result r;
  unsigned* err;
  unsigned long long wait_limit;
  int halves = 0;          // 1: tiles of 128 columns (256 otherwise)
  int splits = 1;          // PART: parts of K
  float4* part = nullptr;  // their sums, [part][tile][256 / 128 rows][64 quads of columns][128 rows]
};

struct Tile {
  int e, i, j, row0, n0;
  int split, index;  // PART: part of K, and tile of all matrices
};
template <int MODE>
__host__ __device__ inline int tiles_per_matrix(int m, int n) {
  const int mt = (m + 255) / 256, nt = (n + 255) / 256;
  return MODE == GRAM || MODE == POLY || MODE == PART ? mt * (mt + 1) / 2 : mt * nt;
}
template <int MODE>
__device__ __forceinline__ Tile tile_of(int t, const Params& p, int per, uint32_t rank) {
  Tile w;
  w.split = 0;
  if (MODE == PART) {
    const int tiles = p.E * per;
    w.split = t / tiles;
    t -= w.split * tiles;
  }
  w.index = t;
  w.e = t / per;
  int r = t - w.e * per;
  const int half = r & p.halves;
  r >>= p.halves;
  if (MODE == GRAM || MODE == POLY || MODE == PART) {  // column blocks from the left, i <= j in each
    int j = (int)((sqrtf(8.f * r + 1.f) - 1.f) * 0.5f);
    while (j * (j + 1) / 2 > r) --j;
    while ((j + 1) * (j + 2) / 2 <= r) ++j;
    w.j = j;
    w.i = r - j * (j + 1) / 2;
  } else {
    const int mt = (p.m + 255) / 256;
    w.i = r % mt;
    w.j = r / mt;
  }
  w.row0 = w.i * 2 * BM + (int)rank * BM;
  w.n0 = w.j * BN + half * (BN / 2);
  return w;
}

// A warp's tile of 32 rows x 32 columns of fp16 is read and written in whole pieces of 64 bytes of a row, four
// lanes to a piece; a lane's own row comes and goes through 2 KB of shared memory, where the four 16-byte
// parts of a row are exchanged by the row's bits 1 and 2 (no bank conflicts).  (With a row to a lane in global
// memory too, each access touched 32 lines, and the L1's tag stage took as long as the products: POLY at
// 64 x 1408 x 1408 210 us, so 140.)
struct Piece {
  uint4 v[4];
};
__device__ __forceinline__ uint4* part_of(uint8_t* stg, int row, int part) {
  return reinterpret_cast<uint4*>(stg + row * 64 + ((part ^ (row >> 1 & 3)) << 4));
}
// rows row0 + lane / 4 + 8 k, columns col0 + 8 (lane % 4) .. of a matrix with `rows` rows (columns up to the row's
// padding)
__device__ __forceinline__ void load_piece(Piece& q, const __half* plane, long long ld, int row0, int col0, int rows,
                                           int lane) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = row0 + (lane >> 2) + 8 * k;
    if (r < rows) q.v[k] = *reinterpret_cast<const uint4*>(plane + r * ld + col0 + 8 * (lane & 3));
  }
}
__device__ __forceinline__ void own_row(const Piece& q, uint8_t* stg, int lane, uint4 (&row)[4]) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) *part_of(stg, (lane >> 2) + 8 * k, lane & 3) = q.v[k];
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) row[k] = *part_of(stg, lane, k);
}
__device__ __forceinline__ void store_tile(__half* plane, long long ld, int row0, int col0, int rows, uint8_t* stg,
                                           int lane, const float (&v)[32]) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint4 q;
    __half2* h = reinterpret_cast<__half2*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[8 * k + 2 * i], v[8 * k + 2 * i + 1]);
    *part_of(stg, lane, k) = q;
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = row0 + (lane >> 2) + 8 * k;
    if (r < rows)
      *reinterpret_cast<uint4*>(plane + r * ld + col0 + 8 * (lane & 3)) = *part_of(stg, (lane >> 2) + 8 * k, lane & 3);
  }
}

// v[at], which becomes 0; nothing where `at` is outside 0..31
__device__ __forceinline__ float take_diagonal(float (&v)[32], int at) {
  float own = 0.f;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    own = j == at ? v[j] : own;
    v[j] = j == at ? 0.f : v[j];
  }
  return own;
}

// ---- the result.  A warp's tile lies in shared memory by rows of the result (turned around for a tall one); in round
// k a lane has four neighbours of row lane / 8 + 4 k.
struct Place {  // the tile's corner in a matrix of `rows` rows of `len`, which begins at `plane`
  long long plane;
  int row0, col0, rows, len;
};
template <int KIND>
struct Old {  // the old weights of a tile, asked for a tile ahead
  static constexpr int N = KIND == ORTHO ? 1 : KIND == MUON_BF16 ? 2 : 4;
  unsigned v[8][N];
  __device__ __forceinline__ void load(const Result& r, const Place& p, int lane) {
    if (KIND == ORTHO || !r.vec) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int row = p.row0 + (lane >> 3) + 4 * k, col = p.col0 + 4 * (lane & 7);
      if (row >= p.rows || col >= p.len) continue;
      const long long at = p.plane + (long long)row * p.len + col;
      if (KIND == MUON_BF16) {
        const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const bf16*>(r.w) + at);
        v[k][0] = q.x, v[k][1 % N] = q.y;
      } else {
        const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const float*>(r.w) + at);
        v[k][0] = q.x, v[k][1 % N] = q.y, v[k][2 % N] = q.z, v[k][3 % N] = q.w;
      }
    }
  }
  __device__ __forceinline__ float at(int k, int i) const {
    if (KIND == MUON_F32) return __uint_as_float(v[k][i % N]);
    return __uint_as_float(i & 1 ? v[k][i / 2 % N] & 0xffff0000u : v[k][i / 2 % N] << 16);
  }
};
__device__ __forceinline__ unsigned pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const unsigned*>(&h);
}
template <int KIND>
__device__ __forceinline__ void put_tile(const Result& r, const Place& p, const Old<KIND>& old, const float* stg,
                                         int lane) {
  using T = typename std::conditional<KIND == MUON_F32, float, bf16>::type;
  bf16* low = KIND == ORTHO ? r.o : KIND == MUON_BF16 ? static_cast<bf16*>(r.w_out) : r.w_low;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int row = p.row0 + (lane >> 3) + 4 * k, col = p.col0 + 4 * (lane & 7);
    if (row >= p.rows || col >= p.len) continue;
    const float4 q = *reinterpret_cast<const float4*>(stg + ((lane >> 3) + 4 * k) * STG + 4 * (lane & 7));
    float y[4] = {q.x, q.y, q.z, q.w};
    const long long at = p.plane + (long long)row * p.len + col;
    if (r.vec) {
      if (KIND != ORTHO)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = r.keep * old.at(k, i) - r.step * y[i];
      const uint2 h = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
      if (KIND == MUON_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(r.w_out) + at) = make_float4(y[0], y[1], y[2], y[3]);
      if (KIND != MUON_F32 || low) *reinterpret_cast<uint2*>(low + at) = h;
      if (KIND == MUON_BF16 && r.w_low) *reinterpret_cast<uint2*>(r.w_low + at) = h;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (col + i >= p.len) break;
        if (KIND == ORTHO) {
          r.o[at + i] = __float2bfloat16_rn(y[i]);
        } else {
          const float w = r.keep * to_f32(static_cast<const T*>(r.w)[at + i]) - r.step * y[i];
          static_cast<T*>(r.w_out)[at + i] = from_f32<T>(w);
          if (r.w_low) r.w_low[at + i] = __float2bfloat16_rn(w);
        }
      }
    }
  }
}

// The products on pairs of SMs: 256 x 256 tiles by the two-CTA MMA, TMA operands in a ring of
// five or six stages, two accumulators in tensor memory so that the epilogue of a tile runs under the
// next one's products.  Measured, 64 x 2048 x 1408 (m padded to 1536 by the tiles): GRAM 187 us, POLY 140, APPLY 325, the
// tensor pipe 76, 63 and 88% busy; FINAL, whose epilogue reads and writes the weights, 440 with bf16 ones; the
// whole momentum step 4.5 ms, of which its passes over gradient and momentum take 0.64 (at a copy's rate).  Barriers as in the expert products' pair kernel: `full` the leader's
// (both CTAs' bytes), `empty` and `accf` each CTA's own, `acce` the leader's.  All waits are bounded.
template <int MODE, int KIND = ORTHO>
__global__ void __launch_bounds__(THREADS, 1) __cluster_dims__(2, 1, 1)
ns_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmT,
               const __grid_constant__ CUtensorMap tmA2, const Params p) {
  constexpr bool SYM = MODE == GRAM || MODE == POLY || MODE == PART;
  constexpr bool FIRST = MODE == GRAM || MODE == PART;  // X X^T
  constexpr int STAGES = Cfg<MODE>::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stage_out = smem + STAGES * STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES + EPI_WARPS * Cfg<MODE>::WARP_BYTES);
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int per = tiles_per_matrix<MODE>(p.m, p.n) << p.halves;
  const int total = p.E * per * (MODE == PART ? p.splits : 1);
  const int K = FIRST ? p.n : p.m;
  const int cols = SYM ? p.m : p.n;
  const int kbs = (K + BK - 1) / BK;
  // the blocks of K that a tile sums over
  auto k_begin = [&](const Tile& w) { return MODE == PART ? (int)((long long)kbs * w.split / p.splits) : 0; };
  auto k_end = [&](const Tile& w) { return MODE == PART ? (int)((long long)kbs * (w.split + 1) / p.splits) : kbs; };
  // a tile with no more than 128 columns takes MMAs of half the width, and half of the second operand
  auto narrow = [&](const Tile& w) { return p.halves || cols - w.n0 <= BN / 2; };
  // Whether a block of the first operand (rows of tile row i) or of the second is read as it lies in the transposed
  // place, [64 of K][rows] in two boxes of 64 rows: D and P below the diagonal, and X as APPLY's second operand.
  auto a_turned = [&](int i, int kb) { return !FIRST && kb / 4 < i; };
  auto b_turned = [&](int j, int kb) { return MODE == POLY ? kb / 4 < j : !SYM; };

  auto full_bar = [&](int s) { return smem_u32(&bars[s]); };
  auto empty_bar = [&](int s) { return smem_u32(&bars[STAGES + s]); };
  auto accf_bar = [&](int a) { return smem_u32(&bars[2 * STAGES + a]); };
  auto acce_bar = [&](int a) { return smem_u32(&bars[2 * STAGES + 2 + a]); };
  const uint32_t drain_bar = smem_u32(&bars[2 * STAGES + 4]);

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf_bar(a), 1);
      mbar_init(acce_bar(a), 2 * EPI_WARPS);  // the epilogue warps of both CTAs
    }
    mbar_init(drain_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmT);
    if (!SYM) prefetch_tmap(&tmA2);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_slot)),
                 "r"(2u * BN));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised before anything arrives on them
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // one thread issues, but the warp walks along: see elect_one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int stage = 0, filled = 0;  // stages filled so far
    uint32_t phase = 0;
    bool ok = true;
    const uint32_t full0 = cluster_addr(full_bar(0), 0);  // the leader's, 8 bytes apart
    for (int t = pair; ok && t < total; t += n_pairs) {
      const Tile w = tile_of<MODE>(t, p, per, rank);
      const bool half = narrow(w);
      const int b0 = w.n0 + (int)rank * (half ? BN / 4 : BN / 2);
      for (int kb = k_begin(w); kb < k_end(w); ++kb) {
        ok = __all_sync(0xffffffffu, wait_bounded(empty_bar(stage), phase ^ 1u, &abort_flag, p));
        if (!ok) break;
        const uint32_t a_dst = smem_u32(smem + stage * STAGE_BYTES), b_dst = a_dst + OPERAND_BYTES;
        const uint32_t fb = full0 + 8 * stage;
        const bool at = a_turned(w.i, kb), bt = b_turned(w.j, kb);
        if (elect_one()) {
          if (leader) mbar_expect_tx(full_bar(stage), half ? 2 * (STAGE_BYTES - OPERAND_BYTES / 2) : 2 * STAGE_BYTES);
          // the maps of the turned boxes: of D (POLY), of P and of X (APPLY: P's is tmA2)
          if (at) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
              tma_load_3d_pair(a_dst + c * (64 * BK * 2), SYM ? &tmT : &tmA2, fb, w.row0 + c * 64, kb * BK, w.e);
          } else {
            tma_load_3d_pair(a_dst, &tmA, fb, kb * BK, w.row0, w.e);
          }
          if (bt) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (c == 0 || !half) tma_load_3d_pair(b_dst + c * (64 * BK * 2), &tmT, fb, b0 + c * 64, kb * BK, w.e);
          } else if (half) {  // the map of 64 rows, as it lies
            tma_load_3d_pair(b_dst, &tmT, fb, kb * BK, b0, w.e);
          } else {
            tma_load_3d_pair(b_dst, &tmA, fb, kb * BK, b0, w.e);
          }
        }
        __syncwarp();
        ++filled;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (leader && lane == 0) {  // every stage filled must have landed, both CTAs' bytes
      for (int k = max(0, filled - STAGES); k < filled; ++k) {
        const long long t0 = clock64();
        while (!mbar_try_wait(full_bar(k % STAGES), (uint32_t)(k / STAGES) & 1u)) {
          if ((unsigned long long)(clock64() - t0) > DRAIN_LIMIT) { set_error(p.err, DEV_TIMEOUT); break; }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------- MMA issuer (leader only)
    if (leader) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false;
      int i = 0;
      for (int t = pair; ok && t < total; t += n_pairs, ++i) {
        const int acc = i & 1;
        ok = __all_sync(0xffffffffu,
                        wait_bounded_cluster(acce_bar(acc), (((uint32_t)i >> 1) & 1u) ^ 1u, &abort_flag, p));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        const Tile w = tile_of<MODE>(t, p, per, 0);
        const int kb0 = k_begin(w);
        for (int kb = kb0; kb < k_end(w); ++kb) {
          const bool at = a_turned(w.i, kb), bt = b_turned(w.j, kb);
          const uint32_t idesc = instr_desc(2 * BM, narrow(w) ? BN / 2 : BN, false, false, true) |
                                 (at ? 1u << 15 : 0u) | (bt ? 1u << 16 : 0u);
          ok = __all_sync(0xffffffffu, wait_bounded(full_bar(stage), phase, &abort_flag, p));
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_t = smem_u32(smem + stage * STAGE_BYTES), b_t = a_t + OPERAND_BYTES;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < BK / 16; ++k) {
              // as it lies: +32 bytes for 16 of K in the 128-byte row; turned: +16 rows, 64-wide boxes 8 KB apart
              const uint64_t adesc =
                  at ? smem_desc(a_t + k * 16 * 128, 64 * BK * 2, 1024) : smem_desc(a_t + k * 32, 16, 1024);
              const uint64_t bdesc =
                  bt ? smem_desc(b_t + k * 16 * 128, 64 * BK * 2, 1024) : smem_desc(b_t + k * 32, 16, 1024);
              tc_mma_pair(d_tmem, adesc, bdesc, idesc, (kb > kb0 || k > 0) ? 1u : 0u);
            }
            tc_commit_pair(empty_bar(stage), 3);
          }
          __syncwarp();
          issued = true;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (ok && elect_one()) tc_commit_pair(accf_bar(acc), 3);
        __syncwarp();
      }
      if (issued) {
        if (elect_one()) tc_commit_pair(drain_bar, 1);
        __syncwarp();
        const long long t0 = clock64();
        while (!mbar_try_wait(drain_bar, 0)) {
          if ((unsigned long long)(clock64() - t0) > DRAIN_LIMIT) { set_error(p.err, DEV_TIMEOUT); break; }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int CHUNKS = BN / 32 / 2;  // of 32 columns, of a warp
    const int q = warp & 3;  // TMEM lane quadrant of this warp
    const int n_chunks = CHUNKS >> p.halves, c_begin = ((warp - 2) >> 2) * n_chunks;
    uint8_t* stg = stage_out + (warp - 2) * Cfg<MODE>::WARP_BYTES;
    float* diag = reinterpret_cast<float*>(stg + 2048);  // POLY
    float* wide = reinterpret_cast<float*>(stg);         // FINAL
    constexpr bool ALL = MODE == POLY || MODE == APPLY;  // all that the epilogue reads is asked for at once
    int i = 0;
    for (int t = pair; t < total; t += n_pairs, ++i) {
      const int acc = i & 1;
      const Tile w = tile_of<MODE>(t, p, per, rank);
      const int row0 = w.row0 + q * 32, row = row0 + lane;
      const bool row_ok = row < p.m;
      const int c_end = min(c_begin + n_chunks, (cols - w.n0 + 31) / 32);
      // What the epilogue reads is asked for before the sums are waited for.
      const long long ldi = MODE == POLY ? p.lda : p.ldx;
      const __half* in = p.in + (long long)w.e * p.m * ldi;
      Piece piece[ALL ? CHUNKS : FIRST ? 1 : 2];
      float s_row = 0.f, d_row = 0.f;
      if (!FIRST) {
#pragma unroll
        for (int c = 0; c < (ALL ? CHUNKS : 1); ++c)
          if (c_begin + c < c_end) load_piece(piece[c], in, ldi, row0, w.n0 + (c_begin + c) * 32, p.m, lane);
        if (row_ok) {
          if (MODE == POLY) s_row = p.s[(long long)w.e * p.lda + row];
          else d_row = p.d[(long long)w.e * p.lda + row];
        }
      }
      if (MODE == POLY) {  // the diagonal at the warp's columns (lda is a multiple of 64)
        const float* sc = p.s + (long long)w.e * p.lda + w.n0 + c_begin * 32;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) diag[c * 32 + lane] = c_begin + c < c_end ? sc[c * 32 + lane] : 0.f;
        __syncwarp();
      }
      // FINAL: where the result of chunk c lies
      auto place = [&](int c) {
        const int col0 = w.n0 + c * 32;
        const long long plane = (long long)w.e * p.m * p.n;
        return p.r.tall ? Place{plane, col0, row0, p.n, p.m} : Place{plane, row0, col0, p.m, p.n};
      };
      Old<KIND> old[2];
      if (MODE == FINAL && c_begin < c_end) old[0].load(p.r, place(c_begin), lane);
      // all lanes or none: what follows is for the whole warp
      if (!__all_sync(0xffffffffu, wait_bounded(accf_bar(acc), ((uint32_t)i >> 1) & 1u, &abort_flag, p))) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + acc * BN + ((uint32_t)(q * 32) << 16);
#pragma unroll
      for (int cc = 0; cc < CHUNKS; ++cc) {
        const int c = c_begin + cc;
        if (c >= c_end) break;
        if (MODE == FINAL && c + 1 < c_end) {
          load_piece(piece[(cc + 1) % 2], in, ldi, row0, w.n0 + (c + 1) * 32, p.m, lane);
          old[(cc + 1) % 2].load(p.r, place(c + 1), lane);
        }
        const int col0 = w.n0 + c * 32;
        uint4 mine[4];
        if (!FIRST) own_row(piece[ALL ? cc : FIRST ? 0 : cc % 2], stg, lane, mine);
        const __half2* h = reinterpret_cast<const __half2*>(mine);
        float v[32];
        tmem_ld32(tbase + c * 32, v);
        if (MODE == PART) {
          float4* dst = p.part + (((long long)w.split * (p.E * per) + w.index) * 2 + rank) * (64 * BM) + q * 32 + lane;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[(c * 8 + j) * BM] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else if (MODE == GRAM) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= INV;  // A, held times 2^10
          if (w.i == w.j) {
            const float own = take_diagonal(v, row - col0);
            if (row_ok && row >= col0 && row < col0 + 32) p.s[(long long)w.e * p.lda + row] = own * INV;
          }
        } else if (MODE == POLY) {
          const float k0 = p.b + p.c * s_row, k1 = p.c * INV;
          if (w.i == w.j) {
            const float own = take_diagonal(v, row - col0);  // (D D)_ii; D_ii is 0, and so is P_ii then
            if (row_ok && row >= col0 && row < col0 + 32)
              p.d[(long long)w.e * p.lda + row] = p.a + (p.b + p.c * s_row) * s_row + k1 * INV * own;
          }
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 sj = *reinterpret_cast<const float4*>(diag + cc * 32 + j);
            const float2 x0 = __half22float2(h[j / 2]), x1 = __half22float2(h[j / 2 + 1]);
            v[j] = fmaf(k1, v[j], fmaf(p.c, sj.x, k0) * x0.x);
            v[j + 1] = fmaf(k1, v[j + 1], fmaf(p.c, sj.y, k0) * x0.y);
            v[j + 2] = fmaf(k1, v[j + 2], fmaf(p.c, sj.z, k0) * x1.x);
            v[j + 3] = fmaf(k1, v[j + 3], fmaf(p.c, sj.w, k0) * x1.y);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 x = __half22float2(h[j]);
            v[2 * j] = fmaf(d_row, x.x, v[2 * j] * INV);
            v[2 * j + 1] = fmaf(d_row, x.y, v[2 * j + 1] * INV);
          }
        }
        if (MODE == FINAL) {
          __syncwarp();
          if (p.r.tall) {
#pragma unroll
            for (int j = 0; j < 32; ++j) wide[j * STG + lane] = v[j] * INV;
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4*>(wide + lane * STG + j) =
                  make_float4(v[j] * INV, v[j + 1] * INV, v[j + 2] * INV, v[j + 3] * INV);
          }
          __syncwarp();
          put_tile<KIND>(p.r, place(c), old[cc % 2], wide, lane);
        } else if (MODE != PART) {
          const long long ldo = SYM ? p.lda : p.ldx;
          store_tile(p.out + (long long)w.e * p.m * ldo, ldo, row0, col0, p.m, stg, lane, v);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(acce_bar(acc));
        else mbar_arrive_remote(cluster_addr(acce_bar(acc), 0));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs are done with tensor memory and with each other's barriers
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(2u * BN));
  }
}

// GRAM's parts added in order, and its epilogue: a block takes 4 columns x 128 rows of a tile, a thread a row of them.
__global__ void __launch_bounds__(BM) ns_join_kernel(const Params p, int per) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int quad = blockIdx.x, rank = blockIdx.y, tiles = p.E * per;
  const Tile w = tile_of<GRAM>(blockIdx.z, p, per, rank);
  const int row = w.row0 + threadIdx.x, col = w.n0 + 4 * quad;
  if (row >= p.m || col >= p.m) return;
  const float4* src = p.part + ((long long)w.index * 2 + rank) * (64 * BM) + quad * BM + threadIdx.x;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < p.splits; ++k) {
    const float4 x = src[(long long)k * tiles * (2 * 64 * BM)];
    v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
  }
  float a[4] = {v.x * INV, v.y * INV, v.z * INV, v.w * INV};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (col + j == row) {
      p.s[(long long)w.e * p.lda + row] = a[j] * INV;
      a[j] = 0.f;
    }
  uint2 q;
  reinterpret_cast<__half2*>(&q)[0] = __floats2half2_rn(a[0], a[1]);
  reinterpret_cast<__half2*>(&q)[1] = __floats2half2_rn(a[2], a[3]);
  *reinterpret_cast<uint2*>(p.out + ((long long)w.e * p.m + row) * p.lda + col) = q;
}

// ------------------------------------------------------- norm and first X ---
// |U|_F without over- or underflow: the squares are summed in three scales, of u, 2^-80 u and
// 2^80 u, in fp32 for a thread's values and in fp64 from there on, and the scale that holds the
// sum is taken at the end.
constexpr int PARTS = 256;   // most partial sums of a matrix
constexpr int SUM_NT = 256;
constexpr float BIG = 1.2089258196146292e24f;  // 2^80

struct Source {
  const void* x = nullptr;  // the matrices, dtype; or the momentum step's:
  const float* g = nullptr;
  const float* m = nullptr;
  float* m_out = nullptr;
  float beta = 0.f;
  bool nesterov = false;
};

enum From { FROM_F32 = 0, FROM_BF16 = 1, FROM_MOMENTUM = 2 };

// u at `at`, and with FIRST the momentum written
template <int FROM, bool FIRST>
__device__ __forceinline__ float u_at(const Source& s, long long at) {
  if (FROM == FROM_F32) return static_cast<const float*>(s.x)[at];
  if (FROM == FROM_BF16) return __bfloat162float(static_cast<const bf16*>(s.x)[at]);
  if (FIRST) {
    const float g = s.g[at], m = fmaf(s.beta, s.m[at], g);
    s.m_out[at] = m;
    return s.nesterov ? fmaf(s.beta, m, g) : m;
  }
  const float m = s.m_out[at];
  return s.nesterov ? fmaf(s.beta, m, s.g[at]) : m;
}
// four neighbours, 16-byte aligned (8 for bf16)
template <int FROM, bool FIRST>
__device__ __forceinline__ float4 u4_at(const Source& s, long long at) {
  if (FROM == FROM_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(s.x) + at);
  if (FROM == FROM_BF16) {
    const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const bf16*>(s.x) + at);
    const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q.x));
    const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q.y));
    return make_float4(lo.x, lo.y, hi.x, hi.y);
  }
  float4 m, g = make_float4(0.f, 0.f, 0.f, 0.f);
  if (FIRST || s.nesterov) g = *reinterpret_cast<const float4*>(s.g + at);
  if (FIRST) {
    m = *reinterpret_cast<const float4*>(s.m + at);
    m = make_float4(fmaf(s.beta, m.x, g.x), fmaf(s.beta, m.y, g.y), fmaf(s.beta, m.z, g.z), fmaf(s.beta, m.w, g.w));
    *reinterpret_cast<float4*>(s.m_out + at) = m;
  } else {
    m = *reinterpret_cast<const float4*>(s.m_out + at);
  }
  if (!s.nesterov) return m;
  return make_float4(fmaf(s.beta, m.x, g.x), fmaf(s.beta, m.y, g.y), fmaf(s.beta, m.z, g.z), fmaf(s.beta, m.w, g.w));
}

struct Sums {
  float mid = 0.f, high = 0.f, low = 0.f;
  __device__ __forceinline__ void add(float u) {
    const float h = u * (1.f / BIG), l = u * BIG;
    mid = fmaf(u, u, mid);
    high = fmaf(h, h, high);
    low = fmaf(l, l, low);
  }
};

// block `blockIdx.x` of a matrix's `gridDim.x` takes `span` neighbours (a multiple of 4)
template <int FROM, bool VEC>
__global__ void __launch_bounds__(SUM_NT) ns_sum_kernel(const Source s, long long size, long long span,
                                                        double* __restrict__ part) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long base = (long long)blockIdx.y * size, lo = blockIdx.x * span, hi = min(size, lo + span);
  Sums a;
  if (VEC) {
#pragma unroll 4
    for (long long i = lo + 4 * threadIdx.x; i < hi; i += 4 * SUM_NT) {
      const float4 u = u4_at<FROM, true>(s, base + i);
      a.add(u.x), a.add(u.y), a.add(u.z), a.add(u.w);
    }
  } else {
#pragma unroll 4
    for (long long i = lo + threadIdx.x; i < hi; i += SUM_NT) a.add(u_at<FROM, true>(s, base + i));
  }
  __shared__ double red[3][SUM_NT / 32];
  double v[3] = {a.mid, a.high, a.low};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if ((threadIdx.x & 31) == 0) red[k][threadIdx.x >> 5] = v[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    double sum = 0;
    for (int w = 0; w < SUM_NT / 32; ++w) sum += red[threadIdx.x][w];
    part[((long long)blockIdx.y * PARTS + blockIdx.x) * 3 + threadIdx.x] = sum;
  }
}

// 2^10 / (|U| + eps) as the product of two floats, neither of which leaves the range, from the three sums; NaN for
// a matrix that holds a NaN or an infinity, 0 for one of zeros
__device__ __forceinline__ float2 factor_of(const double (&v)[3], double eps) {
  const double norm = v[0] > 0x1p100 ? sqrt(v[1]) * 0x1p80 : v[0] > 0x1p-60 ? sqrt(v[0]) : sqrt(v[2]) * 0x1p-80;
  if (!(v[1] < HUGE_VAL)) return make_float2(NAN, NAN);
  if (norm == 0) return make_float2(0.f, 0.f);
  int e;
  const double x = frexp(norm + eps, &e);  // norm + eps = x 2^e
  return make_float2(ldexpf(1.f, -(e / 2)), (float)ldexp(1024.0 / x, -(e - e / 2)));
}

// The factor of each matrix, a warp a matrix.  (Here and in what follows, what the kernel before wrote is read by plain
// loads: it may still have been writing when this one began.)
__global__ void __launch_bounds__(32) ns_factor_kernel(const double* part, int parts, double eps, float2* factor) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x;
  part += (long long)blockIdx.x * PARTS * 3;
  double v[3] = {0, 0, 0};
  for (int i = lane; i < parts; i += 32)
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] += part[i * 3 + k];
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (lane == 0) factor[blockIdx.x] = factor_of(v, eps);
}

// First X (fp16, times 2^10) from U, turned around where M > N: 64 x 64 tiles through shared
// memory, read along U's rows and written along X's.  VEC: N is a multiple of 4.
constexpr int LT = 64;
constexpr int LOAD_NT = 256;
template <int FROM, bool VEC>
__global__ void __launch_bounds__(LOAD_NT) ns_load_kernel(const Source s, int M, int N, bool tall, long long ldx,
                                                          const float2* factor, __half* x) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ __align__(16) __half tile[LT][LT + 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.z;
  const int r0 = blockIdx.y * LT, c0 = blockIdx.x * LT;
  const long long base = (long long)e * M * N;
  const float2 f = factor[e];
  if (VEC) {
    const int rr = threadIdx.x >> 4, cc = (threadIdx.x & 15) * 4;
    float4 u[LT / 16];
#pragma unroll
    for (int k = 0; k < LT / 16; ++k) {
      const int r = r0 + rr + 16 * k, c = c0 + cc;
      u[k] = r < M && c < N ? u4_at<FROM, false>(s, base + (long long)r * N + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = 0; k < LT / 16; ++k) {
      __half2* dst = reinterpret_cast<__half2*>(&tile[rr + 16 * k][cc]);
      dst[0] = __floats2half2_rn(u[k].x * f.x * f.y, u[k].y * f.x * f.y);
      dst[1] = __floats2half2_rn(u[k].z * f.x * f.y, u[k].w * f.x * f.y);
    }
  } else {
    float u[LT / 8][2];
#pragma unroll
    for (int k = 0; k < LT / 8; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = r0 + warp + 8 * k, c = c0 + lane + 32 * h;
        u[k][h] = r < M && c < N ? u_at<FROM, false>(s, base + (long long)r * N + c) : 0.f;
      }
#pragma unroll
    for (int k = 0; k < LT / 8; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) tile[warp + 8 * k][lane + 32 * h] = __float2half_rn(u[k][h] * f.x * f.y);
  }
  __syncthreads();
  const int m = tall ? N : M, n = tall ? M : N, xr0 = tall ? c0 : r0, xc0 = tall ? r0 : c0;
  __half* plane = x + (long long)e * m * ldx;
#pragma unroll
  for (int k = 0; k < LT / 8; ++k) {
    const int r = warp + 8 * k, c = 2 * lane;
    const __half2 v = tall ? __halves2half2(tile[c][r], tile[c + 1][r]) : __halves2half2(tile[r][c], tile[r][c + 1]);
    // a column behind the last one lies in the row's padding
    if (xr0 + r < m && xc0 + c < n) *reinterpret_cast<__half2*>(plane + (long long)(xr0 + r) * ldx + xc0 + c) = v;
  }
}

// ------------------------------------------------------- small matrices ---
// m <= 128 and n <= 512: a CTA takes a matrix from U to the result, X and D (then P) in shared memory and the sums in
// tensor memory.  A step is a few thousand cycles of products and epilogues one after the other, where the chain of
// kernels above costs three launches.  Measured in us, here and in the chain, for 1, 8, 152 and 1024 matrices:
//   128 x 512   61, 56, 58, 418   110, 118, 227, 1208
//   128 x 256   39, 39, 41, 300   106, 112, 173, 859
//   16 x 512    41, 41, 43, 276   82, 88, 153, 743
// X lies as 64-column blocks of 128 rows of 128 bytes, 16-byte parts exchanged by the row's low bits: the tensor core
// reads such a block along its rows (GRAM) and down its columns (APPLY).
constexpr int SM_ROWS = 128, SM_COLS = 512;
constexpr int SM_WARPS = 16;
constexpr int SM_NT = 32 * SM_WARPS;
constexpr int SM_BLOCK = SM_ROWS * 128;  // bytes of 64 columns
constexpr size_t small_smem(int n) {     // X, D, and the result's staging tiles over and behind D
  return (size_t)(n + 63) / 64 * SM_BLOCK + SM_WARPS * 32 * STG * 4 + 1024;
}

struct SmallParams {
  Source src;
  int M, N, steps;
  float a, b, c;
  double eps;
  Result r;
  unsigned* err;
  unsigned long long wait_limit;
};

// 16-byte part of a row
__device__ __forceinline__ uint4* small_part(uint8_t* base, int row, int part) {
  return reinterpret_cast<uint4*>(base + (part >> 3) * SM_BLOCK + row * 128 + (((part & 7) ^ (row & 7)) << 4));
}
__device__ __forceinline__ void small_row(uint8_t* base, int row, int col0, uint4 (&q)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) q[k] = *small_part(base, row, col0 / 8 + k);
}
__device__ __forceinline__ void small_store(uint8_t* base, int row, int col0, const float (&v)[32]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint4 q;
    __half2* h = reinterpret_cast<__half2*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[8 * k + 2 * i], v[8 * k + 2 * i + 1]);
    *small_part(base, row, col0 / 8 + k) = q;
  }
}

template <int FROM, int KIND>
__global__ void __launch_bounds__(SM_NT, 1) ns_small_kernel(const SmallParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* X = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ __align__(16) float s_of[SM_ROWS], d_of[SM_ROWS];
  __shared__ float red[3][SM_WARPS];
  __shared__ float2 factor;
  const bool tall = p.M > p.N;
  const int m = tall ? p.N : p.M, n = tall ? p.M : p.N, blocks = (n + 63) / 64;
  uint8_t* D = X + blocks * SM_BLOCK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, part = warp >> 2, row = q * 32 + lane;
  const long long size = (long long)p.M * p.N, base = blockIdx.x * size;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(smem_u32(&bar), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // ---- norm (and the momentum): a warp takes every SM_WARPS-th row.  fp32 sums of at most 65536 squares: their
  // rounding moves X by a common factor alone.
  const bool vec = p.N % 4 == 0;
  Sums sums;
  for (int r = warp; r < p.M; r += SM_WARPS) {
    const long long at = base + (long long)r * p.N;
    if (vec) {
#pragma unroll 4
      for (int c = 4 * lane; c < p.N; c += 128) {
        const float4 u = u4_at<FROM, true>(p.src, at + c);
        sums.add(u.x), sums.add(u.y), sums.add(u.z), sums.add(u.w);
      }
    } else {
#pragma unroll 4
      for (int c = lane; c < p.N; c += 32) sums.add(u_at<FROM, true>(p.src, at + c));
    }
  }
  {
    const float v3[3] = {warp_sum(sums.mid), warp_sum(sums.high), warp_sum(sums.low)};
    if (lane < 3) red[lane][warp] = lane == 0 ? v3[0] : lane == 1 ? v3[1] : v3[2];
  }
  // X's padding takes part in the products: zeros
  for (int i = threadIdx.x; i < blocks * SM_BLOCK / 16; i += SM_NT)
    reinterpret_cast<uint4*>(X)[i] = make_uint4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) {
    float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < SM_WARPS; ++w)
#pragma unroll
      for (int k = 0; k < 3; ++k) sum[k] += red[k][w];
    const double v3[3] = {sum[0], sum[1], sum[2]};
    factor = factor_of(v3, p.eps);
  }
  __syncthreads();
  // ---- first X
  {
    const float2 f = factor;
    auto place = [&](int i, int j) { return reinterpret_cast<__half*>(small_part(X, i, j / 8)) + j % 8; };
    for (int r = warp; r < p.M; r += SM_WARPS) {
      const long long at = base + (long long)r * p.N;
      if (vec) {
#pragma unroll 4
        for (int c = 4 * lane; c < p.N; c += 128) {
          const float4 u = u4_at<FROM, false>(p.src, at + c);
          const __half2 lo = __floats2half2_rn(u.x * f.x * f.y, u.y * f.x * f.y);
          const __half2 hi = __floats2half2_rn(u.z * f.x * f.y, u.w * f.x * f.y);
          if (tall) {
            *place(c, r) = __low2half(lo), *place(c + 1, r) = __high2half(lo);
            *place(c + 2, r) = __low2half(hi), *place(c + 3, r) = __high2half(hi);
          } else {
            __half2* dst = reinterpret_cast<__half2*>(place(r, c));
            dst[0] = lo, dst[1] = hi;
          }
        }
      } else {
#pragma unroll 4
        for (int c = lane; c < p.N; c += 32)
          *(tall ? place(c, r) : place(r, c)) = __float2half_rn(u_at<FROM, false>(p.src, at + c) * f.x * f.y);
      }
    }
  }
  const uint32_t tmem = tmem_slot, lanes = tmem + ((uint32_t)(q * 32) << 16);
  const uint32_t xa = smem_u32(X), da = smem_u32(D);
  uint32_t phase = 0;
  // what the threads have written is the tensor core's to read; its sums, once they are there, the threads'
  auto publish = [&]() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };
  auto summed = [&]() {
    const bool ok = wait_bounded(smem_u32(&bar), phase, &abort_flag, p);
    phase ^= 1u;
    tc_fence_after();
    return __syncthreads_and(ok) != 0;
  };
  const int ks = (m + 15) / 16;  // steps of 16 of K = m
  bool ok = true;
  for (int step = 0; step < p.steps && ok; ++step) {
    publish();
    if (warp == 0) {  // A = X X^T
      constexpr uint32_t ID = instr_desc(SM_ROWS, SM_ROWS, false, false, true);
      if (elect_one()) {
        for (int k = 0; k < (n + 15) / 16; ++k) {
          const uint64_t x = smem_desc(xa + k / 4 * SM_BLOCK + k % 4 * 32, 16, 1024);
          tc_mma(tmem, x, x, ID, k > 0);
        }
        tc_commit(smem_u32(&bar));
      }
      __syncwarp();
    }
    ok = summed();
    if (!ok) break;
    float v[32];
    const int col0 = part * 32;
    tmem_ld32(lanes + col0, v);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= INV;
    if (part == q) s_of[row] = take_diagonal(v, lane) * INV;
    small_store(D, row, col0, v);
    publish();
    if (warp == 0) {  // D D
      constexpr uint32_t ID = instr_desc(SM_ROWS, SM_ROWS, false, false, true);
      if (elect_one()) {
        for (int k = 0; k < ks; ++k) {
          const uint64_t d = smem_desc(da + k / 4 * SM_BLOCK + k % 4 * 32, 16, 1024);
          tc_mma(tmem, d, d, ID, k > 0);
        }
        tc_commit(smem_u32(&bar));
      }
      __syncwarp();
    }
    ok = summed();
    if (!ok) break;
    {
      uint4 mine[4];
      small_row(D, row, col0, mine);
      const __half2* h = reinterpret_cast<const __half2*>(mine);
      const float s_row = s_of[row], k0 = p.b + p.c * s_row, k1 = p.c * INV;
      tmem_ld32(lanes + col0, v);
      // D_ii is 0, so P_ii comes out 0 once (D D)_ii has been taken
      if (part == q) d_of[row] = p.a + (p.b + p.c * s_row) * s_row + k1 * INV * take_diagonal(v, lane);
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 sj = *reinterpret_cast<const float4*>(s_of + col0 + j);
        const float2 x0 = __half22float2(h[j / 2]), x1 = __half22float2(h[j / 2 + 1]);
        v[j] = fmaf(k1, v[j], fmaf(p.c, sj.x, k0) * x0.x);
        v[j + 1] = fmaf(k1, v[j + 1], fmaf(p.c, sj.y, k0) * x0.y);
        v[j + 2] = fmaf(k1, v[j + 2], fmaf(p.c, sj.z, k0) * x1.x);
        v[j + 3] = fmaf(k1, v[j + 3], fmaf(p.c, sj.w, k0) * x1.y);
      }
      small_store(D, row, col0, v);
    }
    publish();
    if (warp == 0) {  // P X, up to 256 columns an MMA
      if (elect_one()) {
        for (int c = 0; c < n; c += 256) {
          const uint32_t ID = instr_desc(SM_ROWS, min(256, (n - c + 15) / 16 * 16), false, true, true);
          for (int k = 0; k < ks; ++k)
            tc_mma(tmem + c, smem_desc(da + k / 4 * SM_BLOCK + k % 4 * 32, 16, 1024),
                   smem_desc(xa + c / 64 * SM_BLOCK + k * 16 * 128, SM_BLOCK, 1024), ID, k > 0);
        }
        tc_commit(smem_u32(&bar));
      }
      __syncwarp();
    }
    ok = summed();
    if (!ok) break;
    const float d_row = d_of[row];
    const bool last = step + 1 == p.steps;
    for (int c0 = part * 32; c0 < n; c0 += 32 * (SM_WARPS / 4)) {
      uint4 mine[4];
      small_row(X, row, c0, mine);
      const __half2* h = reinterpret_cast<const __half2*>(mine);
      tmem_ld32(lanes + c0, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 x = __half22float2(h[j]);
        // a column behind the last one has no sums
        v[2 * j] = c0 + 2 * j < n ? fmaf(d_row, x.x, v[2 * j] * INV) : 0.f;
        v[2 * j + 1] = c0 + 2 * j + 1 < n ? fmaf(d_row, x.y, v[2 * j + 1] * INV) : 0.f;
      }
      if (!last) {
        small_store(X, row, c0, v);
        continue;
      }
      float* wide = reinterpret_cast<float*>(D) + warp * 32 * STG;
      const Place place = tall ? Place{base, c0, q * 32, n, m} : Place{base, q * 32, c0, m, n};
      Old<KIND> old;
      old.load(p.r, place, lane);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 32; ++j) wide[tall ? j * STG + lane : lane * STG + j] = v[j] * INV;
      __syncwarp();
      put_tile<KIND>(p.r, place, old, wide, lane);
    }
  }
  if (!ok && warp == 0) {  // after a wait that gave up: nothing may still write the tensor memory that is freed
    const long long t0 = clock64();
    while (!mbar_try_wait(smem_u32(&bar), phase ^ 1u)) {
      if ((unsigned long long)(clock64() - t0) > DRAIN_LIMIT) { set_error(p.err, DEV_TIMEOUT); break; }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

// ------------------------------------------------------------------ host ----
inline long long up(long long v, long long k) { return (v + k - 1) / k * k; }

struct Layout {
  long long ldx, lda;
  size_t x[2], d, p, s, diag, part, factor, grams, bytes;
  int splits;
};
Layout layout(int E, int M, int N) {
  Layout l;
  const long long m = M < N ? M : N, n = M < N ? N : M;
  l.ldx = up(n, 64);
  l.lda = up(m, 64);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  for (int k = 0; k < 2; ++k) l.x[k] = take((size_t)E * m * l.ldx * 2);
  l.d = take((size_t)E * m * l.lda * 2);
  l.p = take((size_t)E * m * l.lda * 2);
  l.s = take((size_t)E * l.lda * 4);
  l.diag = take((size_t)E * l.lda * 4);
  l.part = take((size_t)E * PARTS * 3 * 8);
  l.factor = take((size_t)E * 8);
  // Few and long sums X X^T are shared out along K where at least three pairs of SMs can take one, eight blocks of
  // 64 or more each: 1 x 7168 x 384 281 -> 164 us.  With two to a sum the parts' way through memory eats the gain.
  const long long tiles = (long long)E * tiles_per_matrix<GRAM>((int)m, (int)n);
  const long long by_sms = sm_count() / 2 / tiles, by_k = up(n, BK) / BK / 8;
  l.splits = (int)(by_sms < by_k ? by_sms : by_k);
  if (l.splits < 3) l.splits = 1;
  l.grams = take(l.splits > 1 ? (size_t)l.splits * tiles * (2 * 64 * BM) * sizeof(float4) : 0);
  l.bytes = at;
  return l;
}

bool map_half(CUtensorMap* t, const void* base, long long inner, long long ld, long long rows, long long depth,
              int box_rows) {
  cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)depth};
  cuuint64_t str[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * rows * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  return make_map(t, base, 3, dims, str, box, CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
}

// Each kernel of the chain is set up while the one before it finishes, and waits for that one's end before it
// touches memory (griddepcontrol).
template <typename... P, typename... A>
int launch_next(void (*k)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, k, args...) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

template <int MODE, int KIND = ORTHO>
int launch_gemm(const CUtensorMap& a, const CUtensorMap& t, const CUtensorMap& a2, Params p, cudaStream_t s) {
  auto k = ns_gemm_kernel<MODE, KIND>;
  constexpr size_t smem = Cfg<MODE>::SMEM;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return MOE_ERR_CUDA;
  const long long whole = (long long)p.E * tiles_per_matrix<MODE>(p.m, p.n);
  long long pairs = sm_count() / 2;
  // Tiles of half the columns where each still finds a pair of its own.  Five steps, in us, with whole tiles and so:
  // 1 x 777 x 1001 178 and 139, 4 x 768 x 768 171 and 138, 1 x 512 x 512 143 and 114; with halves of up to as many
  // whole tiles as pairs 2 x 2048 x 1408 288 against 260, 3 x 1001 x 777 166 against 162.
  p.halves = MODE != PART && 2 * whole <= pairs;
  const long long tiles = (whole << p.halves) * (MODE == PART ? p.splits : 1);
  if (tiles < pairs) pairs = tiles;
  return launch_next(k, dim3((unsigned)(2 * pairs)), THREADS, smem, s, a, t, a2, p);
}

template <int FROM, int KIND>
int run(const Source& src, int E, int M, int N, int steps, float a, float b, float c, float eps, const Result& result,
        void* ws, cudaStream_t st) {
  const int m = M < N ? M : N, n = M < N ? N : M;
  if (m <= SM_ROWS && n <= SM_COLS) {
    SmallParams sp;
    sp.src = src, sp.M = M, sp.N = N, sp.steps = steps, sp.a = a, sp.b = b, sp.c = c, sp.eps = eps, sp.r = result;
    sp.err = device_error_word(), sp.wait_limit = g_wait_limit;
    auto k = ns_small_kernel<FROM, KIND>;
    static_assert(small_smem(SM_COLS) + 2048 <= 227 * 1024, "shared memory");
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)small_smem(SM_COLS)) != cudaSuccess)
      return MOE_ERR_CUDA;
    k<<<E, SM_NT, small_smem(n), st>>>(sp);
    return launch_status();
  }
  const Layout l = layout(E, M, N);
  uint8_t* base = static_cast<uint8_t*>(ws);
  double* part = reinterpret_cast<double*>(base + l.part);
  const long long size = (long long)M * N;
  // partial sums: enough blocks to fill the GPU, 4096 values or more to a block
  long long parts = up(8LL * sm_count(), E) / E;
  if (parts > up(size, 4096) / 4096) parts = up(size, 4096) / 4096;
  if (parts > PARTS) parts = PARTS;
  const long long span = up(up(size, parts) / parts, 4);
  const dim3 sum_grid((unsigned)parts, (unsigned)E);
  if (size % 4 == 0) ns_sum_kernel<FROM, true><<<sum_grid, SUM_NT, 0, st>>>(src, size, span, part);
  else ns_sum_kernel<FROM, false><<<sum_grid, SUM_NT, 0, st>>>(src, size, span, part);
  int r = launch_status();
  if (r != MOE_OK) return r;
  __half* x = reinterpret_cast<__half*>(base + l.x[0]);
  __half* x2 = reinterpret_cast<__half*>(base + l.x[1]);
  __half* D = reinterpret_cast<__half*>(base + l.d);
  __half* P = reinterpret_cast<__half*>(base + l.p);
  const dim3 load_grid((unsigned)((N + LT - 1) / LT), (unsigned)((M + LT - 1) / LT), (unsigned)E);
  float2* factor = reinterpret_cast<float2*>(base + l.factor);
  r = launch_next(ns_factor_kernel, dim3((unsigned)E), 32, 0, st, part, (int)parts, (double)eps, factor);
  if (r != MOE_OK) return r;
  r = launch_next(N % 4 == 0 ? ns_load_kernel<FROM, true> : ns_load_kernel<FROM, false>, load_grid, LOAD_NT, 0, st, src,
                  M, N, result.tall, l.ldx, factor, x);
  if (r != MOE_OK) return r;

  Params p;
  p.E = E, p.m = m, p.n = n, p.ldx = l.ldx, p.lda = l.lda;
  p.s = reinterpret_cast<float*>(base + l.s), p.d = reinterpret_cast<float*>(base + l.diag);
  p.a = a, p.b = b, p.c = c;
  p.r = result;
  p.err = device_error_word(), p.wait_limit = g_wait_limit;
  p.splits = l.splits, p.part = reinterpret_cast<float4*>(base + l.grams);
  // by 128 rows of 64 of K, and (_t) turned: by 64 of K
  CUtensorMap mx, mx_t, md, md_t, mp, mp_t;
  if (!map_half(&md, D, m, l.lda, m, E, 128) || !map_half(&md_t, D, m, l.lda, m, E, 64) ||
      !map_half(&mp, P, m, l.lda, m, E, 128) || !map_half(&mp_t, P, m, l.lda, m, E, 64))
    return MOE_ERR_CUDA;
  for (int k = 0; k < steps; ++k) {
    if (!map_half(&mx, x, n, l.ldx, m, E, 128) || !map_half(&mx_t, x, n, l.ldx, m, E, 64)) return MOE_ERR_CUDA;
    p.in = nullptr, p.out = D;
    if (l.splits > 1) {
      if ((r = launch_gemm<PART>(mx, mx_t, mx, p, st)) != MOE_OK) return r;
      const int per = tiles_per_matrix<GRAM>(m, n);
      r = launch_next(ns_join_kernel, dim3(64, 2, (unsigned)(E * per)), BM, 0, st, p, per);
    } else {
      r = launch_gemm<GRAM>(mx, mx_t, mx, p, st);
    }
    if (r != MOE_OK) return r;
    p.in = D, p.out = P;
    if ((r = launch_gemm<POLY>(md, md_t, md, p, st)) != MOE_OK) return r;
    p.in = x, p.out = x2;
    r = k + 1 < steps ? launch_gemm<APPLY>(mp, mx_t, mp_t, p, st)
                      : launch_gemm<FINAL, KIND>(mp, mx_t, mp_t, p, st);
    if (r != MOE_OK) return r;
    __half* t = x;
    x = x2;
    x2 = t;
  }
  return MOE_OK;
}

}  // namespace ns

size_t orthogonalize_ws_bytes(int E, int M, int N) { return ns::layout(E, M, N).bytes; }

int launch_orthogonalize(const void* x, int E, int M, int N, int dtype, int steps, float a, float b, float c, float eps,
                         void* out, void* ws, cudaStream_t s) {
  ns::Source src;
  src.x = x;
  ns::Result r;
  r.o = static_cast<bf16*>(out);
  r.tall = M > N, r.vec = N % 4 == 0;
  return dtype == MOE_BF16 ? ns::run<ns::FROM_BF16, ns::ORTHO>(src, E, M, N, steps, a, b, c, eps, r, ws, s)
                           : ns::run<ns::FROM_F32, ns::ORTHO>(src, E, M, N, steps, a, b, c, eps, r, ws, s);
}

int launch_muon_step(const void* w, const float* dw, const float* m, int E, int M, int N, int dtype, float beta,
                     bool nesterov, float lr, float decay, float scale, int steps, float a, float b, float c, float eps,
                     void* w_out, void* w_low, float* m_out, void* ws, cudaStream_t s) {
  ns::Source src;
  src.g = dw, src.m = m, src.m_out = m_out, src.beta = beta, src.nesterov = nesterov;
  ns::Result r;
  r.w = w, r.w_out = w_out, r.w_low = static_cast<bf16*>(w_low);
  r.keep = (float)(1.0 - (double)lr * decay), r.step = (float)((double)lr * scale);
  r.tall = M > N, r.vec = N % 4 == 0;
  return dtype == MOE_BF16 ? ns::run<ns::FROM_MOMENTUM, ns::MUON_BF16>(src, E, M, N, steps, a, b, c, eps, r, ws, s)
                           : ns::run<ns::FROM_MOMENTUM, ns::MUON_F32>(src, E, M, N, steps, a, b, c, eps, r, ws, s);
}

}  // namespace moe
