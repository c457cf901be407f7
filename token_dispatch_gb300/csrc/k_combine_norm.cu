// Combine fused with the RMS norms around the block, its gate and its residual
// scale (moe_combine_norm), and the backward of all of it.
//
// Both kernels stream rows: a CTA takes a token, a thread the same 16-byte columns
// of every row of it, and persistent CTAs walk the tokens.  What bounds them is the
// memory bus (K + 1 rows in and 2 out a token; K + 3 in and K + 1 out backward), so
// the work is keeping it busy across the row reductions: every thread copies its own
// columns of the rows to come into its own places of a ring in shared memory
// (cp.async, 16 bytes) and waits for its own copies alone.  No thread reads what
// another copied, so the ring needs no barrier; the only ones are those of the
// reductions, while the copies of the rows behind are under way.
//
// Of a copy's 6.77 TB/s: forward 8192 x 7168 bf16, K = 8: 195 us, 0.98; 8192 x 4096, K = 2
// without the norm after the block: 58 us, 0.86 (the launch and the first rows' latency are
// the rest); backward 16384 x 2048, K = 6: 183 us, 0.87; 8192 x 4096, K = 2: 110 us, 0.72,
// where the norms' instructions are more of a token (issue slots 61%, 16 warps to an SM).  Seven
// tokens forward take 8 us, most of them the launch.
#include <math.h>

#include <atomic>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int META = 16, AHEAD = 15;  // tokens whose row addresses and gates are at hand; how far ahead they are read
constexpr int MAXK = 16, MAXA = 3;    // rows of h, and of y, dxn and dy, of a token
constexpr int MAXW = 16;              // warps of a CTA

__device__ __forceinline__ void copy16(uint4* dst, const void* src, int bytes) {  // 16, or 0 for zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A thread's values in pairs: the packed fp32 operations of this architecture take two at
// a time, and instructions are what these kernels run short of first.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
template <typename T> struct Pairs;
template <> struct Pairs<bf16> {
  static constexpr int N = 4;
  __device__ __forceinline__ static void unpack(const uint4& q, float2* v) {
    const unsigned w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ static uint4 pack(const float2* v) {
    uint4 q;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[i].x, v[i].y);
    return q;
  }
};
template <> struct Pairs<float> {
  static constexpr int N = 2;
  __device__ __forceinline__ static void unpack(const uint4& q, float2* v) {
    v[0] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
    v[1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
  }
  __device__ __forceinline__ static uint4 pack(const float2* v) {
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
  }
};

// N pairs of a weight vector from column c on; 1 without one, 0 beside the row
template <int N> __device__ __forceinline__ void load_w(const float* w, int c, bool live, float2* v) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
    if (!live) f = make_float4(0.f, 0.f, 0.f, 0.f);
    else if (w) f = __ldg(reinterpret_cast<const float4*>(w + c + 2 * i));
    v[i] = make_float2(f.x, f.y);
    v[i + 1] = make_float2(f.z, f.w);
  }
}

// Sums of four values over the warp's lanes by halving: every step gives half of the
// values to half of the lanes.  Value i ends in the lanes with (lane >> 3) == i.
__device__ __forceinline__ float warp_sum4(const float (&v)[4]) {
  const int lane = threadIdx.x & 31;
  const bool a = lane & 16, b = lane & 8;
  float x = (a ? v[2] : v[0]) + __shfl_xor_sync(FULL, a ? v[0] : v[2], 16);
  float y = (a ? v[3] : v[1]) + __shfl_xor_sync(FULL, a ? v[1] : v[3], 16);
  x = (b ? y : x) + __shfl_xor_sync(FULL, b ? x : y, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
  return x;
}

__device__ __forceinline__ void team_sync(int id, int warps) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(warps * 32) : "memory");
}

// Sums over the CTA, in a fixed order and the same in every thread.  Two buffers in
// turn: one barrier for each call.
struct CtaSum {
  float buf[2][MAXW];
  __device__ __forceinline__ float run(float v, int turn) {
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    v = warp_sum(v);
    if (lane == 0) buf[turn & 1][threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < nw ? buf[turn & 1][lane] : 0.f;
#pragma unroll
    for (int o = MAXW / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return __shfl_sync(FULL, v, 0);
  }
};
// of up to eight values over the nw warps of a team, which barrier `id` holds together; buf [2][nw][8]
__device__ __forceinline__ void team_sum8(float (&v)[8], float* buf, int turn, int warp, int nw, int id) {
  const int lane = threadIdx.x & 31;
  buf += (turn & 1) * nw * 8;
  const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
  const float x = warp_sum4(lo), y = warp_sum4(hi);
  if ((lane & 7) == 0) {
    buf[warp * 8 + (lane >> 3)] = x;
    buf[warp * 8 + 4 + (lane >> 3)] = y;
  }
  team_sync(id, nw);
  float s = 0.f;  // value lane % 8 of warps lane / 8, + 4, + 8, + 12
  for (int w = lane >> 3; w < nw; w += 4) s += buf[w * 8 + (lane & 7)];
  s += __shfl_xor_sync(FULL, s, 8);
  s += __shfl_xor_sync(FULL, s, 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(FULL, s, i);
}

// gates and row numbers of the tokens: row -1 for an index outside [0, R)
struct MetaSource {
  const float* gate;
  const int32_t* dst_row;
  long long T, R;
  int K;
  unsigned* err;
  __device__ __forceinline__ void get(long long t, int k, int& row, float& g) const {
    row = -1;
    g = 0.f;
    if (t >= T || k >= K) return;
    const long long i = t * K + k;
    const long long r = dst_row ? __ldg(dst_row + i) : i;
    g = gate ? __ldg(gate + i) : 1.f;
    if (r >= 0 && r < R) row = (int)r;
    else set_error(err, DEV_BOUNDS);
  }
};

// the address to copy a row from; the lowest bit marks a row of zeros (rows are 16-byte aligned)
__device__ __forceinline__ unsigned long long row_address(const void* base, long long row, long long row_bytes) {
  return row < 0 ? (unsigned long long)base | 1ull : (unsigned long long)base + row * row_bytes;
}

struct FwdArgs {
  const void* h;
  MetaSource meta;
  const float* row_scale;
  const void* residual;
  const float *w_post, *res_scale, *w_next;
  float eps, inv_h;  // inv_h: 1 / H
  int T, H, K;
  void *y, *xn;
};

// X values of a row for each thread, S rows of ring, CTAS of at most MAXT threads to an SM.
// Order of a token's rows: its K rows of h, then residual.  ALL: h, residual, w_post and w_next
// are there, as in a block.
template <typename T, int X, int S, int MAXT, int CTAS, bool ALL>
__global__ void __launch_bounds__(MAXT, CTAS) combine_norm_kernel(const FwdArgs a) {
  extern __shared__ uint4 ring[];
  __shared__ unsigned long long src[META * (MAXK + 1)];
  __shared__ float2 gates[META][MAXK];  // twice, as a pair
  __shared__ CtaSum sum;
  constexpr int N = Pairs<T>::N, V = 2 * N, VPT = X / V, P = X / 2;
  constexpr bool HOLD_W = X <= 16;  // the weights fit in registers beside the row
  const int tid = threadIdx.x, NT = blockDim.x, nvec = a.H / V, K = a.K;
  const bool residual = ALL || a.residual, post = ALL || a.w_post, next = ALL || a.w_next;
  const int R = K + (residual ? 1 : 0);
  const long long row_bytes = (long long)a.H * sizeof(T);
  int offset[VPT];
  bool live[VPT];  // columns beside the row read as zeros
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = tid + v * NT;
    live[v] = i < nvec;
    offset[v] = live[v] ? 16 * i : 0;
  }
  auto note = [&](int j, int k, long long t, int row, float g) {  // row k of token t, which is at place j
    src[j * R + k] = k < K ? row_address(a.h, row, row_bytes) : row_address(a.residual, t < a.T ? t : -1, row_bytes);
    if (k < K) gates[j][k] = both(g);
  };
  for (int i = tid; i < AHEAD * R; i += NT) {
    const int k = i / AHEAD, j = i - k * AHEAD;
    const long long t = blockIdx.x + (long long)j * gridDim.x;
    int row = -1;
    float g = 0.f;
    a.meta.get(t, k, row, g);
    note(j, k, t, row, g);
  }
  float2 aw[HOLD_W ? P : 1], wn[HOLD_W ? P : 1];
  auto weights = [&](int v, float2* p, float2* n) {
    float2 r[N];
    load_w<N>(a.w_post, offset[v] / 16 * V, live[v], p);
    load_w<N>(a.res_scale, offset[v] / 16 * V, live[v], r);
    load_w<N>(a.w_next, offset[v] / 16 * V, live[v], n);
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = __fmul2_rn(p[i], r[i]);
  };
  if (HOLD_W) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) weights(v, aw + v * N, wn + v * N);
  }
  __syncthreads();

  const int step = VPT * NT, total = S * step, QN = META * R;
  int qn = 0, at = tid;  // the next row to be copied; the thread's place of the oldest row in the ring
  auto issue = [&](int place) {
    const unsigned long long p = src[qn];
    qn = qn + 1 == QN ? 0 : qn + 1;
    const char* from = reinterpret_cast<const char*>(p & ~1ull);
#pragma unroll
    for (int v = 0; v < VPT; ++v) copy16(ring + place + v * NT, from + offset[v], live[v] && !(p & 1) ? 16 : 0);
    copies_commit();
  };
  for (int i = 0; i < S; ++i) issue(tid + i * step);
  auto next_row = [&]() {  // the oldest row has been read: its place takes the next one
    issue(at);
    at += step;
    if (at >= total) at -= total;
  };

  int turn = 0, j = 0;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const long long t_ahead = t + (long long)AHEAD * gridDim.x;
    int m_row = -1;
    float m_gate = 0.f;
    if (tid < K) a.meta.get(t_ahead, tid, m_row, m_gate);
    float f = a.row_scale ? __ldg(a.row_scale + t) : 1.f;

    float2 z[P];
#pragma unroll
    for (int i = 0; i < P; ++i) z[i] = both(0.f);
    for (int k = 0; k < K; ++k) {
      const float2 g = gates[j][k];
      copies_wait<S - 1>();
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        float2 x[N];
        Pairs<T>::unpack(ring[at + v * NT], x);
#pragma unroll
        for (int i = 0; i < N; ++i) z[v * N + i] = __ffma2_rn(g, x[i], z[v * N + i]);
      }
      next_row();
    }
    if (post) {
      float2 s = both(0.f);
#pragma unroll
      for (int i = 0; i < P; ++i) s = __ffma2_rn(z[i], z[i], s);
      f *= rsqrtf(sum.run(s.x + s.y, turn++) * a.inv_h + a.eps);
    }
    if (residual) copies_wait<S - 1>();
    float2 s = both(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float2 x[N], p[N], n[N];
      if (HOLD_W) {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = aw[(v * N + i) % (HOLD_W ? P : 1)];
      } else {
        weights(v, p, n);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = both(0.f);
      if (residual) Pairs<T>::unpack(ring[at + v * NT], x);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[i] = __ffma2_rn(__fmul2_rn(both(f), z[v * N + i]), p[i], x[i]);
        z[v * N + i] = x[i];
        s = __ffma2_rn(x[i], x[i], s);
      }
      if ((ALL || a.y) && live[v])
        *reinterpret_cast<uint4*>(static_cast<char*>(a.y) + t * row_bytes + offset[v]) = Pairs<T>::pack(x);
    }
    if (residual) next_row();
    if (next) {
      const float q = rsqrtf(sum.run(s.x + s.y, turn++) * a.inv_h + a.eps);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        float2 x[N], p[N], n[N];
        if (HOLD_W) {
#pragma unroll
          for (int i = 0; i < N; ++i) n[i] = wn[(v * N + i) % (HOLD_W ? P : 1)];
        } else {
          weights(v, p, n);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = __fmul2_rn(__fmul2_rn(z[v * N + i], both(q)), n[i]);
        if (live[v])
          *reinterpret_cast<uint4*>(static_cast<char*>(a.xn) + t * row_bytes + offset[v]) = Pairs<T>::pack(x);
      }
    } else if (!post) {
      __syncthreads();  // a token takes one barrier at least: the addresses below are read behind it
    }
    if (tid < R) note(j == 0 ? META - 1 : j - 1, tid, t_ahead, m_row, m_gate);
    j = j + 1 == META ? 0 : j + 1;
  }
  copies_wait<0>();
}

struct BwdArgs {
  const void *dy, *dxn, *h, *y;
  MetaSource meta;
  const float *row_scale, *w_post, *res_scale, *w_next;
  float eps, inv_h;  // inv_h: 1 / H
  int T, H, K;
  void *d_res, *dh;
  float *d_gate, *d_scale;
  float* part;  // [gridDim.x][2][H]: this CTA's sums over its tokens of s D u and of dxn v
  int S;        // rows of ring of a team
  int teams;
};

// What a team keeps beside its ring, in 16-byte pieces from its place in shared memory on: the
// sums' shares [2][nw][8] of its nw warps, the gate gradients' [2][MAXK][nw + 1], the tokens'
// row addresses [META][R], gates [META][K] and row numbers [META][K].
__host__ __device__ constexpr int beside_dots(int nw) { return 4 * nw; }
__host__ __device__ constexpr int beside_src(int nw) { return beside_dots(nw) + 2 * MAXK * (nw + 1) / 4; }
__host__ __device__ constexpr int beside_gates(int nw, int R) { return beside_src(nw) + META * R / 2; }
__host__ __device__ constexpr int beside_rows(int nw, int R, int K) { return beside_gates(nw, R) + META * K / 2; }
__host__ __device__ constexpr int beside_all(int nw, int R, int K) { return beside_rows(nw, R, K) + META * K / 4; }

__device__ __forceinline__ void wait_all_but(int n) {  // 4, 2 or none
  if (n >= 4) copies_wait<4>();
  else if (n >= 2) copies_wait<2>();
  else copies_wait<0>();
}

// TEAMS: a CTA has several teams of threads, each with a ring and a barrier of its own, and each
// takes a token; they meet at the end, where the CTA's column sums are added.  Otherwise a
// CTA is one team.
//
// HOLD: a token's rows (y, dxn, dy, then h) stay in the ring from the sums to the
// gradients, and the ring holds S - R rows of the next tokens behind them.  Otherwise
// (rows too many or too wide for that) a token's rows pass through the ring twice, h and
// y, dxn, dy for the sums, then y, dxn, dy and h for the gradients; the second time
// they come from L2.
//
// One reduction serves both norms.  With D = dy + q (w_next dxn - q vm y):
//   <aw D, z> = <aw dy, z> + q <aw w_next dxn, z> - q^2 vm <aw y, z>,
// so its three products are summed along with y^2, w_next dxn y and z^2.
//
// NEXT, DY: dxn (with w_next and y) and dy are there.  Registers are what a thread runs out of
// (128, where 170 would take a quarter fewer instructions): the two are no arguments, and
// w_next is read again for each token, from L1 (8192 x 4096, K = 2: 123 us to 110 for both; in
// shared memory 106, but without the room for the rows of K = 8: 256 us instead of 230).
template <typename T, int X, bool HOLD, bool TEAMS, bool NEXT, bool DY>
__global__ void __launch_bounds__(512) combine_norm_bwd_kernel(const BwdArgs a) {
  extern __shared__ uint4 smem[];
  asm volatile("griddepcontrol.launch_dependents;");  // the column sums may get ready
  constexpr int N = Pairs<T>::N, V = 2 * N, VPT = X / V, P = X / 2;
  constexpr bool HOLD_W = X <= 16;
  const int teams = TEAMS ? a.teams : 1;
  const int NT = blockDim.x / teams, team = TEAMS ? threadIdx.x / NT : 0, tid = threadIdx.x - team * NT;
  const int nvec = a.H / V, K = a.K, S = a.S;
  const int lane = tid & 31, warp = tid >> 5, nw = NT >> 5, bar = TEAMS ? 1 + team : 0;
  uint4* ring = smem + team * S * VPT * NT;
  // T < 2^31: a token's number, and those of the ones ahead, fit in 32 bits without sign
  const unsigned first = blockIdx.x * teams + team, stride = gridDim.x * teams;
  constexpr int A = (NEXT ? 2 : 0) + (DY ? 1 : 0);
  const int R = HOLD ? A + K : 2 * (A + K);
  const int beside = teams * S * VPT * NT + team * beside_all(nw, R, K);
  unsigned long long* src = reinterpret_cast<unsigned long long*>(smem + beside + beside_src(nw));
  float2* gates = reinterpret_cast<float2*>(smem + beside + beside_gates(nw, R));  // twice, as a pair
  int* rows = reinterpret_cast<int*>(smem + beside + beside_rows(nw, R, K));
  float* sums = reinterpret_cast<float*>(smem + beside);
  float* dots = reinterpret_cast<float*>(smem + beside + beside_dots(nw));
  const long long row_bytes = (long long)a.H * sizeof(T);
  int offset[VPT];
  bool live[VPT];  // columns beside the row read as zeros
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = tid + v * NT;
    live[v] = i < nvec;
    offset[v] = live[v] ? 16 * i : 0;
  }
  auto note = [&](int j, int k, unsigned t, int row, float g) {  // row k (of h, then y, dxn, dy) of token t, at place j
    unsigned long long p;
    if (k < K) {
      p = row_address(a.h, row, row_bytes);
      gates[j * K + k] = both(g);
      rows[j * K + k] = row;
    } else {
      const int x = k - K;
      p = row_address(NEXT && x < 2 ? (x == 0 ? a.y : a.dxn) : a.dy, t < (unsigned)a.T ? (long long)t : -1ll, row_bytes);
    }
    unsigned long long* q = src + j * R;
    if (HOLD) {
      q[k < K ? A + k : k - K] = p;
    } else {
      q[k] = p;
      q[K + A + (k < K ? A + k : k - K)] = p;
    }
  };
  for (int i = tid; i < AHEAD * (K + A); i += NT) {
    const int k = i / AHEAD, j = i - k * AHEAD;
    const unsigned t = first + j * stride;
    int row = -1;
    float g = 0.f;
    a.meta.get(t, k, row, g);
    note(j, k, t, row, g);
  }
  float2 aw[HOLD_W ? P : 1];
  auto post_weights = [&](int v, float2* p) {
    float2 r[N];
    load_w<N>(a.w_post, offset[v] / 16 * V, live[v], p);
    load_w<N>(a.res_scale, offset[v] / 16 * V, live[v], r);
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = __fmul2_rn(p[i], r[i]);
  };
  if (HOLD_W) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) post_weights(v, aw + v * N);
  }
  auto weights_of = [&](int v, float2* p, float2* n) {
    if (NEXT) load_w<N>(a.w_next, offset[v] / 16 * V, true, n);  // beside the row dxn is 0
    if (HOLD_W) {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = aw[(v * N + i) % (HOLD_W ? P : 1)];
    } else {
      post_weights(v, p);
    }
  };
  team_sync(bar, nw);

  const int step = VPT * NT, total = S * step, QN = META * R;
  int qn = 0, at = tid;  // the next row to be copied; the thread's place of the oldest row in the ring
  auto issue = [&](int place) {
    const unsigned long long p = src[qn];
    qn = qn + 1 == QN ? 0 : qn + 1;
    const char* from = reinterpret_cast<const char*>(p & ~1ull);
#pragma unroll
    for (int v = 0; v < VPT; ++v) copy16(ring + place + v * NT, from + offset[v], live[v] && !(p & 1) ? 16 : 0);
    copies_commit();
  };
  for (int i = 0; i < S; ++i) issue(tid + i * step);
  auto next_row = [&]() {
    issue(at);
    at += step;
    if (at >= total) at -= total;
  };
  auto behind = [&](int rows_on) {  // the thread's place of the row that many behind the oldest
    const int p = at + rows_on * step;
    return p >= total ? p - total : p;
  };

  float2 Q[P], M[P];
#pragma unroll
  for (int i = 0; i < P; ++i) Q[i] = M[i] = both(0.f);
  int turn = 0, j = 0;
  auto write_gates = [&](unsigned t, int b) {  // of token t, from the shares in `dots`
    if (a.d_gate && tid < K) {
      float d = 0.f;
      for (int w = 0; w < nw; ++w) d += dots[(b * MAXK + tid) * (nw + 1) + w];
      a.d_gate[(long long)t * K + tid] = d;
    }
  };

  for (unsigned t = first; t < (unsigned)a.T; t += stride) {
    const unsigned t_ahead = t + AHEAD * stride;
    int m_row = -1;
    float m_gate = 0.f;
    if (tid < K) a.meta.get(t_ahead, tid, m_row, m_gate);
    const float rs = a.row_scale ? __ldg(a.row_scale + t) : 1.f;

    float2 z[P];
#pragma unroll
    for (int i = 0; i < P; ++i) z[i] = both(0.f);
    if (HOLD) wait_all_but(S - R);
    int place = HOLD ? behind(A) : at;
    for (int k = 0; k < K; ++k) {
      const float2 g = gates[j * K + k];
      if (!HOLD) copies_wait<2>();  // three rows are on their way: the oldest is here
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        float2 x[N];
        Pairs<T>::unpack(ring[place + v * NT], x);
#pragma unroll
        for (int i = 0; i < N; ++i) z[v * N + i] = __ffma2_rn(g, x[i], z[v * N + i]);
      }
      if (!HOLD) next_row();
      place += step;
      if (place >= total) place -= total;
    }
    if (!HOLD) copies_wait<0>();
    const int at_y = at, at_x = behind(1), at_d = behind(A - 1);
    float2 s2[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) s2[i] = both(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float2 p[N], n[N], x[N], y[N];
      weights_of(v, p, n);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        p[i] = __fmul2_rn(p[i], z[v * N + i]);
        s2[2] = __ffma2_rn(z[v * N + i], z[v * N + i], s2[2]);
      }
      if (NEXT) {
        Pairs<T>::unpack(ring[at_y + v * NT], y);
        Pairs<T>::unpack(ring[at_x + v * NT], x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float2 e = __fmul2_rn(n[i], x[i]);
          s2[0] = __ffma2_rn(y[i], y[i], s2[0]);
          s2[1] = __ffma2_rn(e, y[i], s2[1]);
          s2[4] = __ffma2_rn(p[i], e, s2[4]);
          s2[5] = __ffma2_rn(p[i], y[i], s2[5]);
        }
      }
      if (DY) {
        Pairs<T>::unpack(ring[at_d + v * NT], x);
#pragma unroll
        for (int i = 0; i < N; ++i) s2[3] = __ffma2_rn(p[i], x[i], s2[3]);
      }
    }
    if (!HOLD)
      for (int i = 0; i < A; ++i) next_row();
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 6; ++i) s[i] = s2[i].x + s2[i].y;
    team_sum8(s, sums, turn++, warp, nw, bar);
    if (t != first) write_gates(t - stride, (j & 1) ^ 1);
    const float q = NEXT ? rsqrtf(s[0] * a.inv_h + a.eps) : 0.f, vm = s[1] * q * a.inv_h;
    const float r = a.w_post ? rsqrtf(s[2] * a.inv_h + a.eps) : 1.f;
    const float sd = r * (s[3] + q * (s[4] - q * vm * s[5]));
    const float um = a.w_post ? rs * sd * a.inv_h : 0.f;
    const float2 rsr = both(rs * r), zu = both(-um * r * r), q2 = both(q), qvm = both(-q * vm);
    if (tid == 0 && a.d_scale) a.d_scale[t] = sd;

    if (!HOLD) copies_wait<0>();
    const int by_x = HOLD ? at_x : behind(1), by_d = HOLD ? at_d : behind(A - 1);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float2 p[N], n[N], d[N];
      weights_of(v, p, n);
      if (DY) {
        Pairs<T>::unpack(ring[by_d + v * NT], d);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = both(0.f);
      }
      if (NEXT) {
        float2 x[N], y[N];
        Pairs<T>::unpack(ring[at + v * NT], y);
        Pairs<T>::unpack(ring[by_x + v * NT], x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float2 u = __fmul2_rn(y[i], q2);
          d[i] = __ffma2_rn(u, qvm, __ffma2_rn(q2, __fmul2_rn(x[i], n[i]), d[i]));
          M[v * N + i] = __ffma2_rn(x[i], u, M[v * N + i]);
        }
      }
      if (a.d_res && live[v])
        *reinterpret_cast<uint4*>(static_cast<char*>(a.d_res) + t * row_bytes + offset[v]) = Pairs<T>::pack(d);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 u = __fmul2_rn(z[v * N + i], rsr);
        Q[v * N + i] = __ffma2_rn(d[i], u, Q[v * N + i]);
        z[v * N + i] = __ffma2_rn(rsr, __fmul2_rn(d[i], p[i]), __fmul2_rn(z[v * N + i], zu));  // dz
      }
    }
    for (int i = 0; i < A; ++i) next_row();
    for (int k0 = 0; k0 < K; k0 += 4) {
      float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const int k = k0 + kk;
        if (k >= K) break;
        const float2 g = gates[j * K + k];
        const int row = rows[j * K + k];
        if (!HOLD) copies_wait<2>();
        float2 c = both(0.f);
        char* out = static_cast<char*>(a.dh) + row * row_bytes;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          float2 x[N];
          Pairs<T>::unpack(ring[at + v * NT], x);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            c = __ffma2_rn(z[v * N + i], x[i], c);
            x[i] = __fmul2_rn(g, z[v * N + i]);
          }
          if (a.dh && row >= 0 && live[v]) *reinterpret_cast<uint4*>(out + offset[v]) = Pairs<T>::pack(x);
        }
        dot[kk] = c.x + c.y;
        next_row();
      }
      if (a.d_gate) {
        const float d = warp_sum4(dot);
        if ((lane & 7) == 0) dots[((j & 1) * MAXK + k0 + (lane >> 3)) * (nw + 1) + warp] = d;
      }
    }
    if (tid < K + A) note(j == 0 ? META - 1 : j - 1, tid, t_ahead, m_row, m_gate);
    j = j + 1 == META ? 0 : j + 1;
  }
  copies_wait<0>();
  team_sync(bar, nw);
  if (first < (unsigned)a.T) write_gates(first + ((unsigned)a.T - 1 - first) / stride * stride, (j & 1) ^ 1);
  if (!a.part) return;
  // a team alone writes its sums; several put them into their rings (2 H floats, at most four
  // rows of bf16) and the CTA adds them in the order of the teams
  float* part = a.part + (size_t)blockIdx.x * 2 * a.H;
  float* to = !TEAMS ? part : reinterpret_cast<float*>(ring);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (!live[v]) continue;
    const int c = offset[v] / 16 * V;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 *e = Q + v * N + i, *f = M + v * N + i;
      *reinterpret_cast<float4*>(to + c + 2 * i) = make_float4(e[0].x, e[0].y, e[1].x, e[1].y);
      *reinterpret_cast<float4*>(to + a.H + c + 2 * i) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    }
  }
  if (!TEAMS) return;
  __syncthreads();
  for (int i = threadIdx.x; i < a.H / 2; i += blockDim.x) {
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < teams; ++w) {
      const float4 x = reinterpret_cast<const float4*>(smem + (size_t)w * S * VPT * NT)[i];
      sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
    }
    reinterpret_cast<float4*>(part)[i] = sum;
  }
}

// The column sums: a CTA takes 32 columns of [2][H], its 32 warps the parts w, w + 32, ...
// in order; the warps' sums are added in warp order and multiplied by their column factors.
// Latency bounds it; it is set up while the kernel before it runs (16384 x 2048, K = 6: 186 us
// to 183 for both; 1001 x 1000 fp32: 22.5 to 20).
__global__ void __launch_bounds__(1024)
column_sums_kernel(const float* part, int parts, int H, const float* __restrict__ w_post,
                   const float* __restrict__ res_scale, float* dw_post, float* d_res_scale, float* dw_next) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the launch before it has ended and its writes are visible
  float acc = 0.f;
  if (i < 2 * H) {
#pragma unroll 8
    for (int p = w; p < parts; p += 32) acc += part[(size_t)p * 2 * H + i];
  }
  red[w][lane] = acc;
  __syncthreads();
  if (w > 0 || i >= 2 * H) return;
#pragma unroll
  for (int k = 1; k < 32; ++k) acc += red[k][lane];
  if (i >= H) {
    if (dw_next) dw_next[i - H] = acc;
  } else {
    if (dw_post) dw_post[i] = acc * (res_scale ? res_scale[i] : 1.f);
    if (d_res_scale) d_res_scale[i] = acc * (w_post ? w_post[i] : 1.f);
  }
}

constexpr int RING_BYTES = 200 * 1024;  // of a CTA with one team; its 227 KB also hold what is beside the ring
constexpr int SM_BYTES = 227 * 1024;

int threads_for(int nvec, int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; }

// CTAs of a persistent grid: as many as fit, at most `cap` to an SM, at most one a token.
// The answer to the last question is kept for each kernel (asking the runtime takes 0.7 us):
// one word holds device, threads, shared memory and CTAs to an SM.
template <typename F> int persistent_grid(F kernel, std::atomic<unsigned long long>& known, int threads, int smem,
                                          int limit, int cap, int T, int* grid) {
  int dev = 0, per_sm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const unsigned long long ask = (unsigned long long)(dev + 1) << 48 | (unsigned long long)threads << 32 |
                                 (unsigned long long)smem << 8;
  const unsigned long long k = known.load(std::memory_order_relaxed);
  if ((k & ~0xffull) == ask) {
    per_sm = (int)(k & 0xff);
  } else {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, limit) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1)
      return MOE_ERR_CUDA;
    known.store(ask | (unsigned)per_sm, std::memory_order_relaxed);
  }
  const long long n = (long long)sm_count() * (per_sm < cap ? per_sm : cap);
  *grid = (int)(T < n ? T : n);
  return MOE_OK;
}

template <typename T, int X, int S, int MAXT, int CTAS, bool ALL> int fwd_a(const FwdArgs& a, cudaStream_t s) {
  constexpr int VPT = X / Vec16<T>::N;
  const int threads = threads_for(a.H / Vec16<T>::N, VPT), smem = S * VPT * threads * 16;
  int grid = 0;
  static std::atomic<unsigned long long> known{0};
  const int st = persistent_grid(combine_norm_kernel<T, X, S, MAXT, CTAS, ALL>, known, threads, smem, RING_BYTES, 32, a.T,
                                 &grid);
  if (st != MOE_OK) return st;
  combine_norm_kernel<T, X, S, MAXT, CTAS, ALL><<<grid, threads, smem, s>>>(a);
  return launch_status();
}

// A block's whole call has instances of its own: instructions count where K is small (16384 x 512,
// K = 1 to 3: 17 to 19 us instead of 19 to 23; 16384 x 1024: 26 to 37 instead of 32 to 38; 8192 x
// 7168, K = 2: 110 instead of 114, K = 8 the same).
template <typename T, int X, int S, int MAXT, int CTAS> int fwd_v(const FwdArgs& a, cudaStream_t s) {
  return a.K > 0 && a.residual && a.w_post && a.w_next ? fwd_a<T, X, S, MAXT, CTAS, true>(a, s)
                                                       : fwd_a<T, X, S, MAXT, CTAS, false>(a, s);
}

// 16 values a thread up to H = 8192, where the registers still hold weights beside the row, 32
// beyond (32 for 8192 x 4096, K = 2: 70 us instead of 60; 4096 x 8192: 72 instead of 66).  Rows
// of up to 8 KB: three CTAs or more to an SM, 8 rows of ring each, so that some stream while
// others reduce (with 12 rows and as many CTAs as then fit, 16384 x 4096, K = 1: 111 us instead of
// 98, 11650 x 2880, K = 2: 78 instead of 59; K = 8 is within 3% either way); wider rows: one CTA
// with 12 rows of up to 16 KB, 6 of up to 32 KB, 3 beyond.
template <typename T> int fwd_t(const FwdArgs& a, cudaStream_t s) {
  constexpr bool WIDE = sizeof(T) == 4;
  const int row = a.H * (int)sizeof(T);
  if (row <= 8192 && a.H <= 4096) return fwd_v<T, 16, 8, 256, 3>(a, s);
  if (row <= 16384 && a.H <= 8192) return fwd_v<T, 16, 12, 512, 1>(a, s);
  if constexpr (WIDE) {
    if (a.H <= 8192) return fwd_v<T, 16, 6, 512, 1>(a, s);
    return fwd_v<T, 32, 3, 512, 1>(a, s);
  } else {
    return fwd_v<T, 32, 6, 512, 1>(a, s);
  }
}

// column sums kept per CTA: at most this many CTAs to an SM
int bwd_ctas_per_sm(int H) { return H >= 8192 ? 2 : H >= 1024 ? 16384 / H : 16; }

int bwd_rows(const BwdArgs& a) { return a.K + (a.w_next ? 2 : 0) + (a.dy ? 1 : 0); }

// 128 registers leave room for 512 threads to an SM
constexpr int BWD_THREADS = 512, MAX_TEAMS = 8;

template <typename T, int X, bool HOLD, bool TEAMS, bool NEXT, bool DY>
int bwd_n(BwdArgs& a, int threads, int smem, int* grid, cudaStream_t s) {
  static std::atomic<unsigned long long> known{0};
  const int tokens = (a.T + a.teams - 1) / a.teams;
  const int st = persistent_grid(combine_norm_bwd_kernel<T, X, HOLD, TEAMS, NEXT, DY>, known, threads, smem, SM_BYTES,
                                 bwd_ctas_per_sm(a.H), tokens, grid);
  if (st != MOE_OK) return st;
  combine_norm_bwd_kernel<T, X, HOLD, TEAMS, NEXT, DY><<<*grid, threads, smem, s>>>(a);
  return launch_status();
}

template <typename T, int X, bool HOLD, bool TEAMS> int bwd_v(BwdArgs& a, int threads, int smem, int* grid, cudaStream_t s) {
  if (!a.w_next) return bwd_n<T, X, HOLD, TEAMS, false, true>(a, threads, smem, grid, s);
  return a.dy ? bwd_n<T, X, HOLD, TEAMS, true, true>(a, threads, smem, grid, s)
              : bwd_n<T, X, HOLD, TEAMS, true, false>(a, threads, smem, grid, s);
}

template <typename T, int X, bool HOLD> int bwd_x(BwdArgs& a, int* grid, cudaStream_t s) {
  constexpr int VPT = X / Vec16<T>::N;
  const int threads = threads_for(a.H / Vec16<T>::N, VPT), row = VPT * threads * 16, R = bwd_rows(a);
  const int beside = 16 * beside_all(threads / 32, HOLD ? R : 2 * R, a.K);
  a.teams = 1;
  a.S = 3;
  if constexpr (HOLD) {
    // As many teams as there are tokens to an SM, where the GPU holds them all at once: a CTA's
    // one set of column sums instead of one for each token (1001 tokens of 1000 fp32 columns:
    // 24.5 us without, 21 with, both before the second launch overlapped the first).  A ring
    // then holds a token's rows, and the team's 2 H sums.
    const int per_sm = (a.T + sm_count() - 1) / sm_count(), sums = (8 * a.H + row - 1) / row, S = R > sums ? R : sums;
    if (per_sm > 1 && per_sm <= MAX_TEAMS && per_sm * threads <= BWD_THREADS && per_sm * (S * row + beside) <= SM_BYTES) {
      a.teams = per_sm;
      a.S = S;
      return bwd_v<T, X, HOLD, true>(a, a.teams * threads, a.teams * (S * row + beside), grid, s);
    }
    // Otherwise CTAs, as many as the registers have room for, and behind a token's own rows 4, 2 or
    // none of the next ones, what shared memory has room for (with 8, w_next would lose its place
    // in L1: 4096 x 7168, K = 2: 119 us instead of 113).  A quarter of the CTAs go for 4 rows where
    // that is enough (13104 x 2048, K = 8: 3 CTAs 179 us, 4 with 2 rows 194), not more (8192 x
    // 4096, K = 8: 2 CTAs with 2 rows 225 us, one with 4 264).
    auto ahead = [&](int ctas) {
      const int room = (SM_BYTES / ctas - beside - 1024) / row - R;
      return room >= 4 ? 4 : room >= 2 ? 2 : room >= 0 ? 0 : -1;
    };
    int ctas = BWD_THREADS / threads;
    while (ctas > 1 && ahead(ctas) < 4 && 4 * (ctas - 1) * threads >= 3 * BWD_THREADS) --ctas;
    if (ahead(ctas) < 4) ctas = BWD_THREADS / threads;
    while (ctas > 1 && ahead(ctas) < 0) --ctas;
    a.S = R + ahead(ctas);
  }
  return bwd_v<T, X, HOLD, false>(a, threads, a.S * row + beside, grid, s);
}

// 16 values a thread up to H = 8192, 32 beyond (32 for 16384 x 2048, K = 6: 291 us instead of
// 186); a token's rows are held where they fit (read twice instead: 226 us;
// 4096 x 7168, K = 8: 290 instead of 214)
template <typename T> int bwd_t(BwdArgs& a, int* grid, cudaStream_t s) {
  constexpr int VPT = 16 / Vec16<T>::N;
  if (a.H > 8192) return bwd_x<T, 32, false>(a, grid, s);
  const long long row = VPT * threads_for(a.H / Vec16<T>::N, VPT) * 16;
  return bwd_rows(a) * row <= RING_BYTES ? bwd_x<T, 16, true>(a, grid, s) : bwd_x<T, 16, false>(a, grid, s);
}

long long bwd_max_ctas(int T, int H) {
  const long long cap = (long long)sm_count() * bwd_ctas_per_sm(H);
  return T < cap ? (T > 0 ? T : 1) : cap;
}

}  // namespace

size_t combine_norm_bwd_ws_bytes(int T, int H) { return (size_t)bwd_max_ctas(T, H) * 2 * H * 4; }

int launch_combine_norm(const void* h, const float* gate, const int32_t* dst_row, const float* row_scale,
                        const void* residual, const float* w_post, const float* res_scale, const float* w_next,
                        float eps, int T, int H, int K, int dtype, void* y, void* xn, cudaStream_t s) {
  if (T == 0) return MOE_OK;
  const FwdArgs a{h, MetaSource{gate, dst_row, T, (long long)T * K, K, device_error_word()}, row_scale, residual,
                  w_post, res_scale, w_next, eps, 1.f / H, T, H, K, y, xn};
  return dtype == MOE_BF16 ? fwd_t<bf16>(a, s) : fwd_t<float>(a, s);
}

int launch_combine_norm_bwd(const void* dy, const void* dxn, const void* h, const float* gate, const int32_t* dst_row,
                            const float* row_scale, const void* y, const float* w_post, const float* res_scale,
                            const float* w_next, float eps, int T, int H, int K, int dtype, void* d_res, void* dh,
                            float* d_gate, float* d_scale, float* dw_post, float* d_res_scale, float* dw_next, void* ws,
                            cudaStream_t s) {
  const bool sums = dw_post || d_res_scale || dw_next;
  if (T == 0) {
    for (float* p : {dw_post, d_res_scale, dw_next})
      if (p && cudaMemsetAsync(p, 0, (size_t)H * 4, s) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  BwdArgs a{dy, dxn, h, y, MetaSource{gate, dst_row, T, (long long)T * K, K, device_error_word()}, row_scale, w_post,
            res_scale, w_next, eps, 1.f / H, T, H, K, d_res, dh, d_gate, d_scale, sums ? static_cast<float*>(ws) : nullptr, 0, 1};
  int grid = 0;
  const int st = dtype == MOE_BF16 ? bwd_t<bf16>(a, &grid, s) : bwd_t<float>(a, &grid, s);
  if (st != MOE_OK || !sums) return st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3((2 * H + 31) / 32);
  config.blockDim = dim3(1024);
  config.stream = s;
  config.attrs = &early;
  config.numAttrs = 1;
  const float* part = a.part;
  if (cudaLaunchKernelEx(&config, column_sums_kernel, part, grid, H, w_post, res_scale, dw_post, d_res_scale, dw_next) !=
      cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace moe
