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
#include <math.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int META = 16, AHEAD = 15;  // tokens whose row numbers and gates are at hand; how far ahead they are read
constexpr int MAXK = 16, MAXW = 32;

__device__ __forceinline__ void copy16(uint4* dst, const void* src, bool live) {  // zeros where not live
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T> __device__ __forceinline__ void unpack(const uint4& q, float* v) { Vec16<T>::load_raw_unpack(q, v); }

// 4 or 8 floats of a weight vector from column c on, 1 without one
template <int V> __device__ __forceinline__ void load_w(const float* w, int c, float* v) {
#pragma unroll
  for (int j = 0; j < V; j += 4) {
    const float4 f = w ? __ldg(reinterpret_cast<const float4*>(w + c + j)) : make_float4(1.f, 1.f, 1.f, 1.f);
    v[j] = f.x; v[j + 1] = f.y; v[j + 2] = f.z; v[j + 3] = f.w;
  }
}

// Sums over the CTA, in a fixed order and the same in every thread.  Two buffers in
// turn: one barrier for each call.
template <int N> struct CtaSum {
  float buf[2][N][MAXW];
  __device__ __forceinline__ void run(float (&v)[N], int turn) {
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if (nw == 1) {
      __syncthreads();
      return;
    }
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[turn & 1][i][threadIdx.x >> 5] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < nw ? buf[turn & 1][i][lane] : 0.f);
  }
};

// row numbers and gates of the tokens to come; row -1 for an index outside [0, R)
struct Meta {
  int row[META][MAXK];
  float gate[META][MAXK];
};
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

struct FwdArgs {
  const void* h;
  MetaSource meta;
  const float* row_scale;
  const void* residual;
  const float *w_post, *res_scale, *w_next;
  float eps;
  int T, H, K;
  void *y, *xn;
};

// VPT vectors of a row for each thread, S rows of ring.  Order of a token's rows: its
// K rows of h, then residual.
template <typename T, int VPT, int S>
__global__ void __launch_bounds__(896) combine_norm_kernel(const FwdArgs a) {
  extern __shared__ uint4 ring[];
  __shared__ Meta meta;
  __shared__ CtaSum<1> sum;
  constexpr int V = Vec16<T>::N, X = VPT * V;
  constexpr bool HOLD_W = X <= 8;  // the weights fit in registers beside the row
  const int tid = threadIdx.x, NT = blockDim.x, nvec = a.H / V, K = a.K, R = K + (a.residual ? 1 : 0);
  const uint4* h = static_cast<const uint4*>(a.h);
  const uint4* residual = static_cast<const uint4*>(a.residual);
  for (int i = tid; i < AHEAD * MAXK; i += NT) {
    const int j = i / MAXK, k = i % MAXK;
    a.meta.get(blockIdx.x + (long long)j * gridDim.x, k, meta.row[j][k], meta.gate[j][k]);
  }
  float aw[HOLD_W ? X : 1], wn[HOLD_W ? X : 1];
  auto weights = [&](int v, float* p, float* n) {
    const int c = (tid + v * NT) * V;
    float r[V];
    load_w<V>(c < a.H ? a.w_post : nullptr, c, p);
    load_w<V>(c < a.H ? a.res_scale : nullptr, c, r);
    load_w<V>(c < a.H ? a.w_next : nullptr, c, n);
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] *= r[j];
  };
  if (HOLD_W) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) weights(v, aw + v * V, wn + v * V);
  }
  __syncthreads();

  // the next row to be copied: row qk of the CTA's qj-th token, into place qs
  int qj = 0, qk = 0, qs = 0;
  long long qt = blockIdx.x;
  auto issue = [&]() {
    if (qt < a.T) {
      const int row = qk < K ? meta.row[qj % META][qk] : 0;
      const uint4* src = qk < K ? h + (long long)max(row, 0) * nvec : residual + qt * nvec;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int i = tid + v * NT;
        if (i < nvec) copy16(ring + (qs * VPT + v) * NT + tid, src + i, row >= 0);
      }
      if (++qk == R) {
        qk = 0;
        ++qj;
        qt += gridDim.x;
      }
    }
    copies_commit();
    qs = qs + 1 == S ? 0 : qs + 1;
  };
#pragma unroll
  for (int i = 0; i < S; ++i) issue();

  int slot = 0, turn = 0, j = 0;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x, ++j) {
    int m_row = -1;
    float m_gate = 0.f;
    if (tid < MAXK) a.meta.get(t + (long long)AHEAD * gridDim.x, tid, m_row, m_gate);
    const float rs = a.row_scale ? __ldg(a.row_scale + t) : 1.f;

    float z[X];
#pragma unroll
    for (int i = 0; i < X; ++i) z[i] = 0.f;
    for (int k = 0; k < K; ++k) {
      const float g = meta.gate[j % META][k];
      copies_wait<S - 1>();
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        if (tid + v * NT >= nvec) continue;
        float x[V];
        unpack<T>(ring[(slot * VPT + v) * NT + tid], x);
#pragma unroll
        for (int i = 0; i < V; ++i) z[v * V + i] = fmaf(g, x[i], z[v * V + i]);
      }
      issue();
      slot = slot + 1 == S ? 0 : slot + 1;
    }
    float s[1];
    float f = rs;
    if (a.w_post) {
      s[0] = 0.f;
#pragma unroll
      for (int i = 0; i < X; ++i) s[0] = fmaf(z[i], z[i], s[0]);
      sum.run(s, turn++);
      f *= 1.f / sqrtf(s[0] / a.H + a.eps);
    }
    if (residual) copies_wait<S - 1>();
    s[0] = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (tid + v * NT >= nvec) continue;
      float x[V], p[V], n[V];
      if (HOLD_W) {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = aw[(v * V + i) % (HOLD_W ? X : 1)];
      } else {
        weights(v, p, n);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = 0.f;
      if (residual) unpack<T>(ring[(slot * VPT + v) * NT + tid], x);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[i] = fmaf(f * z[v * V + i], p[i], x[i]);
        z[v * V + i] = x[i];
        s[0] = fmaf(x[i], x[i], s[0]);
      }
      if (a.y) Vec16<T>::store(static_cast<T*>(a.y) + t * a.H + (long long)(tid + v * NT) * V, x);
    }
    if (residual) {
      issue();
      slot = slot + 1 == S ? 0 : slot + 1;
    }
    if (a.w_next) {
      sum.run(s, turn++);
      const float q = 1.f / sqrtf(s[0] / a.H + a.eps);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        if (tid + v * NT >= nvec) continue;
        float x[V], p[V], n[V];
        if (HOLD_W) {
#pragma unroll
          for (int i = 0; i < V; ++i) n[i] = wn[(v * V + i) % (HOLD_W ? X : 1)];
        } else {
          weights(v, p, n);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = z[v * V + i] * q * n[i];
        Vec16<T>::store(static_cast<T*>(a.xn) + t * a.H + (long long)(tid + v * NT) * V, x);
      }
    } else if (!a.w_post) {
      __syncthreads();  // a token takes one barrier at least: the numbers below are read behind it
    }
    if (tid < MAXK) {
      meta.row[(j + AHEAD) % META][tid] = m_row;
      meta.gate[(j + AHEAD) % META][tid] = m_gate;
    }
  }
  copies_wait<0>();
}

struct BwdArgs {
  const void *dy, *dxn, *h, *y;
  MetaSource meta;
  const float *row_scale, *w_post, *res_scale, *w_next;
  float eps;
  int T, H, K;
  void *d_res, *dh;
  float *d_gate, *d_scale;
  float* part;  // [gridDim.x][2][H]: this CTA's sums over its tokens of s D u and of dxn v
  int S;        // rows of ring
};

__device__ __forceinline__ void wait_all_but(int n) {  // n of 0, 2, 4, 8
  if (n >= 8) copies_wait<8>();
  else if (n >= 4) copies_wait<4>();
  else if (n >= 2) copies_wait<2>();
  else copies_wait<0>();
}

// HOLD: a token's rows (y, dxn, dy, then h) stay in the ring from the sums to the
// gradients, and the ring holds S - R rows of the next tokens behind them.  Otherwise
// (rows too many or too wide for that) a token's rows pass through the ring twice, h and
// y, dxn, dy for the sums, then y, dxn, dy and h for the gradients; the second time
// they come from L2.
//
// One reduction serves both norms.  With D = dy + q (w_next dxn - q vm y):
//   <aw D, z> = <aw dy, z> + q <aw w_next dxn, z> - q^2 vm <aw y, z>,
// so its three products are summed along with y^2, w_next dxn y and z^2.
template <typename T, int VPT, bool HOLD>
__global__ void __launch_bounds__(512) combine_norm_bwd_kernel(const BwdArgs a) {
  extern __shared__ uint4 ring[];
  __shared__ Meta meta;
  __shared__ CtaSum<6> sum;
  __shared__ float dots[2][MAXK][MAXW / 2 + 1];
  constexpr int V = Vec16<T>::N, X = VPT * V;
  const int tid = threadIdx.x, NT = blockDim.x, nvec = a.H / V, K = a.K, S = a.S;
  const int lane = tid & 31, warp = tid >> 5, nw = NT >> 5;
  const bool next = a.w_next != nullptr;
  const int A = (next ? 2 : 0) + (a.dy ? 1 : 0), R = HOLD ? A + K : 2 * (A + K);
  const uint4 *h = static_cast<const uint4*>(a.h), *dy = static_cast<const uint4*>(a.dy);
  const uint4 *y = static_cast<const uint4*>(a.y), *dxn = static_cast<const uint4*>(a.dxn);
  for (int i = tid; i < AHEAD * MAXK; i += NT) {
    const int j = i / MAXK, k = i % MAXK;
    a.meta.get(blockIdx.x + (long long)j * gridDim.x, k, meta.row[j][k], meta.gate[j][k]);
  }
  __syncthreads();

  int qj = 0, qk = 0, qs = 0;
  long long qt = blockIdx.x;
  auto issue = [&]() {
    if (qt < a.T) {
      int k, x;  // row k of h where k >= 0, otherwise row x of (y, dxn, dy)
      if (HOLD) {
        k = qk - A;
        x = qk;
      } else {
        k = qk < K ? qk : qk - K - 2 * A;
        x = qk - K >= A ? qk - K - A : qk - K;
      }
      const uint4* src;
      bool live = true;
      if (k >= 0) {
        const int row = meta.row[qj % META][k];
        live = row >= 0;
        src = h + (long long)max(row, 0) * nvec;
      } else {
        src = (next && x < 2 ? (x == 0 ? y : dxn) : dy) + qt * nvec;
      }
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int i = tid + v * NT;
        if (i < nvec) copy16(ring + (qs * VPT + v) * NT + tid, src + i, live);
      }
      if (++qk == R) {
        qk = 0;
        ++qj;
        qt += gridDim.x;
      }
    }
    copies_commit();
    qs = qs + 1 == S ? 0 : qs + 1;
  };
  for (int i = 0; i < S; ++i) issue();
  // place of the row i behind the oldest one in the ring
  int slot = 0;
  auto at = [&](int i, int v) -> const uint4& {
    const int p = slot + i;
    return ring[((p >= S ? p - S : p) * VPT + v) * NT + tid];
  };
  auto pass = [&](int n) {
    for (int i = 0; i < n; ++i) issue();
    slot = slot + n >= S ? slot + n - S : slot + n;
  };

  float Q[X], N[X];
#pragma unroll
  for (int i = 0; i < X; ++i) Q[i] = N[i] = 0.f;
  int turn = 0, j = 0;
  long long before = -1;  // the token whose d_gate is still in `dots`
  auto write_gates = [&](long long t, int b) {
    if (a.d_gate && tid < K) {
      float d = 0.f;
      for (int w = 0; w < nw; ++w) d += dots[b][tid][w];
      a.d_gate[t * K + tid] = d;
    }
  };

  for (long long t = blockIdx.x; t < a.T; t += gridDim.x, ++j) {
    int m_row = -1;
    float m_gate = 0.f;
    if (tid < MAXK) a.meta.get(t + (long long)AHEAD * gridDim.x, tid, m_row, m_gate);
    const float rs = a.row_scale ? __ldg(a.row_scale + t) : 1.f;

    float z[X];
#pragma unroll
    for (int i = 0; i < X; ++i) z[i] = 0.f;
    if (HOLD) wait_all_but(S - R);
    for (int k = 0; k < K; ++k) {
      const float g = meta.gate[j % META][k];
      if (!HOLD) copies_wait<2>();  // S >= 3 rows are on their way: the oldest is here
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        if (tid + v * NT >= nvec) continue;
        float x[V];
        unpack<T>(at(HOLD ? A + k : 0, v), x);
#pragma unroll
        for (int i = 0; i < V; ++i) z[v * V + i] = fmaf(g, x[i], z[v * V + i]);
      }
      if (!HOLD) pass(1);
    }
    if (!HOLD) copies_wait<0>();
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (tid + v * NT >= nvec) continue;
      const int c = (tid + v * NT) * V;
      float aw[V], w[V];
      load_w<V>(a.w_post, c, aw);
      load_w<V>(a.res_scale, c, w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        aw[i] *= w[i] * z[v * V + i];
        s[2] = fmaf(z[v * V + i], z[v * V + i], s[2]);
      }
      if (next) {
        float yv[V], xv[V];
        load_w<V>(a.w_next, c, w);
        unpack<T>(at(0, v), yv);
        unpack<T>(at(1, v), xv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float p = w[i] * xv[i];
          s[0] = fmaf(yv[i], yv[i], s[0]);
          s[1] = fmaf(p, yv[i], s[1]);
          s[4] = fmaf(aw[i], p, s[4]);
          s[5] = fmaf(aw[i], yv[i], s[5]);
        }
      }
      if (dy) {
        unpack<T>(at(A - 1, v), w);
#pragma unroll
        for (int i = 0; i < V; ++i) s[3] = fmaf(aw[i], w[i], s[3]);
      }
    }
    if (!HOLD) pass(A);
    sum.run(s, turn++);
    if (before >= 0) write_gates(before, (j & 1) ^ 1);
    const float q = next ? 1.f / sqrtf(s[0] / a.H + a.eps) : 0.f, vm = s[1] * q / a.H;
    const float r = a.w_post ? 1.f / sqrtf(s[2] / a.H + a.eps) : 1.f;
    const float sd = r * (s[3] + q * (s[4] - q * vm * s[5]));
    const float um = a.w_post ? rs * sd / a.H : 0.f;
    if (tid == 0 && a.d_scale) a.d_scale[t] = sd;

    if (!HOLD) copies_wait<0>();
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (tid + v * NT >= nvec) continue;
      const int c = (tid + v * NT) * V;
      float d[V], w[V];
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = 0.f;
      if (dy) unpack<T>(at(A - 1, v), d);
      if (next) {
        float yv[V], xv[V];
        load_w<V>(a.w_next, c, w);
        unpack<T>(at(0, v), yv);
        unpack<T>(at(1, v), xv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float u = yv[i] * q;
          d[i] += q * (xv[i] * w[i] - u * vm);
          N[v * V + i] = fmaf(xv[i], u, N[v * V + i]);
        }
      }
      if (a.d_res) Vec16<T>::store(static_cast<T*>(a.d_res) + t * a.H + c, d);
      if (K > 0) {
        float aw[V];
        load_w<V>(a.w_post, c, aw);
        load_w<V>(a.res_scale, c, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float u = z[v * V + i] * r, e = rs * d[i];
          Q[v * V + i] = fmaf(e, u, Q[v * V + i]);
          z[v * V + i] = r * (e * aw[i] * w[i] - u * um);  // dz
        }
      }
    }
    pass(A);
    for (int k = 0; k < K; ++k) {
      const float g = meta.gate[j % META][k];
      const int row = meta.row[j % META][k];
      if (!HOLD) copies_wait<2>();
      float dot = 0.f;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        if (tid + v * NT >= nvec) continue;
        float x[V];
        unpack<T>(at(0, v), x);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          dot = fmaf(z[v * V + i], x[i], dot);
          x[i] = g * z[v * V + i];
        }
        if (a.dh && row >= 0) Vec16<T>::store(static_cast<T*>(a.dh) + (long long)row * a.H + (tid + v * NT) * V, x);
      }
      pass(1);
      if (a.d_gate) {
        dot = warp_sum(dot);
        if (lane == 0) dots[j & 1][k][warp] = dot;
      }
    }
    before = t;
    if (tid < MAXK) {
      meta.row[(j + AHEAD) % META][tid] = m_row;
      meta.gate[(j + AHEAD) % META][tid] = m_gate;
    }
  }
  copies_wait<0>();
  __syncthreads();
  if (before >= 0) write_gates(before, (j & 1) ^ 1);
  if (a.part) {
    float* p = a.part + (size_t)blockIdx.x * 2 * a.H;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (tid + v * NT >= nvec) continue;
      const int c = (tid + v * NT) * V;
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        *reinterpret_cast<float4*>(p + c + i) = make_float4(Q[v * V + i], Q[v * V + i + 1], Q[v * V + i + 2], Q[v * V + i + 3]);
        *reinterpret_cast<float4*>(p + a.H + c + i) =
            make_float4(N[v * V + i], N[v * V + i + 1], N[v * V + i + 2], N[v * V + i + 3]);
      }
    }
  }
}

// The column sums: a CTA takes 32 columns of [2][H], 16 warps the parts w, w + 16, ... in
// order; the warps' sums are added in warp order and multiplied by their column factors.
__global__ void __launch_bounds__(512)
column_sums_kernel(const float* __restrict__ part, int parts, int H, const float* __restrict__ w_post,
                   const float* __restrict__ res_scale, float* dw_post, float* d_res_scale, float* dw_next) {
  __shared__ float red[16][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float acc = 0.f;
  if (i < 2 * H) {
#pragma unroll 4
    for (int p = w; p < parts; p += 16) acc += __ldg(part + (size_t)p * 2 * H + i);
  }
  red[w][lane] = acc;
  __syncthreads();
  if (w > 0 || i >= 2 * H) return;
  for (int k = 1; k < 16; ++k) acc += red[k][lane];
  if (i >= H) {
    if (dw_next) dw_next[i - H] = acc;
  } else {
    if (dw_post) dw_post[i] = acc * (res_scale ? res_scale[i] : 1.f);
    if (d_res_scale) d_res_scale[i] = acc * (w_post ? w_post[i] : 1.f);
  }
}

constexpr int RING_BYTES = 200 * 1024;  // at most; a CTA's 227 KB also hold the sums and row numbers

int threads_for(int nvec, int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; }

// CTAs of a persistent grid: as many as fit, at most `cap` to an SM, at most one a token
template <typename F> int persistent_grid(F kernel, int threads, int smem, int cap, int T, int* grid) {
  int per_sm = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1)
    return MOE_ERR_CUDA;
  const long long n = (long long)sm_count() * (per_sm < cap ? per_sm : cap);
  *grid = (int)(T < n ? T : n);
  return MOE_OK;
}

template <typename T, int VPT, int S> int fwd_v(const FwdArgs& a, cudaStream_t s) {
  const int threads = threads_for(a.H / Vec16<T>::N, VPT), smem = S * VPT * threads * 16;
  int grid = 0;
  const int st = persistent_grid(combine_norm_kernel<T, VPT, S>, threads, smem, 32, a.T, &grid);
  if (st != MOE_OK) return st;
  combine_norm_kernel<T, VPT, S><<<grid, threads, smem, s>>>(a);
  return launch_status();
}

// The widest rows a thread's vectors reach with at most 896 threads; the ring takes what
// 200 KB hold: 12 rows of up to 14 KB, 6 of up to 28 KB, 3 beyond.
template <typename T> int fwd_t(const FwdArgs& a, cudaStream_t s) {
  const int nvec = a.H / Vec16<T>::N;
  if (nvec <= 896) return fwd_v<T, 1, 12>(a, s);
  if (nvec <= 2 * 896) return fwd_v<T, 2, 6>(a, s);
  if (nvec <= 4 * 896) return fwd_v<T, 4, 3>(a, s);
  return fwd_v<T, 8, 3>(a, s);
}

// column sums kept per CTA: at most this many CTAs to an SM
int bwd_ctas_per_sm(int H) { return H >= 8192 ? 2 : H >= 1024 ? 16384 / H : 16; }

int bwd_rows(const BwdArgs& a) { return a.K + (a.w_next ? 2 : 0) + (a.dy ? 1 : 0); }

template <typename T, int VPT, bool HOLD> int bwd_v(BwdArgs& a, int* grid, cudaStream_t s) {
  const int threads = threads_for(a.H / Vec16<T>::N, VPT), row = VPT * threads * 16, R = bwd_rows(a);
  // rows of the next tokens behind a token's own: 8, or what two CTAs, then one leave room for
  auto fits = [&](int rows, int bytes) { return (long long)rows * row <= bytes; };
  a.S = !HOLD                       ? 3
        : fits(R + 8, RING_BYTES / 2) ? R + 8
        : fits(R + 4, RING_BYTES / 2) ? R + 4
        : fits(R + 8, RING_BYTES)     ? R + 8
        : fits(R + 4, RING_BYTES)     ? R + 4
                                      : R + 2;
  const int smem = a.S * row;
  const int st = persistent_grid(combine_norm_bwd_kernel<T, VPT, HOLD>, threads, smem, bwd_ctas_per_sm(a.H), a.T, grid);
  if (st != MOE_OK) return st;
  combine_norm_bwd_kernel<T, VPT, HOLD><<<*grid, threads, smem, s>>>(a);
  return launch_status();
}

// 8 values a thread up to H = 4096, 16 up to 8192, 32 beyond (their column sums spill a
// little); a token's rows are held where two more fit beside them
template <typename T> int bwd_t(BwdArgs& a, int* grid, cudaStream_t s) {
  constexpr int V = Vec16<T>::N;
  const int nvec = a.H / V;
  auto holds = [&](int vpt) { return (long long)(bwd_rows(a) + 2) * vpt * threads_for(nvec, vpt) * 16 <= RING_BYTES; };
  if (a.H <= 4096 && holds(8 / V)) return bwd_v<T, 8 / V, true>(a, grid, s);
  if (a.H <= 8192) return holds(16 / V) ? bwd_v<T, 16 / V, true>(a, grid, s) : bwd_v<T, 16 / V, false>(a, grid, s);
  return bwd_v<T, 32 / V, false>(a, grid, s);
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
                  w_post, res_scale, w_next, eps, T, H, K, y, xn};
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
            res_scale, w_next, eps, T, H, K, d_res, dh, d_gate, d_scale, sums ? static_cast<float*>(ws) : nullptr, 0};
  int grid = 0;
  const int st = dtype == MOE_BF16 ? bwd_t<bf16>(a, &grid, s) : bwd_t<float>(a, &grid, s);
  if (st != MOE_OK || !sums) return st;
  column_sums_kernel<<<(2 * H + 31) / 32, 512, 0, s>>>(a.part, grid, H, w_post, res_scale, dw_post, d_res_scale, dw_next);
  return launch_status();
}

}  // namespace moe
