// Combine fused with the RMS norms around the block, its gate and its residual
// scale (moe_combine_norm), and the backward of all of it.
//
// One CTA per token: z and y stay in shared memory between the passes over the
// row, so h, residual, y and xn each cross the memory bus once.
#include <math.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int NT = 256;

// sum over the CTA, the same in every thread (a fixed order)
__device__ __forceinline__ float cta_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) v += red[w];
  return v;
}

// z[c] of token t for this thread's vectors into shared memory; returns its share of sum z^2
template <typename T>
__device__ __forceinline__ float block_row(const T* h, const float* gate, const int32_t* dst_row, long long t, int K,
                                           int H, long long R, float* z, unsigned* err) {
  constexpr int V = Vec16<T>::N;
  float sq = 0.f;
  for (int c = threadIdx.x * V; c < H; c += NT * V) {
    float acc[V], v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int k = 0; k < K; ++k) {
      const long long r = dst_row ? dst_row[t * K + k] : t * K + k;
      if (r < 0 || r >= R) {
        set_error(err, DEV_BOUNDS);
        continue;
      }
      const float g = gate ? gate[t * K + k] : 1.f;
      Vec16<T>::load(h + r * H + c, v);
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = fmaf(g, v[j], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      z[c + j] = acc[j];
      sq = fmaf(acc[j], acc[j], sq);
    }
  }
  return sq;
}

template <typename T> __device__ __forceinline__ void load_plain(const T* p, float* v) {
  Vec16<T>::load_raw_unpack(*reinterpret_cast<const uint4*>(p), v);
}

template <typename T>
__global__ void __launch_bounds__(NT)
combine_norm_kernel(const T* h, const float* gate, const int32_t* dst_row, const float* row_scale, const T* residual,
                    const float* w_post, const float* res_scale, const float* w_next, float eps, int Tn, int H, int K,
                    T* y, T* xn, unsigned* err) {
  extern __shared__ float z[];
  __shared__ float red[NT / 32];
  constexpr int V = Vec16<T>::N;
  for (long long t = blockIdx.x; t < Tn; t += gridDim.x) {
    float r = 1.f;
    if (h) {
      const float sq = block_row<T>(h, gate, dst_row, t, K, H, (long long)Tn * K, z, err);
      if (w_post) r = 1.f / sqrtf(cta_sum(sq, red) / H + eps);
    }
    const float s = (row_scale ? row_scale[t] : 1.f) * r;
    float sq = 0.f;
    for (int c = threadIdx.x * V; c < H; c += NT * V) {
      float v[V];
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = 0.f;
      if (residual) load_plain<T>(residual + t * H + c, v);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (h) v[j] = fmaf(s * z[c + j], (w_post ? w_post[c + j] : 1.f) * (res_scale ? res_scale[c + j] : 1.f), v[j]);
        z[c + j] = v[j];
        sq = fmaf(v[j], v[j], sq);
      }
      if (y) Vec16<T>::store(y + t * H + c, v);
    }
    if (w_next) {
      const float q = 1.f / sqrtf(cta_sum(sq, red) / H + eps);
      for (int c = threadIdx.x * V; c < H; c += NT * V) {
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = z[c + j] * q * w_next[c + j];
        Vec16<T>::store(xn + t * H + c, v);
      }
    }
    __syncthreads();
  }
}

// part [gridDim.x][2][H]: this CTA's sums over its tokens of s D u (first) and dxn v (second)
template <typename T>
__global__ void __launch_bounds__(NT)
combine_norm_bwd_kernel(const T* dy, const T* dxn, const T* h, const float* gate, const int32_t* dst_row,
                        const float* row_scale, const T* y, const float* w_post, const float* res_scale,
                        const float* w_next, float eps, int Tn, int H, int K, T* d_res, T* dh, float* d_gate,
                        float* d_scale, float* part, unsigned* err) {
  extern __shared__ float sm[];
  __shared__ float red[NT / 32];
  constexpr int V = Vec16<T>::N;
  float* z = sm;
  float* D = sm + H;
  float* pq = part ? part + (size_t)blockIdx.x * 2 * H : nullptr;
  if (pq)
    for (int c = threadIdx.x; c < 2 * H; c += NT) pq[c] = 0.f;
  __syncthreads();
  const long long R = (long long)Tn * K;
  for (long long t = blockIdx.x; t < Tn; t += gridDim.x) {
    float r = 1.f;
    if (h) {
      const float sq = block_row<T>(h, gate, dst_row, t, K, H, R, z, err);
      if (w_post) r = 1.f / sqrtf(cta_sum(sq, red) / H + eps);
    }
    float q = 0.f, vm = 0.f;
    if (w_next) {
      float sy = 0.f, sa = 0.f;
      for (int c = threadIdx.x * V; c < H; c += NT * V) {
        float yv[V], xv[V];
        load_plain<T>(y + t * H + c, yv);
        load_plain<T>(dxn + t * H + c, xv);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          sy = fmaf(yv[j], yv[j], sy);
          sa = fmaf(xv[j] * w_next[c + j], yv[j], sa);
        }
      }
      q = 1.f / sqrtf(cta_sum(sy, red) / H + eps);
      vm = cta_sum(sa, red) * q / H;  // mean(w_next dxn v)
    }
    const float s = row_scale ? row_scale[t] : 1.f;
    float su = 0.f, sd = 0.f;
    for (int c = threadIdx.x * V; c < H; c += NT * V) {
      float d[V];
#pragma unroll
      for (int j = 0; j < V; ++j) d[j] = 0.f;
      if (dy) load_plain<T>(dy + t * H + c, d);
      if (w_next) {
        float yv[V], xv[V];
        load_plain<T>(y + t * H + c, yv);
        load_plain<T>(dxn + t * H + c, xv);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float v = yv[j] * q;
          d[j] += q * (xv[j] * w_next[c + j] - v * vm);
          if (pq) pq[H + c + j] = fmaf(xv[j], v, pq[H + c + j]);
        }
      }
      if (d_res) Vec16<T>::store(d_res + t * H + c, d);
      if (h) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float u = z[c + j] * r, aw = (w_post ? w_post[c + j] : 1.f) * (res_scale ? res_scale[c + j] : 1.f);
          if (pq) pq[c + j] = fmaf(s * d[j], u, pq[c + j]);
          sd = fmaf(d[j] * aw, u, sd);
          const float P = s * aw * d[j];
          su = fmaf(P, u, su);
          D[c + j] = P;
        }
      }
    }
    if (h) {
      if (d_scale) {
        sd = cta_sum(sd, red);
        if (threadIdx.x == 0) d_scale[t] = sd;
      }
      const float um = w_post ? cta_sum(su, red) / H : 0.f;
      for (int c = threadIdx.x * V; c < H; c += NT * V)
#pragma unroll
        for (int j = 0; j < V; ++j) D[c + j] = w_post ? r * (D[c + j] - z[c + j] * r * um) : D[c + j];
      for (int k = 0; k < K; ++k) {
        const long long row = dst_row ? dst_row[t * K + k] : t * K + k;
        const bool in = row >= 0 && row < R;
        const float g = gate ? gate[t * K + k] : 1.f;
        float dot = 0.f;
        for (int c = threadIdx.x * V; in && c < H; c += NT * V) {
          float v[V], o[V];
          Vec16<T>::load(h + row * H + c, v);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            dot = fmaf(D[c + j], v[j], dot);
            o[j] = g * D[c + j];
          }
          if (dh) Vec16<T>::store(dh + row * H + c, o);
        }
        if (d_gate) {
          dot = cta_sum(dot, red);
          if (threadIdx.x == 0) d_gate[t * K + k] = dot;
        }
      }
    }
    __syncthreads();
  }
}

// the column sums: parts added in CTA order, then their column factors
__global__ void __launch_bounds__(256)
column_sums_kernel(const float* __restrict__ part, int parts, int H, const float* __restrict__ w_post,
                   const float* __restrict__ res_scale, float* dw_post, float* d_res_scale, float* dw_next) {
  for (int c = blockIdx.x * 256 + threadIdx.x; c < H; c += gridDim.x * 256) {
    float a = 0.f, b = 0.f;
    for (int p = 0; p < parts; ++p) {
      a += part[(size_t)p * 2 * H + c];
      b += part[(size_t)p * 2 * H + H + c];
    }
    if (dw_post) dw_post[c] = a * (res_scale ? res_scale[c] : 1.f);
    if (d_res_scale) d_res_scale[c] = a * (w_post ? w_post[c] : 1.f);
    if (dw_next) dw_next[c] = b;
  }
}

int bwd_grid(int T) {
  const int cap = sm_count() * 2;
  return T < cap ? (T > 0 ? T : 1) : cap;
}

template <typename T>
int fwd_t(const void* h, const float* gate, const int32_t* dst_row, const float* row_scale, const void* residual,
          const float* w_post, const float* res_scale, const float* w_next, float eps, int Tn, int H, int K, void* y,
          void* xn, cudaStream_t s) {
  const int smem = H * 4;
  if (cudaFuncSetAttribute(combine_norm_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return MOE_ERR_CUDA;
  const long long cap = (long long)sm_count() * 32;
  combine_norm_kernel<T><<<(int)(Tn < cap ? Tn : cap), NT, smem, s>>>(
      static_cast<const T*>(h), gate, dst_row, row_scale, static_cast<const T*>(residual), w_post, res_scale, w_next,
      eps, Tn, H, K, static_cast<T*>(y), static_cast<T*>(xn), device_error_word());
  return launch_status();
}

template <typename T>
int bwd_t(const void* dy, const void* dxn, const void* h, const float* gate, const int32_t* dst_row,
          const float* row_scale, const void* y, const float* w_post, const float* res_scale, const float* w_next,
          float eps, int Tn, int H, int K, void* d_res, void* dh, float* d_gate, float* d_scale, float* part,
          cudaStream_t s) {
  const int smem = 2 * H * 4;
  if (cudaFuncSetAttribute(combine_norm_bwd_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return MOE_ERR_CUDA;
  combine_norm_bwd_kernel<T><<<bwd_grid(Tn), NT, smem, s>>>(
      static_cast<const T*>(dy), static_cast<const T*>(dxn), static_cast<const T*>(h), gate, dst_row, row_scale,
      static_cast<const T*>(y), w_post, res_scale, w_next, eps, Tn, H, K, static_cast<T*>(d_res), static_cast<T*>(dh),
      d_gate, d_scale, part, device_error_word());
  return launch_status();
}

}  // namespace

size_t combine_norm_bwd_ws_bytes(int T, int H) { return (size_t)bwd_grid(T) * 2 * H * 4; }

int launch_combine_norm(const void* h, const float* gate, const int32_t* dst_row, const float* row_scale,
                        const void* residual, const float* w_post, const float* res_scale, const float* w_next,
                        float eps, int T, int H, int K, int dtype, void* y, void* xn, cudaStream_t s) {
  if (T == 0) return MOE_OK;
  return dtype == MOE_BF16
             ? fwd_t<bf16>(h, gate, dst_row, row_scale, residual, w_post, res_scale, w_next, eps, T, H, K, y, xn, s)
             : fwd_t<float>(h, gate, dst_row, row_scale, residual, w_post, res_scale, w_next, eps, T, H, K, y, xn, s);
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
  float* part = sums ? static_cast<float*>(ws) : nullptr;
  int st = dtype == MOE_BF16 ? bwd_t<bf16>(dy, dxn, h, gate, dst_row, row_scale, y, w_post, res_scale, w_next, eps, T,
                                           H, K, d_res, dh, d_gate, d_scale, part, s)
                             : bwd_t<float>(dy, dxn, h, gate, dst_row, row_scale, y, w_post, res_scale, w_next, eps,
                                            T, H, K, d_res, dh, d_gate, d_scale, part, s);
  if (st != MOE_OK || !sums) return st;
  column_sums_kernel<<<(H + 255) / 256, 256, 0, s>>>(part, bwd_grid(T), H, w_post, res_scale, dw_post, d_res_scale,
                                                     dw_next);
  return launch_status();
}

}  // namespace moe
