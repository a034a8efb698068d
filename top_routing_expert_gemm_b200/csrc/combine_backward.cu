// Gradient of the weighted un-permute y[t] = sum_s w[t,s] y_perm[row_of[t*k+s]]:
//   grad_w[t,s]              = <grad_y[t], y_perm[row]>
//   grad_y_perm[row]         = w[t,s] grad_y[t]
// ("Mixture of Experts Explained: Routers, Active Parameters and VRAM", step
// "Run and combine", differentiated.)  A dropped slot (row -1) has gradient
// zero and no row; rows that no slot points at are left as they were.  The
// shared expert's output enters with weight 1, so its gradient is grad_y.
//
// Bound by HBM: grad_y once, y_perm once, grad_y_perm once.  A token's
// grad_y vector is read once for its k slots; the dot products stay in fp32
// registers (one partial per slot and thread) and are added in a fixed tree.
#include "common.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;

// TPT threads work on one token: a warp where a row has at most 64 vectors,
// the block otherwise.
template <typename T, int KMAX, int TPT>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const CombineBackwardArgs a) {
  constexpr int V = Vec16<T>::N;
  constexpr int kTokens = kThreads / TPT;
  __shared__ float part[KMAX][kThreads / 32];
  const T* __restrict__ gy = static_cast<const T*>(a.grad_y);
  const T* __restrict__ yp = static_cast<const T*>(a.y_perm);
  T* __restrict__ gp = static_cast<T*>(a.grad_y_perm);
  const int nv = a.d / V, k = a.k;
  const int tid = threadIdx.x % TPT, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / TPT; t < a.T; t += (int64_t)gridDim.x * kTokens) {
    int rows[KMAX];
    float w[KMAX], dot[KMAX];
#pragma unroll
    for (int s = 0; s < KMAX; ++s) {
      rows[s] = s < k ? a.row_of[t * k + s] : -1;
      w[s] = s < k && gp ? a.w[t * k + s] : 0.f;
      dot[s] = 0.f;
    }
    for (int v = tid; v < nv; v += TPT) {
      const Vec16<T> g = ld16(gy + t * a.d + (int64_t)v * V);
      Vec16<T> y[KMAX];
      if (yp) {
#pragma unroll
        for (int s = 0; s < KMAX; ++s)
          if (rows[s] >= 0) y[s] = ld16(yp + (int64_t)rows[s] * a.d + (int64_t)v * V);
      }
#pragma unroll
      for (int s = 0; s < KMAX; ++s) {
        if (rows[s] < 0) continue;
        if (yp) {
#pragma unroll
          for (int j = 0; j < V; ++j) dot[s] = fmaf(Elem<T>::to_f(g.v[j]), Elem<T>::to_f(y[s].v[j]), dot[s]);
        }
        if (gp) {
          Vec16<T> o;
#pragma unroll
          for (int j = 0; j < V; ++j) o.v[j] = Elem<T>::from_f(w[s] * Elem<T>::to_f(g.v[j]));
          st16(gp + (int64_t)rows[s] * a.d + (int64_t)v * V, o);
        }
      }
    }
    if (a.grad_w) {
#pragma unroll
      for (int s = 0; s < KMAX; ++s)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot[s] += __shfl_xor_sync(0xffffffffu, dot[s], off);
      if (TPT == 32) {
#pragma unroll
        for (int s = 0; s < KMAX; ++s)
          if (lane == s && s < k) a.grad_w[t * k + s] = dot[s];
      } else {
        if (lane == 0) {
#pragma unroll
          for (int s = 0; s < KMAX; ++s) part[s][warp] = dot[s];
        }
        __syncthreads();
        if (threadIdx.x < k) {
          float v = 0.f;
#pragma unroll
          for (int i = 0; i < kThreads / 32; ++i) v += part[threadIdx.x][i];
          a.grad_w[t * k + threadIdx.x] = v;
        }
        __syncthreads();
      }
    }
  }
}

template <typename T, int KMAX>
cudaError_t launch_k(const CombineBackwardArgs& a, cudaStream_t stream) {
  const bool narrow = a.d / Vec16<T>::N <= 64;
  const int64_t per_block = narrow ? kThreads / 32 : 1;
  int64_t blocks = (a.T + per_block - 1) / per_block;
  const int64_t cap = (int64_t)device_sm_count() * 64;
  if (blocks > cap) blocks = cap;
  if (narrow) combine_backward_kernel<T, KMAX, 32><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  else combine_backward_kernel<T, KMAX, kThreads><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const CombineBackwardArgs& a, cudaStream_t stream) {
  if (a.k <= 2) return launch_k<T, 2>(a, stream);
  if (a.k <= 4) return launch_k<T, 4>(a, stream);
  if (a.k <= 8) return launch_k<T, 8>(a, stream);
  return launch_k<T, kMaxTopK>(a, stream);
}

}  // namespace

cudaError_t launch_combine_backward(const CombineBackwardArgs& args, cudaStream_t stream) {
  CombineBackwardArgs a = args;
  if (a.T == 0 || (!a.grad_w && !a.grad_y_perm)) return cudaSuccess;
  if (!a.grad_w) a.y_perm = nullptr;
  return a.bf16 ? launch_t<__nv_bfloat16>(a, stream) : launch_t<float>(a, stream);
}

}  // namespace moe
