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
// Nothing is used twice, so loads and stores pass through the caches as
// streams: 8192 tokens of 7168, k = 8 (2 GB): 324 against 362 us, 94% of the
// measured copy rate; 8192 of 2880, k = 4: 72 against 77 us (90%); 2048 of 4096,
// k = 2: 18 us either way (70%; about 5 us of it start and end the 2048 blocks).
// A warp per token with several vectors in flight per lane was 1.5 to 2.5 times
// slower, and two or four vectors per thread of a block 1.2 to 1.8 times: what
// counts is that the block reads and writes long pieces of a row at a time.
#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"

namespace moe {
namespace {


template <typename T>
__device__ __forceinline__ Vec16<T> ld16_stream(const T* p) {
  Vec16<T> r;
  *reinterpret_cast<uint4*>(r.v) = __ldcs(reinterpret_cast<const uint4*>(p));
  return r;
}
template <typename T>
__device__ __forceinline__ void st16_stream(T* p, const Vec16<T>& r) {
  __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(r.v));
}

// TPT threads work on one token: a warp where a row has at most 64 vectors, the
// block otherwise.
template <typename T, int KMAX, int TPT, bool ROWS, bool WEIGHTS>
__global__ void __launch_bounds__(TPT == 32 ? 128 : TPT) combine_backward_kernel(const __grid_constant__ CombineBackwardArgs a) {
  constexpr int V = Vec16<T>::N;
  constexpr int kThreads = TPT == 32 ? 128 : TPT, kTokens = kThreads / TPT;
  __shared__ float part[KMAX][kThreads / 32];
  const T* gy = static_cast<const T*>(a.grad_y);
  const T* yp = static_cast<const T*>(a.y_perm);
  T* gp = static_cast<T*>(a.grad_y_perm);
  const int nv = a.d / V, k = a.k;
  const int tid = threadIdx.x % TPT, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / TPT; t < a.T; t += (int64_t)gridDim.x * kTokens) {
    const T* gt = gy + t * a.d;
    Vec16<T> g;  // the first round's does not wait for the rows
    if (tid < nv) g = ld16_stream(gt + (int64_t)tid * V);
    int rows[KMAX];
    float w[KMAX], dot[KMAX];
#pragma unroll
    for (int s = 0; s < KMAX; ++s) {
      rows[s] = s < k ? a.row_of[t * k + s] : -1;
      w[s] = ROWS && s < k ? a.w[t * k + s] : 0.f;
      dot[s] = 0.f;
    }
    for (int v = tid; v < nv; v += TPT) {
      if (v != tid) g = ld16_stream(gt + (int64_t)v * V);
      Vec16<T> y[KMAX];
      if (WEIGHTS) {
#pragma unroll
        for (int s = 0; s < KMAX; ++s)
          if (rows[s] >= 0) y[s] = ld16_stream(yp + (int64_t)rows[s] * a.d + (int64_t)v * V);
      }
      float gf[V];
#pragma unroll
      for (int j = 0; j < V; ++j) gf[j] = Elem<T>::to_f(g.v[j]);
#pragma unroll
      for (int s = 0; s < KMAX; ++s) {
        if (rows[s] < 0) continue;
        if (ROWS) {
          Vec16<T> o;
#pragma unroll
          for (int j = 0; j < V; ++j) o.v[j] = Elem<T>::from_f(w[s] * gf[j]);
          st16_stream(gp + (int64_t)rows[s] * a.d + (int64_t)v * V, o);
        }
        if (WEIGHTS) {
#pragma unroll
          for (int j = 0; j < V; ++j) dot[s] = fmaf(gf[j], Elem<T>::to_f(y[s].v[j]), dot[s]);
        }
      }
    }
    if (WEIGHTS) {
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
  const int64_t per_block = narrow ? 4 : 1;
  int64_t blocks = (a.T + per_block - 1) / per_block;
  const int64_t cap = (int64_t)device_sm_count() * 64;
  if (blocks > cap) blocks = cap;
  auto run = [&](auto kernel, int threads) {
    kernel<<<(unsigned)blocks, threads, 0, stream>>>(a);
    return cudaGetLastError();
  };
  auto parts = [&](auto tpt) {
    constexpr int TPT = decltype(tpt)::value;
    if (!a.grad_w) return run(combine_backward_kernel<T, KMAX, TPT, true, false>, TPT == 32 ? 128 : TPT);
    if (!a.grad_y_perm) return run(combine_backward_kernel<T, KMAX, TPT, false, true>, TPT == 32 ? 128 : TPT);
    return run(combine_backward_kernel<T, KMAX, TPT, true, true>, TPT == 32 ? 128 : TPT);
  };
  if (narrow) return parts(std::integral_constant<int, 32>());
  // many slots take many registers: more threads per token keep as many loads in flight
  if (KMAX > 4 && a.d / Vec16<T>::N >= 512) return parts(std::integral_constant<int, 256>());
  return parts(std::integral_constant<int, 128>());
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
  const CombineBackwardArgs& a = args;
  if (a.T == 0 || (!a.grad_w && !a.grad_y_perm)) return cudaSuccess;
  return a.bf16 ? launch_t<__nv_bfloat16>(a, stream) : launch_t<float>(a, stream);
}

}  // namespace moe
