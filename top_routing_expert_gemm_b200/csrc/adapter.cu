// Low-rank adapters of many requests beside the experts' projections:
//   v[row] = base[row] + s_n B[n, e] (A[n, e] x[row]),   n the adapter of the row's token, e its expert
// followed by the expert's activation for the first projection.  The base
// projection (the weights every request shares) is not touched: base is its
// output.  The layer's pages do not describe adapters; the expert is the one
// of "Mixture of Experts Explained: Routers, Active Parameters and VRAM".
//
// Three kernels:
//   plan    groups the rows of equal (expert, adapter) into tiles of up to TM
//           rows: chunks of 256 rows are sorted inside a block, so no global
//           sort and no histogram over the pairs is needed
//   shrink  U = A x per tile, the reduction over the inputs split over S
//           blocks and the warps of each; partial sums in fp32, added in a
//           fixed order
//   expand  base + s B U per tile and column block, then the activation
// Rows never meet: a row's result does not depend on the tile it falls into.
//
// Bound by bytes: base and result once, x once, the touched adapters' A and B
// once (a tile reads its pair's weights, tiles of one pair meet in L2).  The
// products have a depth or width of rank, 8 to 128, so the tensor work is small
// and mma.sync, whose operands come straight from global memory in fragment
// order, does it without a shared-memory stage; a 128-row tcgen05 tile would
// be mostly empty.  In fp32 layers everything is fmaf on the CUDA cores.
#include <algorithm>

#include "common.cuh"
#include "kernels.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kChunkRows = 256;  // rows a plan block sorts
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;
static_assert((int64_t)(kAdapterMaxPairs + 1) * kChunkRows < (int64_t(1) << 31), "keys of the plan are 31 bits");
constexpr int kSkip = 0x7fffff;  // pair of a row that is not there (kMaxPairs - 1 is below)

struct Tile {
  int start;    // first position in `order`
  int count;    // rows
  int adapter;  // -1: none
  int expert;
};

// ---------------------------------------------------------------- plan
struct PlanParams {
  const int32_t* offsets;  // [E+1] or null: every row is there, expert 0
  const int32_t* perm;     // [rows] or null: row = token
  const int32_t* token_adapter;
  int64_t rows;
  int E, k, N, TM;
  int32_t* order;
  Tile* tiles;
  int* n_tiles;
  int* status;
};

// Four threads per row: each compares the row's key with a quarter of the
// chunk's.  A key holds (expert, adapter) above the row's place in the chunk, so
// all keys differ and one comparison ranks stably.
constexpr int kPlanThreads = 4 * kChunkRows;

__global__ void __launch_bounds__(kPlanThreads) adapter_plan_kernel(const PlanParams p) {
  extern __shared__ int s_off[];  // [E+1]
  __shared__ __align__(16) int keys[kChunkRows];
  __shared__ int sorted[kChunkRows];
  __shared__ int warp_sums[kChunkRows / 32];
  __shared__ int s_base;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  grid_dependency_wait();  // the dispatch (programmatic launch)
  if (tid == 0) grid_launch_dependents();
  const int64_t row0 = (int64_t)blockIdx.x * kChunkRows;
  const int64_t row = row0 + tid;
  const bool mine_to_load = tid < kChunkRows && row < p.rows;
  const int slot = mine_to_load && p.perm ? p.perm[row] : 0;  // garbage behind the last row: not used there
  if (p.offsets)
    for (int e = tid; e <= p.E; e += kPlanThreads) s_off[e] = p.offsets[e];
  __syncthreads();
  const int64_t live = p.offsets ? min((int64_t)s_off[p.E], p.rows) : p.rows;
  if (tid < kChunkRows) {
    int pair = kSkip;
    if (row < live) {
      int a = p.token_adapter[p.perm ? slot / p.k : row];
      if (a >= p.N) {
        set_status(p.status, kDevBadAdapterId);
        a = -1;
      }
      int e = 0;
      if (a >= 0 && p.offsets) {  // the last expert whose rows start at or before this one
        int lo = 0, hi = p.E;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_off[mid] <= row) lo = mid;
          else hi = mid;
        }
        e = lo;
      }
      pair = a < 0 ? 0 : e * p.N + a + 1;  // rows without an adapter form one run, whatever their expert
    }
    keys[tid] = pair * kChunkRows + tid;
  }
  __syncthreads();
  {
    const int i = tid / 4, quarter = tid % 4;
    const int key = keys[i];
    int rank = 0;
    const int4* k4 = reinterpret_cast<const int4*>(keys);
#pragma unroll
    for (int j = 0; j < kChunkRows / 16; ++j) {
      const int4 q = k4[4 * j + quarter];
      rank += (q.x < key) + (q.y < key) + (q.z < key) + (q.w < key);
    }
    rank += __shfl_xor_sync(kFull, rank, 1);
    rank += __shfl_xor_sync(kFull, rank, 2);
    if (quarter == 0) {
      sorted[rank] = key / kChunkRows;
      if (key / kChunkRows != kSkip) p.order[row0 + rank] = (int32_t)(row0 + i);
    }
  }
  __syncthreads();
  // position tid of the sorted chunk starts a tile where its run starts, and
  // every TM rows from there
  const int mine = tid < kChunkRows ? sorted[tid] : kSkip;
  bool head = false;
  int end = 0;
  if (mine != kSkip) {
    int lo = 0, hi = tid;  // first position of the run (the pairs ascend)
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sorted[mid] < mine) lo = mid + 1;
      else hi = mid;
    }
    head = (tid - lo) % p.TM == 0;
    if (head) {
      lo = tid + 1;
      hi = min(kChunkRows, tid + p.TM);
      while (lo < hi) {  // first position behind the tile
        const int mid = (lo + hi) >> 1;
        if (sorted[mid] == mine) lo = mid + 1;
        else hi = mid;
      }
      end = lo;
    }
  }
  const unsigned heads = __ballot_sync(kFull, head);
  if (lane == 0 && tid < kChunkRows) warp_sums[warp] = __popc(heads);
  __syncthreads();
  if (tid == 0) {
    int n = 0;
    for (int w = 0; w < kChunkRows / 32; ++w) {
      const int c = warp_sums[w];
      warp_sums[w] = n;
      n += c;
    }
    s_base = n ? atomicAdd(p.n_tiles, n) : 0;  // the order of the tiles changes no result
  }
  __syncthreads();
  if (head) {
    const int at = s_base + warp_sums[warp] + __popc(heads & ((1u << lane) - 1u));
    const int pair = mine - 1;
    p.tiles[at] = Tile{(int)(row0 + tid), end - tid, pair < 0 ? -1 : pair % p.N, pair < 0 ? 0 : pair / p.N};
  }
}

// ---------------------------------------------------------------- shrink
struct ShrinkParams {
  const void* x;  // [rows, K]
  const void* a;  // [N, E, r, K]
  const int32_t* order;
  const Tile* tiles;
  const int* n_tiles;
  float* u;       // [S][rows][r] by position in `order`
  int64_t rows;
  int K, r, E;
  int k_block;    // inputs per block (blockIdx.y)
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(static_cast<const uint4*>(p)); }

// Asynchronous copies into the warp's own ring in shared memory: a lane reads
// back only what it copied itself, so a wait_group is all the synchronisation
// there is.  Without `on` the destination is zeroed and nothing is read.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Stages of a warp's ring whose stage takes `bytes`: what two blocks per SM
// leave each of their warps (13.5 KiB), one stage at least, four at most
constexpr int ring_stages(int bytes) { return bytes * 4 <= 13824 ? 4 : bytes * 3 <= 13824 ? 3 : bytes * 2 <= 13824 ? 2 : 1; }

// MT row tiles of 16, up to RT rank tiles of 8.  A lane takes 8 consecutive
// inputs of a row with one 16-byte load and uses them as the k indices 2t,
// 2t+1, 2t+8, 2t+9 of two instructions: the sum runs over all inputs, so any
// assignment of inputs to k serves as long as x and A agree.
constexpr int kUnit = 64;  // inputs per warp and round: whole 128-byte lines of every row
template <int MT, int RT>
constexpr int shrink_stage() { return 2 * (2 * MT + RT) * 512; }
template <int MT, int RT>
constexpr int shrink_smem() {
  const int ring = kWarps * ring_stages(shrink_stage<MT, RT>()) * shrink_stage<MT, RT>();
  const int red = kWarps / 2 * MT * 16 * RT * 8 * 4;  // the fold of the warps' sums, over the drained rings
  return ring > red ? ring : red;
}
template <int MT, int RT>
__global__ void __launch_bounds__(kThreads, MT * RT <= 8 ? 2 : 1) adapter_shrink_kernel(const ShrinkParams p) {
  constexpr int kStage = shrink_stage<MT, RT>(), kStages = ring_stages(kStage);
  extern __shared__ __align__(16) uint8_t smem[];
  float(*red)[MT * 16 * RT * 8] = reinterpret_cast<float(*)[MT * 16 * RT * 8]>(smem);
  uint8_t* ring_ptr = smem + threadIdx.x / 32 * (kStages * kStage) + threadIdx.x % 32 * 16;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(ring_ptr);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int g = lane / 4, t4 = lane % 4;
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int n_tiles = *p.n_tiles;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x);
  const int k_lo = blockIdx.y * p.k_block, k_hi = min(p.K, k_lo + p.k_block);
  for (int t = blockIdx.x; t < n_tiles; t += gridDim.x) {
    const Tile tile = p.tiles[t];
    if (tile.adapter < 0) continue;
    const __nv_bfloat16* a =
        static_cast<const __nv_bfloat16*>(p.a) + ((int64_t)tile.adapter * p.E + tile.expert) * p.r * p.K;
    int64_t row[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = m * 16 + h * 8 + g;
        row[m][h] = i < tile.count ? p.order[tile.start + i] : -1;
      }
    float acc[MT][RT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < RT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;

    auto issue = [&](int k0, int slot) {
      const uint32_t dst = ring + slot * kStage;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int k = k0 + 32 * c + 8 * t4;
        const bool in = k < k_hi;  // K and k_block are multiples of 8
#pragma unroll
        for (int n = 0; n < RT; ++n) {
          const bool on = in && n * 8 + g < p.r;
          copy16(dst + (c * RT + n) * 512, on ? a + (int64_t)(n * 8 + g) * p.K + k : a, on);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool on = in && row[m][h] >= 0;
            copy16(dst + (2 * RT + (c * MT + m) * 2 + h) * 512, on ? x + row[m][h] * p.K + k : x, on);
          }
      }
    };
    const int k_first = k_lo + warp * kUnit;
#pragma unroll
    for (int d = 0; d < kStages - 1; ++d) {
      if (k_first + d * kWarps * kUnit < k_hi) issue(k_first + d * kWarps * kUnit, d);
      copies_commit();
    }
    int slot = 0;
    for (int k0 = k_first; k0 < k_hi; k0 += kWarps * kUnit) {
      const int ahead = k0 + (kStages - 1) * kWarps * kUnit;
      if (ahead < k_hi) issue(ahead, slot == 0 ? kStages - 1 : slot - 1);
      copies_commit();
      copies_wait<kStages - 1>();
      const uint4* st = reinterpret_cast<const uint4*>(ring_ptr + slot * kStage);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint4 av[RT];
#pragma unroll
        for (int n = 0; n < RT; ++n) av[n] = st[(c * RT + n) * 32];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint4 x0 = st[(2 * RT + (c * MT + m) * 2) * 32], x1 = st[(2 * RT + (c * MT + m) * 2 + 1) * 32];
#pragma unroll
          for (int n = 0; n < RT; ++n) {
            mma_bf16(acc[m][n], x0.x, x1.x, x0.y, x1.y, av[n].x, av[n].y);
            mma_bf16(acc[m][n], x0.z, x1.z, x0.w, x1.w, av[n].z, av[n].w);
          }
        }
      }
      if (++slot == kStages) slot = 0;
    }
    // the warps' sums: halves are folded, in a fixed order
#pragma unroll
    for (int half = kWarps / 2; half > 0; half >>= 1) {
      __syncthreads();
      if (warp >= half && warp < 2 * half) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < RT; ++n)
            *reinterpret_cast<float4*>(&red[warp - half][((m * RT + n) * 32 + lane) * 4]) =
                make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
      }
      __syncthreads();
      if (warp < half) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < RT; ++n) {
            const float4 o = *reinterpret_cast<const float4*>(&red[warp][((m * RT + n) * 32 + lane) * 4]);
            acc[m][n][0] += o.x;
            acc[m][n][1] += o.y;
            acc[m][n][2] += o.z;
            acc[m][n][3] += o.w;
          }
      }
    }
    if (warp == 0) {
      float* u = p.u + ((int64_t)blockIdx.y * p.rows + tile.start) * p.r;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < RT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int i = m * 16 + h * 8 + g, c = n * 8 + 2 * t4;
            if (i < tile.count && c < p.r)
              *reinterpret_cast<float2*>(u + (int64_t)i * p.r + c) = make_float2(acc[m][n][2 * h], acc[m][n][2 * h + 1]);
          }
    }
    __syncthreads();  // the fold is read before the next tile's copies land there
  }
}

// fp32: a warp takes 4 rows x 8 ranks at a time, the lanes split the inputs
__global__ void __launch_bounds__(kThreads) adapter_shrink_f32_kernel(const ShrinkParams p) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int n_tiles = *p.n_tiles;
  const float* x = static_cast<const float*>(p.x);
  const int k_lo = blockIdx.y * p.k_block, k_hi = min(p.K, k_lo + p.k_block);
  const int ranks = p.r / 8;
  for (int t = blockIdx.x; t < n_tiles; t += gridDim.x) {
    const Tile tile = p.tiles[t];
    if (tile.adapter < 0) continue;
    const float* a = static_cast<const float*>(p.a) + ((int64_t)tile.adapter * p.E + tile.expert) * p.r * p.K;
    const int units = (tile.count + 3) / 4 * ranks;
    for (int unit = warp; unit < units; unit += kWarps) {
      const int i0 = unit / ranks * 4, c0 = unit % ranks * 8;
      const float* xr[4];
      bool on[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        on[i] = i0 + i < tile.count;
        xr[i] = x + (int64_t)p.order[tile.start + (on[i] ? i0 + i : i0)] * p.K;
      }
      float acc[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[i][c] = 0.f;
      for (int k = k_lo + 4 * lane; k < k_hi; k += 128) {
        float4 xv[4], av[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) xv[i] = __ldg(reinterpret_cast<const float4*>(xr[i] + k));
#pragma unroll
        for (int c = 0; c < 8; ++c) av[c] = __ldg(reinterpret_cast<const float4*>(a + (int64_t)(c0 + c) * p.K + k));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            acc[i][c] = fmaf(xv[i].x, av[c].x, acc[i][c]);
            acc[i][c] = fmaf(xv[i].y, av[c].y, acc[i][c]);
            acc[i][c] = fmaf(xv[i].z, av[c].z, acc[i][c]);
            acc[i][c] = fmaf(xv[i].w, av[c].w, acc[i][c]);
          }
      }
      float* u = p.u + ((int64_t)blockIdx.y * p.rows + tile.start + i0) * p.r + c0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) acc[i][c] += __shfl_xor_sync(kFull, acc[i][c], off);
          if (lane == i * 8 + c && on[i]) u[(int64_t)i * p.r + c] = acc[i][c];
        }
    }
  }
}

// ---------------------------------------------------------------- expand
struct ExpandParams {
  const float* u;  // [S][rows][r]
  const void* b;   // [N, E, n_out, r]
  const float* scale;
  const void* base;  // [rows, n_out]
  void* out;         // [rows, f] (SwiGLU: n_out = 2 f) or [rows, n_out]
  const int32_t* order;
  const Tile* tiles;
  const int* n_tiles;
  int64_t rows;
  int r, E, S;
  int n_out, n_res;  // columns of base and of the result
  int col_block;     // result columns per block (blockIdx.x), whole rounds of the block's warps
  bool in_place;     // base is the result and nothing is applied to it: rows without an adapter are right
};

template <int EPI>
__device__ __forceinline__ float finish(float v, float up) {
  return EPI == kEpiSwiGLU ? silu_f(v) * up : EPI == kEpiGELU ? gelu_f(v) : v;
}

// SiLU for results that are rounded to bf16: __expf and __fdividef are off by
// under 2^-19 of the value for any argument that leaves one above 2^-126,
// against half a bf16 step of 2^-9; expf and the IEEE division made the kernel
// issue bound (285 against 94 us for the 2048-token batch below).
__device__ __forceinline__ float silu_fast(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

template <int EPI>
__device__ __forceinline__ float finish_bf16(float v, float up) {
  return EPI == kEpiSwiGLU ? silu_fast(v) * up : EPI == kEpiGELU ? gelu_f(v) : v;
}

// A warp takes 16 rows of the tile and 32 result columns (and, for SwiGLU, the
// matching 32 up columns) per round; the block's warps cover the tile's WR row
// groups side by side, so they share B through L1.  Column 2t+i of instruction
// j stands for result column 8t + 2j + i, so a lane ends with 8 consecutive
// columns of a row: base comes and the result leaves in 16-byte vectors.  U
// enters as a sum of two bf16 values (16 bits of mantissa), so its rounding
// does not show beside the result's own.
template <int RK, int EPI>
constexpr int expand_stage() { return (EPI == kEpiSwiGLU ? 2 : 1) * (2 * 512 + 4 * RK * 256); }
template <int RK, int EPI>
constexpr int expand_smem() { return kWarps * ring_stages(expand_stage<RK, EPI>()) * expand_stage<RK, EPI>(); }
template <int WR, int RK, int EPI>
__global__ void __launch_bounds__(kThreads, RK <= 2 ? 2 : 1) adapter_expand_kernel(const ExpandParams p) {
  constexpr int H = EPI == kEpiSwiGLU ? 2 : 1;
  constexpr int kStage = expand_stage<RK, EPI>(), kStages = ring_stages(kStage);
  constexpr int kB = 2 * H * 512;  // base first, then B
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* ring_ptr = smem + threadIdx.x / 32 * (kStages * kStage);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(ring_ptr);
  constexpr int CG = kWarps / WR;  // column groups of a round
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int g = lane / 4, t4 = lane % 4;
  const int i0 = warp % WR * 16;
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int n_tiles = *p.n_tiles;
  const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(p.base);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
  for (int t = blockIdx.y; t < n_tiles; t += gridDim.y) {
    const Tile tile = p.tiles[t];
    const bool has = tile.adapter >= 0;
    if ((!has && p.in_place) || i0 >= tile.count) continue;
    int64_t row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) row[h] = i0 + h * 8 + g < tile.count ? p.order[tile.start + i0 + h * 8 + g] : -1;
    const __nv_bfloat16* b = static_cast<const __nv_bfloat16*>(p.b) +
                             ((int64_t)(has ? tile.adapter : 0) * p.E + tile.expert) * p.n_out * p.r;
    const int c_first = blockIdx.x * p.col_block + warp / WR * 32;
    const int c_end = min(p.n_res, (int)((blockIdx.x + 1) * p.col_block));
    auto issue = [&](int c0, int slot) {
      const int col = c0 + 8 * t4;  // this lane's 8 result columns
      const uint32_t dst = ring + slot * kStage;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < H; ++q) {
          const bool on = col < p.n_res && row[h] >= 0;
          copy16(dst + (h * H + q) * 512 + lane * 16, on ? base + row[h] * p.n_out + q * p.n_res + col : base, on);
        }
#pragma unroll
      for (int q = 0; q < H; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = c0 + 8 * (g / 2) + 2 * j + (g & 1);
#pragma unroll
          for (int c = 0; c < RK; ++c) {
            const int k = 16 * c + 4 * t4;
            const bool on = has && n < p.n_res && k < p.r;
            copy8(dst + kB + ((q * 4 + j) * RK + c) * 256 + lane * 8,
                  on ? b + (int64_t)(q * p.n_res + n) * p.r + k : base, on);
          }
        }
    };
#pragma unroll
    for (int d = 0; d < kStages - 1; ++d) {
      if (c_first + d * CG * 32 < c_end) issue(c_first + d * CG * 32, d);
      copies_commit();
    }
    uint32_t hi[RK][4], lo[RK][4];  // U fragments: rows g, g+8; ranks 16 c + 4 t4 + {0,1} and {2,3}
    const float sc = has ? p.scale[tile.adapter] : 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int c = 0; c < RK; ++c) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        const int k = 16 * c + 4 * t4;
        if (has && row[h] >= 0 && k < p.r) {
          const float* u = p.u + (int64_t)(tile.start + i0 + h * 8 + g) * p.r + k;
#pragma unroll 4
          for (int s = 0; s < p.S; ++s) {
            const float4 w = __ldg(reinterpret_cast<const float4*>(u + (int64_t)s * p.rows * p.r));
            v.x += w.x;
            v.y += w.y;
            v.z += w.z;
            v.w += w.w;
          }
          v = make_float4(v.x * sc, v.y * sc, v.z * sc, v.w * sc);
        }
        hi[c][h] = pack_bf16x2(v.x, v.y);
        hi[c][2 + h] = pack_bf16x2(v.z, v.w);
        const __nv_bfloat162 p0 = *reinterpret_cast<__nv_bfloat162*>(&hi[c][h]);
        const __nv_bfloat162 p1 = *reinterpret_cast<__nv_bfloat162*>(&hi[c][2 + h]);
        lo[c][h] = pack_bf16x2(v.x - __low2float(p0), v.y - __high2float(p0));
        lo[c][2 + h] = pack_bf16x2(v.z - __low2float(p1), v.w - __high2float(p1));
      }
    }
    int slot = 0;
    for (int c0 = c_first; c0 < c_end; c0 += CG * 32) {
      const int ahead = c0 + (kStages - 1) * CG * 32;
      if (ahead < c_end) issue(ahead, slot == 0 ? kStages - 1 : slot - 1);
      copies_commit();
      copies_wait<kStages - 1>();
      const int col = c0 + 8 * t4;
      const bool in = col < p.n_res;
      const uint8_t* st = ring_ptr + slot * kStage;
      const uint4* st_base = reinterpret_cast<const uint4*>(st) + lane;
      const uint2* st_b = reinterpret_cast<const uint2*>(st + kB) + lane;
      if (++slot == kStages) slot = 0;
      float acc[H][4][4];
#pragma unroll
      for (int q = 0; q < H; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float(&d)[4] = acc[q][j];
          d[0] = d[1] = d[2] = d[3] = 0.f;
#pragma unroll
          for (int c = 0; c < RK; ++c) {
            const uint2 bv = st_b[((q * 4 + j) * RK + c) * 32];
            mma_bf16(d, lo[c][0], lo[c][1], lo[c][2], lo[c][3], bv.x, bv.y);
            mma_bf16(d, hi[c][0], hi[c][1], hi[c][2], hi[c][3], bv.x, bv.y);
          }
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!in || row[h] < 0) continue;
        uint4 bs[H];
#pragma unroll
        for (int q = 0; q < H; ++q) bs[q] = st_base[(h * H + q) * 32];
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[H][2];
#pragma unroll
          for (int q = 0; q < H; ++q) {
            const uint32_t w = j == 0 ? bs[q].x : j == 1 ? bs[q].y : j == 2 ? bs[q].z : bs[q].w;
            v[q][0] = __uint_as_float(w << 16) + acc[q][j][2 * h];
            v[q][1] = __uint_as_float(w & 0xffff0000u) + acc[q][j][2 * h + 1];
          }
          o[j] = pack_bf16x2(finish_bf16<EPI>(v[0][0], v[H - 1][0]), finish_bf16<EPI>(v[0][1], v[H - 1][1]));
        }
        *reinterpret_cast<uint4*>(out + row[h] * p.n_res + col) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// fp32: a thread takes one result column of the tile's (at most 16) rows; U
// is broadcast from shared memory
constexpr int kF32Rows = 16;
template <int EPI>
__global__ void __launch_bounds__(kThreads) adapter_expand_f32_kernel(const ExpandParams p) {
  constexpr int H = EPI == kEpiSwiGLU ? 2 : 1;
  __shared__ __align__(16) float su[kF32Rows][128];
  __shared__ int srow[kF32Rows];
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int n_tiles = *p.n_tiles;
  const float* base = static_cast<const float*>(p.base);
  float* out = static_cast<float*>(p.out);
  for (int t = blockIdx.y; t < n_tiles; t += gridDim.y) {
    const Tile tile = p.tiles[t];
    const bool has = tile.adapter >= 0;
    if (!has && p.in_place) continue;
    __syncthreads();
    for (int i = threadIdx.x; i < kF32Rows * p.r; i += kThreads) {
      const int rr = i / p.r, k = i % p.r;
      float v = 0.f;
      if (has && rr < tile.count) {
        const float* u = p.u + (int64_t)(tile.start + rr) * p.r + k;
        for (int s = 0; s < p.S; ++s) v += __ldg(u + (int64_t)s * p.rows * p.r);
        v *= p.scale[tile.adapter];
      }
      su[rr][k] = v;
    }
    if (threadIdx.x < tile.count) srow[threadIdx.x] = p.order[tile.start + threadIdx.x];
    __syncthreads();
    const float* b = static_cast<const float*>(p.b) + ((int64_t)(has ? tile.adapter : 0) * p.E + tile.expert) * p.n_out * p.r;
    const int c_end = min(p.n_res, (int)((blockIdx.x + 1) * p.col_block));
    for (int col = blockIdx.x * p.col_block + threadIdx.x; col < c_end; col += kThreads) {
      float acc[kF32Rows][H];
#pragma unroll
      for (int i = 0; i < kF32Rows; ++i)
#pragma unroll
        for (int q = 0; q < H; ++q) acc[i][q] = 0.f;
      if (has) {
        for (int k = 0; k < p.r; k += 4) {
          float4 bv[H];
#pragma unroll
          for (int q = 0; q < H; ++q)
            bv[q] = __ldg(reinterpret_cast<const float4*>(b + (int64_t)(q * p.n_res + col) * p.r + k));
#pragma unroll
          for (int i = 0; i < kF32Rows; ++i) {
            const float4 uv = *reinterpret_cast<const float4*>(&su[i][k]);
#pragma unroll
            for (int q = 0; q < H; ++q) {
              acc[i][q] = fmaf(uv.x, bv[q].x, acc[i][q]);
              acc[i][q] = fmaf(uv.y, bv[q].y, acc[i][q]);
              acc[i][q] = fmaf(uv.z, bv[q].z, acc[i][q]);
              acc[i][q] = fmaf(uv.w, bv[q].w, acc[i][q]);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kF32Rows; ++i) {
        if (i >= tile.count) break;
        const int64_t row = srow[i];
        float v[H];
#pragma unroll
        for (int q = 0; q < H; ++q) v[q] = base[row * p.n_out + q * p.n_res + col] + acc[i][q];
        out[row * p.n_res + col] = finish<EPI>(v[0], v[H - 1]);
      }
    }
  }
}

// ---------------------------------------------------------------- host side
// Rows of a tile: 16 (one MMA tile) where a pair has few rows or the rank's
// accumulators leave no room, more where the reuse of A and B pays
int tile_rows(const AdapterShape& s) {
  if (!s.bf16) return kF32Rows;
  const int64_t pairs = (int64_t)s.E * std::min<int64_t>(s.N, s.T);
  const int64_t per_pair = s.rows / std::max<int64_t>(1, pairs);
  return per_pair >= 24 && s.r <= 64 ? 32 : 16;
}

int64_t tiles_guess(const AdapterShape& s) {  // a likely number of tiles, for the grids only
  const int tm = tile_rows(s);
  const int64_t pairs = std::min<int64_t>(s.rows, (int64_t)s.E * std::min<int64_t>(s.N, s.T));
  return std::max<int64_t>(1, std::min<int64_t>(s.rows, s.rows / tm + pairs));
}

// Blocks that share one reduction of K inputs, and the inputs of each: enough
// for about four blocks per SM, at least 512 inputs (64 per warp) each
void split(const AdapterShape& s, int K, int* S, int* k_block) {
  const int64_t want = (4 * 148 + tiles_guess(s) - 1) / tiles_guess(s);
  const int most = (K + 511) / 512;
  const int n = (int)std::max<int64_t>(1, std::min<int64_t>(want, most));
  *k_block = ((K + n - 1) / n + 63) / 64 * 64;
  *S = (K + *k_block - 1) / *k_block;
}

constexpr size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct PlanLayout {
  size_t order, tiles, u, total;
};
PlanLayout layout(const AdapterShape& s) {
  int s1, s2, kb;
  split(s, s.d, &s1, &kb);
  split(s, s.f, &s2, &kb);
  PlanLayout l;
  l.order = kAdapterHeader;  // status word, number of tiles
  l.tiles = l.order + up256(sizeof(int32_t) * (size_t)s.rows);
  l.u = l.tiles + up256(sizeof(Tile) * (size_t)s.rows);
  l.total = l.u + up256(sizeof(float) * (size_t)std::max(s1, s2) * (size_t)s.rows * s.r);
  return l;
}

template <typename K>
cudaError_t allow_smem(K kernel, int smem) {
  return smem <= 48 * 1024 ? cudaSuccess
                           : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <int MT, int RT>
cudaError_t run_shrink(const ShrinkParams& p, dim3 grid, bool chained, cudaStream_t stream) {
  const cudaError_t e = allow_smem(adapter_shrink_kernel<MT, RT>, shrink_smem<MT, RT>());
  if (e != cudaSuccess) return e;
  return launch_maybe_chained(adapter_shrink_kernel<MT, RT>, grid, dim3(kThreads), shrink_smem<MT, RT>(), stream, chained, p);
}

cudaError_t launch_shrink(const ShrinkParams& p, int tm, bool bf16, dim3 grid, bool chained, cudaStream_t stream) {
  if (!bf16)
    return launch_maybe_chained(adapter_shrink_f32_kernel, grid, dim3(kThreads), 0, stream, chained, p);
  if (tm == 32) {
    if (p.r <= 8) return run_shrink<2, 1>(p, grid, chained, stream);
    if (p.r <= 16) return run_shrink<2, 2>(p, grid, chained, stream);
    if (p.r <= 32) return run_shrink<2, 4>(p, grid, chained, stream);
    return run_shrink<2, 8>(p, grid, chained, stream);
  }
  if (p.r <= 8) return run_shrink<1, 1>(p, grid, chained, stream);
  if (p.r <= 16) return run_shrink<1, 2>(p, grid, chained, stream);
  if (p.r <= 32) return run_shrink<1, 4>(p, grid, chained, stream);
  if (p.r <= 64) return run_shrink<1, 8>(p, grid, chained, stream);
  return run_shrink<1, 16>(p, grid, chained, stream);
}

template <int WR, int RK, int EPI>
cudaError_t run_expand(const ExpandParams& p, dim3 grid, cudaStream_t stream) {
  const int smem = expand_smem<RK, EPI>();
  const cudaError_t e = allow_smem(adapter_expand_kernel<WR, RK, EPI>, smem);
  if (e != cudaSuccess) return e;
  return launch_maybe_chained(adapter_expand_kernel<WR, RK, EPI>, grid, dim3(kThreads), smem, stream, true, p);
}

template <int WR, int EPI>
cudaError_t launch_expand_r(const ExpandParams& p, dim3 grid, cudaStream_t stream) {
  if (p.r <= 16) return run_expand<WR, 1, EPI>(p, grid, stream);
  if (p.r <= 32) return run_expand<WR, 2, EPI>(p, grid, stream);
  if (p.r <= 64) return run_expand<WR, 4, EPI>(p, grid, stream);
  return run_expand<WR, 8, EPI>(p, grid, stream);
}

template <int EPI>
cudaError_t launch_expand(const ExpandParams& p, int tm, bool bf16, dim3 grid, cudaStream_t stream) {
  if (!bf16)
    return launch_maybe_chained(adapter_expand_f32_kernel<EPI>, grid, dim3(kThreads), 0, stream, true, p);
  if (tm == 32) return launch_expand_r<2, EPI>(p, grid, stream);
  return launch_expand_r<1, EPI>(p, grid, stream);
}

}  // namespace

size_t adapter_plan_bytes(const AdapterShape& s) { return layout(s).total; }

cudaError_t launch_adapter_plan(const AdapterShape& s, const int32_t* offsets, const int32_t* perm,
                                const int32_t* token_adapter, void* plan, int* status, bool chained,
                                cudaStream_t stream) {
  uint8_t* base = static_cast<uint8_t*>(plan);
  const PlanLayout l = layout(s);
  if (s.rows == 0) return cudaSuccess;
  PlanParams p{offsets, perm, token_adapter, s.rows, s.E, s.k, s.N, tile_rows(s),
               reinterpret_cast<int32_t*>(base + l.order), reinterpret_cast<Tile*>(base + l.tiles),
               reinterpret_cast<int*>(base + kAdapterTilesAt), status};
  const unsigned blocks = (unsigned)((s.rows + kChunkRows - 1) / kChunkRows);
  return launch_maybe_chained(adapter_plan_kernel, dim3(blocks), dim3(kPlanThreads), sizeof(int) * (size_t)(s.E + 1),
                              stream, chained, p);
}

cudaError_t launch_adapter_apply(const AdapterShape& s, const AdapterApply& a, bool chained, cudaStream_t stream) {
  if (s.rows == 0) return cudaSuccess;
  uint8_t* base = static_cast<uint8_t*>(a.plan);
  const PlanLayout l = layout(s);
  const int tm = tile_rows(s);
  const int K = a.gate_up ? s.d : s.f;
  const int n_res = a.gate_up ? s.f : s.d;
  const int n_out = a.gate_up && s.act == kEpiSwiGLU ? 2 * s.f : n_res;
  const int32_t* order = reinterpret_cast<const int32_t*>(base + l.order);
  const Tile* tiles = reinterpret_cast<const Tile*>(base + l.tiles);
  const int* n_tiles = reinterpret_cast<const int*>(base + kAdapterTilesAt);
  float* u = reinterpret_cast<float*>(base + l.u);
  int S, k_block;
  split(s, K, &S, &k_block);
  const int64_t guess = tiles_guess(s);
  const unsigned tiles_grid = (unsigned)std::min<int64_t>(guess, 4096);
  ShrinkParams sp{a.x, a.a, order, tiles, n_tiles, u, s.rows, K, s.r, s.E, k_block};
  cudaError_t e = launch_shrink(sp, tm, s.bf16, dim3(tiles_grid, (unsigned)S), chained, stream);
  if (e != cudaSuccess) return e;
  // columns per block: one round of the warps, more where there are enough tiles to fill the SMs
  const int kRound = 32 * kWarps / (s.bf16 ? tm / 16 : 1);
  const int64_t rounds = (n_res + kRound - 1) / kRound;
  const int64_t per = std::max<int64_t>(1, std::min<int64_t>(rounds, rounds * guess / (148 * 8)));
  const int col_block = (int)std::min<int64_t>(per, 16) * kRound;
  ExpandParams ep{u, a.b, a.scale, a.base, a.out, order, tiles, n_tiles, s.rows, s.r, s.E, S, n_out, n_res, col_block,
                  !a.gate_up && a.base == a.out};
  const dim3 grid((unsigned)((n_res + col_block - 1) / col_block), tiles_grid);
  if (!a.gate_up) return launch_expand<kEpiNone>(ep, tm, s.bf16, grid, stream);
  return s.act == kEpiSwiGLU ? launch_expand<kEpiSwiGLU>(ep, tm, s.bf16, grid, stream)
                             : launch_expand<kEpiGELU>(ep, tm, s.bf16, grid, stream);
}

}  // namespace moe
