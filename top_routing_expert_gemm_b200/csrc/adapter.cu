// Low-rank adapters of many requests beside the experts' projections:
//   v[row] = base[row] + s_n B[n, e] (A[n, e] x[row]),   n the adapter of the row's token, e its expert
// followed by the expert's activation for the first projection.  The base
// projection (the weights every request shares) is not touched: base is its
// output.  The layer's pages do not describe adapters; the expert is the one
// of "Mixture of Experts Explained: Routers, Active Parameters and VRAM".
//
// Three kernels:
//   plan    groups the rows of equal (expert, adapter) into tiles of up to 16
//           rows: chunks of 256 rows are sorted inside a block, so no global
//           sort and no histogram over the pairs is needed
//   shrink  U = A x per tile, the reduction over the inputs split over
//           blocks and the warps of each; partial sums in fp32, added in a
//           fixed order
//   expand  base + s B U per tile and column block, then the activation
// Measured (plan, shrink, expand): 2048 tokens, k = 2, 4096 -> 14336, 12 requests,
// rank 16: 8, 12, 86 us; 8192 tokens, k = 4, 2880 -> 2880, 24 requests, rank 8: 12,
// 41, 75; 64 tokens of 64 adapters, k = 2, 14336 -> 4096, rank 16: 6, 13, 12; one
// token, k = 2, 4096 -> 14336: 5, 4.5, 7.5.  Chained, a call takes 2 to 5 us less
// than their sum.
// Rows never meet; of the others in its batch a row's result depends by the
// order of U's partial sums at most, and equal calls give equal results.
//
// Bound by bytes: base and result once, x once, the touched adapters' A and B
// once (a tile reads its pair's weights, tiles of one pair meet in L2).  The
// products have a depth or width of rank, 8 to 128, so the tensor work is small
// and mma.sync does it, on tiles of 16 rows; a 128-row tcgen05 tile would be
// mostly empty.  In fp32 layers everything is fmaf on the CUDA cores.
#include <algorithm>

#include "common.cuh"
#include "kernels.cuh"
#include "pdl.cuh"
#include "tc_primitives.cuh"

namespace moe {
namespace {

constexpr int kChunkRows = 256;  // rows a plan block sorts
// Rows of a tile: one MMA tile.  Tiles of 32 rows (half the reads of A and B
// from L2) left too many of them half empty: the expand of the 2048-token
// batch of 12 requests took 100 us with them, 87 us with 16 rows.
constexpr int kTileRows = 16;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;
static_assert((int64_t)(kAdapterMaxPairs + 1) * kChunkRows < (int64_t(1) << 31), "keys of the plan are 31 bits");
constexpr int kSkip = 0x7fffff;  // pair of a row that is not there (kMaxPairs - 1 is below)

struct __align__(16) Tile {
  int start;    // position of its first row among the grouped rows: where its U lies
  int count;    // rows
  int adapter;  // -1: none
  int expert;
  int rows[kTileRows];
};
struct TileHead {  // in registers
  int start, count, adapter, expert;
};
__device__ __forceinline__ TileHead head_of(const Tile* t) {
  const int4 v = *reinterpret_cast<const int4*>(t);
  return TileHead{v.x, v.y, v.z, v.w};
}

// ---------------------------------------------------------------- plan
struct PlanParams {
  const int32_t* offsets;  // [E+1] or null: every row is there, expert 0
  const int32_t* perm;     // [rows] or null: row = token
  const int32_t* token_adapter;
  int64_t rows;
  int E, k, N;
  Tile* tiles;
  int2* n_tiles;             // the number of tiles; not 0: a chunk gave up
  int* turn;                 // several blocks: which chunk is next,
  unsigned long long* state; // and what is known of each (kKnown...)
  int* status;
  uint64_t wait_limit_ns;
  bool clear;  // one block: the status word is this call's own
};

// Four threads per row: each compares the row's key with a quarter of the
// chunk's.  A key holds (expert, adapter) above the row's place in the chunk, so
// all keys differ and one comparison ranks stably.
constexpr int kPlanThreads = 4 * kChunkRows;

// The tiles stand in the order of the chunks, so that equal calls cut them into
// equal runs and give equal results.  A chunk's place is the number of tiles
// before it (a scan with decoupled look-back): every block publishes its own
// number, and its first warp adds up those before it, 32 at a time, down to one
// that has published its total.
// Blocks take their chunks in turn, so whoever waits waits for running blocks.
// (Places from one atomic counter took 6.3 us against 8 for 16 chunks and 7 against
// 12 for 128, but then the order of the tiles, and with it the last bits of U,
// changed from call to call.)
constexpr unsigned long long kKnownOwn = 1, kKnownTotal = 2, kGivenUp = 3;  // low bits; the number above them
__device__ __forceinline__ int64_t tiles_before(const PlanParams& p, int64_t chunk, int64_t own, int lane) {
  volatile unsigned long long* state = p.state;
  if (lane == 0 && chunk > 0) state[chunk] = (unsigned long long)own << 2 | kKnownOwn;
  int64_t before = 0;
  bool over = chunk == 0, lost = false;
  uint64_t t0 = 0;
  for (int64_t last = chunk - 1; !over;) {
    const unsigned long long v = last >= lane ? state[last - lane] : +kKnownTotal;
    const unsigned total = __ballot_sync(kFull, (v & 3) == kKnownTotal), none = __ballot_sync(kFull, (v & 3) == 0);
    const unsigned upto = total ? (2u << (__ffs(total) - 1)) - 1 : kFull;  // the lanes that count
    lost = __any_sync(kFull, (v & 3) == kGivenUp);
    if (!(none & upto) && !lost) {
      int64_t n = upto >> lane & 1u ? (int64_t)(v >> 2) : 0;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(kFull, n, off);
      before += n;
      over = total != 0;
      last -= 32;
      continue;
    }
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    lost = __any_sync(kFull, lost || now - t0 > p.wait_limit_ns);
    if (lost) break;
  }
  if (lane == 0) {
    if (lost) {
      // This chunk's tiles will be missing, and a later chunk that has already
      // read its number counts them: the whole plan is void.
      p.n_tiles->y = 1;
      set_status(p.status, kDevTimeout);
    }
    state[chunk] = lost ? kGivenUp : (unsigned long long)(before + own) << 2 | kKnownTotal;
  }
  return lost ? -1 : before;
}

__global__ void __launch_bounds__(kPlanThreads) adapter_plan_kernel(const PlanParams p) {
  extern __shared__ int s_off[];  // [E+1]
  __shared__ __align__(16) int keys[kChunkRows];
  __shared__ int sorted[kChunkRows], s_row[kChunkRows];
  __shared__ int warp_sums[kChunkRows / 32];
  __shared__ int s_base, s_chunk;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  grid_dependency_wait();  // the dispatch (programmatic launch)
  if (tid == 0) grid_launch_dependents();
  const bool alone = gridDim.x == 1;
  if (!alone && tid == 0) s_chunk = atomicAdd(p.turn, 1);
  bool bad = false;
  if (p.offsets)
    for (int e = tid; e <= p.E; e += kPlanThreads) s_off[e] = p.offsets[e];
  __syncthreads();
  const int chunk = alone ? 0 : s_chunk;
  const int64_t row0 = (int64_t)chunk * kChunkRows;
  const int64_t row = row0 + tid;
  const int64_t live = p.offsets ? min((int64_t)s_off[p.E], p.rows) : p.rows;
  if (tid < kChunkRows) {
    int pair = kSkip;
    if (row < live) {
      int a = p.token_adapter[p.perm ? p.perm[row] / p.k : row];
      if (a >= p.N) {
        bad = true;
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
      s_row[rank] = (int)(row0 + i);
    }
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    if (p.clear) *p.status = bad ? kDevBadAdapterId : 0;
    else if (bad) set_status(p.status, kDevBadAdapterId);
  }
  // position tid of the sorted chunk starts a tile where its run starts, and
  // every kTileRows from there
  const int mine = tid < kChunkRows ? sorted[tid] : kSkip;
  bool head = false;
  int end = 0, place = 0;  // place: in its tile
  if (mine != kSkip) {
    int lo = 0, hi = tid;  // first position of the run (the pairs ascend)
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sorted[mid] < mine) lo = mid + 1;
      else hi = mid;
    }
    place = (tid - lo) % kTileRows;
    head = place == 0;
    if (head) {
      lo = tid + 1;
      hi = min(kChunkRows, tid + kTileRows);
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
  if (warp == 0) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kChunkRows / 32; ++w) n += warp_sums[w];
    const int64_t before = gridDim.x > 1 ? tiles_before(p, chunk, n, lane) : 0;
    __syncwarp();
    if (lane == 0) {
      if (chunk == (int)gridDim.x - 1) p.n_tiles->x = before < 0 ? 0 : (int)before + n;
      if (gridDim.x == 1) p.n_tiles->y = 0;  // otherwise cleared ahead of the launch
      s_base = (int)before;
      n = 0;
      for (int w = 0; w < kChunkRows / 32; ++w) {
        const int c = warp_sums[w];
        warp_sums[w] = n;
        n += c;
      }
    }
  }
  __syncthreads();
  if (mine != kSkip && s_base >= 0) {
    // the tile of a position: the heads up to it, less one
    Tile* tile = p.tiles + s_base + warp_sums[warp] + __popc(heads & (0xffffffffu >> (31 - lane))) - 1;
    tile->rows[place] = s_row[tid];
    if (head) {
      const int pair = mine - 1;
      *reinterpret_cast<int4*>(tile) =
          make_int4((int)(row0 + tid), end - tid, pair < 0 ? -1 : pair % p.N, pair < 0 ? 0 : pair / p.N);
    }
  }
}

// The tiles of a plan as the kernels that use it see them: none if a chunk gave
// up, since some of those counted were then never written.
__device__ __forceinline__ int planned_tiles(const int2* n_tiles) {
  const int2 n = *n_tiles;
  return n.y ? 0 : n.x;
}

// ---------------------------------------------------------------- shrink
struct ShrinkParams {
  const void* x;  // [rows, K]
  const void* a;  // [N, E, r, K]
  const Tile* tiles;
  const int2* n_tiles;
  float* u;       // [rows][r]: a tile's first partial sum, by tile.start
  float* more;    // [blocks][16][r]: the partial sums that continue a tile
  int K, r, E;
};

// The work is a list of units, kUnits of 512 inputs per tile, and every block
// takes an equal run of it.  A run holds whole tiles, and perhaps the end of a
// tile that an earlier block began and the beginning of one that a later block
// ends: the partial sum of a beginning goes to the tile's place in u, that of a
// continuation (a block has one at most) to the block's place in more, and the
// expand adds them in the order of the blocks.  While a block computes a piece it
// looks at the next one, and fetches its first inputs before it adds up the
// warps' sums: 41 against 45.5 us for 32768 rows of 2880, rank 8 (189 MB of x:
// 4.6 TB/s).
constexpr int kUnitInputs = 64 * kWarps;
// a / b for a >= 0: 64-bit divisions are slow, and the numbers seldom need them
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
  return a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
struct Run {
  int64_t lo, hi;
};
// With fewer units than blocks only so many blocks take part: no run between two
// others is empty.
__device__ __forceinline__ Run run_of(int64_t total, int block, int blocks) {
  blocks = (int)min((int64_t)blocks, total);
  if (block >= blocks) return Run{0, 0};
  return Run{quotient(total * block, blocks), quotient(total * (block + 1), blocks)};
}
// the block whose run holds a unit
__device__ __forceinline__ int block_of(int64_t unit, int64_t total, int blocks) {
  blocks = (int)min((int64_t)blocks, total);
  return (int)quotient((unit + 1) * blocks - 1, total);
}
// a tile's run of blocks that hold partial sums of it: first..last
struct Parts {
  int first, last;
};
__device__ __forceinline__ Parts parts_of(int tile, int n_tiles, int units, int blocks) {
  const int64_t total = (int64_t)n_tiles * units, at = (int64_t)tile * units;
  return Parts{block_of(at, total, blocks), block_of(at + units - 1, total, blocks)};
}
// U[i, k..k+3] of a tile, all partial sums.  Ordinary loads: the shrink may still
// write them when this kernel starts (pdl.cuh), and the read-only path is for
// what nobody writes as long as a kernel lives.
__device__ __forceinline__ float4 sum_parts(const float* u, const float* more, int start, Parts parts, int r,
                                            int i, int k) {
  float4 v = *reinterpret_cast<const float4*>(u + (int64_t)(start + i) * r + k);
#pragma unroll 4
  for (int b = parts.first + 1; b <= parts.last; ++b) {
    const float4 w = *reinterpret_cast<const float4*>(more + ((int64_t)b * kTileRows + i) * r + k);
    v.x += w.x;
    v.y += w.y;
    v.z += w.z;
    v.w += w.w;
  }
  return v;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Asynchronous copies into the warp's own ring in shared memory: a lane reads
// back only what it copied itself, so a wait_group is all the synchronisation
// there is.  Without `on` the destination is zeroed and nothing is read.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Stages of a warp's ring whose stage takes `bytes`: what two blocks per SM
// leave each of their warps (13.5 KiB), one stage at least, four at most
constexpr int ring_stages(int bytes) { return bytes * 4 <= 13824 ? 4 : bytes * 3 <= 13824 ? 3 : bytes * 2 <= 13824 ? 2 : 1; }

// 16 rows, up to RT rank tiles of 8.  A lane takes 8 consecutive inputs of a
// row with one 16-byte copy and uses them as the k indices 2t, 2t+1, 2t+8, 2t+9
// of two instructions: the sum runs over all inputs, so any assignment of inputs
// to k serves as long as x and A agree.  The warps of a block take 64 inputs each
// in turn and are added up at the end.
constexpr int kUnit = 64;  // inputs per warp and round: whole 128-byte lines of every row
template <int RT>
constexpr int shrink_stage() { return 2 * (2 + RT) * 512; }
template <int RT>
constexpr int shrink_smem() {
  return kWarps * (ring_stages(shrink_stage<RT>()) * shrink_stage<RT>() + RT * 512);  // the rings and the warps' sums
}
template <int RT>
__global__ void __launch_bounds__(kThreads, RT <= 8 ? 2 : 1) adapter_shrink_kernel(const ShrinkParams p) {
  constexpr int kStage = shrink_stage<RT>(), kStages = ring_stages(kStage);
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int g = lane / 4, t4 = lane % 4;
  uint8_t* ring_ptr = smem + warp * (kStages * kStage) + lane * 16;
  const uint32_t ring = tc::smem_u32(ring_ptr);
  float4* sums = reinterpret_cast<float4*>(smem + kWarps * kStages * kStage);  // [warps][RT][32]
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x);
  const int units = (p.K + kUnitInputs - 1) / kUnitInputs;
  const Run run = run_of((int64_t)planned_tiles(p.n_tiles) * units, blockIdx.x, gridDim.x);

  // a piece of the run is a tile's units, or what the run has of them.  The one
  // that starts at `at` is looked at while the one before it is computed:
  int64_t at = run.lo;
  TileHead next;
  int next_row[2], next_lo = 0, next_hi = 0;
  auto look = [&] {
    const int t = (int)quotient(at, units);
    next = head_of(&p.tiles[t]);
#pragma unroll
    for (int h = 0; h < 2; ++h) next_row[h] = p.tiles[t].rows[h * 8 + g];
    next_lo = (int)(at - (int64_t)t * units);
    next_hi = (int)min((int64_t)units, next_lo + (run.hi - at));
    at += next_hi - next_lo;
  };
  const __nv_bfloat16* a = nullptr;
  int count = 0, row[2], k_first = 0, k_hi = 0, slot = 0;
  float* u = nullptr;  // where the piece's sums go
  auto issue = [&](int k0, int to) {
    const uint32_t dst = ring + to * kStage;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int k = k0 + 32 * c + 8 * t4;
      const bool in = k < k_hi;  // K is a multiple of 8
#pragma unroll
      for (int n = 0; n < RT; ++n) {
        const bool on = in && n * 8 + g < p.r;
        copy16(dst + (c * RT + n) * 512, on ? a + (int64_t)(n * 8 + g) * p.K + k : a, on);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool on = in && h * 8 + g < count;
        copy16(dst + (2 * RT + c * 2 + h) * 512, on ? x + (int64_t)row[h] * p.K + k : x, on);
      }
    }
  };
  // the first copies of the piece that was looked at
  auto begin = [&] {
    count = next.count;
    row[0] = next_row[0];
    row[1] = next_row[1];
    a = static_cast<const __nv_bfloat16*>(p.a) + ((int64_t)next.adapter * p.E + next.expert) * p.r * p.K;
    u = next_lo == 0 ? p.u + (int64_t)next.start * p.r : p.more + (int64_t)blockIdx.x * kTileRows * p.r;
    k_hi = min(p.K, next_hi * kUnitInputs);
    k_first = next_lo * kUnitInputs + warp * kUnit;
#pragma unroll
    for (int d = 0; d < kStages - 1; ++d) {
      if (k_first + d * kWarps * kUnit < k_hi) issue(k_first + d * kWarps * kUnit, slot + d < kStages ? slot + d : slot + d - kStages);
      copies_commit();
    }
  };
  // the next piece with an adapter, from what is looked at; false at the run's end
  auto settle = [&](bool any) {
    while (any && next.adapter < 0) {
      any = at < run.hi;
      if (any) look();
    }
    return any;
  };
  bool any = at < run.hi;
  if (any) look();
  any = settle(any);
  if (any) begin();
  while (any) {
    any = at < run.hi;
    if (any) look();
    float acc[RT][4];
#pragma unroll
    for (int n = 0; n < RT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    for (int k0 = k_first; k0 < k_hi; k0 += kWarps * kUnit) {
      const int ahead = k0 + (kStages - 1) * kWarps * kUnit;
      if (ahead < k_hi) issue(ahead, slot == 0 ? kStages - 1 : slot - 1);
      copies_commit();
      copies_wait<kStages - 1>();
      const uint4* st = reinterpret_cast<const uint4*>(ring_ptr + slot * kStage);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4 x0 = st[(2 * RT + c * 2) * 32], x1 = st[(2 * RT + c * 2 + 1) * 32];
#pragma unroll
        for (int n = 0; n < RT; ++n) {
          const uint4 av = st[(c * RT + n) * 32];
          mma_bf16(acc[n], x0.x, x1.x, x0.y, x1.y, av.x, av.y);
          mma_bf16(acc[n], x0.z, x1.z, x0.w, x1.w, av.z, av.w);
        }
      }
      if (++slot == kStages) slot = 0;
    }
    // the next piece's first copies go out before the warps' sums are added up
    const int n_rows = count;
    float* to = u;
    any = settle(any);
    if (any) begin();
#pragma unroll
    for (int n = 0; n < RT; ++n)
      sums[(warp * RT + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
    __syncthreads();
    for (int i = threadIdx.x; i < RT * 32; i += kThreads) {  // in a fixed order
      float4 v[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v[w] = sums[w * RT * 32 + i];
#pragma unroll
      for (int half = kWarps / 2; half > 0; half >>= 1)
#pragma unroll
        for (int w = 0; w < half; ++w) {
          v[w].x += v[w + half].x;
          v[w].y += v[w + half].y;
          v[w].z += v[w + half].z;
          v[w].w += v[w + half].w;
        }
      const int i0 = i % 32 / 4, c = i / 32 * 8 + 2 * (i % 4);
      if (i0 < n_rows && c < p.r) *reinterpret_cast<float2*>(to + (int64_t)i0 * p.r + c) = make_float2(v[0].x, v[0].y);
      if (i0 + 8 < n_rows && c < p.r)
        *reinterpret_cast<float2*>(to + (int64_t)(i0 + 8) * p.r + c) = make_float2(v[0].z, v[0].w);
    }
    __syncthreads();
  }
}

// fp32: a warp takes 4 rows x 8 ranks at a time, the lanes split the inputs
__global__ void __launch_bounds__(kThreads) adapter_shrink_f32_kernel(const ShrinkParams p) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const float* x = static_cast<const float*>(p.x);
  const int ranks = p.r / 8;
  const int k_units = (p.K + kUnitInputs - 1) / kUnitInputs;
  const Run run = run_of((int64_t)planned_tiles(p.n_tiles) * k_units, blockIdx.x, gridDim.x);
  for (int64_t at = run.lo; at < run.hi;) {
    const int t = (int)quotient(at, k_units);
    const int* rows = p.tiles[t].rows;
    const TileHead tile = head_of(&p.tiles[t]);
    const int u_lo = (int)(at - (int64_t)t * k_units), u_hi = (int)min((int64_t)k_units, u_lo + (run.hi - at));
    at += u_hi - u_lo;
    if (tile.adapter < 0) continue;
    const int k_lo = u_lo * kUnitInputs, k_hi = min(p.K, u_hi * kUnitInputs);
    const float* a = static_cast<const float*>(p.a) + ((int64_t)tile.adapter * p.E + tile.expert) * p.r * p.K;
    const int units = (tile.count + 3) / 4 * ranks;
    for (int unit = warp; unit < units; unit += kWarps) {
      const int i0 = unit / ranks * 4, c0 = unit % ranks * 8;
      const float* xr[4];
      bool on[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        on[i] = i0 + i < tile.count;
        xr[i] = x + (int64_t)rows[on[i] ? i0 + i : i0] * p.K;
      }
      float acc[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[i][c] = 0.f;
      for (int k = k_lo + 4 * lane; k < k_hi; k += 128) {
        float4 xv[4], av[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) xv[i] = *reinterpret_cast<const float4*>(xr[i] + k);
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
      float* u = (u_lo == 0 ? p.u + (int64_t)tile.start * p.r : p.more + (int64_t)blockIdx.x * kTileRows * p.r) +
                 (int64_t)i0 * p.r + c0;
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
  const float* u;     // as the shrink left them
  const float* more;
  const void* b;   // [N, E, n_out, r]
  const float* scale;
  const void* base;  // [rows, n_out]
  void* out;         // [rows, f] (SwiGLU: n_out = 2 f) or [rows, n_out]
  const Tile* tiles;
  const int2* n_tiles;
  int64_t rows;
  int r, E;
  int units, shrink_blocks;  // the shrink's units per tile and its blocks
  int n_out, n_res;  // columns of base and of the result
  int col_block;     // fp32: result columns per block (blockIdx.x)
  bool in_place;     // base is the result and nothing is applied to it: rows without an adapter are right
  int stages, stage_bytes;  // bf16: the ring
  int* status;
  uint64_t wait_limit_ns;
};

template <int EPI>
__device__ __forceinline__ float finish(float v, float up) {
  return EPI == kEpiSwiGLU ? silu_f(v) * up : EPI == kEpiGELU ? gelu_f(v) : v;
}

// SiLU for results that are rounded to bf16, z / (1 + 2^(-z log2 e)) with the
// hardware's approximate exponential and reciprocal: their 2^-22 and the
// argument's rounding (|z| 2^-24 of the exponential) are lost under half a bf16
// step, 2^-9.  With expf and the IEEE division the kernel was issue bound.
// Denormals are flushed: the results there are below 2^-119.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {  // two products in one instruction
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 silu_fast2(float2 z) {
  float2 e = mul2(z, make_float2(-1.4426950408889634f, -1.4426950408889634f));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
  e = add2(e, make_float2(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
  return mul2(z, e);
}

// two results of one row, rounded to bf16
template <int EPI>
__device__ __forceinline__ uint32_t finish_bf16(float2 v, float2 up) {
  if (EPI == kEpiSwiGLU) v = mul2(silu_fast2(v), up);
  if (EPI == kEpiGELU) v = make_float2(gelu_f(v.x), gelu_f(v.y));
  return pack_bf16x2(v.x, v.y);
}

// The work is a list of rounds: a tile times two groups of 256 result columns
// (SwiGLU: one group and its up columns), tile after tile; every block takes an equal
// run of it, so the blocks end together whatever the tiles are.  A producer warp
// goes ahead of eight consumer warps: per tile it sums U, scales it and leaves it
// as MMA fragments in shared memory with the tile's rows (the eight would
// otherwise do it eight times, and wait for it), and per round it fetches the
// columns' rows of B (one contiguous piece per group) with bulk copies into a ring of
// stages under mbarriers.  A consumer warp takes 32 columns of each group and
// fetches its part of base itself, each lane its own 16-byte vectors, a
// round ahead and on into the next tile.  (base by bulk copies as well, a
// segment of each row, measured 186 against 117 us for 16-byte copies: at 256
// bytes a bulk copy costs more than it moves.)  One group per round and three
// blocks per SM instead of two took 83 against 76 us for 32768 rows of 2880, rank 8:
// the second group hides the first one's latencies.
//
// Measured: 4096 rows of 14336, SwiGLU, rank 16 (352 MB of base and result): 87 us,
// 4.1 TB/s; 32768 rows of 2880, rank 8 (377 MB): 76 us, 5.0 TB/s, of 6.5 that a copy
// reaches.  Not memory but the issue of dependent instructions bounds it (half the
// issue slots are used; without its activation the first takes 78 us, without
// its MMAs 73, without base or stores 88).
//
// Column 2t+i of instruction j stands for column 8t + 2j + i of the warp's 32, so
// a lane ends with 8 consecutive columns of a row: base is read and the result
// leaves in 16-byte vectors.  base is the accumulators' first value.  U enters
// as a sum of two bf16 values (16 bits of mantissa), so its rounding does not
// show beside the result's own.
//
// The first of the two values is kept finite, so that the second, what is left
// of U, is infinite or NaN where U is, and not inf - inf.
__device__ __forceinline__ float in_bf16(float v) {
  constexpr float kMost = 3.38953138925153547590e38f;
  return fminf(fmaxf(v, -kMost), kMost);
}
constexpr int kMaxStages = 8;
constexpr int kInfos = 4;  // tiles the producer may be ahead
struct ExpandHeader {
  uint64_t full[kMaxStages], empty[kMaxStages];  // stages of B
  uint64_t ifull[kInfos], iempty[kInfos];        // tiles
  int fill_par[kMaxStages];
  int abort;
};
template <int RK>
struct __align__(16) TileInfo {
  int q0, q_end;  // rounds of this block's run
  int count;      // rows; -1: the run is over
  int has;        // an adapter
  int rows[kTileRows];
  uint4 hi[RK][32], lo[RK][32];  // U, lane by lane: rows g, g + 8; ranks 16 c + 4 t4 + {0, 1} and {2, 3}
};
constexpr int kExpandHead = 256;
static_assert(sizeof(ExpandHeader) <= kExpandHead, "header of the expand ring");
constexpr int kExpandThreads = kThreads + 32;

template <int EPI>
struct ExpandShape {
  static constexpr int H = 2;             // column groups of a round: gate and up, or neighbours
  static constexpr int GW = 32 * kWarps;  // columns of a group
  static constexpr int CW = EPI == kEpiSwiGLU ? GW : H * GW;  // result columns of a round
  static constexpr int kAhead = 2;           // rounds of base in flight per warp, the current one included
  static constexpr int kSlot = 2 * H * 512;  // a warp's part of base
  static constexpr int kBase = kWarps * kAhead * kSlot;
  static int stage_bytes(int r) { return H * GW * r * 2; }
};

// Blocks per SM that the registers (and, below, the rings) leave room for
template <int RK, int EPI>
constexpr int expand_blocks() { return RK > 2 ? 1 : 2; }

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, int bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

template <int RK, int EPI>
__global__ void __launch_bounds__(kExpandThreads, expand_blocks<RK, EPI>())
    adapter_expand_kernel(const __grid_constant__ ExpandParams p) {
  using Sh = ExpandShape<EPI>;
  constexpr int H = Sh::H, CW = Sh::CW, GW = Sh::GW;
  constexpr bool kPair = EPI == kEpiSwiGLU;  // the groups are gate and up
  extern __shared__ __align__(16) uint8_t smem[];
  ExpandHeader* hd = reinterpret_cast<ExpandHeader*>(smem);
  TileInfo<RK>* infos = reinterpret_cast<TileInfo<RK>*>(smem + kExpandHead);
  uint8_t* bases = smem + kExpandHead + kInfos * sizeof(TileInfo<RK>);
  uint8_t* ring = bases + Sh::kBase;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int g = lane / 4, t4 = lane % 4;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      tc::mbar_init(tc::smem_u32(&hd->full[i]), 1);
      tc::mbar_init(tc::smem_u32(&hd->empty[i]), kWarps);
      hd->fill_par[i] = -1;
    }
    for (int i = 0; i < kInfos; ++i) {
      tc::mbar_init(tc::smem_u32(&hd->ifull[i]), 1);
      tc::mbar_init(tc::smem_u32(&hd->iempty[i]), kWarps);
    }
    hd->abort = 0;
    tc::fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  volatile int* abort_flag = &hd->abort;
  const int b_bytes = GW * p.r * 2;
  const int apart = kPair ? p.n_res : GW;  // columns between the groups, in base and B
  int stage = 0, info = 0;  // stages and tiles in turn, with their parities
  uint32_t phase = 0, info_phase = 0;

  if (warp == kWarps) {
    // ------------------------------------------------ producer
    const int rounds = (p.n_res + CW - 1) / CW;  // per tile
    const int n_tiles = planned_tiles(p.n_tiles);
    const Run run = run_of((int64_t)n_tiles * rounds, blockIdx.x, gridDim.x);
    for (int64_t at = run.lo;;) {
      const bool over = at >= run.hi;
      const int t = over ? 0 : (int)quotient(at, rounds);
      const TileHead tile = over ? TileHead{0, -1, -1, 0} : head_of(&p.tiles[t]);
      const int q0 = over ? 0 : (int)(at - (int64_t)t * rounds);
      const int q_end = over ? 0 : (int)min((int64_t)rounds, q0 + (run.hi - at));
      at += q_end - q0;
      const bool has = tile.adapter >= 0;
      if (!over && !has && p.in_place) continue;
      const int row = !over && lane < tile.count ? p.tiles[t].rows[lane & (kTileRows - 1)] : 0;
      float4 u[RK][2];
      if (has) {
        const Parts parts = parts_of(t, n_tiles, p.units, p.shrink_blocks);
        const float sc = p.scale[tile.adapter];
#pragma unroll
        for (int c = 0; c < RK; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            u[c][h] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int i = h * 8 + g, k = 16 * c + 4 * t4;
            if (i < tile.count && k < p.r) {
              const float4 v = sum_parts(p.u, p.more, tile.start, parts, p.r, i, k);
              u[c][h] = make_float4(v.x * sc, v.y * sc, v.z * sc, v.w * sc);
            }
          }
      }
      int ok = 0;
      if (lane == 0)
        ok = tc::mbar_wait_bounded(tc::smem_u32(&hd->iempty[info]), info_phase ^ 1u, abort_flag, p.wait_limit_ns,
                                   p.status);
      if (!__shfl_sync(kFull, ok, 0)) break;
      __syncwarp();  // what lane 0 has seen holds for the warp
      TileInfo<RK>& to = infos[info];
      if (lane == 0) *reinterpret_cast<int4*>(&to) = make_int4(q0, q_end, tile.count, has);
      if (lane < kTileRows) to.rows[lane] = row;
      if (has) {
#pragma unroll
        for (int c = 0; c < RK; ++c) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 v = u[c][h];
            hi[h] = pack_bf16x2(in_bf16(v.x), in_bf16(v.y));
            hi[2 + h] = pack_bf16x2(in_bf16(v.z), in_bf16(v.w));
            const __nv_bfloat162 p0 = *reinterpret_cast<__nv_bfloat162*>(&hi[h]);
            const __nv_bfloat162 p1 = *reinterpret_cast<__nv_bfloat162*>(&hi[2 + h]);
            lo[h] = pack_bf16x2(v.x - __low2float(p0), v.y - __high2float(p0));
            lo[2 + h] = pack_bf16x2(v.z - __low2float(p1), v.w - __high2float(p1));
          }
          to.hi[c][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          to.lo[c][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&hd->ifull[info]));
      if (++info == kInfos) {
        info = 0;
        info_phase ^= 1u;
      }
      if (over) break;
      if (!has) continue;
      ok = 1;
      if (lane == 0) {
        const __nv_bfloat16* b =
            static_cast<const __nv_bfloat16*>(p.b) + ((int64_t)tile.adapter * p.E + tile.expert) * p.n_out * p.r;
        for (int q = q0; q < q_end; ++q) {
          const int c0 = q * CW, cols = min(CW, p.n_res - c0);
          const uint32_t full = tc::smem_u32(&hd->full[stage]);
          ok = tc::mbar_wait_bounded(tc::smem_u32(&hd->empty[stage]), phase ^ 1u, abort_flag, p.wait_limit_ns,
                                     p.status);
          if (!ok) break;
          tc::mbar_expect_tx(full, (kPair ? 2 : 1) * cols * p.r * 2);
          hd->fill_par[stage] = (int)phase;
          const uint32_t dst = tc::smem_u32(ring + stage * p.stage_bytes);
#pragma unroll
          for (int h = 0; h < (kPair ? 2 : 1); ++h)
            bulk_copy(dst + h * b_bytes, b + (int64_t)(h * p.n_res + c0) * p.r, cols * p.r * 2, full);
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!__shfl_sync(kFull, ok, 0)) break;
    }
  } else {
    // ------------------------------------------------ consumers
    const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(p.base);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
    const int w0 = warp * 32 + 8 * t4;  // this lane's first column of a round
    const uint8_t* mine = bases + warp * (Sh::kAhead * Sh::kSlot) + lane * 16;
    const uint32_t mine32 = tc::smem_u32(mine);
    // fetching runs ahead of computing: its own place in the tiles
    int f_info = 0, f_q = 0, f_end = 0, f_slot = 0, ahead = 0;  // ahead: rounds fetched and not yet computed
    uint32_t f_phase = 0;
    bool f_over = false, f_on[2] = {false, false};
    const __nv_bfloat16* src[2][H];
    // one more round of base, if its tile is known; a group of copies of its own
    auto fetch = [&]() -> bool {
      if (f_q == f_end) {
        const int known = lane == 0 ? (int)tc::mbar_try_wait(tc::smem_u32(&hd->ifull[f_info]), f_phase) : 0;
        if (!__shfl_sync(kFull, known, 0)) return false;
        __syncwarp();  // what lane 0 has seen holds for the warp
        const TileInfo<RK>& ti = infos[f_info];
        if (ti.count < 0) {
          f_over = true;
          return false;
        }
        f_q = ti.q0;
        f_end = ti.q_end;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          f_on[i] = i * 8 + g < ti.count;
          const int64_t row = f_on[i] ? ti.rows[i * 8 + g] : 0;
#pragma unroll
          for (int h = 0; h < H; ++h) src[i][h] = base + row * p.n_out + h * apart + f_q * CW + w0;
        }
        if (++f_info == kInfos) {
          f_info = 0;
          f_phase ^= 1u;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const bool in = f_q * CW + (kPair ? 0 : h * GW) + w0 < p.n_res;
          copy16(mine32 + f_slot * Sh::kSlot + (i * H + h) * 512, src[i][h], in && f_on[i]);
          src[i][h] += CW;
        }
      copies_commit();
      ++f_q;
      ++ahead;
      f_slot = (f_slot + 1) % Sh::kAhead;
      return true;
    };
    // The lanes wait each for itself (so each sees what the barrier guards) and
    // go on or leave together: one whose limit expired must not part from those
    // that the shuffles, the MMAs and the block's barrier below wait for.
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(kFull, tc::mbar_wait_bounded(tc::smem_u32(bar), parity, abort_flag, p.wait_limit_ns, p.status));
    };
    int slot = 0;
    bool ok = true;
    while (ok) {
      ok = wait(&hd->ifull[info], info_phase);
      if (!ok) break;
      const TileInfo<RK>& ti = infos[info];
      const int4 head = *reinterpret_cast<const int4*>(&ti);
      if (head.z < 0) break;
      const bool has = head.w != 0;
      __nv_bfloat16* orow[2];
      bool on[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        on[i] = i * 8 + g < head.z;
        orow[i] = out + (on[i] ? (int64_t)ti.rows[i * 8 + g] * p.n_res : 0) + w0;
      }
      uint4 hi[RK], lo[RK];
#pragma unroll
      for (int c = 0; c < RK; ++c) {
        hi[c] = has ? ti.hi[c][lane] : make_uint4(0, 0, 0, 0);
        lo[c] = has ? ti.lo[c][lane] : make_uint4(0, 0, 0, 0);
      }
      for (int q = head.x; q < head.y; ++q) {
        if (ahead < Sh::kAhead && !f_over) fetch();
        if (ahead < Sh::kAhead && !f_over) fetch();  // until it is as far ahead as it may be
        // the copies of round q are the oldest of `ahead` groups
        static_assert(Sh::kAhead == 2, "one wait per depth");
        if (ahead == 2) copies_wait<1>();
        else copies_wait<0>();
        const int c0 = q * CW;
        const bool work = c0 + warp * 32 < p.n_res;  // else the second group has none either
        float acc[H][4][4];
        if (work) {
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const uint4 r0 = *reinterpret_cast<const uint4*>(mine + slot * Sh::kSlot + h * 512);
            const uint4 r1 = *reinterpret_cast<const uint4*>(mine + slot * Sh::kSlot + (H + h) * 512);
            const uint32_t w[2][4] = {{r0.x, r0.y, r0.z, r0.w}, {r1.x, r1.y, r1.z, r1.w}};
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                acc[h][j][2 * i] = __uint_as_float(w[i][j] << 16);
                acc[h][j][2 * i + 1] = __uint_as_float(w[i][j] & 0xffff0000u);
              }
          }
        }
        slot = (slot + 1) % Sh::kAhead;
        --ahead;
        if (has) {
          ok = wait(&hd->full[stage], phase);
          if (!ok) break;
          if (work) {
            const uint8_t* st =
                ring + stage * p.stage_bytes + (warp * 32 + 8 * (g / 2) + (g & 1)) * p.r * 2 + 8 * t4;
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint8_t* sb = st + h * b_bytes + j * 4 * p.r;
#pragma unroll
                for (int c = 0; c < RK; ++c) {
                  const uint2 bv = 16 * c + 4 * t4 < p.r ? *reinterpret_cast<const uint2*>(sb + 32 * c) : make_uint2(0, 0);
                  mma_bf16(acc[h][j], lo[c].x, lo[c].y, lo[c].z, lo[c].w, bv.x, bv.y);
                  mma_bf16(acc[h][j], hi[c].x, hi[c].y, hi[c].z, hi[c].w, bv.x, bv.y);
                }
              }
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(tc::smem_u32(&hd->empty[stage]));
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
#pragma unroll
        for (int h = 0; h < (kPair ? 1 : H); ++h) {
          if (!work || c0 + h * GW + w0 >= p.n_res) break;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!on[i]) continue;
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              o[j] = finish_bf16<EPI>(make_float2(acc[h][j][2 * i], acc[h][j][2 * i + 1]),
                                      make_float2(acc[H - 1][j][2 * i], acc[H - 1][j][2 * i + 1]));
            *reinterpret_cast<uint4*>(orow[i] + c0 + h * GW) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&hd->iempty[info]));
      if (++info == kInfos) {
        info = 0;
        info_phase ^= 1u;
      }
    }
  }
  copies_wait<0>();  // an aborted round may have left some
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // let the copies in flight land before the block's shared memory goes
    for (int i = 0; i < p.stages; ++i)
      if (hd->fill_par[i] >= 0) tc::drain_wait(tc::smem_u32(&hd->full[i]), (uint32_t)hd->fill_par[i]);
  }
  __syncthreads();
}

// fp32: a thread takes one result column of the tile's (at most 16) rows; U
// is broadcast from shared memory
template <int EPI>
__global__ void __launch_bounds__(kThreads) adapter_expand_f32_kernel(const ExpandParams p) {
  constexpr int H = EPI == kEpiSwiGLU ? 2 : 1;
  __shared__ __align__(16) float su[kTileRows][128];
  __shared__ int srow[kTileRows];
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int n_tiles = planned_tiles(p.n_tiles);
  const float* base = static_cast<const float*>(p.base);
  float* out = static_cast<float*>(p.out);
  for (int t = blockIdx.y; t < n_tiles; t += gridDim.y) {
    const int* rows = p.tiles[t].rows;
    const TileHead tile = head_of(&p.tiles[t]);
    const bool has = tile.adapter >= 0;
    if (!has && p.in_place) continue;
    __syncthreads();
    const Parts parts = parts_of(t, n_tiles, p.units, p.shrink_blocks);
    for (int i = threadIdx.x; i < kTileRows * p.r / 4; i += kThreads) {
      const int rr = i / (p.r / 4), k = i % (p.r / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (has && rr < tile.count) {
        const float sc = p.scale[tile.adapter];
        v = sum_parts(p.u, p.more, tile.start, parts, p.r, rr, k);
        v = make_float4(v.x * sc, v.y * sc, v.z * sc, v.w * sc);
      }
      *reinterpret_cast<float4*>(&su[rr][k]) = v;
    }
    if (threadIdx.x < tile.count) srow[threadIdx.x] = rows[threadIdx.x];
    __syncthreads();
    const float* b = static_cast<const float*>(p.b) + ((int64_t)(has ? tile.adapter : 0) * p.E + tile.expert) * p.n_out * p.r;
    const int c_end = min(p.n_res, (int)((blockIdx.x + 1) * p.col_block));
    for (int col = blockIdx.x * p.col_block + threadIdx.x; col < c_end; col += kThreads) {
      float acc[kTileRows][H];
#pragma unroll
      for (int i = 0; i < kTileRows; ++i)
#pragma unroll
        for (int q = 0; q < H; ++q) acc[i][q] = 0.f;
      if (has) {
        for (int k = 0; k < p.r; k += 4) {
          float4 bv[H];
#pragma unroll
          for (int q = 0; q < H; ++q)
            bv[q] = __ldg(reinterpret_cast<const float4*>(b + (int64_t)(q * p.n_res + col) * p.r + k));
#pragma unroll
          for (int i = 0; i < kTileRows; ++i) {
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
      for (int i = 0; i < kTileRows; ++i) {
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
int64_t tiles_guess(const AdapterShape& s) {  // a likely number of tiles, for the grids only
  const int64_t pairs = std::min<int64_t>(s.rows, (int64_t)s.E * std::min<int64_t>(s.N, s.T));
  return std::max<int64_t>(1, std::min<int64_t>(s.rows, s.rows / kTileRows + pairs));
}

// Blocks of the shrink: what the registers let be resident.  The plan's size
// does not depend on the device.
constexpr int kMaxShrinkBlocks = 512;
int shrink_blocks(const AdapterShape& s) {
  return std::min(kMaxShrinkBlocks, device_sm_count() * (s.bf16 && s.r > 64 ? 1 : 2));
}

constexpr size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct PlanLayout {
  size_t state, tiles, u, more, total;
};
int64_t chunks_of(const AdapterShape& s) { return (s.rows + kChunkRows - 1) / kChunkRows; }
PlanLayout layout(const AdapterShape& s) {
  PlanLayout l;
  l.state = kAdapterHeader;  // behind the status word, the number of tiles and the chunks' turn
  l.tiles = l.state + (s.rows > kChunkRows ? up256(sizeof(unsigned long long) * (size_t)chunks_of(s)) : 0);
  l.u = l.tiles + up256(sizeof(Tile) * (size_t)s.rows);
  l.more = l.u + up256(sizeof(float) * (size_t)s.rows * s.r);
  l.total = l.more + up256(sizeof(float) * (size_t)kMaxShrinkBlocks * kTileRows * s.r);
  return l;
}

template <typename K>
cudaError_t allow_smem(K kernel, int smem) {
  return smem <= 48 * 1024 ? cudaSuccess
                           : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <int RT>
cudaError_t run_shrink(const ShrinkParams& p, dim3 grid, cudaStream_t stream) {
  const cudaError_t e = allow_smem(adapter_shrink_kernel<RT>, shrink_smem<RT>());
  if (e != cudaSuccess) return e;
  return launch_maybe_chained(adapter_shrink_kernel<RT>, grid, dim3(kThreads), shrink_smem<RT>(), stream, true, p);
}

cudaError_t launch_shrink(const ShrinkParams& p, bool bf16, dim3 grid, cudaStream_t stream) {
  if (!bf16)
    return launch_maybe_chained(adapter_shrink_f32_kernel, grid, dim3(kThreads), 0, stream, true, p);
  if (p.r <= 8) return run_shrink<1>(p, grid, stream);
  if (p.r <= 16) return run_shrink<2>(p, grid, stream);
  if (p.r <= 32) return run_shrink<4>(p, grid, stream);
  if (p.r <= 64) return run_shrink<8>(p, grid, stream);
  return run_shrink<16>(p, grid, stream);
}

// As many blocks per SM as leave each a ring of two stages
template <int RK, int EPI>
cudaError_t run_expand(const ExpandParams& params, cudaStream_t stream) {
  using Sh = ExpandShape<EPI>;
  ExpandParams p = params;
  p.stage_bytes = Sh::stage_bytes(p.r);
  constexpr int kFixed = kExpandHead + kInfos * (int)sizeof(TileInfo<RK>) + Sh::kBase;
  int per_sm = expand_blocks<RK, EPI>(), room = 0;
  for (;; --per_sm) {
    room = 227 * 1024 / per_sm - (per_sm > 1 ? 1024 : 0) - kFixed;
    if (per_sm == 1 || room >= 2 * p.stage_bytes) break;
  }
  p.stages = std::min(kMaxStages, room / p.stage_bytes);
  const int smem = kFixed + p.stages * p.stage_bytes;
  const cudaError_t e = allow_smem(adapter_expand_kernel<RK, EPI>, smem);
  if (e != cudaSuccess) return e;
  const int64_t most = p.rows * ((p.n_res + Sh::CW - 1) / Sh::CW);  // rounds, if every row were a tile
  const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)device_sm_count() * per_sm);
  return launch_maybe_chained(adapter_expand_kernel<RK, EPI>, dim3(grid), dim3(kExpandThreads), smem, stream, true,
                              p);
}

template <int EPI>
cudaError_t launch_expand_r(const ExpandParams& p, cudaStream_t stream) {
  if (p.r <= 16) return run_expand<1, EPI>(p, stream);
  if (p.r <= 32) return run_expand<2, EPI>(p, stream);
  if (p.r <= 64) return run_expand<4, EPI>(p, stream);
  return run_expand<8, EPI>(p, stream);
}

template <int EPI>
cudaError_t launch_expand(const ExpandParams& p, bool bf16, dim3 grid, cudaStream_t stream) {
  if (!bf16)
    return launch_maybe_chained(adapter_expand_f32_kernel<EPI>, grid, dim3(kThreads), 0, stream, true, p);
  return launch_expand_r<EPI>(p, stream);
}

}  // namespace

size_t adapter_plan_bytes(const AdapterShape& s) { return layout(s).total; }

cudaError_t launch_adapter_plan(const AdapterShape& s, const int32_t* offsets, const int32_t* perm,
                                const int32_t* token_adapter, void* plan, int* status, uint64_t wait_limit_ns,
                                cudaStream_t stream) {
  uint8_t* base = static_cast<uint8_t*>(plan);
  const PlanLayout l = layout(s);
  if (s.rows == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)chunks_of(s);
  PlanParams p{offsets, perm, token_adapter, s.rows, s.E, s.k, s.N, reinterpret_cast<Tile*>(base + l.tiles),
               reinterpret_cast<int2*>(base + kAdapterTilesAt), reinterpret_cast<int*>(base + kAdapterTurnAt),
               reinterpret_cast<unsigned long long*>(base + l.state), status, wait_limit_ns, blocks == 1 && status == plan};
  return launch_maybe_chained(adapter_plan_kernel, dim3(blocks), dim3(kPlanThreads), sizeof(int) * (size_t)(s.E + 1),
                              stream, true, p);
}

size_t adapter_plan_clear_bytes(const AdapterShape& s) {
  return s.rows == 0 ? kAdapterHeader : s.rows > kChunkRows ? layout(s).tiles : 0;
}

cudaError_t launch_adapter_apply(const AdapterShape& s, const AdapterApply& a, cudaStream_t stream) {
  if (s.rows == 0) return cudaSuccess;
  uint8_t* base = static_cast<uint8_t*>(a.plan);
  const PlanLayout l = layout(s);
  const int K = a.gate_up ? s.d : s.f;
  const int n_res = a.gate_up ? s.f : s.d;
  const int n_out = a.gate_up && s.act == kEpiSwiGLU ? 2 * s.f : n_res;
  const Tile* tiles = reinterpret_cast<const Tile*>(base + l.tiles);
  const int2* n_tiles = reinterpret_cast<const int2*>(base + kAdapterTilesAt);
  float* u = reinterpret_cast<float*>(base + l.u);
  float* more = reinterpret_cast<float*>(base + l.more);
  const int blocks = shrink_blocks(s), units = (K + kUnitInputs - 1) / kUnitInputs;
  ShrinkParams sp{a.x, a.a, tiles, n_tiles, u, more, K, s.r, s.E};
  cudaError_t e = launch_shrink(sp, s.bf16, dim3((unsigned)blocks), stream);
  if (e != cudaSuccess) return e;
  // fp32: one round of the block's threads, more where there are enough tiles to fill the SMs
  const int64_t guess = tiles_guess(s);
  const int64_t rounds = (n_res + kThreads - 1) / kThreads;
  const int64_t per = std::max<int64_t>(1, std::min<int64_t>(rounds, rounds * guess / (device_sm_count() * 8)));
  const int col_block = (int)std::min<int64_t>(per, 16) * kThreads;
  ExpandParams ep{u, more, a.b, a.scale, a.base, a.out, tiles, n_tiles, s.rows, s.r, s.E, units, blocks, n_out, n_res,
                  col_block, !a.gate_up && a.base == a.out, 0, 0, a.status, a.wait_limit_ns};
  const dim3 grid((unsigned)((n_res + col_block - 1) / col_block), (unsigned)std::min<int64_t>(guess, 4096));
  if (!a.gate_up) return launch_expand<kEpiNone>(ep, s.bf16, grid, stream);
  return s.act == kEpiSwiGLU ? launch_expand<kEpiSwiGLU>(ep, s.bf16, grid, stream)
                             : launch_expand<kEpiGELU>(ep, s.bf16, grid, stream);
}

}  // namespace moe
