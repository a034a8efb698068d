// Routing from logits: scores, selection bias, expert groups, top-k and the
// routing weights (forward), and the gradient of the weights and of the two
// router penalties with respect to the logits (backward).
//
// "Mixture of Experts: why a model with 671 billion parameters uses only 37",
// "How many experts to pick and how to score them: top-k, softmax, sigmoid"
// (independent sigmoid scores, normalised over the selected set); "Mixture of
// experts: how MoE works and what it costs", "Why load balancing is the hard
// part of MoE" (a bias steers the selection, not the gate values).  Groups: a
// token first keeps the best Gk of G equal blocks of experts and picks inside
// them; the pages do not describe them.
//
// Mathematics, per row (token), over the experts that are available (logit
// above the lowest finite value of its type; -inf, NaN and that value mask):
//   s_i = sigmoid(l_i)  or  e^{l_i} / sum_j e^{l_j},      c_i = s_i + b_i
//   group score: the largest c, or the sum of the two largest, of the group
//   picked: the k largest c of the Gk best groups, ties to the lower index
//   w_i = scale * s_i  or  scale * s_i / sum over the picked
//
// A choice between two experts is an integer decided by floating point, so it
// must not depend on how s was rounded.  Without a bias c is increasing in l
// and the logits themselves are compared: exact.  Otherwise a row is decided
// in fp32 with a bound on its error, and where two neighbours in the order
// (or the last kept and the first dropped group) are closer than the bound,
// the warp decides the row again in binary64.  Measured on N(0, 1) logits with
// 256 experts: well under one row in a hundred.
//
// One warp per row: lane L holds the NC consecutive columns from L * NC, so an
// aligned group is a run of lanes.  Choices are compared as order-preserving
// integers, the picks come from a few candidates (pick_candidates).  Measured (8192 x 256, sigmoid, 8 groups, k = 8): RANK_US us,
// against 33 us for k rounds of maximum, owner and removal; 65536 x 128 in bf16
// with k = 4: RANK2_US against 61 us.  (A thread per row over a tile in shared
// memory, two-level maxima per thread: 75 and 39 us.)
#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxGroups = 32;  // a lane per group (the host check's limit)

template <typename T>
__device__ __forceinline__ float lowest();
template <>
__device__ __forceinline__ float lowest<float>() { return -3.40282346638528859812e38f; }
template <>
__device__ __forceinline__ float lowest<__nv_bfloat16>() { return __uint_as_float(0xff7f0000u); }

// -inf for an expert the row must not use; +inf counts as the largest finite value
template <typename T>
__device__ __forceinline__ float usable(float l) {
  return l > lowest<T>() ? fminf(l, 3.40282346638528859812e38f) : -INFINITY;
}

// Order-preserving integer of a float: 0 for -inf and NaN (what must not be
// picked), -0 and +0 alike.
__device__ __forceinline__ uint32_t key_of(float f) {
  const int b = __float_as_int(f + 0.0f);
  return f > -INFINITY ? (uint32_t)(b ^ (b >> 31 | (int)0x80000000)) : 0u;
}
__device__ __forceinline__ float float_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// 1 / (1 + e^-l) for the comparisons: the hardware's exponential (2^-22, and
// 2^-24 |l| from its argument, both weighted with s (1 - s)), one rounded sum
// and the hardware's reciprocal (2^-23) leave less than 2^-21.8.
__device__ __forceinline__ float sigmoid_fast(float l) {
  float e, q;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.0f + e));
  return q;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
  return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

// The NC columns of this lane; vec: rows start on 16 bytes (wide loads)
template <typename T, int NC>
__device__ __forceinline__ void load_cols(const T* row, int c0, int E, bool vec, float (&v)[NC]) {
  constexpr int V = 16 / sizeof(T);
  if (vec && c0 + NC <= E && NC * sizeof(T) >= 4) {
    if constexpr (NC % V == 0) {
#pragma unroll
      for (int i = 0; i < NC / V; ++i) {
        const Vec16<T> x = ld16(row + c0 + i * V);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i * V + j] = Elem<T>::to_f(x.v[j]);
      }
      return;
    } else if constexpr (NC * sizeof(T) == 8) {
      union { uint2 u; T t[NC]; } x;
      x.u = __ldg(reinterpret_cast<const uint2*>(row + c0));
#pragma unroll
      for (int j = 0; j < NC; ++j) v[j] = Elem<T>::to_f(x.t[j]);
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) v[j] = c0 + j < E ? Elem<T>::to_f(row[c0 + j]) : -INFINITY;
}

template <typename T, int NC>
__device__ __forceinline__ void store_cols(T* row, int c0, int E, bool vec, const float (&v)[NC]) {
  constexpr int V = 16 / sizeof(T);
  if (vec && c0 + NC <= E) {
    if constexpr (NC % V == 0) {
#pragma unroll
      for (int i = 0; i < NC / V; ++i) {
        Vec16<T> x;
#pragma unroll
        for (int j = 0; j < V; ++j) x.v[j] = Elem<T>::from_f(v[i * V + j]);
        st16(row + c0 + i * V, x);
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < NC; ++j)
    if (c0 + j < E) row[c0 + j] = Elem<T>::from_f(v[j]);
}

template <typename F>
__device__ __forceinline__ F neg_inf();
template <> __device__ __forceinline__ float neg_inf<float>() { return -INFINITY; }
template <> __device__ __forceinline__ double neg_inf<double>() { return -(double)INFINITY; }

// The picks of one row for any group shape, from the choices c (-inf: not to
// be picked) of the warp's columns.  Lane s < k returns slot s (-1: none
// left).  near: two values whose order decides something were within eps
// (group scores: 2 eps).  Used in fp32 where a group is no aligned run of
// lanes, and in binary64 for the rows whose fp32 decision was too close.
template <typename F, int NC>
__device__ __noinline__ int pick_any(F (&c)[NC], const RouteArgs& p, int lane, F eps, bool* near) {
  bool close = false;
  const int c0 = lane * NC;
  if (p.G > 1) {
    const int gs = p.E / p.G;
    F mine = neg_inf<F>();  // lane g: the score of group g
    for (int g = 0; g < p.G; ++g) {
      F a = neg_inf<F>(), b = neg_inf<F>();
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const F v = c0 + j >= g * gs && c0 + j < (g + 1) * gs ? c[j] : neg_inf<F>();
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        const F oa = __shfl_xor_sync(kFull, a, off), ob = __shfl_xor_sync(kFull, b, off);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
      }
      if (p.group_top == 2 && b > neg_inf<F>()) a += b;
      if (lane == g) mine = a;
    }
    int rank = 0;
    for (int g = 0; g < p.G; ++g) {
      const F o = __shfl_sync(kFull, mine, g);
      rank += o > mine || (o == mine && g < lane);
    }
    const unsigned kept = __ballot_sync(kFull, lane < p.G && rank < p.Gk);
    F lo = lane < p.G && rank < p.Gk ? mine : (F)INFINITY, hi = lane < p.G && rank >= p.Gk ? mine : neg_inf<F>();
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      lo = fmin(lo, __shfl_xor_sync(kFull, lo, off));
      hi = fmax(hi, __shfl_xor_sync(kFull, hi, off));
    }
    close = hi > neg_inf<F>() && lo - hi < 2 * eps;
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (c0 + j < p.E && !(kept >> ((c0 + j) / gs) & 1u)) c[j] = neg_inf<F>();
  }
  int id = -1;
  F prev = (F)INFINITY;
  for (int s = 0; s <= p.k; ++s) {  // the round after the last only looks how close the next one was
    F best = c[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < NC; ++j)
      if (c[j] > best) {
        best = c[j];
        at = j;
      }
    at += c0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const F ob = __shfl_xor_sync(kFull, best, off);
      const int oa = __shfl_xor_sync(kFull, at, off);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    if (!(best > neg_inf<F>())) break;
    close |= s > 0 && prev - best < eps;
    prev = best;
    if (s < p.k && lane == s) id = at;
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (c0 + j == at) c[j] = neg_inf<F>();
  }
  *near = close;
  return id;
}

// The k largest of the warp's columns from a few candidates.  key orders the
// columns as val does or more coarsely (equal keys of different values), 0 is
// not to be picked.  The k + 1 largest lane maxima give a threshold that at
// least k + 1 columns reach and hardly more; those are gathered in shared
// memory, one per lane, and each counts the candidates before it (larger val,
// or equal and a lower column): its rank.  Returns the number of candidates, over
// 32 if ties leave too many (then nothing else is done); lane s holds the
// candidate of rank s.
template <typename V>
struct Picks {
  V val[32];
  int col[32];
};
template <typename V, int NC>
__device__ __forceinline__ int pick_candidates(const uint32_t (&key)[NC], const V (&val)[NC], int k, int c0, int lane,
                                               Picks<V>* cand, Picks<V>* order) {
  uint32_t left = key[0], tau = 0;
#pragma unroll
  for (int j = 1; j < NC; ++j) left = max(left, key[j]);
  for (int s = 0; s <= k; ++s) {
    tau = __reduce_max_sync(kFull, left);
    if (left == tau) left = 0;  // lanes that tie leave together: tau only falls lower
  }
  tau = max(tau, 1u);
  int mine = 0;
#pragma unroll
  for (int j = 0; j < NC; ++j) mine += key[j] >= tau;
  int at = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(kFull, at, off);
    if (lane >= off) at += o;
  }
  const int n = __shfl_sync(kFull, at, 31);
  if (n > 32) return n;
  at -= mine;
#pragma unroll
  for (int j = 0; j < NC; ++j)
    if (key[j] >= tau) {
      cand->val[at] = val[j];
      cand->col[at] = c0 + j;
      ++at;
    }
  __syncwarp();
  const V v = lane < n ? cand->val[lane] : V(0);
  const int c = lane < n ? cand->col[lane] : 0;
  int rank = 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const V o = cand->val[i];
    // the candidates of a lane, and the lanes, come in ascending columns
    rank += o > v || (o == v && i < lane);
  }
  if (lane < n) {
    order->val[rank] = v;
    order->col[rank] = c;
  }
  __syncwarp();
  return n;
}

// The row again in binary64: scores from the fp32 or bf16 logits as stored.
// runs: groups are aligned runs of lanes_g lanes.
template <typename T, int NC>
__device__ __noinline__ int pick_exact(const RouteArgs& p, const T* row, int lane, bool runs, int lanes_g,
                                       Picks<double>* cand, Picks<double>* order) {
  const int c0 = lane * NC;
  double c[NC];
  double m = -(double)INFINITY;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    c[j] = c0 + j < p.E ? (double)usable<T>(Elem<T>::to_f(row[c0 + j])) : -(double)INFINITY;
    m = fmax(m, c[j]);
  }
  double z = 0.0;
  if (!p.sigmoid) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmax(m, __shfl_xor_sync(kFull, m, off));
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (c[j] > -(double)INFINITY) z += exp(c[j] - m);
    z = warp_sum(z);
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const double s = p.sigmoid ? 1.0 / (1.0 + exp(-c[j])) : exp(c[j] - m) / z;
    const double v = s + (p.bias && c0 + j < p.E ? (double)p.bias[c0 + j] : 0.0);
    c[j] = c[j] > -(double)INFINITY && v == v ? v : -(double)INFINITY;
  }
  if (p.G == 1 || runs) {
    bool kept = true;
    if (p.G > 1) {
      double a = -(double)INFINITY, b = a;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        b = fmax(b, fmin(a, c[j]));
        a = fmax(a, c[j]);
      }
      for (int off = 1; off < lanes_g; off <<= 1) {
        const double oa = __shfl_xor_sync(kFull, a, off), ob = __shfl_xor_sync(kFull, b, off);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
      }
      if (p.group_top == 2 && b > -(double)INFINITY) a += b;
      int rank = 0;
      for (int g = 0; g < p.G; ++g) {
        const double o = __shfl_sync(kFull, a, g * lanes_g);
        rank += o > a || (o == a && g < lane / lanes_g);
      }
      kept = c0 < p.E && rank < p.Gk;
    }
    uint32_t key[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) key[j] = kept ? key_of(fmaxf((float)c[j], c[j] > -(double)INFINITY ? lowest<float>() : -INFINITY)) : 0u;
    const int n = pick_candidates<double, NC>(key, c, p.k, c0, lane, cand, order);
    if (n <= 32) {
      const int id = lane < min(n, p.k) ? order->col[lane] : -1;
      __syncwarp();
      return id;
    }
  }
  double v[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) v[j] = c[j];
  bool unused;
  return pick_any<double, NC>(v, p, lane, 0.0, &unused);
}

// lanes < k of the warp hold a picked expert's logit l (-inf: empty slot):
// the weight before scaling and renormalisation, relative to a factor shared
// by the row's picks (which the renormalisation divides out): sigmoid scores
// far below zero are scaled by e^{-max l}, so that none underflows.
__device__ __forceinline__ float picked_score(bool sigmoid, bool renorm, float l, float top, float m, float z) {
  if (!(l > -INFINITY)) return 0.f;
  if (sigmoid) {
    if (renorm && top < 0.f) return expf(l - top) / (1.0f + expf(l));
    return 1.0f / (1.0f + expf(-l));
  }
  return renorm ? expf(l - top) : expf(l - m) / z;
}

template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) route_topk_kernel(const RouteArgs p) {
  const int lane = threadIdx.x % 32;
  const int c0 = lane * NC;
  const T* __restrict__ logits = static_cast<const T*>(p.logits);
  __shared__ Picks<double> s_picks[kWarps][2];  // candidates, and in order (also as floats)
  Picks<double>* exact = s_picks[threadIdx.x / 32];
  Picks<float>* cand = reinterpret_cast<Picks<float>*>(&exact[0]);
  Picks<float>* order = reinterpret_cast<Picks<float>*>(&exact[1]);
  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t t = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  if (threadIdx.x == 0) grid_launch_dependents();  // the dispatch may be scheduled (it waits for these ids)
  if (t >= p.T) return;

  float next[NC];
  load_cols<T, NC>(logits + t * p.stride, c0, p.E, p.vec, next);
  float b[NC];
  float bmax = 0.f;  // the largest |bias|: part of the bound on the choices' error
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    b[j] = p.bias && c0 + j < p.E ? p.bias[c0 + j] : 0.f;
    if (b[j] > -INFINITY) bmax = fmaxf(bmax, fabsf(b[j]));
  }
  bmax = warp_max(bmax);
  // groups as aligned runs of lanes, a power-of-two number of whole lanes each
  const int gs = p.E / p.G;
  const int lanes_g = gs / NC;
  const bool runs = p.G > 1 && gs % NC == 0 && (lanes_g & (lanes_g - 1)) == 0;
  // (otherwise pick_any decides)
  // c is increasing in l (no bias or a zero one, no sum over a group's two
  // best): compare logits
  bool zero = true;
#pragma unroll
  for (int j = 0; j < NC; ++j) zero &= b[j] == 0.f;
  const bool by_logit = __all_sync(kFull, zero) && (p.G == 1 || p.group_top == 1);
  const bool need_z = !p.sigmoid && (!by_logit || !p.renorm);

  for (; t < p.T; t += step) {
    const T* row = logits + t * p.stride;
    float c[NC];
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      c[j] = usable<T>(next[j]);
      m = fmaxf(m, c[j]);
    }
    if (t + step < p.T) load_cols<T, NC>(row + step * p.stride, c0, p.E, p.vec, next);

    // ---- choices and the bound on the error of a difference of two of them.
    // sigmoid: s is off by less than 2^-21 (sigmoid_fast), the sum with b by
    // 2^-24 (1 + |b|).  softmax: every
    // probability is off by less than 2^-18 of the largest (the terms'
    // errors and the up to 37 additions of the denominator).
    float eps = 0.f, z = 1.f;
    if (need_z) {
      m = warp_max(m);
      z = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) z += c[j] > -INFINITY ? __expf(c[j] - m) : 0.f;
      z = warp_sum(z);
    }
    if (!by_logit) {
      if (p.sigmoid) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
          c[j] = c[j] > -INFINITY ? sigmoid_fast(c[j]) + b[j] : -INFINITY;
        eps = 0x1p-19f * (1.0f + bmax);
      } else {
        const float inv = 1.0f / z;
#pragma unroll
        for (int j = 0; j < NC; ++j)
          if (c[j] > -INFINITY) c[j] = fmaf(__expf(c[j] - m), inv, b[j]);
        eps = 0x1p-17f * inv + 0x1p-22f * (bmax + 1.0f * inv);
      }
    }

    int id = -1;
    float l = -INFINITY;  // lane s < k: the logit of slot s
    bool near = false;
    if (p.G > 1 && !runs) {
      float v[NC];  // pick_any takes its values by address: c stays in registers
#pragma unroll
      for (int j = 0; j < NC; ++j) v[j] = c[j] == c[j] ? c[j] : -INFINITY;  // a NaN bias masks too
      id = pick_any<float, NC>(v, p, lane, eps, &near);
    } else {
      uint32_t key[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j) key[j] = key_of(c[j]);
      if (p.G > 1) {
        // ---- the best two of each group inside its run of lanes, then its rank
        uint32_t a = 0, a2 = 0;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          a2 = max(a2, min(a, key[j]));
          a = max(a, key[j]);
        }
        for (int off = 1; off < lanes_g; off <<= 1) {
          const uint32_t oa = __shfl_xor_sync(kFull, a, off), ob = __shfl_xor_sync(kFull, a2, off);
          a2 = max(min(a, oa), max(a2, ob));
          a = max(a, oa);
        }
        uint32_t gk = a;
        if (p.group_top == 2 && a2) gk = key_of(float_of(a) + float_of(a2));
        if (c0 >= p.E) gk = 0;
        const int mine = lane / lanes_g;
        int rank = 0;
        for (int g = 0; g < p.G; ++g) {
          const uint32_t o = __shfl_sync(kFull, gk, g * lanes_g);
          rank += o > gk || (o == gk && g < mine);
        }
        const bool kept = c0 < p.E && rank < p.Gk;
        const uint32_t lo = __reduce_min_sync(kFull, kept ? gk : 0xffffffffu);
        const uint32_t hi = __reduce_max_sync(kFull, kept ? 0u : gk);
        near = hi && float_of(lo) - float_of(hi) < 2.0f * eps;
        if (!kept) {
#pragma unroll
          for (int j = 0; j < NC; ++j) key[j] = 0;
        }
      }
      const int n = pick_candidates<float, NC>(key, c, p.k, c0, lane, cand, order);
      if (n <= 32) {
        if (lane < min(n, p.k)) {
          id = order->col[lane];
          l = order->val[lane];
          near |= lane + 1 < n && l - order->val[lane + 1] < eps;
        }
        near = __any_sync(kFull, near);
      } else {
        // more columns tie than a warp has lanes: k rounds of the largest key,
        // the lowest lane that holds it, and its lowest column
        uint32_t best = key[0];
#pragma unroll
        for (int j = 1; j < NC; ++j) best = max(best, key[j]);
        float prev = INFINITY;
        for (int s = 0; s <= p.k; ++s) {  // the round after the last only looks how close the next one was
          const uint32_t top = __reduce_max_sync(kFull, best);
          if (top == 0) break;
          const float v = float_of(top);
          near |= prev - v < eps;
          prev = v;
          const int owner = __ffs(__ballot_sync(kFull, best == top)) - 1;
          int at = 0;
          if (lane == owner) {
#pragma unroll
            for (int j = NC - 1; j >= 0; --j) at = key[j] == top ? j : at;
            best = 0;
#pragma unroll
            for (int j = 0; j < NC; ++j) {
              key[j] = j == at ? 0u : key[j];
              best = max(best, key[j]);
            }
            at += c0;
          }
          at = __shfl_sync(kFull, at, owner);
          if (lane == s && s < p.k) {
            id = at;
            l = v;
          }
        }
      }
      __syncwarp();  // the candidates are read before the next row's are written
    }
    if (near) id = pick_exact<T, NC>(p, row, lane, runs, lanes_g, &exact[0], &exact[1]);

    // ---- weights: lane s < k holds slot s (its choice is its logit, or the row is read again)
    if (!by_logit || (p.G > 1 && !runs)) l = id >= 0 ? usable<T>(Elem<T>::to_f(row[id])) : -INFINITY;
    const float top = p.renorm ? warp_max(l) : 0.f;
    float zw = z;
    if (!p.sigmoid && !p.renorm) {  // probabilities as they are: the denominator with expf
      zw = 0.f;
      float lr[NC];
      load_cols<T, NC>(row, c0, p.E, p.vec, lr);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const float lu = usable<T>(lr[j]);
        zw += lu > -INFINITY ? expf(lu - m) : 0.f;
      }
      zw = warp_sum(zw);
    }
    float w = picked_score(p.sigmoid, p.renorm, l, top, m, zw);
    if (p.renorm) {
      const float sum = warp_sum(w);
      w = sum > 0.f ? w / sum : 0.f;
    }
    if (lane < p.k) {
      p.ids[t * p.k + lane] = id;
      p.w[t * p.k + lane] = w * p.scale;
    }
  }
}

// Gradient with respect to the logits of
//   sum_s grad_w[t,s] w[t,s]                       (the routing weights)
//   + cb * E sum_e f_e mean_t p[t,e]               (balance loss; f = counts / sum counts, a constant)
//   + cz * mean_t (log sum_e e^{l[t,e]})^2         (z-loss)
// with p the softmax over the available experts.  Per row, g = scale grad_w,
// q the picked scores over their sum S:
//   sigmoid, renormalised:  picked s += q_s (1 - sigma_s)(g_s - sum q g)
//   sigmoid:                picked s += g_s sigma_s (1 - sigma_s)
//   softmax, renormalised:  picked s += q_s (g_s - sum q g)
//   softmax:                i        += p_i ([i picked] g_i - sum over picked p g)
//   balance:                i        += (cb E / T) p_i (f_i - sum f p)
//   z-loss:                 i        += (2 cz / T) lse p_i
// The ids carry no gradient, and neither does the bias.  One warp per row,
// everything in fp32, one rounding to the logits' type at the store.  Bound by
// the row's bytes: the logits are read whole only where p is needed.
template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const RouteBackwardArgs p) {
  const int lane = threadIdx.x % 32;
  const int c0 = lane * NC;
  const T* __restrict__ logits = static_cast<const T*>(p.logits);
  T* __restrict__ grad = static_cast<T*>(p.grad);
  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t t = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  if (t >= p.T) return;

  const bool dense = p.balance != 0.f || p.z != 0.f || (!p.sigmoid && !p.renorm && p.grad_w);
  float f[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) f[j] = 0.f;
  if (p.balance != 0.f) {
    int64_t n = 0;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = c0 + j < p.E ? p.counts[c0 + j] : 0;
      f[j] = (float)c;
      n += c;
    }
    n = warp_sum(n);
    const float inv = n > 0 ? (float)(1.0 / (double)n) : 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) f[j] *= inv;
  }
  const float cb = p.balance * (float)p.E / (float)p.T, cz = 2.0f * p.z / (float)p.T;

  for (; t < p.T; t += step) {
    const T* row = logits + t * p.stride;
    int id = lane < p.k && p.grad_w ? p.ids[t * p.k + lane] : -1;
    if (id >= p.E) id = -1;
    const float g = id >= 0 ? p.grad_w[t * p.k + lane] * p.scale : 0.f;
    const float l = id >= 0 ? usable<T>(Elem<T>::to_f(row[id])) : -INFINITY;

    float v[NC];
    float m = 0.f, z = 1.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) v[j] = 0.f;
    if (dense) {
      load_cols<T, NC>(row, c0, p.E, p.vec, v);
      m = -INFINITY;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        v[j] = usable<T>(v[j]);
        m = fmaxf(m, v[j]);
      }
      m = warp_max(m);
      z = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        v[j] = v[j] > -INFINITY ? expf(v[j] - m) : 0.f;
        z += v[j];
      }
      z = warp_sum(z);
    }

    // ---- the picked slots (lane s < k)
    float part = 0.f, shared = 0.f;  // shared: what every p_i is multiplied with
    if (p.grad_w) {
      if (!p.sigmoid && !p.renorm) {
        const float pw = z > 0.f && l > -INFINITY ? expf(l - m) / z : 0.f;
        part = pw * g;
        shared = -warp_sum(part);
      } else {
        const float top = warp_max(l);
        float q = picked_score(p.sigmoid, p.renorm, l, top, 0.f, 1.f);
        const float rest = p.sigmoid && l > -INFINITY ? 1.0f / (1.0f + expf(l)) : 1.0f;  // 1 - sigmoid(l)
        if (p.renorm) {
          const float sum = warp_sum(q);
          q = sum > 0.f ? q / sum : 0.f;
          part = q * rest * (g - warp_sum(q * g));
        } else {
          part = q * rest * g;
        }
      }
    }
    if (dense) {
      const float inv = z > 0.f ? 1.0f / z : 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) v[j] *= inv;
      float fp = 0.f;
      if (p.balance != 0.f) {
#pragma unroll
        for (int j = 0; j < NC; ++j) fp = fmaf(f[j], v[j], fp);
        fp = warp_sum(fp);
      }
      if (p.z != 0.f && z > 0.f) shared += cz * (m + logf(z));
#pragma unroll
      for (int j = 0; j < NC; ++j) v[j] *= fmaf(cb, f[j] - fp, shared);
    }
    if (p.grad_w) {
      for (int s = 0; s < p.k; ++s) {
        const int at = __shfl_sync(kFull, id, s) - c0;
        const float add = __shfl_sync(kFull, part, s);
#pragma unroll
        for (int j = 0; j < NC; ++j) v[j] += at == j ? add : 0.f;
      }
    }
    store_cols<T, NC>(grad + t * p.stride, c0, p.E, p.vec, v);
  }
}

// Blocks: a warp per row up to a few resident blocks per SM, then rows in turn
unsigned blocks_for(int64_t T) {
  const int64_t cap = (int64_t)device_sm_count() * 12;
  const int64_t n = (T + kWarps - 1) / kWarps;
  return (unsigned)(n < cap ? n : cap);
}

template <typename T, typename F>
cudaError_t by_columns(int E, F&& run) {
  if (E <= 32) return run(std::integral_constant<int, 1>());
  if (E <= 64) return run(std::integral_constant<int, 2>());
  if (E <= 128) return run(std::integral_constant<int, 4>());
  if (E <= 256) return run(std::integral_constant<int, 8>());
  if (E <= 512) return run(std::integral_constant<int, 16>());
  return run(std::integral_constant<int, 32>());
}

bool rows_on_16(const void* p, int64_t stride, int eb) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * eb % 16 == 0;
}

}  // namespace

cudaError_t launch_route_topk(const RouteArgs& args, cudaStream_t stream) {
  if (args.T == 0) return cudaSuccess;
  if (args.G > kMaxGroups || args.k > kMaxTopK || args.E > kMaxExperts) return cudaErrorInvalidValue;
  RouteArgs a = args;
  a.vec = rows_on_16(a.logits, a.stride, a.bf16 ? 2 : 4);
  auto typed = [&](auto tag) {
    using T = decltype(tag);
    return by_columns<T>(a.E, [&](auto nc) {
      route_topk_kernel<T, decltype(nc)::value><<<blocks_for(a.T), kThreads, 0, stream>>>(a);
      return cudaGetLastError();
    });
  };
  return a.bf16 ? typed(__nv_bfloat16()) : typed(float());
}

cudaError_t launch_route_backward(const RouteBackwardArgs& args, cudaStream_t stream) {
  if (args.T == 0) return cudaSuccess;
  if (args.k > kMaxTopK || args.E > kMaxExperts) return cudaErrorInvalidValue;
  RouteBackwardArgs a = args;
  const int eb = a.bf16 ? 2 : 4;
  a.vec = rows_on_16(a.logits, a.stride, eb) && rows_on_16(a.grad, a.stride, eb);
  auto typed = [&](auto tag) {
    using T = decltype(tag);
    return by_columns<T>(a.E, [&](auto nc) {
      route_backward_kernel<T, decltype(nc)::value><<<blocks_for(a.T), kThreads, 0, stream>>>(a);
      return cudaGetLastError();
    });
  };
  return a.bf16 ? typed(__nv_bfloat16()) : typed(float());
}

}  // namespace moe
