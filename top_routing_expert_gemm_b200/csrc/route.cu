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
// the warp decides it again in binary64, as a rule over the few columns within
// reach (pick_near): about one row in three thousand of N(0, 1) logits, 256
// experts and a bias, and some 5 us for a warp that meets one.
//
// One warp per row: lane L holds the NC consecutive columns from L * NC, so an
// aligned group is a run of lanes.  Choices are compared as order-preserving
// integers, the picks come from a few candidates (pick_candidates).
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
// (2^-24 s) and the hardware's reciprocal (2^-23 s) leave less than 1.65 2^-23.
__device__ __forceinline__ float sigmoid_fast(float l) {
  float e, q;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.0f + e));
  return q;
}

__device__ __forceinline__ float warp_max(float v) {
  asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v));
  return v;
}
// e^x: the hardware's 2^t (2^-22) of the rounded t = x log2 e, corrected by what the rounding left out,
// about 2^-21.5 of the value.  From 88 on the correction is left out, since 2^t becomes infinite at 88.72
// and inf * left is no number (such x only occur in 1 / (1 + e^x), below 2^-126 and flushed to 0);
// below -87.34 the value is flushed to 0 and there is nothing to correct.
__device__ __forceinline__ float exp_near(float x) {
  const float t = x * 1.4426950408889634f;
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  const float left = fmaf(x, 1.4426950408889634f, -t);
  return fabsf(x) < 88.0f ? fmaf(e, left * 0.6931471805599453f, e) : e;
}
// 1 / x to 2^-23 (x of ordinary size, or infinite: 0)
__device__ __forceinline__ float rcp_near(float x) {
  float q;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(x));
  return q;
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

// A group's two largest choices added up.  In fp32 the sum stays above -inf,
// which is a group without experts: sums of biases below the range meet at its
// end, where they are close (the bound grows with the biases) and binary64 decides.
__device__ __forceinline__ float sum_of_two(float a, float b) { return fmaxf(a + b, lowest<float>()); }
__device__ __forceinline__ double sum_of_two(double a, double b) { return a + b; }

// The picks of one row for any group shape, from the choices c (-inf: not to
// be picked) of the warp's columns; the groups kept, the experts rank by them, or
// by their logits (row, not null).  G: the groups, 1 if they are chosen already.
// Lane s < k returns slot s (-1: none left).  near: two values whose order decides
// something were within eps (group scores: 2 eps).  Used in fp32 where a group is
// no aligned run of lanes, and in binary64 for the rows whose fp32 decision was
// too close.
template <typename T, typename F, int NC>
__device__ __noinline__ int pick_any(F (&c)[NC], const T* row, int G, const RouteArgs& p, int lane, F eps, bool* near) {
  bool close = false;
  const int c0 = lane * NC;
  if (G > 1) {
    const int gs = p.E / G;
    F mine = neg_inf<F>();  // lane g: the score of group g
    for (int g = 0; g < G; ++g) {
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
      if (p.group_top == 2 && b > neg_inf<F>()) a = sum_of_two(a, b);
      if (lane == g) mine = a;
    }
    int rank = 0;
    for (int g = 0; g < G; ++g) {
      const F o = __shfl_sync(kFull, mine, g);
      rank += o > mine || (o == mine && g < lane);
    }
    const unsigned kept = __ballot_sync(kFull, lane < G && rank < p.Gk);
    F lo = lane < G && rank < p.Gk ? mine : (F)INFINITY, hi = lane < G && rank >= p.Gk ? mine : neg_inf<F>();
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      lo = fmin(lo, __shfl_xor_sync(kFull, lo, off));
      hi = fmax(hi, __shfl_xor_sync(kFull, hi, off));
    }
    close = hi > neg_inf<F>() && !(lo - hi >= 2 * eps);  // or both infinite
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (c0 + j < p.E && !(kept >> ((c0 + j) / gs) & 1u)) c[j] = neg_inf<F>();
  }
  if (row) {
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (c[j] > neg_inf<F>()) c[j] = (F)usable<T>(Elem<T>::to_f(row[c0 + j]));
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

// No bias, or zeros
__device__ __forceinline__ bool no_bias(const RouteArgs& p, int lane) {
  bool zero = true;
  if (p.bias) {
#pragma unroll 1
    for (int c = lane; c < p.E; c += 32) zero &= p.bias[c] == 0.f;
  }
  return __all_sync(kFull, zero);
}

// The row again in binary64: scores from the fp32 or bf16 logits as stored.
// runs: groups are aligned runs of lanes_g lanes.  Without a bias, or with zeros
// (and groups by sums of two, or nothing would be close), the groups kept, the
// experts rank by their logits, which differ where saturated scores do not.
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
    const bool zero = no_bias(p, lane);
    uint32_t key[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if (!kept) c[j] = -(double)INFINITY;
      if (zero && c[j] > -(double)INFINITY) c[j] = (double)usable<T>(Elem<T>::to_f(row[c0 + j]));
      key[j] = c[j] > -(double)INFINITY ? key_of(fmaxf((float)c[j], lowest<float>())) : 0u;
    }
    const int n = pick_candidates<double, NC>(key, c, p.k, c0, lane, cand, order);
    if (n <= 32) {
      const int id = lane < min(n, p.k) ? order->col[lane] : -1;
      __syncwarp();
      return id;
    }
  }
  bool unused;
  const bool chosen = p.G == 1 || runs;
  return pick_any<T, double, NC>(c, !chosen && no_bias(p, lane) ? row : nullptr, chosen ? 1 : p.G, p, lane, 0.0, &unused);
}

// The picks of a row whose kept groups are certain but whose order is not: only
// the columns within reach of the k-th best, vk, can be picked, so only those
// (one per lane, seldom more than k + 2) are computed in binary64.  thr: vk less
// the bound; m, inv: the softmax's maximum and 1 / denominator.  Without a bias
// they rank by their logits (pick_exact).  Returns the
// number of candidates; over 32, nothing is decided.  Not unrolled: it runs for
// one row in a thousand, and its instructions come from far away.
template <typename T>
__device__ __noinline__ int pick_near(const RouteArgs& p, const T* row, int lane, uint32_t kept, float thr, float m,
                                      float inv, Picks<double>* cand, int* id) {
  const int gs = p.E / p.G;
  int n = 0;
  double z = 0.0;
#pragma unroll 1
  for (int c0 = 0; c0 < p.E; c0 += 256) {  // 256 columns' loads in flight: the row is in L2 at best
    float l[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + 32 * j + lane;
      l[j] = c < p.E ? usable<T>(Elem<T>::to_f(row[c])) : -INFINITY;
      b[j] = p.bias && c < p.E ? p.bias[c] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + 32 * j + lane;
      const float v = (p.sigmoid ? sigmoid_fast(l[j]) : __expf(l[j] - m) * inv) + b[j];
      const bool in = l[j] > -INFINITY && v > -INFINITY && v >= thr && (p.G == 1 || kept >> (c / gs) & 1u);
      const unsigned who = __ballot_sync(kFull, in);
      const int at = n + __popc(who & ((1u << lane) - 1u));
      if (in && at < 32) cand->col[at] = c;
      n += __popc(who);
    }
    if (!p.sigmoid) {
#pragma unroll 1
      for (int j = 0; j < 8; ++j)
        if (c0 + 32 * j + lane < p.E) {
          const float lj = usable<T>(Elem<T>::to_f(row[c0 + 32 * j + lane]));
          if (lj > -INFINITY) z += exp((double)lj - (double)m);
        }
    }
  }
  if (n > 32) return n;
  const bool zero = no_bias(p, lane);
  z = warp_sum(z);
  __syncwarp();
  const int c = lane < n ? cand->col[lane] : 0;
  const double l = (double)usable<T>(Elem<T>::to_f(row[c]));
  const double num = p.sigmoid ? 1.0 : exp(l - (double)m);
  const double v = zero ? l : num / (p.sigmoid ? 1.0 + exp(-l) : z) + (p.bias ? (double)p.bias[c] : 0.0);
  cand->val[lane] = v;
  __syncwarp();
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const double o = cand->val[i];
    rank += o > v || (o == v && i < lane);
  }
  __syncwarp();
  if (lane < n) cand->col[rank] = c;
  __syncwarp();
  *id = lane < min(n, p.k) ? cand->col[lane] : -1;
  __syncwarp();
  return n;
}

// lanes < k of the warp hold a picked expert's logit l (-inf: empty slot):
// the weight before scaling and renormalisation, relative to a factor shared
// by the row's picks (which the renormalisation divides out): sigmoid scores
// far below zero are scaled by e^{-max l}, so that none underflows.
__device__ __forceinline__ float picked_score(bool sigmoid, bool renorm, float l, float top, float m, float z) {
  if (!(l > -INFINITY)) return 0.f;
  if (sigmoid) {
    if (renorm && top < 0.f) return exp_near(l - top) * rcp_near(1.0f + exp_near(l));
    return rcp_near(1.0f + exp_near(-l));
  }
  return renorm ? exp_near(l - top) : exp_near(l - m) * rcp_near(z);
}

template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) route_topk_kernel(const __grid_constant__ RouteArgs p) {
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

    // ---- choices and eps, the bound on the error of a difference of two of them
    // (of two group scores: 2 eps).  sigmoid: s is off by less than 1.65 2^-23
    // (sigmoid_fast), the sum with b by 2^-24 (1 + |b|), so a difference of two
    // by less than 2^-22 (2.15 + 0.5 |b|); a sum of two adds its own rounding,
    // 2^-23 (1 + |b|): 2^-22 (5.3 + 2 |b|) for a difference of group scores.  softmax: every
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
        eps = 0x1p-22f * (2.75f + bmax);
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
    bool near = false, near_group = false;
    uint32_t groups = 0xffffffffu;  // the kept ones
    float vk = INFINITY;            // the last pick's choice
    if (p.G > 1 && !runs) {
      float v[NC];  // pick_any takes its values by address: c stays in registers
#pragma unroll
      for (int j = 0; j < NC; ++j) v[j] = c[j] == c[j] ? c[j] : -INFINITY;  // a NaN bias masks too
      id = pick_any<T, float, NC>(v, nullptr, p.G, p, lane, eps, &near_group);  // which of the two was close is not told
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
        if (p.group_top == 2 && a2) gk = key_of(sum_of_two(float_of(a), float_of(a2)));
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
        near_group = hi && !(float_of(lo) - float_of(hi) >= 2.0f * eps);  // or both infinite
        groups = __reduce_or_sync(kFull, kept ? 1u << mine : 0u);
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
        vk = n > 0 ? order->val[min(n, p.k) - 1] : INFINITY;
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
          vk = s < p.k ? v : vk;
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
    if (near && !near_group && pick_near<T>(p, row, lane, groups, vk - eps, m, 1.0f / z, &exact[0], &id) > 32)
      near_group = true;
    if (near_group) id = pick_exact<T, NC>(p, row, lane, runs, lanes_g, &exact[0], &exact[1]);

    // ---- weights: lane s < k holds slot s (its choice is its logit, or the row is read again)
    if (!by_logit || (p.G > 1 && !runs)) l = id >= 0 ? usable<T>(Elem<T>::to_f(row[id])) : -INFINITY;
    const float top = p.renorm ? warp_max(l) : 0.f;
    float zw = z;
    if (!p.sigmoid && !p.renorm) {  // probabilities as they are: the denominator with exp_near
      zw = 0.f;
      float lr[NC];
      load_cols<T, NC>(row, c0, p.E, p.vec, lr);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const float lu = usable<T>(lr[j]);
        zw += lu > -INFINITY ? exp_near(lu - m) : 0.f;
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

// Four threads per row, 32 rows per block, so that every instruction serves 8
// rows.  A row's columns are cut into blocks of up to 16 inside its groups;
// thread q takes the blocks q, q + 4, ...: it loads them (16-byte loads where rows
// and blocks are aligned), computes their choices, leaves them in shared memory
// and keeps the block maxima in registers.  A pick is the maximum of the block
// maxima (the first of equals) over the four threads; together they search that
// block for the column and for what its maximum is without it.
constexpr int kTileRows = 32;

struct TileShape {
  int gs, nbg, bl, blp, nb;  // columns of a group, blocks of it, columns of a block and their pitch, blocks
  int pitch, bmp;            // floats per row of the choices, and of the block maxima
};
__host__ __device__ inline TileShape tile_shape(int E, int G) {
  TileShape s;
  s.gs = E / G;
  s.nbg = (s.gs + 15) / 16;
  s.bl = (s.gs + 4 * s.nbg - 1) / (4 * s.nbg) * 4;
  s.blp = s.bl + 4;
  s.nb = G * s.nbg;
  // rows 16 floats apart modulo 32 and blocks 20: the four threads' 16-byte writes of two rows meet no bank conflict
  s.pitch = (s.nb * s.blp + 15) / 32 * 32 + 16;
  if (s.pitch < s.nb * s.blp) s.pitch += 32;
  s.bmp = s.nb | 1;
  return s;
}
__host__ __device__ inline size_t tile_smem(int E, int G) {
  const TileShape s = tile_shape(E, G);
  return sizeof(float) * (kTileRows * (size_t)(s.pitch + (G > 1 ? 2 * s.bmp + G : 0) + kMaxTopK) + 16 * s.nb) +
         kWarps * 2 * sizeof(Picks<double>);
}
// blocks of a row per thread, for E <= 32 NC
template <int NC>
constexpr int kTileBlocks = NC <= 4 ? 2 : NC / 2;

// n <= 16 columns as stored, -inf behind them (vec: in 16-byte loads)
template <typename T>
__device__ __forceinline__ void load_block(const T* row, int n, bool vec, float (&v)[16]) {
  constexpr int V = 16 / sizeof(T);
  if (vec) {  // n is a multiple of V
#pragma unroll
    for (int i = 0; i < 16 / V; ++i) {
      Vec16<T> x;
      if (i * V < n) x = ld16(row + i * V);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i * V + e] = i * V < n ? Elem<T>::to_f(x.v[e]) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = j < n ? Elem<T>::to_f(row[j]) : -INFINITY;
  }
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(kFull, v, 1));
  return fmaxf(v, __shfl_xor_sync(kFull, v, 2));
}

// BY_LOGIT: no bias and no sums over a group's two best, known at the launch, so
// no row is close and the calls that decide those are not in the kernel: 65536
// rows of 128, bf16, softmax: 13.3 against 17.0 us.
template <typename T, int NC, bool BY_LOGIT>
__global__ void __launch_bounds__(kThreads) route_tile_kernel(const __grid_constant__ RouteArgs p) {
  constexpr int NB = kTileBlocks<NC>;
  extern __shared__ __align__(16) float sm[];
  const TileShape sh = tile_shape(p.E, p.G);
  const int lane = threadIdx.x % 32, r = threadIdx.x / 4, q = threadIdx.x % 4;
  float* row_c = sm + r * sh.pitch;                                      // the row's choices, block after block
  float* s_bias = sm + kTileRows * sh.pitch;                             // [nb][16] bias, 0 behind a block
  float* row_id = s_bias + 16 * sh.nb + r * kMaxTopK;                    // the row's picks
  float* grp = s_bias + 16 * sh.nb + kTileRows * kMaxTopK;               // G > 1:
  float* bm = grp + r * (2 * sh.bmp + p.G);                              //   block maxima,
  float* bm2 = bm + sh.bmp;                                              //   and seconds,
  float* score = bm2 + sh.bmp;                                           //   group scores
  const size_t head = tile_smem(p.E, p.G) - kWarps * 2 * sizeof(Picks<double>);
  Picks<double>* exact = reinterpret_cast<Picks<double>*>(reinterpret_cast<uint8_t*>(sm) + head) + threadIdx.x / 32 * 2;
  if (threadIdx.x == 0) grid_launch_dependents();  // the dispatch may be scheduled (it waits for these ids)
  const int64_t t = (int64_t)blockIdx.x * kTileRows + r;
  const bool live = t < p.T;
  const T* row = static_cast<const T*>(p.logits) + (live ? t : 0) * p.stride;

  // ---- the bias: in shared memory, zero throughout?, and its largest
  float bmax = 0.f;
  bool zero = true;
  if (!BY_LOGIT && p.bias) {
    for (int i = threadIdx.x; i < 16 * sh.nb; i += kThreads) {
      const int b = i / 16, j = i % 16, at = b % sh.nbg * sh.bl + j;
      const float v = j < sh.bl && at < sh.gs ? p.bias[b / sh.nbg * sh.gs + at] : 0.f;
      s_bias[i] = v == v ? v : -INFINITY;  // a NaN bias masks too
      if (v > -INFINITY) bmax = fmaxf(bmax, fabsf(v));
      zero &= v == 0.f;
    }
    zero = __syncthreads_and(zero);
  }
  const bool by_logit = BY_LOGIT || (zero && (p.G == 1 || p.group_top == 1));
  const bool need_z = !p.sigmoid && (!by_logit || !p.renorm);
  if (!BY_LOGIT && !zero) {
    bmax = warp_max(bmax);
    float* part = reinterpret_cast<float*>(exact - threadIdx.x / 32 * 2);
    if (lane == 0) part[threadIdx.x / 32] = bmax;
    __syncthreads();
    bmax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    __syncthreads();
  }
  // whole vectors: rows on 16 bytes, groups and blocks of whole vectors
  const bool vec = p.vec && sh.gs * sizeof(T) % 16 == 0 && sh.bl * sizeof(T) % 16 == 0;

  float m = -INFINITY, z = 0.f, inv = 1.f;
  if (need_z) {
    for (int b = q; b < sh.nb; b += 4) {
      const int at = b % sh.nbg * sh.bl;
      float v[16];
      load_block<T>(row + b / sh.nbg * sh.gs + at, min(sh.bl, sh.gs - at), vec, v);
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        v[j] = usable<T>(v[j]);
        top = fmaxf(top, v[j]);
      }
      if (top > m) {
        z *= exp_near(m - top);
        m = top;
      }
      // a block's terms in a tree: few roundings, whatever the number of experts
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = v[j] > -INFINITY ? exp_near(v[j] - m) : 0.f;
#pragma unroll
      for (int half = 8; half > 0; half >>= 1)
#pragma unroll
        for (int j = 0; j < half; ++j) v[j] += v[j + half];
      z += v[0];
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      const float om = __shfl_xor_sync(kFull, m, off), oz = __shfl_xor_sync(kFull, z, off);
      const float top = fmaxf(m, om);
      z = (m > -INFINITY ? z * exp_near(m - top) : 0.f) + (om > -INFINITY ? oz * exp_near(om - top) : 0.f);
      m = top;
    }
    inv = 1.0f / z;
  }
  // the bounds of route_topk_kernel (the denominator here: up to 8 rescalings
  // of 2^-21.5 and 15 additions, together below 2^-18)
  const float eps = by_logit    ? 0.f
                    : p.sigmoid ? 0x1p-22f * (2.75f + bmax)
                                : 0x1p-17f * inv + 0x1p-22f * (bmax + 1.0f * inv);

  // ---- choices and block maxima; four blocks are loaded at a time
  const bool seconds = !BY_LOGIT && p.G > 1 && p.group_top == 2;
  float top[NB];
  constexpr int NL = NB < 4 ? NB : 4;
#pragma unroll
  for (int i0 = 0; i0 < NB; i0 += NL) {
    float v[NL][16];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int b = q + 4 * (i0 + i), at = b % sh.nbg * sh.bl;
      load_block<T>(row + b / sh.nbg * sh.gs + at, live && b < sh.nb ? min(sh.bl, sh.gs - at) : 0, vec, v[i]);
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int b = q + 4 * (i0 + i);
      float best = -INFINITY;
      if (b < sh.nb) {
        if (by_logit) {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[i][j] = usable<T>(v[i][j]);
        } else {
          float add[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 f = zero ? make_float4(0.f, 0.f, 0.f, 0.f) : reinterpret_cast<const float4*>(s_bias + 16 * b)[j];
            add[4 * j] = f.x;
            add[4 * j + 1] = f.y;
            add[4 * j + 2] = f.z;
            add[4 * j + 3] = f.w;
          }
          if (p.sigmoid) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[i][j] = v[i][j] > lowest<T>() ? sigmoid_fast(v[i][j]) + add[j] : -INFINITY;
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              v[i][j] = v[i][j] > lowest<T>() ? fmaf(__expf(usable<T>(v[i][j]) - m), inv, add[j]) : -INFINITY;
          }
        }
        float second = -INFINITY;
        if (seconds) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            second = fmaxf(second, fminf(best, v[i][j]));
            best = fmaxf(best, v[i][j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) best = fmaxf(best, v[i][j]);
        }
        float4* dst = reinterpret_cast<float4*>(row_c + b * sh.blp);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * j < sh.bl) dst[j] = make_float4(v[i][4 * j], v[i][4 * j + 1], v[i][4 * j + 2], v[i][4 * j + 3]);
        if (p.G > 1) {
          bm[b] = best;
          bm2[b] = second;
        }
      }
      top[i0 + i] = best;
    }
  }
  __syncwarp();

  bool near = false, near_group = false;
  uint32_t kept = 0xffffffffu;  // groups
  if (p.G > 1) {  // thread q scores and ranks the groups q, q + 4, ...
    for (int g = q; g < p.G; g += 4) {
      float a = -INFINITY, a2 = -INFINITY;
      for (int i = g * sh.nbg; i < (g + 1) * sh.nbg; ++i) {
        a2 = fmaxf(fminf(a, bm[i]), fmaxf(a2, bm2[i]));
        a = fmaxf(a, bm[i]);
      }
      score[g] = seconds && a2 > -INFINITY ? sum_of_two(a, a2) : a;
    }
    __syncwarp();
    kept = 0;
    float lo = INFINITY, hi = -INFINITY;
    for (int g = q; g < p.G; g += 4) {
      const float v = score[g];
      int rank = 0;
#pragma unroll 4
      for (int o = 0; o < p.G; ++o) rank += score[o] > v || (score[o] == v && o < g);
      if (rank < p.Gk) {
        kept |= 1u << g;
        lo = fminf(lo, v);
      } else {
        hi = fmaxf(hi, v);
      }
    }
    kept |= __shfl_xor_sync(kFull, kept, 1);
    kept |= __shfl_xor_sync(kFull, kept, 2);
    lo = -quad_max(-lo);
    hi = quad_max(hi);
    near_group = hi > -INFINITY && !(lo - hi >= 2.0f * eps);  // or both infinite
#pragma unroll
    for (int i = 0; i < NB; ++i)
      if (q + 4 * i < sh.nb && !(kept >> ((q + 4 * i) / sh.nbg) & 1u)) top[i] = -INFINITY;
  }

  // ---- k picks; the round after the last only looks how close the next one was
  int* ids = reinterpret_cast<int*>(row_id);
  float prev = INFINITY, vk = INFINITY;  // the pick before; the last one
  for (int s = 0; s <= p.k; ++s) {
    float best = top[0];
    int wb = q;
#pragma unroll
    for (int i = 1; i < NB; ++i) {
      wb = top[i] > best ? q + 4 * i : wb;
      best = fmaxf(best, top[i]);
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      const float ob = __shfl_xor_sync(kFull, best, off);
      const int ow = __shfl_xor_sync(kFull, wb, off);
      if (ob > best || (ob == best && ow < wb)) {
        best = ob;
        wb = ow;
      }
    }
    const bool any = best > -INFINITY;
    near |= any && prev - best < eps;
    prev = best;
    if (s == p.k) break;
    vk = any ? best : vk;
    // the block, four columns per thread (a row without candidates looks at its own block 0)
    if (!any) wb = 0;
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (4 * q < sh.bl) v = *reinterpret_cast<const float4*>(row_c + wb * sh.blp + 4 * q);
    int at = v.x == best ? 0 : v.y == best ? 1 : v.z == best ? 2 : v.w == best ? 3 : 99;
    at += 4 * q;
    at = min(at, __shfl_xor_sync(kFull, at, 1));
    at = min(at, __shfl_xor_sync(kFull, at, 2));
    const int mine = at - 4 * q;
    const float rest = quad_max(fmaxf(fmaxf(mine == 0 ? -INFINITY : v.x, mine == 1 ? -INFINITY : v.y),
                                      fmaxf(mine == 2 ? -INFINITY : v.z, mine == 3 ? -INFINITY : v.w)));
    if (any && mine >= 0 && mine < 4) row_c[wb * sh.blp + at] = -INFINITY;
#pragma unroll
    for (int i = 0; i < NB; ++i)
      if (any && wb == q + 4 * i) top[i] = rest;
    if (q == 0) ids[s] = any ? 16 * wb + at : -1;
    __syncwarp();
  }
  __syncwarp();
  for (int s = q; s < p.k; s += 4)  // places -> columns
    if (ids[s] >= 0) ids[s] = ids[s] / 16 / sh.nbg * sh.gs + ids[s] / 16 % sh.nbg * sh.bl + ids[s] % 16;
  __syncwarp();
  // rows that fp32 could not decide: the warp takes them one by one
  if (!BY_LOGIT && __any_sync(kFull, (near || near_group) && live)) {
    const int lanes_g = sh.gs / NC;
    const bool runs = p.G > 1 && sh.gs % NC == 0 && (lanes_g & (lanes_g - 1)) == 0;
    for (unsigned todo = __ballot_sync(kFull, (near || near_group) && live && q == 0); todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;  // the row's first lane
      const int rr = (threadIdx.x - lane + from) / 4;
      const T* other = static_cast<const T*>(p.logits) + (t - r + rr) * p.stride;
      bool whole = __shfl_sync(kFull, near_group, from);
      int id = -1;
      const uint32_t groups = __shfl_sync(kFull, kept, from);
      const float thr = __shfl_sync(kFull, vk - eps, from), om = __shfl_sync(kFull, m, from);
      const float oinv = __shfl_sync(kFull, inv, from);
      if (!whole) whole = pick_near<T>(p, other, lane, groups, thr, om, oinv, &exact[0], &id) > 32;
      if (whole) id = pick_exact<T, NC>(p, other, lane, runs, lanes_g, &exact[0], &exact[1]);
      if (lane < p.k) reinterpret_cast<int*>(s_bias + 16 * sh.nb)[rr * kMaxTopK + lane] = id;
      __syncwarp();
    }
  }

  // ---- weights: thread q takes the slots q, q + 4, ...
  float l[kMaxTopK / 4], most = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxTopK / 4; ++i) {
    const int s = q + 4 * i;
    l[i] = s < p.k && ids[s] >= 0 ? usable<T>(Elem<T>::to_f(row[ids[s]])) : -INFINITY;
    most = fmaxf(most, l[i]);
  }
  most = quad_max(most);
#pragma unroll
  for (int i = 0; i < kMaxTopK / 4; ++i)
    if (4 * i < p.k) {
      l[i] = picked_score(p.sigmoid, p.renorm, l[i], most, m, z);
      sum += l[i];
    }
  sum += __shfl_xor_sync(kFull, sum, 1);
  sum += __shfl_xor_sync(kFull, sum, 2);
  const float f = !p.renorm ? p.scale : sum > 0.f ? p.scale / sum : 0.f;
#pragma unroll
  for (int i = 0; i < kMaxTopK / 4; ++i) {
    const int s = q + 4 * i;
    if (live && s < p.k) {
      p.ids[t * p.k + s] = ids[s];
      p.w[t * p.k + s] = l[i] * f;
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
template <int NC>
constexpr int kBackwardBlocks = NC <= 2 ? 12 : NC <= 4 ? 10 : NC == 8 ? 8 : NC == 16 ? 5 : 3;  // resident per SM
template <typename T, int NC>
__global__ void __launch_bounds__(kThreads, kBackwardBlocks<NC>) route_backward_kernel(const __grid_constant__ RouteBackwardArgs p) {
  const int lane = threadIdx.x % 32;
  const int c0 = lane * NC;
  __shared__ __align__(16) float s_row[kWarps][32 * NC];
  float* row_sm = s_row[threadIdx.x / 32];
  const T* __restrict__ logits = static_cast<const T*>(p.logits);
  T* __restrict__ grad = static_cast<T*>(p.grad);
  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t t = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  if (t >= p.T) return;

  const bool dense = p.balance != 0.f || p.z != 0.f || (!p.sigmoid && !p.renorm && p.grad_w);
  const float cb = p.balance * (float)p.E / (float)p.T, cz = 2.0f * p.z / (float)p.T;
  // a row's inputs, fetched one row ahead
  float nv[NC], ng = 0.f;
  int nid = -1;
  auto fetch = [&](int64_t row_t) {
    if (dense) load_cols<T, NC>(logits + row_t * p.stride, c0, p.E, p.vec, nv);
    if (p.grad_w) {
      nid = lane < p.k ? p.ids[row_t * p.k + lane] : -1;
      ng = lane < p.k ? p.grad_w[row_t * p.k + lane] * p.scale : 0.f;
    }
  };
  fetch(t);

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
    // in two parts that the warp's integer sum takes
    n = ((int64_t)__reduce_add_sync(kFull, (int)(n >> 16)) << 16) + __reduce_add_sync(kFull, (unsigned)(n & 0xffff));
    const float inv = n > 0 ? (float)(1.0 / (double)n) : 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) f[j] *= inv;
  }

  for (; t < p.T; t += step) {
    const T* row = logits + t * p.stride;
    const int id = nid >= 0 && nid < p.E ? nid : -1;
    float v[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) v[j] = dense ? usable<T>(nv[j]) : 0.f;
    const float l = id >= 0 ? usable<T>(Elem<T>::to_f(row[id])) : -INFINITY;
    const float g = l > -INFINITY ? ng : 0.f;  // whatever it is at an empty slot or a masked expert
    if (t + step < p.T) fetch(t + step);

    // ---- maxima of the row and of the picks, then all sums in one pass
    float m = 0.f, top = 0.f, z = 0.f, fp = 0.f;
    if (dense) {
      m = v[0];
#pragma unroll
      for (int j = 1; j < NC; ++j) m = fmaxf(m, v[j]);
      m = warp_max(m);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        v[j] = v[j] > -INFINITY ? exp_near(v[j] - m) : 0.f;
        z += v[j];
        fp = fmaf(f[j], v[j], fp);
      }
    }
    // picked slots (lane s < k): q its score, up to a factor of the row where the weights are renormalised
    const bool whole = !p.sigmoid && !p.renorm;  // probabilities as they are
    float q = 0.f;
    if (p.grad_w) {
      if (!whole) top = p.renorm ? warp_max(l) : 0.f;
      q = whole ? (l > -INFINITY ? exp_near(l - m) : 0.f) : picked_score(p.sigmoid, p.renorm, l, top, 0.f, 1.f);
    }
    float S = q, D = q * g;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      z += __shfl_xor_sync(kFull, z, off);
      fp += __shfl_xor_sync(kFull, fp, off);
      S += __shfl_xor_sync(kFull, S, off);
      D += __shfl_xor_sync(kFull, D, off);
    }
    const float inv = z > 0.f ? rcp_near(z) : 0.f;
    float part = 0.f, shared = 0.f;  // shared: what every p_i is multiplied with
    if (p.grad_w) {
      const float rest = p.sigmoid && l > -INFINITY ? rcp_near(1.0f + exp_near(l)) : 1.0f;  // 1 - sigmoid(l)
      if (whole) {
        part = q * inv * g;
        shared = -D * inv;
      } else if (p.renorm) {
        const float is = S > 0.f ? rcp_near(S) : 0.f;
        part = q * is * rest * (g - D * is);
      } else {
        part = q * rest * g;
      }
      part = l > -INFINITY ? part : 0.f;  // also where the other slots' sums are infinite or NaN
    }
    if (dense) {
      if (p.z != 0.f && z > 0.f) shared += cz * (m + logf(z));
      const float mean = fp * inv;
#pragma unroll
      for (int j = 0; j < NC; ++j) v[j] = v[j] * inv * fmaf(cb, f[j] - mean, shared);
      if (!(fabsf(shared) < INFINITY)) {  // 0 times that is NaN, and a masked expert's gradient 0
#pragma unroll 1
        for (int j = 0; j < NC; ++j) {
          const bool in = c0 + j < p.E && usable<T>(Elem<T>::to_f(row[c0 + j])) > -INFINITY;
#pragma unroll
          for (int i = 0; i < NC; ++i) v[i] = i == j && !in ? 0.f : v[i];
        }
      }
    }
    if (p.grad_w) {
      // the picks' parts join the row in shared memory, repeated ids one after the other
      float* mine = row_sm + c0;
#pragma unroll
      for (int j = 0; j < NC; ++j) mine[j] = v[j];
      const unsigned same = __match_any_sync(kFull, id) & ((1u << lane) - 1u);
      const bool valid = id >= 0;
      __syncwarp();
      if (valid && same == 0) row_sm[id] += part;
      __syncwarp();
      if (__any_sync(kFull, valid && same != 0)) {
        for (int s = 1; s < p.k; ++s) {
          if (lane == s && valid && same != 0) row_sm[id] += part;
          __syncwarp();
        }
      }
#pragma unroll
      for (int j = 0; j < NC; ++j) v[j] = mine[j];
    }
    store_cols<T, NC>(grad + t * p.stride, c0, p.E, p.vec, v);
  }
}

// From this many rows (and up to 512 experts) four threads per row instead of a
// warp: fewer instructions, a longer chain.  Measured, us, warp / four threads:
//   rows    256 fp32,            512 bf16,        128 bf16,      8 fp32,
//           sigmoid in groups,   sigmoid, bias,   softmax, k 4   softmax, k 2
//           bias, k 8            k 16
//   16      4.3 / 8.7            5.2 / 15.8       3.4 / 3.8      3.0 / 2.8
//   1024    5.8 / 11.2           10.6 / 21.0      3.5 / 3.9      3.2 / 3.0
//   4096    11.7 / 13.8          19.3 / 26.1      6.3 / 4.0      3.9 / 3.0
//   8192    17.5 / 17.3          30.3 / 28.3      10.4 / 5.4     6.6 / 3.1
//   65536   96 / 53              152 / 150        68 / 13.2      41 / 9.0
// One bound for all: it is where the widest rows change over; narrow rows
// without a bias would at 4096 already, for 1 to 2 us.
constexpr int64_t kTileMinRows = 8192;

// Blocks: a warp per row up to a few resident blocks per SM, then rows in turn
unsigned blocks_for(int64_t T, int per_sm) {
  const int64_t cap = (int64_t)device_sm_count() * per_sm;
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
      constexpr int NC = decltype(nc)::value;
      if constexpr (NC <= 16) {
        if (a.T >= kTileMinRows && tile_shape(a.E, a.G).nb <= 4 * kTileBlocks<NC>) {
          const size_t smem = tile_smem(a.E, a.G);
          auto run = [&](auto kernel) {
            if (smem > 48 * 1024) {
              const cudaError_t e =
                  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
              if (e != cudaSuccess) return e;
            }
            kernel<<<(unsigned)((a.T + kTileRows - 1) / kTileRows), kThreads, smem, stream>>>(a);
            return cudaGetLastError();
          };
          if (!a.bias && (a.G == 1 || a.group_top == 1)) return run(route_tile_kernel<T, NC, true>);
          return run(route_tile_kernel<T, NC, false>);
        }
      }
      route_topk_kernel<T, decltype(nc)::value><<<blocks_for(a.T, 12), kThreads, 0, stream>>>(a);
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
      route_backward_kernel<T, decltype(nc)::value><<<blocks_for(a.T, kBackwardBlocks<decltype(nc)::value>), kThreads, 0, stream>>>(a);
      return cudaGetLastError();
    });
  };
  return a.bf16 ? typed(__nv_bfloat16()) : typed(float());
}

}  // namespace moe
