// The router in front of the layer: each token's k experts and their weights from
// its E logits, and the gradient of the logits from that of the weights.
//
//   score = softmax(logits) or sigmoid(logits), per token
//   key   = the logit; with a bias or a group limit: score + bias (in 64 bits)
//   limit: only the `limit` groups with the largest sum of their two largest keys stay, of which
//          a closed expert's counts as less than any number: those with two open experts before
//          those with one, and these before those with none
//   ids   = the k largest keys, the larger first, ties to the lower id
//   w_j   = factor * score of id j, or factor * score / (sum of the chosen scores)
// A logit of -inf is never chosen; slots with no expert left get id -1 and weight 0.
//
// A wave takes a token: lane l holds the R consecutive experts from l R on, so the
// first lane that holds the largest key also holds the lowest id.  Keys are compared
// as unsigned integers in the order of the numbers, 0 below them all.  The two
// numbers that a choice depends on have to order as they do in exact arithmetic:
// logits are compared as they are, and scores, which a float32 sigmoid rounds onto
// each other, in 64 bits.
//
// What is read and written is little (a token of 256 fp32 logits: 1 KB).  64 tokens, 8 of 256
// experts by sigmoid with a bias and a group limit: 6.4 us, a launch's latency and the k rounds of a
// wave's maximum, one after the other.  16384 tokens, 8 of 128 experts: 10.6 us for 5 MB; 16 waves
// to a SIMD hide the rounds' latency there, and the issue of some 400 vector instructions (counted in
// the source) of four cycles for each token takes the time.
#include <algorithm>
#include <type_traits>

#include "wave.h"

namespace moe {

namespace {

constexpr int kWaves = 4;        // tokens of a workgroup
constexpr int kMaxLimitGroups = 64;  // groups under a limit: one per lane

struct RouterArgs {
  const void* logits;       // [T][E]
  const float* bias;        // [E] or null
  const float* grad_w;      // backward: [T][k]
  int32_t* idx;             // [T][k]
  float* w;                 // [T][k]
  void* grad;               // backward: [T][E]
  int T, E, k, G, limit;
  int renorm;
  float factor;
};

// Numbers as unsigned integers of the same order, all above 0 (-0 as 0; no NaN).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
  return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = wave_max((uint32_t)(v >> 32));
  const uint32_t lo = wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ float wave_max_float(float x) {  // no NaN
  const uint32_t m = wave_max(ordered(x));
  return __uint_as_float(m & 0x80000000u ? m & 0x7fffffffu : ~m);
}

// Elements of the vectors that R consecutive ones of `bytes` each are moved in: at most
// 16 bytes (rows start on 16 bytes or on R elements, whichever is less).
template <int R, int bytes>
constexpr int kVecOf = R * bytes <= 16 ? R : 16 / bytes;

// R logits from expert e0 on (kVec: E is a multiple of R, and they are read as
// vectors); -inf past the last expert.
template <int R, bool kBf16, bool kVec>
__device__ __forceinline__ void load_logits(const RouterArgs& a, int t, int e0, float (&x)[R]) {
  typedef std::conditional_t<kBf16, uint16_t, uint32_t> raw_t;
  const raw_t* p = (const raw_t*)a.logits + (int64_t)t * a.E + e0;
  raw_t raw[R];
  if constexpr (kVec) {
    constexpr int C = kVecOf<R, sizeof(raw_t)>;
    typedef raw_t vec __attribute__((ext_vector_type(C)));
#pragma unroll
    for (int c = 0; c < R; c += C) {
      vec v{};
      if (e0 < a.E) v = *(const vec*)(p + c);
#pragma unroll
      for (int r = 0; r < C; ++r) raw[c + r] = v[r];
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) raw[r] = e0 + r < a.E ? p[r] : 0;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float f = __uint_as_float(kBf16 ? (uint32_t)raw[r] << 16 : (uint32_t)raw[r]);
    x[r] = e0 + r < a.E ? f : -INFINITY;
  }
}

// 1 / (1 + e^-x)
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Whether the wave's token holds a NaN or +inf.
template <int R>
__device__ __forceinline__ bool not_finite(const float (&x)[R]) {
  bool bad = false;
#pragma unroll
  for (int r = 0; r < R; ++r) bad |= !(x[r] < INFINITY);
  return __ballot(bad) != 0;
}

template <int R>
__device__ __forceinline__ float max_of(const float (&x)[R]) {
  float m = x[0];
#pragma unroll
  for (int r = 1; r < R; ++r) m = fmaxf(m, x[r]);
  return wave_max_float(m);
}

// The chosen logits' scores over their sum, for a lane with `kept` (0 otherwise).  All
// scores are divided by e^m, m the largest of those logits (for the sigmoid only where
// m < 0), so that it holds where they leave float32's range.
template <bool kSigmoid>
__device__ __forceinline__ float renormalized(float l, bool kept) {
  const float m = wave_max_float(kept ? l : -INFINITY);
  float s = 0.0f;
  if (kept) {
    if constexpr (kSigmoid) {
      const float m0 = fminf(m, 0.0f);  // (0 where there is an l > 0)
      s = l > 0.0f ? sigmoid(l) : expf(l - m0) / (1.0f + expf(l));
    } else {
      s = expf(l - m);
    }
  }
  const float total = wave_sum(s);
  return kept ? s / total : 0.0f;
}

template <int R, bool kBf16, bool kVec, bool kSigmoid, bool kScored>
__global__ void __launch_bounds__(64 * kWaves) router_top_k(RouterArgs a) {
  typedef std::conditional_t<kScored, uint64_t, uint32_t> key_t;
  extern __shared__ double group_keys[];  // kScored with a limit: [kWaves][E]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kWaves + wave;
  if (t >= a.T) return;
  const int e0 = lane * R;
  float x[R];
  load_logits<R, kBf16, kVec>(a, t, e0, x);
  int id = -1;          // lane j: slot j's expert and its logit
  float logit = -INFINITY;
  if (not_finite(x)) {
    // no order: the first k experts, with NaN for weights
    if (lane < a.k) {
      a.idx[(int64_t)t * a.k + lane] = lane < a.E ? lane : -1;
      a.w[(int64_t)t * a.k + lane] = __uint_as_float(0x7fc00000u);
    }
    return;
  }
  key_t key[R];
  if constexpr (kScored) {
    double score[R];
    if constexpr (kSigmoid) {
#pragma unroll
      for (int r = 0; r < R; ++r) score[r] = 1.0 / (1.0 + exp(-(double)x[r]));
    } else {
      const float m = max_of(x);
      double sum = 0.0;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        score[r] = x[r] > -INFINITY ? exp((double)x[r] - (double)m) : 0.0;
        sum += score[r];
      }
      sum = wave_sum(sum);
#pragma unroll
      for (int r = 0; r < R; ++r) score[r] /= sum;  // (a row of -inf: never used)
    }
    double k64[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float b = a.bias && e0 + r < a.E ? a.bias[e0 + r] : 0.0f;
      // (a bias that is no number closes its expert as -inf does)
      k64[r] = x[r] > -INFINITY && fabsf(b) < INFINITY ? score[r] + (double)b : -(double)INFINITY;
    }
    uint64_t kept = ~0ull;
    if (a.limit > 0) {
      double* mine = group_keys + wave * a.E;
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (e0 + r < a.E) mine[e0 + r] = k64[r];
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the wave reads its own writes
      __builtin_amdgcn_wave_barrier();
      const int size = a.E / a.G;
      double first = -(double)INFINITY, second = -(double)INFINITY;
      if (lane < a.G)
        for (int i = 0; i < size; ++i) {
          const double v = mine[lane * size + i];
          second = fmax(second, fmin(first, v));
          first = fmax(first, v);
        }
      double sum = size > 1 ? first + second : first;
      int before = 0;  // groups that come before the lane's
      // where a group has a closed expert among its two, those with more open ones come first
      if (size > 1 && __ballot(lane < a.G && sum == -(double)INFINITY) != 0) {
        const int open = (first > -(double)INFINITY ? 1 : 0) + (second > -(double)INFINITY ? 1 : 0);
        if (open < 2) sum = open == 1 ? first : 0.0;
        for (int g = 0; g < a.G; ++g) {
          const int n = __builtin_amdgcn_readlane(open, g);
          const double o = __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(sum), g),
                                            __builtin_amdgcn_readlane(__double2loint(sum), g));
          before += n > open || (n == open && (o > sum || (o == sum && g < lane))) ? 1 : 0;
        }
      } else {  // those with more, or as much and a lower number
        for (int g = 0; g < a.G; ++g) {
          const double o = __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(sum), g),
                                            __builtin_amdgcn_readlane(__double2loint(sum), g));
          before += o > sum || (o == sum && g < lane) ? 1 : 0;
        }
      }
      kept = __ballot(lane < a.G && before < a.limit);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (e0 + r < a.E && !(kept >> ((e0 + r) / size) & 1)) k64[r] = -(double)INFINITY;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) key[r] = k64[r] > -(double)INFINITY ? ordered(k64[r]) : 0;
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) key[r] = x[r] > -INFINITY ? ordered(x[r]) : 0;
  }
  for (int j = 0; j < a.k; ++j) {
    key_t best = key[0];
#pragma unroll
    for (int r = 1; r < R; ++r) best = key[r] > best ? key[r] : best;
    const key_t top = wave_max(best);
    if (top == 0) break;
    const int owner = __ffsll((unsigned long long)__ballot(best == top)) - 1;
    // the owner's first expert with that key, and its logit
    int at = 0;
    float l = x[0];
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
      if (key[r] == top) {
        at = r;
        l = x[r];
      }
    const int won = __builtin_amdgcn_readlane(e0 + at, owner);
    const float won_l =
        __int_as_float(__builtin_amdgcn_readlane(__float_as_int(l), owner));
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (e0 + r == won) key[r] = 0;
    if (lane == j) {
      id = won;
      logit = won_l;
    }
  }
  float w;
  if (a.renorm) {
    w = renormalized<kSigmoid>(logit, id >= 0);
  } else if constexpr (kSigmoid) {
    w = id >= 0 ? sigmoid(logit) : 0.0f;
  } else {
    const float m = max_of(x);
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) sum += x[r] > -INFINITY ? expf(x[r] - m) : 0.0f;
    sum = wave_sum(sum);
    w = id >= 0 ? expf(logit - m) / sum : 0.0f;
  }
  if (lane < a.k) {
    a.idx[(int64_t)t * a.k + lane] = id;
    a.w[(int64_t)t * a.k + lane] = w * a.factor;
  }
}

// Gradient.  With c = factor, g_j the gradient of w_j and q_j = w_j / c:
//   softmax            grad_e = sum_{j: id_j = e} p_e c g_j - p_e S,  S = sum_j p_j c g_j
//   softmax, renorm.   grad at id_j: q_j (c g_j - S),  S = sum_j q_j c g_j
//   sigmoid            grad at id_j: s_j (1 - s_j) c g_j
//   sigmoid, renorm.   grad at id_j: q_j (c g_j - S) (1 - s_j)
// Only the first is dense; slots with an id outside [0, E) or a logit of -inf were
// given no weight and add nothing.  16384 tokens of 256 experts: 35 MB in 15 us, 2.3 TB/s, half of
// what a copy reaches: two exponentials and a division an element, and the k R comparisons that place
// the slots' values, take the rest.
template <int R, bool kBf16, bool kVec, bool kSigmoid>
__global__ void __launch_bounds__(64 * kWaves) router_top_k_backward(RouterArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kWaves + wave;
  if (t >= a.T) return;
  const int e0 = lane * R;
  float x[R], grad[R];
  load_logits<R, kBf16, kVec>(a, t, e0, x);
  int id = -1;
  float g = 0.0f, l = -INFINITY;
  if (lane < a.k) {
    id = a.idx[(int64_t)t * a.k + lane];
    if (id >= 0 && id < a.E) {
      g = a.grad_w[(int64_t)t * a.k + lane] * a.factor;
      const int64_t at = (int64_t)t * a.E + id;
      l = kBf16 ? __uint_as_float((uint32_t)((const uint16_t*)a.logits)[at] << 16)
                : ((const float*)a.logits)[at];
    }
  }
  const bool kept = l > -INFINITY;
  if (!kept) {
    id = -1;
    g = 0.0f;
  }
  const bool bad = not_finite(x);
  float own;            // slot's contribution at its expert
  float dense = 0.0f;   // S where every expert gets -p_e S
  float m = 0.0f, total = 1.0f;
  if (a.renorm) {
    const float q = renormalized<kSigmoid>(l, kept);
    const float S = wave_sum(q * g);
    own = kept ? q * (g - S) : 0.0f;
    if (kSigmoid && kept) own *= sigmoid(-l);
  } else if constexpr (kSigmoid) {
    own = kept ? sigmoid(l) * sigmoid(-l) * g : 0.0f;
  } else {
    m = max_of(x);
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) sum += x[r] > -INFINITY ? expf(x[r] - m) : 0.0f;
    total = wave_sum(sum);
    own = kept ? expf(l - m) / total * g : 0.0f;
    dense = wave_sum(own);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    grad[r] = 0.0f;
    if constexpr (!kSigmoid)
      if (!a.renorm && x[r] > -INFINITY) grad[r] = -(expf(x[r] - m) / total) * dense;
  }
  for (int j = 0; j < a.k; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(own), j));
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (e0 + r == e) grad[r] += v;
  }
  if (bad) {
#pragma unroll
    for (int r = 0; r < R; ++r) grad[r] = __uint_as_float(0x7fc00000u);
  }
  typedef std::conditional_t<kBf16, uint16_t, float> out_t;
  out_t* dst = (out_t*)a.grad + (int64_t)t * a.E + e0;
  out_t o[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if constexpr (kBf16)
      o[r] = __builtin_bit_cast(uint16_t, (__bf16)grad[r]);
    else
      o[r] = grad[r];
  }
  if constexpr (kVec) {
    constexpr int C = kVecOf<R, sizeof(out_t)>;
    typedef out_t vec __attribute__((ext_vector_type(C)));
    if (e0 >= a.E) return;
#pragma unroll
    for (int c = 0; c < R; c += C) {
      vec v;
#pragma unroll
      for (int r = 0; r < C; ++r) v[r] = o[c + r];
      *(vec*)(dst + c) = v;
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (e0 + r < a.E) dst[r] = o[r];
  }
}

// fn(R, kBf16, kVec) as compile-time constants: R experts to a lane, the fewest that
// hold E, read as vectors where E allows.
template <class F>
hipError_t with_layout(int E, bool bf16, F fn) {
  auto pick = [&](auto r) {
    constexpr int R = decltype(r)::value;
    const bool vec = E % R == 0;
    std::true_type yes;
    std::false_type no;
    if (bf16) return vec ? fn(r, yes, yes) : fn(r, yes, no);
    return vec ? fn(r, no, yes) : fn(r, no, no);
  };
  if (E <= 64) return pick(std::integral_constant<int, 1>{});
  if (E <= 128) return pick(std::integral_constant<int, 2>{});
  if (E <= 256) return pick(std::integral_constant<int, 4>{});
  if (E <= 512) return pick(std::integral_constant<int, 8>{});
  return pick(std::integral_constant<int, 16>{});
}

RouterArgs router_args(const Shape& s, const RouterIO& io) {
  RouterArgs a{};
  a.logits = io.logits;
  a.bias = io.bias;
  a.grad_w = io.grad_w;
  a.idx = io.idx;
  a.w = io.w;
  a.grad = io.grad;
  a.T = s.T;
  a.E = s.E;
  a.k = s.k;
  a.G = s.G;
  a.limit = io.limit;
  a.renorm = io.renorm;
  a.factor = io.factor;
  return a;
}

// A launch has less than 2^32 threads, 64 for every token: launch(first, tokens) for at most
// kMostTokens of them at a time, with the arguments of the first.
constexpr int kMostTokens = 1 << 25;
template <class F>
hipError_t in_launches(const RouterArgs& all, bool bf16, F launch) {
  for (int64_t t = 0; t < all.T; t += kMostTokens) {
    RouterArgs a = all;
    const int64_t logits = t * all.E * (bf16 ? 2 : 4), slots = t * all.k;
    a.T = (int)std::min<int64_t>(all.T - t, kMostTokens);
    a.logits = (const char*)all.logits + logits;
    a.idx = all.idx + slots;
    if (all.w) a.w = all.w + slots;
    if (all.grad_w) a.grad_w = all.grad_w + slots;
    if (all.grad) a.grad = (char*)all.grad + logits;
    const hipError_t e = launch(a, dim3((unsigned)((a.T + kWaves - 1) / kWaves)));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

bool router_limit_ok(const Shape& s, int limit) {
  return limit <= 0 || limit >= s.G || s.G <= kMaxLimitGroups;
}

hipError_t launch_router_top_k(const Shape& s, const RouterIO& io, hipStream_t st) {
  RouterArgs a = router_args(s, io);
  if (a.limit >= a.G) a.limit = 0;  // every group stays
  const bool scored = a.bias || a.limit > 0;
  const size_t lds = a.limit > 0 ? sizeof(double) * kWaves * s.E : 0;
  return with_layout(s.E, io.bf16, [&](auto r, auto bf16, auto vec) {
    constexpr int R = decltype(r)::value;
    constexpr bool B = decltype(bf16)::value, V = decltype(vec)::value;
    auto go = [&](auto kernel) {
      return in_launches(a, io.bf16, [&](const RouterArgs& part, dim3 grid) {
        hipLaunchKernelGGL(kernel, grid, dim3(64 * kWaves), lds, st, part);
        return hipGetLastError();
      });
    };
    if (io.sigmoid)
      return scored ? go(router_top_k<R, B, V, true, true>) : go(router_top_k<R, B, V, true, false>);
    return scored ? go(router_top_k<R, B, V, false, true>) : go(router_top_k<R, B, V, false, false>);
  });
}

hipError_t launch_router_top_k_backward(const Shape& s, const RouterIO& io, hipStream_t st) {
  const RouterArgs a = router_args(s, io);
  return with_layout(s.E, io.bf16, [&](auto r, auto bf16, auto vec) {
    constexpr int R = decltype(r)::value;
    constexpr bool B = decltype(bf16)::value, V = decltype(vec)::value;
    auto go = [&](auto kernel) {
      return in_launches(a, io.bf16, [&](const RouterArgs& part, dim3 grid) {
        hipLaunchKernelGGL(kernel, grid, dim3(64 * kWaves), 0, st, part);
        return hipGetLastError();
      });
    };
    return io.sigmoid ? go(router_top_k_backward<R, B, V, true>)
                      : go(router_top_k_backward<R, B, V, false>);
  });
}

}  // namespace moe
