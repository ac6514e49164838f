// Routing of tokens to experts: each token's top-k experts by score, their
// weights, and the counting sort of the T k choices by expert that the grouped
// product's offsets describe.
//
//   p = softmax(l) or sigmoid(l),  key = p + bias
//   groups of consecutive experts are ranked by the sum of their one or two
//   largest keys, and only experts of the best ones can be chosen
//   the k largest keys, the lower number first among equals
//   w = p of the chosen, divided by their sum or not, times a factor
//
// Both scores rise with the logit, so without a bias the experts are compared by
// their logits, exactly.  Keys and groups' sums are compared in FP32 where they
// are further apart than FP32 can be wrong, and the row is done again in FP64
// where two that matter are not (about one row in a thousand), so that a choice
// is that of FP64 without its rate (GB300 issues an FP64 instruction of a warp
// every 16 cycles an SM).  A NaN compares above everything.
//
// A warp takes a token, expert e in lane e % 32.  A CTA takes a run of tokens, 32
// at a time: the choices set one bit for each token in a word for each expert, so
// that a choice's rank among the run's is a count of bits below its own, whatever
// order the warps came in.  The runs' counts go to the workspace, and a second
// kernel adds what lies before each run (a single run needs none).  Up to 64 experts
// two CTAs share an SM; above, their 101 to 128 registers a thread leave room for one,
// and above 256 a token's keys spill.
//
// Bytes are next to nothing (4 an expert and token): it is bound by the chain of a
// token's steps, a warp's maximum and the lowest lane that has it for each choice.
// One token 3.2 us; 226 over 256 experts, 4 of 8 groups, top 8: 10.6; 17,776 over 64,
// top 2: 16; 4,444 over 256 in groups 29, 17,776 66.
#include <cstdint>

#include "common.cuh"
#include "ctx_cache.h"
#include "internal.h"

namespace sixbit {
namespace route {

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kBlock = kRouteTurn;  // tokens of a turn: bits of a word
constexpr unsigned kAll = 0xFFFFFFFFu;

// Bits in the order of the values; a NaN above all, an absent expert (0) below.
__device__ __forceinline__ uint32_t ordered(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(v + 0.f);  // (-0 is 0)
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double v) {
  if (v != v) return ~0ull;
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return b ^ ((b >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o >> 31) ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ double value_of(uint64_t o) {
  return __longlong_as_double(static_cast<long long>((o >> 63) ? o ^ 0x8000000000000000ull : ~o));
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

template <typename F>
struct OrdOf;
template <>
struct OrdOf<float> {
  using type = uint32_t;
};
template <>
struct OrdOf<double> {
  using type = uint64_t;
};
__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
__device__ __forceinline__ float inverse(float v) {  // to 2^-23
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ double inverse(double v) { return 1.0 / v; }

// The k largest of the warp's keys (N a lane, 0: absent), lower numbers first
// among equals: lane j's `mine` is the j-th expert.  CHECK: true if no two
// consecutive ones, the last chosen and the next included, are within `tol` +
// `rel` |key|, and the last chosen in `least`.
template <int N, bool CHECK, typename O>
__device__ __forceinline__ bool top_k_in_turn(O (&key)[N], int k, float tol, float rel, int* mine, float* least) {
  const int lane = threadIdx.x & 31;
  O best = 0;
  int slot = 0;
  auto refresh = [&] {
    best = 0;
    slot = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (key[i] > best) {
        best = key[i];
        slot = i;
      }
  };
  refresh();
  bool clear = true;
  float last = 0.f;
  const int turns = CHECK ? k + 1 : k;
  for (int j = 0; j < turns; ++j) {
    const O top = warp_max(best);
    if (CHECK) {
      if (top == 0) break;  // (nothing is left beyond the last)
      const float v = value_of(static_cast<uint32_t>(top));
      if (j > 0 && !(last - v > tol + rel * fabsf(last))) clear = false;
      if (j == k) break;
      last = v;
    }
    const unsigned who = best == top ? static_cast<unsigned>(lane + 32 * slot) : kAll;
    const int e = static_cast<int>(__reduce_min_sync(kAll, who));
    if (lane == j) *mine = e;
    if ((e & 31) == lane) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i == (e >> 5)) key[i] = 0;
      refresh();
    }
  }
  *least = last;
  return clear;
}

// Lanes sorted by v, the largest first.
template <typename V>
__device__ __forceinline__ V sorted(V v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int h = size >> 1; h > 0; h >>= 1) {
      const V o = __shfl_xor_sync(kAll, v, h);
      const bool larger = ((lane & size) == 0) == ((lane & h) == 0);  // this lane keeps the larger of the two
      v = (v > o) == larger ? v : o;
    }
  return v;
}
// The same by sorting: keys that are not clearly below the k-th largest of the
// lanes' own largest are nearly all of the k largest; up to 32 of them are put side
// by side and sorted.  Up to four in turn: 17776 tokens over 64, k = 2, 17 us where
// sorting takes 20; over 256 in groups, k = 8, 100 and 90.  list: the warp's [32].
template <int N, bool CHECK>
__device__ __forceinline__ bool top_k(const uint32_t (&key)[N], int k, float tol, float rel, int* mine, float* least, uint2* list) {
  const int lane = threadIdx.x & 31;
  uint64_t pair;
  if (k <= 4) {
    uint32_t left[N];
#pragma unroll
    for (int i = 0; i < N; ++i) left[i] = key[i];
    return top_k_in_turn<N, CHECK>(left, k, tol, rel, mine, least);
  }
  if constexpr (N == 1) {
    pair = key[0] == 0 ? 0 : (static_cast<uint64_t>(key[0]) << 32) | (kAll - lane);
  } else {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) best = max(best, key[i]);
    uint32_t from = __shfl_sync(kAll, sorted(best), k - 1);
    if (CHECK && from != 0) {
      const float v = value_of(from), below = v - (tol + rel * fabsf(v));
      from = below == below ? ordered(below) : 0;  // (an infinity or a NaN: all)
    }
    if (from == 0) from = 1;
    int total = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool in = key[i] >= from;
      const uint32_t all = __ballot_sync(kAll, in);
      const int at = total + __popc(all & ((1u << lane) - 1));
      if (in && at < 32) list[at] = make_uint2(key[i], kAll - (lane + 32 * i));
      total += __popc(all);
    }
    if (total > 32) {
      uint32_t left[N];
#pragma unroll
      for (int i = 0; i < N; ++i) left[i] = key[i];
      return top_k_in_turn<N, CHECK>(left, k, tol, rel, mine, least);
    }
    __syncwarp();
    const uint2 l = list[lane];
    pair = lane < total ? (static_cast<uint64_t>(l.x) << 32) | l.y : 0;
    __syncwarp();
  }
  pair = sorted(pair);
  *mine = static_cast<int>(kAll - static_cast<uint32_t>(pair));
  if (!CHECK) return true;
  const uint32_t o = static_cast<uint32_t>(pair >> 32), next = __shfl_down_sync(kAll, o, 1);
  const float v = value_of(o);
  *least = __shfl_sync(kAll, v, k - 1);
  // (what is not on the list is further away; lane 31 has no next)
  const bool apart = lane == 31 || next == 0 || v - value_of(next) > tol + rel * fabsf(v);
  return __all_sync(kAll, lane >= k || (o != 0 && apart));
}

// Bits of the groups that are kept.  keys: the warp's E keys in shared memory.
template <bool CHECK, typename O>
__device__ __forceinline__ bool keep_groups(const RouteParams& p, const O* keys, float tol, uint32_t* kept) {
  const int lane = threadIdx.x & 31, size = p.E / p.groups;
  __syncwarp();
  // 1 << p.team lanes a group, each every so many keys of it; their two largest are joined in a tree
  const int team = 1 << p.team, g = lane >> p.team, sub = lane & (team - 1);
  O a = 0, b = 0;
  if (g < p.groups) {
#pragma unroll 4
    for (int i = sub; i < size; i += team) {
      const O o = keys[g * size + i];
      b = max(b, min(a, o));
      a = max(a, o);
    }
  }
  for (int h = team >> 1; h > 0; h >>= 1) {
    const O oa = __shfl_xor_sync(kAll, a, h), ob = __shfl_xor_sync(kAll, b, h);
    b = max(max(b, ob), min(a, oa));
    a = max(a, oa);
  }
  // lane g: group g's
  const int from = (lane << p.team) & 31;
  a = __shfl_sync(kAll, a, from), b = __shfl_sync(kAll, b, from);
  const bool two = p.best > 1 && size > 1;
  O score = lane < p.groups ? (two ? ordered(value_of(a) + value_of(b)) : a) : O(0);
  const O sum = score;
  uint32_t bits = 0;
  for (int j = 0; j < p.top_groups; ++j) {
    const O top = warp_max(score);
    const int g = __ffs(__ballot_sync(kAll, score == top)) - 1;
    bits |= 1u << g;
    if (lane == g) score = 0;
  }
  bool clear = true;
  if constexpr (CHECK) {
    if (p.top_groups < p.groups) {  // (which of the kept comes first does not matter)
      // A key is off by its score's error and 2^-24 of its own size, however small the sum that it cancels in, and the sum
      // by that of both keys and 2^-24 of its own; a quarter more, and the sum's once more, for the arithmetic here.
      // An infinite bias is exact.  (What overflows leaves a NaN, which is not clear.)
      const float fa = value_of(a), fb = two ? value_of(b) : 0.f, s = value_of(sum);
      const float off = fa == -INFINITY || fb == -INFINITY ? 0.f : 0x1.4p-24f * (fabsf(fa) + fabsf(fb) + 2.f * fabsf(s));
      const bool in = (bits >> lane) & 1;
      const float least = value_of(__reduce_min_sync(kAll, in ? ordered(s - off) : kAll));
      const float next = value_of(__reduce_max_sync(kAll, in || lane >= p.groups ? 0u : ordered(s + off)));
      clear = least - next > 2.f * tol;
    }
  }
  __syncwarp();
  *kept = bits;
  return clear;
}

// e / (E / groups): p.per is 2^20 over the group's size, rounded up, and e times the
// size is below 2^20.
__device__ __forceinline__ uint32_t group_of(const RouteParams& p, int e) { return (static_cast<uint32_t>(e) * p.per) >> 20; }

// A token's logits, expert lane + 32 i's in l[i]; -infinity beyond the last.
template <int N>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t t, float (&l)[N]) {
  const int lane = threadIdx.x & 31;
  const size_t at = static_cast<size_t>(t) * p.E;  // (loads under no condition, so that they are on their way at once)
  if (p.logits_bf16 != nullptr) {
    uint16_t w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(p.logits_bf16 + at + min(lane + 32 * i, p.E - 1));
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = __uint_as_float(static_cast<uint32_t>(w[i]) << 16);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = __ldg(p.logits + at + min(lane + 32 * i, p.E - 1));
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane + 32 * i >= p.E) l[i] = -INFINITY;
}

// What FP32 left open of a token: everything (all), or the order of the experts
// whose keys are not clearly below the last chosen (bit i: expert lane + 32 i).
struct Open {
  bool all;
  uint32_t listed;
};

// One token's experts (lane j: the j-th), from its logits l and the experts' biases.
// F: the type that keys are computed in; CHECK: false is returned where F is too
// narrow.
template <int N, bool CHECK, typename F>
__device__ __forceinline__ bool choose(const RouteParams& p, const float (&l)[N], const float (&bias)[N], float lmax,
                                       typename OrdOf<F>::type* keys, uint2* list, int* mine, Open* open) {
  using O = typename OrdOf<F>::type;
  const int lane = threadIdx.x & 31;
  const bool by_logit = p.bias == nullptr;
  F v[N];
  float tol = 0.f;
  if (!by_logit || p.groups > 1) {
    if (p.score == SIXBIT_SCORE_SOFTMAX) {
      F sum = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = lane + 32 * i < p.E && l[i] != -INFINITY ? exp_of(static_cast<F>(l[i]) - static_cast<F>(lmax)) : F(0);
        sum += v[i];
      }
      sum = warp_sum(sum);
      const F by = sum == F(0) ? F(0) : inverse(sum);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= by;
      // units of 2^-24: a term is 2 off by its exponential and 0.4 by its argument, the sum by that and its N + 5
      // additions, its reciprocal 2 and the product 1
      tol = 0x1p-24f * 2.f * (N + 14);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = inverse(F(1) + exp_of(-static_cast<F>(l[i])));
      tol = 0x1p-24f * 8.f;  // (0.5 by the exponential, 1 by the sum, 2 by the reciprocal)
    }
    if (!by_logit) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += static_cast<F>(bias[i]);
    }
  }
  const float rel = 0x1p-24f * 3;  // (the bias joins with half a unit of the key)
  bool clear = true;
  uint32_t kept = kAll;
  O key[N];
  if (!by_logit || p.groups > 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = lane + 32 * i < p.E ? ordered(v[i]) : O(0);
  }
  if (p.groups > 1) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane + 32 * i < p.E) keys[lane + 32 * i] = key[i];
    clear = keep_groups<CHECK>(p, keys, tol, &kept);
  }
  float least = 0.f;
  if (by_logit) {
    uint32_t lk[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = lane + 32 * i;
      lk[i] = e < p.E && (p.groups == 1 || ((kept >> group_of(p, e)) & 1)) ? ordered(l[i]) : 0u;
    }
    top_k<N, false>(lk, p.k, 0.f, 0.f, mine, &least, list);
    if (CHECK) open->all = true;
    return clear;
  }
  if (p.groups > 1) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!((kept >> group_of(p, lane + 32 * i)) & 1)) key[i] = 0;
  }
  bool order;
  if constexpr (CHECK)
    order = top_k<N, true>(key, p.k, tol, rel, mine, &least, list);
  else
    order = top_k_in_turn<N, false>(key, p.k, tol, rel, mine, &least);
  if (CHECK && !(order && clear)) {
    const float below = least - (tol + rel * fabsf(least));
    open->all = !clear || p.score == SIXBIT_SCORE_SOFTMAX || !(fabsf(below) < INFINITY);
    open->listed = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (key[i] != 0 && !(v[i] < F(below))) open->listed |= 1u << i;
    }
  }
  return order && clear;
}

__device__ __forceinline__ float logit_at(const RouteParams& p, int64_t t, int e) {
  const size_t at = static_cast<size_t>(t) * p.E + e;
  return p.logits_bf16 != nullptr ? __uint_as_float(static_cast<uint32_t>(__ldg(p.logits_bf16 + at)) << 16)
                                  : __ldg(p.logits + at);
}

template <int N>
__device__ __forceinline__ void load_bias(const RouteParams& p, float (&bias)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < N; ++i) bias[i] = 0.f;
  if (p.bias == nullptr) return;
#pragma unroll
  for (int i = 0; i < N; ++i) bias[i] = __ldg(p.bias + min(lane + 32 * i, p.E - 1));
}

// A token again in FP64, a call of its own: its registers (two a key) are not the
// fast path's.  With sigmoid scores only the listed experts, up to four a lane (an
// exponential is some 60 FP64 instructions).
template <int N>
__device__ __noinline__ int choose64(const RouteParams& p, int64_t t, float lmax, uint64_t* keys, uint2* list, bool all,
                                     uint32_t listed) {
  const int lane = threadIdx.x & 31;
  int mine = 0;
  if (!all && !__any_sync(kAll, __popc(listed) > 4)) {
    uint64_t key[4] = {};
    int number[4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (__all_sync(kAll, listed == 0)) break;
      if (listed != 0) {
        const int e = lane + 32 * (__ffs(listed) - 1);
        listed &= listed - 1;
        number[j] = e;
        key[j] = ordered(1.0 / (1.0 + exp(-static_cast<double>(logit_at(p, t, e)))) + static_cast<double>(__ldg(p.bias + e)));
      }
    }
    for (int j = 0; j < p.k; ++j) {
      uint64_t best = 0;
      int slot = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (key[i] > best) {
          best = key[i];
          slot = i;
        }
      const uint64_t top = warp_max(best);
      int e = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i == slot) e = number[i];
      const int first = static_cast<int>(__reduce_min_sync(kAll, best == top ? static_cast<unsigned>(e) : kAll));
      if (lane == j) mine = first;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (best == top && e == first && i == slot) key[i] = 0;
    }
    return mine;
  }
  float l[N];
  load_logits(p, t, l);
  float bias[N];
  load_bias(p, bias);
  choose<N, false, double>(p, l, bias, lmax, keys, list, &mine, nullptr);
  return mine;
}

// Lane j's weight of the j-th expert.
template <int N>
__device__ __forceinline__ float weight_of(const RouteParams& p, const float (&l)[N], float lmax, float mine, bool live) {
  const int lane = threadIdx.x & 31;
  float w;
  if (p.renorm) {  // relative to the largest chosen, so that small scores keep their ratio
    float m = live ? mine : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    if (p.score == SIXBIT_SCORE_SIGMOID) {
      m = fminf(m, 0.f);
      // e^(l - m) / (1 + e^l); above 0 (m is 0 then) without the large exponential
      w = mine > 0.f ? 1.f / (1.f + expf(-mine)) : expf(mine - m) / (1.f + expf(mine));
    } else {
      w = expf(mine - m);
    }
    if (mine == -INFINITY || !live) w = 0.f;
    const float sum = warp_sum(w);
    w = sum == 0.f ? 0.f : w / sum;
  } else if (p.score == SIXBIT_SCORE_SIGMOID) {
    w = 1.f / (1.f + expf(-mine));
  } else {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += lane + 32 * i < p.E && l[i] != -INFINITY ? expf(l[i] - lmax) : 0.f;
    sum = warp_sum(sum);
    w = mine == -INFINITY ? 0.f * sum : expf(mine - lmax) / sum;
  }
  // (a NaN or an infinite logit makes every probability of its row NaN)
  if (p.score == SIXBIT_SCORE_SOFTMAX && !(lmax < INFINITY)) w = __uint_as_float(0x7FC00000u);
  return w * p.factor;
}

// Exclusive prefix sums of v[0 .. n) in shared memory, n <= 2 kThreads; v[n]
// becomes the total.
__device__ __forceinline__ void scan(int* v, int n, int* part) {
  const int i = 2 * threadIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int a = i < n ? v[i] : 0, b = i + 1 < n ? v[i + 1] : 0;
  int s = a + b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(kAll, s, o);
    if (lane >= o) s += up;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += part[w];
    all += part[w];
  }
  s += before - a - b;
  if (i < n) v[i] = s;
  if (i + 1 < n) v[i + 1] = s + a;
  if (threadIdx.x == 0) v[n] = all;
  __syncthreads();
}

// Shared memory: run [E + 1], mask [E], chosen [kBlock k], then with groups the
// warps' keys, E of 64 bits each.
__host__ __device__ constexpr size_t keys_at(int E, int k) {
  return ((static_cast<size_t>(E) * 2 + 1 + kBlock * k) * 4 + 7) / 8 * 8;
}

// (with the kernel's static shared memory, 4 KB, below what a CTA can have)
constexpr int kSmemBytes = 200 * 1024;
static_assert(keys_at(SIXBIT_MAX_EXPERTS, SIXBIT_MAX_TOP_K) + kWarps * SIXBIT_MAX_EXPERTS * 8 <= kSmemBytes, "the largest launch");

template <int N>
__global__ void __launch_bounds__(kThreads) choose_kernel(const __grid_constant__ RouteParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int part[kWarps];
  __shared__ uint2 lists[kWarps][32];
  int* run = reinterpret_cast<int*>(smem);
  uint32_t* mask = reinterpret_cast<uint32_t*>(run + p.E + 1);
  int* chosen = reinterpret_cast<int*>(mask + p.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* keys = reinterpret_cast<uint64_t*>(smem + keys_at(p.E, p.k)) + static_cast<size_t>(p.groups > 1 ? warp : 0) * p.E;
  float bias[N];
  load_bias(p, bias);
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    run[e] = 0;
    mask[e] = 0;
  }
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens_per_cta;
  const int64_t t1 = min(t0 + p.tokens_per_cta, static_cast<int64_t>(p.T));
  for (int64_t tb = t0; tb < t1; tb += kBlock) {
    for (int j = warp; j < kBlock && tb + j < t1; j += kWarps) {
      const int64_t t = tb + j;
      float l[N];
      load_logits(p, t, l);
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) top = max(top, ordered(l[i]));
      const float lmax = value_of(warp_max(top));
      int mine = 0;
      Open open;
      if (!choose<N, true, float>(p, l, bias, lmax, reinterpret_cast<uint32_t*>(keys), lists[warp], &mine, &open))
        mine = choose64<N>(p, t, lmax, keys, lists[warp], open.all, open.listed);
      const bool live = lane < p.k;
      mine = static_cast<int>(min(static_cast<unsigned>(mine), static_cast<unsigned>(p.E - 1)));  // (lanes beyond k hold anything)
      const float w = weight_of<N>(p, l, lmax, live ? logit_at(p, t, mine) : -INFINITY, live);
      if (live) {
        const size_t at = static_cast<size_t>(t) * p.k + lane;
        p.experts[at] = mine;
        p.weights[at] = w;
        chosen[j * p.k + lane] = mine;
        atomicOr(&mask[mine], 1u << j);
      }
    }
    __syncthreads();
    const int live = static_cast<int>(min(static_cast<int64_t>(kBlock), t1 - tb)) * p.k;
    for (int i = threadIdx.x; i < live; i += kThreads) {
      const int e = chosen[i];
      p.rows[static_cast<size_t>(tb) * p.k + i] = run[e] + __popc(mask[e] & ((1u << (i / p.k)) - 1));
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
      run[e] += __popc(mask[e]);
      mask[e] = 0;
    }
    __syncthreads();
  }
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < p.pitch; e += kThreads) p.counts[static_cast<size_t>(blockIdx.x) * p.pitch + e] = e < p.E ? run[e] : 0;
    return;
  }
  scan(run, p.E, part);
  for (int e = threadIdx.x; e <= p.E; e += kThreads) p.offsets[e] = run[e];
  for (int i = threadIdx.x; i < p.T * p.k; i += kThreads) {  // (this thread wrote rows[i]: one turn of 32 tokens)
    const int r = p.rows[i] + run[p.experts[i]];
    p.rows[i] = r;
    p.token[r] = i / p.k;
  }
}

// Adds what lies before each run: the experts' offsets and the earlier runs' counts.
__global__ void __launch_bounds__(kThreads) place_kernel(const RouteParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int part[kWarps];
  int* all = reinterpret_cast<int*>(smem);  // [E + 1]
  int* before = all + p.E + 1;              // [E]
  for (int e = threadIdx.x; e < p.E; e += kThreads) all[e] = before[e] = 0;
  __syncthreads();
  // four experts a thread and every so many runs of them, eight loads at once
  const int runs = gridDim.x, me = blockIdx.x, quads = p.pitch / 4;
  const int teams = min(kThreads / quads, 16), team = threadIdx.x / quads, q = threadIdx.x % quads;
  if (team < teams) {
    int a[4] = {}, b[4] = {};
    for (int c0 = team; c0 < runs; c0 += 8 * teams) {
      int4 n[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[i] = make_int4(0, 0, 0, 0);
        if (c0 + i * teams < runs) n[i] = *reinterpret_cast<const int4*>(p.counts + static_cast<size_t>(c0 + i * teams) * p.pitch + 4 * q);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int v[4] = {n[i].x, n[i].y, n[i].z, n[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          a[j] += v[j];
          if (c0 + i * teams < me) b[j] += v[j];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (4 * q + j < p.E) {
        atomicAdd(&all[4 * q + j], a[j]);
        atomicAdd(&before[4 * q + j], b[j]);
      }
  }
  __syncthreads();
  scan(all, p.E, part);
  if (me == 0)
    for (int e = threadIdx.x; e <= p.E; e += kThreads) p.offsets[e] = all[e];
  const int64_t t0 = static_cast<int64_t>(me) * p.tokens_per_cta;
  const int64_t t1 = min(t0 + p.tokens_per_cta, static_cast<int64_t>(p.T));
  for (int64_t i = t0 * p.k + threadIdx.x; i < t1 * p.k; i += kThreads) {
    const int e = p.experts[i], r = p.rows[i] + all[e] + before[e];
    p.rows[i] = r;
    p.token[r] = static_cast<int>(i / p.k);
  }
}

template <int N>
cudaError_t launch(const RouteParams& p, int ctas, cudaStream_t st) {
  const size_t smem = keys_at(p.E, p.k) + (p.groups > 1 ? static_cast<size_t>(kWarps) * p.E * 8 : 0);
  cudaError_t e = set_smem_once<choose_kernel<N>>(kSmemBytes);
  if (e != cudaSuccess) return e;
  note_launch();
  choose_kernel<N><<<ctas, kThreads, smem, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || ctas == 1) return e;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (static_cast<size_t>(p.E) * 2 + 1) * 4;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, place_kernel, p);
}

}  // namespace route

cudaError_t launch_moe_route(RouteParams p, cudaStream_t st) {
  // one run up to a turn of 32 tokens, else up to kRouteRuns equal ones of whole rounds of the warps
  int ctas = 1;
  p.tokens_per_cta = p.T;
  if (p.T > route::kBlock) {
    const int64_t per = (static_cast<int64_t>(p.T) + kRouteRuns - 1) / kRouteRuns;
    p.tokens_per_cta = static_cast<int>((per + route::kWarps - 1) / route::kWarps * route::kWarps);
    ctas = static_cast<int>((static_cast<int64_t>(p.T) + p.tokens_per_cta - 1) / p.tokens_per_cta);
  }
  p.pitch = (p.E + 3) / 4 * 4;
  const int size = p.E / p.groups;
  p.per = ((1u << 20) + size - 1) / size;
  p.team = 0;
  while (p.groups << (p.team + 1) <= 32) ++p.team;
  if (p.E <= 32) return route::launch<1>(p, ctas, st);
  if (p.E <= 64) return route::launch<2>(p, ctas, st);
  if (p.E <= 128) return route::launch<4>(p, ctas, st);
  if (p.E <= 256) return route::launch<8>(p, ctas, st);
  if (p.E <= 512) return route::launch<16>(p, ctas, st);
  return route::launch<32>(p, ctas, st);
}

}  // namespace sixbit
