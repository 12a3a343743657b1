// k_route.cu -- the router of the sparse MLP block: for every token the k
// experts with the largest logits, their softmax weights, and the order of
// the (token, expert) entries by expert that the grouped products read.
//
//     p[t,e] = exp(l[t,e] - max_e l) / sum_e exp(l[t,e] - max_e l)
//     ids[t,j]     = expert of the j-th largest logit (ties: lowest number)
//     weights[t,j] = scale * p, or scale * p / (sum of the chosen p)
//     rows, slots  = the entries (t, j) in the order (expert, t k + j)
//
// LPT lanes per token (4 to 32: at least k, and eight experts a lane while that
// is enough): lane l holds the logits of experts l, l + LPT, ... as 32-bit keys
// whose unsigned order is the floats' order.  A key of 0 is no expert: a masked
// logit of -inf, or a lane past E.  A choice is one maximum over the group's
// lanes (log2(LPT) shuffles) of the key with the complement of the expert's
// number below it, so that among equal logits the lowest number wins.  What
// counts is the length of this chain (k rounds of it, each on the one before),
// so nothing in it branches.
//
// The order is a counting sort that keeps entries in sequence, without
// atomics, so its result does not depend on timing: each warp counts its own
// tokens' entries by expert (equal experts within 32 entries are found with
// match_any), the warps' counts are summed in order, and each warp walks its
// entries again and numbers them within the block.
//
// Up to kOneTokens tokens are one launch of one cluster of at most eight blocks: one SM
// issues the choices of 128 tokens in about 6 us, so they are spread over several
// (route_blocks.h), which read each other's counts through distributed shared memory.
// In a graph, 256 experts: 64 tokens by logit 5.5 us, by scores 6.7 (32 tokens a block:
// 9.7 and 10.9); 8 tokens 4.2 and 5.0.  Beyond that a first kernel numbers the entries
// within each block of 32 to 128 tokens (in slots) and writes the block's counts to
// the workspace, and a second one, overlapped by programmatic dependent launch, sums
// the counts of the blocks before its own and adds them (16384 tokens: 14.0 us; in clusters of eight blocks of 32
// tokens about a fifth more).  Every block of the second launch reads the counts
// of all blocks, which is little at such sizes but grows with the square of the
// tokens: 131072 tokens take 89 us with 64 experts and 243 us with 256.
//
// swiglu_moe_route_scored chooses by a score instead of the logit (choose_scored):
//     s = sigmoid(l) or softmax(l),  c = s + bias,
// in the `kept` groups of experts whose largest c (or two largest added) are
// largest.  A warp per token; a group's experts lie in neighbouring lanes.  The
// choice is that of the exact values: FP32 decides where the values compared
// lie further apart than their rounding errors together, and where two do not,
// which is so for about a token in a thousand, FP64 settles the few values
// concerned (without a bias the logits' own order decides, and only sums of two
// scores are compared).  16384 tokens, 256 experts in 8 groups, 33.5 us; a scheduler
// issues for 14 of the first launch's 31, 1042 instructions a token (55 us with all
// scores of such a token in FP64 and a round over all experts for each choice; 8 lanes
// of 32 experts a token instead of a warp 70).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "launch.h"
#include "route_blocks.h"
#include "sm103_ptx.cuh"
#include "swiglu.h"

namespace swiglu {
namespace {

constexpr int kMaxE = 1024;
constexpr int kMaxK = 32;
constexpr int kBlockTokens = 128;        // most tokens per block otherwise
// Warps of a block x experts: 32 warps up to 510 experts, and RouteSmem is the 48 KB
// that a kernel may hold without asking.
constexpr int kCounters = 16320;
constexpr unsigned kAll = 0xffffffffu;

struct RouteParams {
  const void *logits;
  int32_t *ids;
  float *weights;
  int32_t *offsets, *rows, *slots;
  int32_t *counts;  // [blocks][E], two launches only
  int32_t T, E, k, blocks, block_tokens, warp_tokens;
  int32_t renormalize;
  float scale;
  // scored form only
  const float *bias;  // [E] or null
  int32_t sigmoid, fp32, groups, kept, best;
  int32_t group_size, lane_bits;  // E / groups; 2^lane_bits = 32 / groups
};

// Unsigned number with the order of the floats; -inf -> 0 (masked), NaN above
// +inf (it is chosen first and its weight comes out NaN, so it stays visible).
constexpr uint32_t kInfKey = 0x007fffffu;  // -inf's in the plain order (a negative NaN, below it, wraps to the top)
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));  // -0 becomes +0, every NaN the same
  return (b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u)) - kInfKey;
}

__device__ __forceinline__ float key_value(uint32_t key) {
  const uint32_t k = key + kInfKey;
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// The token t of this lane's group of LPT >= k lanes (or none: t >= end), its
// chosen experts to ids16 (shared; 0xffff = none) and global memory.  All
// lanes of the warp call it together.
template <int LPT, int EPL, bool FP32>
__device__ __forceinline__ void choose(const RouteParams &p, int64_t t, int64_t end, int lane,
                                       uint16_t *ids16) {
  using Pick = unsigned long long;  // key above ~expert; 0 in the upper half: none
  const int l = lane & (LPT - 1);
  const bool live = t < end;
  float x[EPL];
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = l + LPT * i;
    x[i] = -INFINITY;
    if (live && e < p.E) {
      const int64_t at = t * p.E + e;
      x[i] = FP32 ? ptx::load(static_cast<const float *>(p.logits) + at)
                  : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[at]);
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = order_key(x[i]);
  // this lane's largest key, the first that holds it
  auto best = [&]() {
    uint32_t b[EPL];
    int w[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) b[i] = key[i], w[i] = i;
#pragma unroll
    for (int st = 1; st < EPL; st <<= 1)
#pragma unroll
      for (int i = 0; i + st < EPL; i += 2 * st) {
        const bool up = b[i + st] > b[i];
        b[i] = up ? b[i + st] : b[i];
        w[i] = up ? w[i + st] : w[i];
      }
    return (Pick(b[0]) << 32) | ~static_cast<uint32_t>(l + LPT * w[0]);
  };
  auto group_max = [](Pick v) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) {
      const Pick u = __shfl_xor_sync(kAll, v, o);
      v = u > v ? u : v;
    }
    return v;
  };
  Pick mx = group_max(best());
  const float m = key_value(static_cast<uint32_t>(mx >> 32));
  float sum = 0.0f;
  if (!p.renormalize) {
    // a masked logit adds exp(-inf) = 0 (where all are, the sum is not used)
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += expf(x[i] - m);
  }
  uint32_t my_key = 0u;  // lane j of the group keeps choice j
  int my_id = -1;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t top = static_cast<uint32_t>(mx >> 32);
    const int e = top != 0u ? static_cast<int>(~static_cast<uint32_t>(mx)) : -1;
    my_key = l == j ? top : my_key;
    my_id = l == j ? e : my_id;
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = l + LPT * i == e ? 0u : key[i];
    mx = group_max(best());
  }
  const float w = my_id < 0 ? 0.0f : expf(key_value(my_key) - m);
  sum = p.renormalize ? w : sum;
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if (live && l < p.k) {
    p.ids[t * p.k + l] = my_id;
    p.weights[t * p.k + l] = my_id < 0 ? 0.0f : p.scale * (w / sum);
    ids16[l] = static_cast<uint16_t>(my_id);  // -1 -> 0xffff
  }
}

// order_key in 64 bits.
__device__ __forceinline__ unsigned long long order_key(double x) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
  const unsigned long long k = b ^ ((b >> 63) ? ~0ull : 1ull << 63);
  return x != x ? ~0ull : x == -CUDART_INF ? 0ull : k;
}

__device__ __forceinline__ double key_value(unsigned long long key) {
  const unsigned long long b = key ^ ((key >> 63) ? 1ull << 63 : ~0ull);
  return key == 0ull ? -CUDART_INF : __longlong_as_double(static_cast<long long>(b));
}

// The largest (key, lowest expert) of the warp's lanes.
__device__ __forceinline__ void warp_best(uint32_t &key, int &e) {
  const uint32_t top = __reduce_max_sync(kAll, key);
  e = static_cast<int>(__reduce_min_sync(kAll, key == top ? static_cast<unsigned>(e) : 0x7fffffffu));
  key = top;
}

__device__ __forceinline__ void warp_best(unsigned long long &key, int &e) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long k = __shfl_xor_sync(kAll, key, o);
    const int f = __shfl_xor_sync(kAll, e, o);
    const bool up = k > key || (k == key && f < e);
    key = up ? k : key;
    e = up ? f : e;
  }
}

// The largest that is left of the warp's keys when the largest has been removed r
// times, equal ones at once: at most the r-th largest (from 0).
__device__ __forceinline__ uint32_t warp_rank(uint32_t key, int r) {
  uint32_t top = __reduce_max_sync(kAll, key);
  for (int i = 0; i < r; ++i) {
    key = key == top ? 0u : key;
    top = __reduce_max_sync(kAll, key);
  }
  return top;
}

__device__ __forceinline__ float score_of(bool sigmoid, float x, float m, float sum) {
  return sigmoid ? __frcp_rn(1.0f + expf(-x)) : __fdiv_rn(expf(x - m), sum);
}
__device__ __forceinline__ double score_of(bool sigmoid, double x, double m, double sum) {
  return sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m) / sum;
}
// The same for the choice: 2^x and the reciprocal of the special-function unit
// (2^-22 of themselves, x's rounding 2^-24 |x|; what would be denormal is 0).
__device__ __forceinline__ float quick_exp(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
  return y;
}
__device__ __forceinline__ double quick_exp(double x) { return exp(x); }
__device__ __forceinline__ float quick_score(bool sigmoid, float x, float m, float by_sum) {
  if (!sigmoid) return quick_exp(x - m) * by_sum;
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + quick_exp(-x)));
  return y;
}
__device__ __forceinline__ double quick_score(bool sigmoid, double x, double m, double by_sum) {
  return sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m) * by_sum;
}

// Largest error of an FP32 score that the choice goes by, as a part of the token's
// largest one.  Sigmoid: s (1 - s) (2^-22 + |x| 2^-24) <= 2^-23 of the exp, a sum
// and a reciprocal.  Softmax: up to 32 additions in a lane and five across, on
// top of two exp.
__device__ __forceinline__ float score_error(bool sigmoid) { return sigmoid ? 0x1p-21f : 0x1p-18f; }

// What a warp keeps from token to token: a lane's group is g = lane / L of L = 32 /
// groups lanes, and its experts are first, first + L, ... below end = (g + 1) E /
// groups; and shared memory for 32 candidates.
struct Candidates {
  uint32_t key[32];
  int e[32];
};
template <int EPL>
struct ScorePlan {
  static constexpr int KEPT = EPL <= 8 ? EPL : 1;  // biases in registers
  int lane, L, g, first, end;
  float bias[KEPT];
  Candidates *found;
  __device__ ScorePlan(const RouteParams &p, int lane_, Candidates *found_) : lane(lane_), found(found_) {
    L = 1 << p.lane_bits;
    g = lane >> p.lane_bits;
    first = g * p.group_size + (lane & (L - 1));
    end = (g + 1) * p.group_size;
    if (EPL <= 8) {
#pragma unroll
      for (int i = 0; i < KEPT; ++i) bias[i] = p.bias && expert(i) < end ? ptx::load(p.bias + expert(i)) : 0.0f;
    }
  }
  __device__ int expert(int i) const { return first + L * i; }
  __device__ float bias_of(const RouteParams &p, int i) const {
    return EPL <= 8 ? bias[EPL <= 8 ? i : 0] : expert(i) < end ? ptx::load(p.bias + expert(i)) : 0.0f;
  }
};

// The `rounds` (at most 33) largest of the warp's keys (0: none), ties to the lowest
// expert: lane j gets the j-th, every lane the last of 33.
// A round takes the largest key and removes it.
template <class Key, int EPL>
__device__ __forceinline__ void choose_by_rounds(const ScorePlan<EPL> &plan, Key (&key)[EPL], int rounds, int k,
                                                 Key &my_key, int &my_id, Key &next_key, int &next_id) {
  my_key = next_key = 0;
  my_id = next_id = -1;
  for (int j = 0; j < rounds; ++j) {
    Key b = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) b = max(b, key[i]);
    // the lane's first expert that holds it; then the warp's lowest
    int at = EPL - 1;
#pragma unroll
    for (int i = EPL - 2; i >= 0; --i) at = key[i] == b ? i : at;
    int e = plan.expert(at);
    const int own = e;
    warp_best(b, e);
    if (b == 0) break;  // none left: nor in the rounds to come
    my_key = plan.lane == j ? b : my_key;
    my_id = plan.lane == j ? e : my_id;
    next_key = j == k ? b : Key(0);
    next_id = j == k ? e : -1;
    const int gone = own == e ? at : -1;
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = i == gone ? Key(0) : key[i];
  }
}

// The same by ranks, for FP32 keys and up to 32 rounds: none of the chosen lies below
// the rounds-th largest of the lanes' own maxima (or, with `margin`, more than that
// below it), and those that do not are few; they are moved to a lane each (all: how
// many, in order), ranked by comparing all with all.  False: more than 32.
// (9 of 256: about 200 instructions instead of 510.)
template <int EPL>
__device__ __forceinline__ bool choose_by_ranks(const ScorePlan<EPL> &plan, const uint32_t (&key)[EPL], int rounds,
                                                int k, float margin, uint32_t &my_key, int &my_id, uint32_t &next_key,
                                                int &next_id, int &all, int &id_of_all) {
  const int lane = plan.lane;
  uint32_t b = key[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) b = max(b, key[i]);
  uint32_t least = max(warp_rank(b, rounds - 1), 1u);
  if (margin > 0.0f && least > 1u) {
    const float v = key_value(least);
    if (v < INFINITY)  // (nothing is within a margin of +inf or NaN but its like)
      least = max(order_key(v - margin - 0x1p-22f * fabsf(v)), 1u);
  }
  int mine = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) mine += key[i] >= least;
  int at = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int w = __shfl_up_sync(kAll, at, o);
    if (lane >= o) at += w;
  }
  const int count = __shfl_sync(kAll, at, 31);
  if (count > 32) return false;
  at -= mine;
  Candidates &found = *plan.found;
  found.key[lane] = 0u;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (key[i] >= least) {
      found.key[at] = key[i];
      found.e[at++] = plan.expert(i);
    }
  __syncwarp();
  const bool there = lane < count;
  const uint32_t c = found.key[lane];
  const int e = found.e[lane];
  int rank = 0;
  for (int j = 0; j < count; j += 4) {
    const uint4 o = *reinterpret_cast<const uint4 *>(found.key + j);
    rank += (o.x > c) + (o.y > c) + (o.z > c) + (o.w > c);
  }
  // equal keys have one rank: the lowest expert is first
  if (__popc(__reduce_or_sync(kAll, there ? 1u << rank : 0u)) != count)
    for (int j = 0; j < count; ++j) rank += found.key[j] == c && found.e[j] < e;
  __syncwarp();
  if (there) {
    found.key[rank] = c;
    found.e[rank] = e;
  }
  __syncwarp();
  const bool more = k < min(count, rounds);
  all = count, id_of_all = there ? found.e[lane] : -1;
  my_key = there && lane < rounds ? found.key[lane] : 0u, my_id = lane < rounds ? id_of_all : -1;
  next_key = more ? found.key[k] : 0u, next_id = more ? found.e[k] : -1;
  __syncwarp();
  return true;
}
// What FP32 leaves open is settled in FP64 for the values concerned alone, one a lane
// at a time: a warp's FP64 instruction takes about 60 cycles here, and all of 256
// experts' scores 17 us.

struct Token {  // where its logits are, and what its scores need
  const float *row32;
  const __nv_bfloat16 *row16;
  double m, sum;  // softmax
  __device__ float logit(bool fp32, int e) const { return fp32 ? ptx::load(row32 + e) : __bfloat162float(row16[e]); }
};

// Expert e's score, with its bias.
__device__ __forceinline__ double worth_in_64(const RouteParams &p, const Token &token, int e) {
  const double s = score_of(p.sigmoid != 0, double(token.logit(p.fp32 != 0, e)), token.m, token.sum);
  return p.bias ? s + double(ptx::load(p.bias + e)) : s;
}

template <int EPL>
__device__ __noinline__ void sum_in_64(const RouteParams &p, const ScorePlan<EPL> &plan, Token &token) {
  double sum = 0;
  for (int i = 0; i < EPL; ++i)
    if (plan.expert(i) < plan.end) sum += exp(double(token.logit(p.fp32 != 0, plan.expert(i))) - token.m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  token.sum = sum;
}

// Whether the lane's group is kept; `close`: which of the lane's experts may be among
// the group's best (one or two).
template <int EPL>
__device__ __noinline__ bool keep_in_64(const RouteParams &p, const ScorePlan<EPL> &plan, const Token &token,
                                        unsigned close) {
  unsigned long long k1 = 0, k2 = 0;
  while (__any_sync(kAll, close != 0)) {
    unsigned long long k = 0;
    if (close != 0) k = order_key(worth_in_64(p, token, plan.expert(__ffs(close) - 1)));
    close &= close - 1;
    k2 = max(k2, min(k1, k));
    k1 = max(k1, k);
  }
  for (int o = 1; o < plan.L; o <<= 1) {
    const unsigned long long j1 = __shfl_xor_sync(kAll, k1, o), j2 = __shfl_xor_sync(kAll, k2, o);
    k2 = max(min(k1, j1), max(k2, j2));
    k1 = max(k1, j1);
  }
  unsigned long long mine = k1;
  if (p.best == 2 && k1 != 0 && k2 != 0) mine = order_key(key_value(k1) + key_value(k2));
  bool keep = false;
  for (int j = 0; j < p.kept; ++j) {
    unsigned long long b = keep ? 0ull : mine;
    int h = plan.g;
    warp_best(b, h);
    if (b == 0) break;
    keep = keep || h == plan.g;
  }
  return keep;
}

// The candidates (lane i < all has expert id) in order: lane j gets the j-th.
__device__ __noinline__ int rank_in_64(const RouteParams &p, const Token &token, Candidates &found, int lane, int all,
                                       int id) {
  const unsigned long long key = lane < all ? order_key(worth_in_64(p, token, id)) : 0ull;
  int rank = 0;
  for (int j = 0; j < all; ++j) {
    const unsigned long long k = __shfl_sync(kAll, key, j);
    const int e = __shfl_sync(kAll, id, j);
    rank += k > key || (k == key && e < id);
  }
  __syncwarp();
  if (lane < all) found.e[rank] = id;
  __syncwarp();
  const int e = lane < all ? found.e[lane] : -1;
  __syncwarp();
  return e;
}

// One token by one warp, in V = float or double: the chosen experts, lane j
// keeping choice j.  Returns whether V decided every comparison (FP64: always).
template <class V, int EPL>
__device__ __forceinline__ bool choose_exactly(const RouteParams &p, const ScorePlan<EPL> &plan, int64_t t,
                                               int &my_id, float &my_weight) {
  using Key = decltype(order_key(V()));
  constexpr bool ROUNDED = sizeof(V) == 4;
  const bool sigmoid = p.sigmoid != 0, fp32 = p.fp32 != 0, biased = p.bias != nullptr;
  const int lane = plan.lane, L = plan.L, g = plan.g;
  const float *row32 = static_cast<const float *>(p.logits) + (fp32 ? t * p.E : 0);
  const __nv_bfloat16 *row16 = static_cast<const __nv_bfloat16 *>(p.logits) + (fp32 ? 0 : t * p.E);
  auto logit = [&](int e) { return fp32 ? ptx::load(row32 + e) : __bfloat162float(row16[e]); };
  float x[EPL];
  if (fp32) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = plan.expert(i) < plan.end ? ptx::load(row32 + plan.expert(i)) : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      x[i] = plan.expert(i) < plan.end ? __bfloat162float(row16[plan.expert(i)]) : -INFINITY;
  }
  V m = 0, sum = 1, by_sum = 1;
  float largest = 1.0f;  // bound of the scores
  if (!sigmoid) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) top = max(top, order_key(x[i]));
    m = key_value(__reduce_max_sync(kAll, top));
    sum = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += x[i] == -INFINITY ? V(0) : quick_exp(V(x[i]) - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    by_sum = V(1) / sum;
    largest = static_cast<float>(by_sum);
  }
  const float err = score_error(sigmoid) * largest;  // of one score
  [[maybe_unused]] Token token = {row32, row16, double(m), 0.0};
  // s + b, or the logit where no bias is given; 0 for no expert
  Key key[EPL];
  auto keys_of = [&](bool sigmoid) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      key[i] = x[i] == -INFINITY ? Key(0)
                                 : order_key(quick_score(sigmoid, V(x[i]), m, by_sum) + V(plan.bias_of(p, i)));
  };
  if (biased && sigmoid) {  // (two loops: a choice within one takes both sides' instructions)
    keys_of(true);
  } else if (biased) {
    keys_of(false);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = order_key(V(x[i]));
  }
  bool sure = true;
  if (p.kept < p.groups) {
    // the group's two largest
    Key k1 = 0, k2 = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      k2 = max(k2, min(k1, key[i]));
      k1 = max(k1, key[i]);
    }
    for (int o = 1; o < L; o <<= 1) {
      const Key j1 = __shfl_xor_sync(kAll, k1, o), j2 = __shfl_xor_sync(kAll, k2, o);
      k2 = max(min(k1, j1), max(k2, j2));
      k1 = max(k1, j1);
    }
    V v1 = key_value(k1), v2 = key_value(k2);
    const bool summed = p.best == 2;
    if (summed && !biased) {  // the logits' order, but the scores are added
      v1 = k1 == 0 ? V(0) : quick_score(sigmoid, v1, m, by_sum);
      v2 = k2 == 0 ? V(0) : quick_score(sigmoid, v2, m, by_sum);
    }
    const V value = summed && k2 != 0 ? v1 + v2 : v1;
    const Key mine = k1 == 0 ? Key(0) : order_key(value);
    const float size12 = fmaxf(fabsf(float(v1)), k2 != 0 ? fabsf(float(v2)) : 0.0f);
    // the best group, kept times over
    bool keep = false;
    for (int j = 0; j < p.kept; ++j) {
      Key b = keep ? Key(0) : mine;
      int h = g;
      warp_best(b, h);
      if (b == 0) break;
      keep = keep || h == g;
    }
    if constexpr (ROUNDED) {
      if (biased || summed) {
        // the least that a kept value can be against the most that another can
        const float off = 2.0f * err + 0x1p-22f * size12;
        const uint32_t low = __reduce_min_sync(kAll, keep ? order_key(value - off) : 0xffffffffu);
        const uint32_t high = __reduce_max_sync(kAll, keep || mine == 0 ? 0u : order_key(value + off));
        if (high >= low) {  // (of the whole warp)
          if (!sigmoid && token.sum == 0.0) sum_in_64(p, plan, token);
          // experts within two errors of the group's last that counts; without a bias
          // the keys are logits, in whose order nothing is open, nor is it below a
          // last that is +inf or NaN
          const Key last = summed && k2 != 0 ? k2 : k1;
          const float v = key_value(last);
          const Key least = biased && v < INFINITY ? order_key(v - 2.0f * err - 0x1p-22f * fabsf(v)) : last;
          unsigned close = 0;
#pragma unroll
          for (int i = 0; i < EPL; ++i) close |= key[i] != 0 && key[i] >= least ? 1u << i : 0u;
          keep = keep_in_64(p, plan, token, close);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = keep ? key[i] : Key(0);
  }
  Key my_key, next_key;
  int next_id;
  const int rounds = ROUNDED && biased ? p.k + 1 : p.k;
  int all = 0, id_of_all = -1;  // of the candidates
  bool ranked = false;
  if constexpr (ROUNDED)
    ranked = rounds <= 32 && choose_by_ranks(plan, key, rounds, p.k, biased ? 2.0f * err : 0.0f, my_key, my_id,
                                             next_key, next_id, all, id_of_all);
  if (!ranked) choose_by_rounds(plan, key, rounds, p.k, my_key, my_id, next_key, next_id);
  if (lane >= p.k) my_id = -1;
  float mx = my_id >= 0 ? logit(my_id) : -INFINITY;
  if (ROUNDED && biased) {
    // each choice against the next one; equal logits with equal biases are a
    // true tie, which the expert's number has settled
    Key ok = __shfl_down_sync(kAll, my_key, 1);
    if (lane == p.k - 1) ok = next_key;
    bool open = false;
    if (lane < p.k && my_key != 0 && ok != 0) {
      const float a = float(key_value(my_key)), b = float(key_value(ok));
      open = a - b <= 2.0f * err + 0x1p-22f * fmaxf(fabsf(a), fabsf(b));
    }
    if (__any_sync(kAll, open)) {
      const float mb = my_id >= 0 ? ptx::load(p.bias + my_id) : 0.0f;
      const float nx = next_id >= 0 ? logit(next_id) : -INFINITY;
      const float nb = next_id >= 0 ? ptx::load(p.bias + next_id) : 0.0f;
      float ox = __shfl_down_sync(kAll, mx, 1), ob = __shfl_down_sync(kAll, mb, 1);
      if (lane == p.k - 1) ox = nx, ob = nb;
      sure = !(open && !(ox == mx && ob == mb));
    }
    if constexpr (ROUNDED) {
      if (ranked && !__all_sync(kAll, sure)) {
        if (!sigmoid && token.sum == 0.0) sum_in_64(p, plan, token);
        my_id = rank_in_64(p, token, *plan.found, lane, all, id_of_all);
        if (lane >= p.k) my_id = -1;
        mx = my_id >= 0 ? logit(my_id) : -INFINITY;
        sure = true;
      }
    }
  }
  V w = my_id >= 0 ? score_of(sigmoid, V(mx), m, sum) : V(0);
  if (p.renormalize) {
    V total = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    if (ROUNDED && my_id >= 0 && total < V(1e-30)) sure = false;  // near underflow
    w = total > V(0) || total != total ? w / total : V(0);
  }
  my_weight = my_id >= 0 ? static_cast<float>(V(p.scale) * w) : 0.0f;
  return __all_sync(kAll, sure);
}

template <int EPL>
__device__ __noinline__ void choose_in_64(const RouteParams &p, const ScorePlan<EPL> &plan, int64_t t, int &id,
                                          float &weight) {
  choose_exactly<double, EPL>(p, plan, t, id, weight);
}

// How a block chooses: by the logits, LPT lanes per token,
template <int LPT, int EPL, bool FP32>
struct ByLogit {
  static constexpr int LANES = LPT, WARPS = 32;  // of a token; most of a block
  static OneLaunch one(const RouteParams &) { return one_by_logit(LPT); }
  __device__ ByLogit(const RouteParams &, int, void *) {}
  __device__ __forceinline__ void choose(const RouteParams &p, int64_t t, int64_t end, int lane, uint16_t *ids16) {
    swiglu::choose<LPT, EPL, FP32>(p, t, end, lane, ids16);
  }
};
// or by scores, a warp per token.  With 32 experts a lane 64 registers (32 warps) do
// not hold the lane's keys: 16 warps (32 warps in brackets) take for sigmoid with a bias
// 3000 x 1024 40.7 us (55.2), 16384 x 1024 101 (157), 16384 x 768 80.6 (81.8),
// 16384 x 576 70.2 (61.8), 65536 x 1024 407 (405).
template <int EPL>
struct ByScore {
  static constexpr int LANES = 32, WARPS = EPL > 16 ? 16 : 32;
  static OneLaunch one(const RouteParams &p) { return one_by_score(EPL, p.k); }
  ScorePlan<EPL> plan;
  __device__ ByScore(const RouteParams &p, int lane, void *spare)
      : plan(p, lane, static_cast<Candidates *>(spare) + (threadIdx.x >> 5)) {}
  __device__ __forceinline__ void choose(const RouteParams &p, int64_t t, int64_t end, int lane, uint16_t *ids16) {
    if (t >= end) return;
    int id;
    float weight;
    if (!choose_exactly<float, EPL>(p, plan, t, id, weight)) choose_in_64<EPL>(p, plan, t, id, weight);
    if (lane < p.k) {
      p.ids[t * p.k + lane] = id;
      p.weights[t * p.k + lane] = weight;
      ids16[lane] = static_cast<uint16_t>(id);
    }
  }
};

// Walks this warp's entries [i0, i1) of the block, 32 at a time, adding them to
// cnt[expert]; number(i, e, before) gets each entry's expert and the entries
// counted before it (e = 0xffff: none).
template <class F>
__device__ __forceinline__ void walk(const uint16_t *ids16, int i0, int i1, uint16_t *cnt, int lane,
                                     F number) {
  for (int b = i0; b < i1; b += 32) {
    const int i = b + lane;
    const unsigned e = i < i1 ? ids16[i] : 0xffffu;
    const unsigned same = __match_any_sync(kAll, e);
    const unsigned before = same & ((1u << lane) - 1u);
    if (i < i1) number(i, e, e != 0xffffu ? cnt[e] + __popc(before) : 0);
    __syncwarp();
    if (e != 0xffffu && before == 0u) cnt[e] += static_cast<uint16_t>(__popc(same));
    __syncwarp();
  }
}

struct RouteSmem {
  uint16_t cnt[kCounters];  // [warp][E]
  alignas(16) int32_t base[kMaxE];     // first place of each expert's entries
  int32_t total[kMaxE];     // entries of this block (read by the cluster's other blocks), or of the blocks before
  uint16_t ids[kBlockTokens * kMaxK];
  int32_t carry[32];
};

static_assert(sizeof(RouteSmem) <= 48 * 1024, "static shared memory");

// Exclusive scan of base[0, E) in place; returns the total.  All threads.
__device__ __forceinline__ int scan_experts(RouteSmem &sm, int E, int32_t *offsets) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int carried = 0;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    const int v = e < E ? sm.base[e] : 0;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(kAll, s, o);
      if (lane >= o) s += w;
    }
    if (lane == 31) sm.carry[warp] = s;
    __syncthreads();
    int c = lane < warps ? sm.carry[lane] : 0;  // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(kAll, c, o);
      if (lane >= o) c += w;
    }
    const int before = __shfl_sync(kAll, c, max(warp - 1, 0));
    const int first = carried + (warp > 0 ? before : 0) + s - v;
    if (e < E) {
      sm.base[e] = first;
      if (offsets) offsets[e] = first;
    }
    carried += __shfl_sync(kAll, c, 31);
    __syncthreads();
  }
  if (offsets && threadIdx.x == 0) offsets[E] = carried;
  return carried;
}

// One block of tokens; ONE: a block of the only cluster, which does the whole
// call, otherwise the first pass of it.
template <class How, bool ONE>
__global__ void __launch_bounds__(32 * How::WARPS, 1) route_choose_kernel(const __grid_constant__ RouteParams p) {
  __shared__ RouteSmem sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int rank = blockIdx.x, ranks = ONE ? gridDim.x : 1;
  const int tokens = p.block_tokens;
  uint16_t *cnt = sm.cnt + warp * p.E;
  ptx::grid_launch_dependents();
  for (int e = lane; e < p.E; e += 32) cnt[e] = 0;
  ptx::grid_dependency_wait();
  const int64_t b0 = int64_t(blockIdx.x) * tokens;
  const int nt = static_cast<int>(max(int64_t(0), min(int64_t(tokens), p.T - b0)));
  // each warp takes a run of tokens, 32 / LPT at a time
  constexpr int SIDE = 32 / How::LANES;
  const int t0 = min(warp * p.warp_tokens, nt), t1 = min(t0 + p.warp_tokens, nt);
  // (base and total, 256 bytes a warp, are not in use yet)
  static_assert(sizeof(sm.base) + sizeof(sm.total) == 32 * sizeof(Candidates), "32 candidates a warp");
  How how(p, lane, sm.base);
  for (int t = t0; t < t1; t += SIDE)
    how.choose(p, b0 + t + lane / How::LANES, b0 + t1, lane, sm.ids + (t + lane / How::LANES) * p.k);
  __syncwarp();
  walk(sm.ids, t0 * p.k, t1 * p.k, cnt, lane, [](int, unsigned, int) {});
  __syncthreads();
  // the warps' counts of each expert, in order
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    int run = 0;
    for (int w = 0; w < warps; ++w) {
      const int c = sm.cnt[w * p.E + e];
      sm.cnt[w * p.E + e] = static_cast<uint16_t>(run);
      run += c;
    }
    if (ONE)
      sm.total[e] = sm.base[e] = run;
    else
      p.counts[int64_t(blockIdx.x) * p.E + e] = run;
  }
  if (ONE && ranks > 1) {
    // the cluster's counts, and those of the blocks before this one
    ptx::cluster_sync();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
      int all = 0, before = 0;
      for (int r = 0; r < ranks; ++r) {
        const int c = static_cast<int>(
            ptx::ld_shared_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sm.total[e]), r)));
        all += c;
        before += r < rank ? c : 0;
      }
      sm.base[e] = all;
      for (int w = 0; w < warps; ++w) sm.cnt[w * p.E + e] += static_cast<uint16_t>(before);
    }
    // the other blocks have read this one's counts: it may end
    ptx::cluster_sync();
  } else {
    __syncthreads();
  }
  const int routed = ONE ? scan_experts(sm, p.E, rank == 0 ? p.offsets : nullptr) : 0;
  walk(sm.ids, t0 * p.k, t1 * p.k, cnt, lane, [&](int i, unsigned e, int before) {
    const int64_t entry = b0 * p.k + i;
    if (ONE && e != 0xffffu) {
      before += sm.base[e];
      p.rows[before] = static_cast<int32_t>(entry) / p.k;
    }
    p.slots[entry] = e == 0xffffu ? -1 : before;
  });
  if (ONE && rank == 0)
    for (int i = routed + threadIdx.x; i < p.T * p.k; i += blockDim.x) p.rows[i] = -1;
}

// Several blocks, second pass: the block's entries get their places.
__global__ void __launch_bounds__(1024) route_place_kernel(const RouteParams p) {
  __shared__ RouteSmem sm;
  const int b = blockIdx.x;
  ptx::grid_launch_dependents();
  int32_t *mine = sm.total;  // [E] entries of the blocks before this one
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    sm.base[e] = 0;
    mine[e] = 0;
  }
  ptx::grid_dependency_wait();
  const int64_t b0 = int64_t(b) * p.block_tokens, entries = int64_t(p.T) * p.k;
  const int64_t end = min(b0 + p.block_tokens, int64_t(p.T)) * p.k;
  // the thread's first entry, on its way while the counts are summed
  int64_t i = b0 * p.k + threadIdx.x;
  int e_next = i < end ? ptx::load(p.ids + i) : -1, s_next = i < end ? p.slots[i] : 0;
  __syncthreads();
  // Thread (g, e) sums blocks g, g + G, ... of expert e, or of four from e on where
  // the blocks' counts are whole pieces of 16 bytes (256 experts: 12.2 -> 9.3 us);
  // integer sums in shared memory: their order does not matter.
  if (p.E % 4 == 0 && (reinterpret_cast<uintptr_t>(p.counts) & 15u) == 0) {
    const int quads = p.E / 4, G4 = static_cast<int>(blockDim.x) / quads, g = threadIdx.x / quads;
    const int e = 4 * (static_cast<int>(threadIdx.x) % quads);
    if (g < G4) {
      int all[4] = {}, before[4] = {};
#pragma unroll 8
      for (int i = g; i < p.blocks; i += G4) {
        const int4 c = ptx::load(reinterpret_cast<const int4 *>(p.counts + int64_t(i) * p.E + e));
        const int v[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          all[j] += v[j];
          before[j] += i < b ? v[j] : 0;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        atomicAdd(&sm.base[e + j], all[j]);
        atomicAdd(&mine[e + j], before[j]);
      }
    }
  } else {
    const int G = max(1, static_cast<int>(blockDim.x) / p.E);
    for (int e0 = 0; e0 < p.E; e0 += blockDim.x) {
      const int e = e0 + static_cast<int>(threadIdx.x) % p.E;  // E > blockDim.x: e0 + threadIdx.x
      const int g = threadIdx.x / p.E;
      if (e < p.E && g < G) {
        int all = 0, before = 0;
#pragma unroll 8
        for (int i = g; i < p.blocks; i += G) {
          const int c = ptx::load(p.counts + int64_t(i) * p.E + e);
          all += c;
          before += i < b ? c : 0;
        }
        atomicAdd(&sm.base[e], all);
        atomicAdd(&mine[e], before);
      }
    }
  }
  __syncthreads();
  const int routed = scan_experts(sm, p.E, b == 0 ? p.offsets : nullptr);
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) sm.base[e] += mine[e];
  __syncthreads();
  while (i < end) {
    if (e_next >= 0) {
      const int pos = sm.base[e_next] + s_next;
      p.slots[i] = pos;
      p.rows[pos] = static_cast<int32_t>(i) / p.k;  // T * k < 2^31
    }
    i += blockDim.x;
    if (i < end) {
      e_next = ptx::load(p.ids + i);
      s_next = p.slots[i];
    }
  }
  for (int64_t n = routed + int64_t(b) * blockDim.x + threadIdx.x; n < entries;
       n += int64_t(p.blocks) * blockDim.x)
    p.rows[n] = -1;
}

cudaError_t launch_pdl(void (*kern)(RouteParams), int grid, int cluster, int threads,
                       const RouteParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// Tokens per block of the two-launch form: as many blocks as SMs (GB300's 152),
// 32 to 128 tokens each, whole groups of eight (4096 tokens in blocks of 32: 11.3
// us, of 128: 12.7; 1024 tokens 7.8 and 12.0).
int block_tokens(int64_t T) {
  const int64_t n = ((T + 151) / 152 + 7) / 8 * 8;
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>(n, 32), kBlockTokens));
}

// Sizes that the call takes (places and offsets are 32-bit).
bool supported(int64_t T, int64_t E, int64_t k) {
  return E <= kMaxE && k <= kMaxK && T <= ((int64_t(1) << 31) - 1) / k;
}

template <class How>
cudaError_t launch_route(const RouteParams &p, cudaStream_t s) {
  // warps: as many as there are groups of tokens, or experts for the scans of a few
  // tokens, and counters for (one token, 256 experts by scores, in a graph: 8.7 us
  // with a warp, 6.7 with 8)
  constexpr int SIDE = 32 / How::LANES;
  auto warps = [&](int tokens) {
    return std::min({How::WARPS, kCounters / p.E, std::max((tokens + SIDE - 1) / SIDE, (p.E + 31) / 32)});
  };
  // a warp's run of tokens
  auto shared_out = [&](RouteParams q, int tokens) {
    q.warp_tokens = (tokens + warps(tokens) * SIDE - 1) / (warps(tokens) * SIDE) * SIDE;
    return q;
  };
  if (p.T <= kOneTokens) {
    RouteParams one = p;
    one.block_tokens = one_block_tokens(p.T, How::one(p));
    one.blocks = one_blocks(p.T, one.block_tokens);
    return launch_pdl(route_choose_kernel<How, true>, one.blocks, one.blocks, 32 * warps(one.block_tokens),
                      shared_out(one, one.block_tokens), s);
  }
  const cudaError_t e = launch_pdl(route_choose_kernel<How, false>, p.blocks, 1, 32 * warps(p.block_tokens),
                                   shared_out(p, p.block_tokens), s);
  return e != cudaSuccess ? e : launch_pdl(route_place_kernel, p.blocks, 1, 1024, p, s);
}

template <int LPT, int EPL>
cudaError_t launch_by_logit(bool fp32, const RouteParams &p, cudaStream_t s) {
  return fp32 ? launch_route<ByLogit<LPT, EPL, true>>(p, s) : launch_route<ByLogit<LPT, EPL, false>>(p, s);
}

// What the two calls share: the checks but those of the choice, and the launch.
template <class Launch>
int run_route(RouteParams p, bool fp32, int64_t T, int64_t E, int64_t k, void *workspace,
              uint64_t workspace_bytes, void *stream, Launch launch) {
  if (!supported(T, E, k)) return SWIGLU_ERR_UNSUPPORTED;
  if (!p.offsets || (T > 0 && (!p.logits || !p.ids || !p.weights || !p.rows || !p.slots)))
    return SWIGLU_ERR_INVALID_ARG;
  if (!ptr_aligned(p.logits, fp32 ? 4 : 2) || !ptr_aligned(p.ids, 4) || !ptr_aligned(p.weights, 4) ||
      !ptr_aligned(p.offsets, 4) || !ptr_aligned(p.rows, 4) || !ptr_aligned(p.slots, 4) ||
      !ptr_aligned(p.bias, 4) || !ptr_aligned(workspace, 4))
    return SWIGLU_ERR_MISALIGNED;
  const uint64_t need = swiglu_moe_route_workspace_size(T, E, k);
  if (need > 0 && (!workspace || workspace_bytes < need)) return SWIGLU_ERR_INVALID_ARG;
  // no output may overlap the inputs, the workspace or another output
  const uint64_t n4 = uint64_t(T) * k * 4;
  const void *ptr[8] = {p.logits, p.bias, p.ids, p.weights, p.rows, p.slots, p.offsets, need ? workspace : nullptr};
  const uint64_t len[8] = {uint64_t(T) * E * (fp32 ? 4 : 2), uint64_t(E) * 4, n4, n4, n4, n4,
                           uint64_t(E + 1) * 4, need};
  for (int i = 2; i < 8; ++i)
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(ptr[i], len[i], ptr[j], len[j])) return SWIGLU_ERR_INVALID_ARG;
  uint32_t *err = nullptr;
  int sms = 0;
  uint64_t timeout_ns = 0, gen = 0;
  int rc = device_info(&err, &sms, &timeout_ns, &gen);
  if (rc != SWIGLU_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0)
    return cudaMemsetAsync(p.offsets, 0, uint64_t(E + 1) * 4, s) == cudaSuccess ? SWIGLU_OK
                                                                                : SWIGLU_ERR_CUDA;
  p.counts = static_cast<int32_t *>(workspace);
  p.T = int32_t(T);
  p.E = int32_t(E);
  p.k = int32_t(k);
  p.block_tokens = block_tokens(T);
  p.blocks = int32_t((T + p.block_tokens - 1) / p.block_tokens);
  return launch(p, s) == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA;
}

}  // namespace
}  // namespace swiglu

extern "C" uint64_t swiglu_moe_route_workspace_size(int64_t T, int64_t E, int64_t k) {
  using namespace swiglu;
  if (T <= kOneTokens || E < 1 || k < 1 || !supported(T, E, k)) return 0;
  const int n = block_tokens(T);
  return uint64_t((T + n - 1) / n) * E * 4;
}

extern "C" int swiglu_moe_route(const void *logits, int32_t logits_fp32, int32_t renormalize,
                                float scale, int32_t *ids, float *weights, int32_t *offsets,
                                int32_t *rows, int32_t *slots, int64_t T, int64_t E, int64_t k,
                                void *workspace, uint64_t workspace_bytes, void *stream) {
  using namespace swiglu;
  if (T < 0 || E < 1 || k < 1 || k > E || (logits_fp32 != 0 && logits_fp32 != 1) ||
      (renormalize != 0 && renormalize != 1) || !std::isfinite(scale))
    return SWIGLU_ERR_INVALID_ARG;
  RouteParams p = {};
  p.logits = logits;
  p.ids = ids;
  p.weights = weights;
  p.offsets = offsets;
  p.rows = rows;
  p.slots = slots;
  p.renormalize = renormalize;
  p.scale = scale;
  const bool f = logits_fp32 != 0;
  const int64_t lanes = std::max((E + 7) / 8, k);  // per token
  return run_route(p, f, T, E, k, workspace, workspace_bytes, stream, [=](const RouteParams &q, cudaStream_t s) {
    return lanes <= 4    ? launch_by_logit<4, 8>(f, q, s)
           : lanes <= 8  ? launch_by_logit<8, 8>(f, q, s)
           : lanes <= 16 ? launch_by_logit<16, 8>(f, q, s)
           : E <= 256    ? launch_by_logit<32, 8>(f, q, s)
           : E <= 512    ? launch_by_logit<32, 16>(f, q, s)
                         : launch_by_logit<32, 32>(f, q, s);
  });
}

extern "C" int swiglu_moe_route_scored(const void *logits, int32_t logits_fp32, int32_t score,
                                       const float *bias, int32_t groups, int32_t kept_groups,
                                       int32_t group_best, int32_t renormalize, float scale,
                                       int32_t *ids, float *weights, int32_t *offsets, int32_t *rows,
                                       int32_t *slots, int64_t T, int64_t E, int64_t k, void *workspace,
                                       uint64_t workspace_bytes, void *stream) {
  using namespace swiglu;
  if (T < 0 || E < 1 || k < 1 || (logits_fp32 != 0 && logits_fp32 != 1) || (score != 0 && score != 1) ||
      (renormalize != 0 && renormalize != 1) || !std::isfinite(scale) || groups < 1 || E % groups != 0 ||
      kept_groups < 1 || kept_groups > groups || (group_best != 1 && group_best != 2) ||
      k > E / groups * kept_groups)
    return SWIGLU_ERR_INVALID_ARG;
  if (groups > 32 || (groups & (groups - 1)) != 0) return SWIGLU_ERR_UNSUPPORTED;
  RouteParams p = {};
  p.logits = logits;
  p.ids = ids;
  p.weights = weights;
  p.offsets = offsets;
  p.rows = rows;
  p.slots = slots;
  p.renormalize = renormalize;
  p.scale = scale;
  p.bias = bias;
  p.groups = groups;
  p.kept = kept_groups;
  p.best = group_best;
  p.sigmoid = score;
  p.fp32 = logits_fp32;
  // experts of a lane: a group's lie in 32 / groups lanes
  const int64_t lanes = 32 / groups, per_lane = (E / groups + lanes - 1) / lanes;
  p.group_size = static_cast<int32_t>(E / groups);
  while ((1 << p.lane_bits) < lanes) ++p.lane_bits;
  return run_route(p, logits_fp32 != 0, T, E, k, workspace, workspace_bytes, stream, [=](const RouteParams &q, cudaStream_t s) {
    return per_lane <= 2    ? launch_route<ByScore<2>>(q, s)
           : per_lane <= 8  ? launch_route<ByScore<8>>(q, s)
           : per_lane <= 16 ? launch_route<ByScore<16>>(q, s)
                            : launch_route<ByScore<32>>(q, s);
  });
}
