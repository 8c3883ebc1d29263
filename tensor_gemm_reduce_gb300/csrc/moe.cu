// moe.cu -- routing to experts and the experts' row-parallel layer in 8-bit
// floating point (gemm_rs_moe_* in include/gemm_rs_ops.h).
//
//   score = softmax(logits) or sigmoid(logits)         choice = score + bias
//   the top_groups groups with the largest sums of their two best choices stay,
//   of their experts the top_k best; weight = scale * score / (sum of the chosen)
//   rows: the token-expert pairs in the order of their experts, then tokens
//   out[t] = sum_j weight[t][j] (A[row] W[expert])     row = rows[t][j]
//
// Eight lanes or a whole warp route a token, lane l of them the experts l, l + 8 (or 32), ...  What is
// chosen does not depend on rounding: without a bias the order of scores is that of the logits;
// with one, or between groups, two fp32 values that are nearer than their errors
// send the token through the same code in 64 bits, by the whole warp.
#include <cfloat>
#include <cstring>

#include "fp8.cuh"

using namespace grs;

namespace {

constexpr int kMaxTopK = GEMM_RS_MOE_MAX_TOP_K;
constexpr int kMaxGroups = 32;
constexpr int kRouteWarps = 4;
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct RouteParams {
  const void* logits;
  const float* bias;
  const uint8_t* mask;
  int* ids;
  float* weights;
  int T, E, top_k, groups, top_groups, group_size;
  int bf16, sigmoid, renormalize;
  float scale;
  Divider by_group;
};

__device__ __forceinline__ float load_logit(const void* logits, int bf16, long long at) {
  if (bf16) {
    uint16_t v;
    asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(static_cast<const uint16_t*>(logits) + at) : "memory");
    return __uint_as_float((uint32_t)v << 16);
  }
  return load_f32(static_cast<const float*>(logits) + at);
}

// Integers in the order of the values: NaN 1, below every value; 0 is free for what is excluded.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 counts as 0
  return v != v ? 1u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long ordered(double v) {
  // in integers: an instruction in 64-bit floating point takes a warp 16 cycles
  const unsigned long long u = (unsigned long long)__double_as_longlong(v), size = u & ~(1ull << 63);
  return size > 0x7FF0000000000000ull ? 1ull : (u >> 63) && size ? ~u : u | (1ull << 63);
}
// Reductions over the W lanes of a token; W lanes are 32 or 8 of a warp.
template <int W, typename F>
__device__ __forceinline__ F lanes_sum(F v) {
#pragma unroll
  for (int d = W / 2; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
template <int W>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int d = W / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
template <int W>
__device__ __forceinline__ uint32_t lanes_ballot(bool v, int lane) {
  const uint32_t all = __ballot_sync(kAll, v);
  return W == 32 ? all : (all >> (lane & (32 - W))) & ((1u << (W & 31)) - 1u);
}
// The largest key of the token's lanes and the least index that has it.
template <int W>
__device__ __forceinline__ void lanes_best(uint32_t& key, int& index) {
  if constexpr (W == 32) {
    const uint32_t best = __reduce_max_sync(kAll, key);
    index = __reduce_min_sync(kAll, key == best ? index : 0x7FFFFFFF);
    key = best;
  } else {
#pragma unroll
    for (int d = W / 2; d > 0; d >>= 1) {
      const uint32_t k = __shfl_xor_sync(kAll, key, d);
      const int i = __shfl_xor_sync(kAll, index, d);
      const bool better = k > key || (k == key && i < index);
      key = better ? k : key;
      index = better ? i : index;
    }
  }
}
template <int W>
__device__ __forceinline__ void lanes_best(unsigned long long& key, int& index) {
  static_assert(W == 32, "the whole warp");
  const uint32_t high = __reduce_max_sync(kAll, (uint32_t)(key >> 32));
  const uint32_t low = __reduce_max_sync(kAll, (uint32_t)(key >> 32) == high ? (uint32_t)key : 0u);
  const unsigned long long best = (unsigned long long)high << 32 | low;
  index = __reduce_min_sync(kAll, key == best ? index : 0x7FFFFFFF);
  key = best;
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// sigmoid(x) / e^top where top, no less than x, is negative, else sigmoid(x): scores that are divided by
// their sum keep their ratios where each would underflow.
__device__ __forceinline__ float sigmoid_over(float x, float top) {
  if (x >= 0.f) return 1.f / (1.f + expf(-x));
  return top == -INFINITY ? 0.f : expf(x - fminf(top, 0.f)) / (1.f + expf(x));
}

// e^(x - top) for top no less than x; infinities that are the largest are equal.
template <typename F>
__device__ __forceinline__ F exp_below(F x, F top) {
  return x == top ? F(1) : exp_of(x - top);
}

// Scores of a token from its logits (E of them, slots behind E hold -inf).  A NaN counts as -inf; of logits
// of +inf each takes the same share of a softmax, and the others nothing.
template <int W, typename F, int kPer>
__device__ __forceinline__ void scores_of(const float (&logit)[kPer], bool sigmoid, F (&score)[kPer]) {
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) score[i] = logit[i] != logit[i] ? F(0) : F(1) / (F(1) + exp_of(-(F)logit[i]));
    return;
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) top = fmaxf(top, logit[i]);
  top = lanes_max<W>(top);
  F sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    score[i] = top == -INFINITY || logit[i] != logit[i] ? F(0) : exp_below((F)logit[i], (F)top);
    sum += score[i];
  }
  sum = lanes_sum<W>(sum);
#pragma unroll
  for (int i = 0; i < kPer; ++i) score[i] = top == -INFINITY ? F(0) : score[i] / sum;
}

// A choice is a score plus a bias.  In units of 2^-24, a softmax score is off by at most 32 of the
// token's largest score: its exponential by 4 (two units in the last place) and by 1 for its argument x
// (|x| e^x is at most 1/e), the sum by the 4 of its terms' exponentials, by 3.4 for their arguments (the mean of
// |x| weighted by e^x, of 255 experts beside the largest, is below that) and by 18 for adding up slots
// and lanes, the quotient by 1; a sigmoid s by 5 (4 s (1 - s) for its exponential, sum 1, quotient 1, the
// rest to spare); the choice by another 1 of itself.  `slack` is
// twice the multiple for the score.  With a quarter more for the bound's own roundings, two choices may
// be in the wrong order where they are this near.  (A bound for scores of 1 sent 20 to 30 times as many
// tokens of 96 experts to 64 bits.)
__device__ __forceinline__ bool near_values(float a, float b, float slack) {
  const float d = fabsf(a - b);
  return d <= 7.5e-8f * (slack + fabsf(a) + fabsf(b)) && d <= FLT_MAX;
}

// Chooses a token's experts: its lane j < top_k returns the j-th one's index.  In fp32, false
// where the choice may depend on rounding.  `scratch`: the token's, W * kPer doubles.  Every lane
// of the warp takes part throughout, whatever its token.
template <int W, typename F, int kPer>
__device__ __forceinline__ bool choose(const RouteParams& p, const float (&logit)[kPer], int lane, double* scratch, int* id) {
  constexpr bool kCheck = sizeof(F) == 4;
  const int sub = lane & (W - 1);
  F choice[kPer];
  F* values = reinterpret_cast<F*>(scratch);
  bool sure = true;
  uint32_t kept = kAll;
  float slack = 0.f;
  if (p.bias || p.groups > 1) {
    scores_of<W>(logit, p.sigmoid, choice);
    if constexpr (kCheck) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) top = fmaxf(top, choice[i]);
      slack = p.sigmoid ? 2 * 5.f : 2 * 32.f * lanes_max<W>(top);
    }
    if (p.bias)
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (sub + W * i < p.E) choice[i] += (F)load_f32(p.bias + sub + W * i);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kPer; ++i) values[sub + W * i] = choice[i];
    __syncwarp();
  }
  if (p.groups > 1) {
    F sum = -INFINITY;
    float error = 0.f;  // of a sum of two: as two choices, and its own rounding
    if (sub < p.groups) {  // its group's two best
      F a = -INFINITY, b = -INFINITY;
      // lanes start at different places of their groups: from the first on, groups of 16 lie in two banks
      int at = lane & (p.group_size - 1);
#pragma unroll 4
      for (int i = 0; i < p.group_size; ++i) {
        const F v = values[sub * p.group_size + at];
        at = at + 1 < p.group_size ? at + 1 : 0;
        if (v > a) {
          b = a;
          a = v;
        } else if (v > b) {
          b = v;
        }
      }
      sum = p.group_size > 1 ? a + b : a;
      if (sum != sum) sum = a;  // inf - inf: the group of an expert that a bias forces
      if constexpr (kCheck) {
        error = 7.5e-8f * (slack + fabsf(a) + fabsf(b) + fabsf(sum));
        if (!(error <= FLT_MAX)) error = 0.f;  // infinite sums are exact
      }
    }
    if constexpr (kCheck) error = 2.f * lanes_max<W>(error);
    int rank = 0;
    bool close = false;
    for (int g = 0; g < p.groups; ++g) {
      const F other = __shfl_sync(kAll, sum, g, W);
      rank += g != sub && (other > sum || (other == sum && g < sub));
      if constexpr (kCheck) close |= g != sub && fabsf(other - sum) <= error;
    }
    kept = lanes_ballot<W>(sub < p.groups && rank < p.top_groups, lane);
    if constexpr (kCheck) {
      // a close pair matters where one of its groups stays and the other does not
      const uint32_t closes = lanes_ballot<W>(close && sub < p.groups, lane);
      if ((closes & kept) && (closes & ~kept)) sure = false;
    }
  }
  using Key = decltype(ordered(F(0)));
  Key key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = sub + W * i;
    const bool in = e < p.E && (p.groups == 1 || (kept >> divided((uint32_t)e, p.by_group)) & 1u);
    key[i] = !in ? Key(0) : p.bias ? ordered(choice[i]) : ordered((F)logit[i]);
  }
  const bool check = kCheck && p.bias;
  const int picks = check ? p.top_k + 1 : p.top_k;
  int found = -1;
  auto next = [&](Key& best, int& e) {  // the best of those that are left
    best = key[0];
    e = sub;
#pragma unroll
    for (int i = 1; i < kPer; ++i)
      if (key[i] > best) {
        best = key[i];
        e = sub + W * i;
      }
    lanes_best<W>(best, e);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (e == sub + W * i) key[i] = 0;
  };
  Key best;
  int e;
  for (int j = 0; j < picks; ++j) {
    next(best, e);
    if (j == sub && best != 0) found = e;  // 0: only behind the last of the experts that there are
  }
  if (check) {  // is one nearer to the one before than the errors, and not its equal?
    float v = 0.f, l = 0.f, b = 0.f;
    if (found >= 0) {
      v = (float)values[found];
      b = load_f32(p.bias + found);
    }
    float* logits = reinterpret_cast<float*>(scratch) + W * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) logits[sub + W * i] = logit[i];
    __syncwarp();
    if (found >= 0) l = logits[found];
    const float pv = __shfl_up_sync(kAll, v, 1, W), pl = __shfl_up_sync(kAll, l, 1, W), pb = __shfl_up_sync(kAll, b, 1, W);
    const bool same = l == pl && b == pb;
    if (lanes_ballot<W>(sub > 0 && found >= 0 && near_values(v, pv, slack) && !same, lane)) sure = false;
    // where the last that is chosen and the first that is not are equals, the first behind them that is none
    bool equals = (lanes_ballot<W>(found >= 0 && same, lane) >> p.top_k) & 1u;
    const float lv = __shfl_sync(kAll, v, p.top_k, W), ll = __shfl_sync(kAll, l, p.top_k, W), lb = __shfl_sync(kAll, b, p.top_k, W);
    while (__any_sync(kAll, equals)) {
      next(best, e);
      if (!equals) continue;
      equals = best != 0 && logits[e] == ll && load_f32(p.bias + e) == lb;
      if (best != 0 && !equals && near_values((float)values[e], lv, slack)) sure = false;
    }
  }
  *id = found >= 0 ? found : 0;
  return sure;
}

template <int W, int kPer>
__device__ __forceinline__ void load_logits(const RouteParams& p, int t, int sub, float (&logit)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = sub + W * i;
    logit[i] = e < p.E ? load_logit(p.logits, p.bf16, (long long)t * p.E + e) : -INFINITY;
  }
}

// One token by the whole warp.  Reads the logits again: an argument in memory would keep them there
// for every token.
template <int kPer>
__device__ __noinline__ int choose_in_64_bits(const RouteParams& p, int t, int lane, double* scratch) {
  float logit[kPer];
  load_logits<32>(p, t, lane, logit);
  int id = 0;
  choose<32, double>(p, logit, lane, scratch, &id);
  return id;
}

// A warp's tokens, 32 / W of them from t0 on.  scratch: the warp's 32 * kPer doubles.
template <int W, int kPer>
__device__ __forceinline__ void route_tokens(const RouteParams& p, int t0, int lane, double* scratch) {
  const int sub = lane & (W - 1);
  const bool exists = t0 + lane / W < p.T;
  const int t = exists ? t0 + lane / W : p.T - 1;
  double* const all_scratch = scratch;
  scratch += (lane / W) * (W * kPer);
  bool masked = false;
  if (p.mask) {
    uint32_t m;
    asm volatile("ld.global.u8 %0, [%1];" : "=r"(m) : "l"(p.mask + t) : "memory");
    masked = m == 0;
  }
  float logit[kPer];
  load_logits<W>(p, t, sub, logit);
  bool nan = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) nan |= logit[i] != logit[i];
  int id = 0;
  const bool sure = choose<W, float>(p, logit, lane, scratch, &id) || masked;
  for (uint32_t unsure = __ballot_sync(kAll, !sure); unsure;) {  // token by token
    const int first = (__ffs(unsure) - 1) & ~(W - 1);
    const int exact = choose_in_64_bits<(W * kPer + 31) / 32>(p, __shfl_sync(kAll, t, first), lane, all_scratch);
    const int mine = __shfl_sync(kAll, exact, sub);
    if (lane / W == first / W) id = mine;
    unsure &= W == 32 ? 0u : ~(((1u << (W & 31)) - 1u) << first);
  }
  nan = lanes_ballot<W>(nan, lane) != 0;
  // lane j: the j-th chosen one's score, from its logit where the others do not count or cancel
  float score[kPer];
  const bool of_all = !p.sigmoid && !p.renormalize;
  if (of_all) scores_of<W>(logit, false, score);
  float* values = reinterpret_cast<float*>(scratch);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPer; ++i) values[sub + W * i] = of_all ? score[i] : logit[i];
  __syncwarp();
  float mine = values[id];
  __syncwarp();
  const bool in = sub < p.top_k;
  if (p.sigmoid || p.renormalize) {
    const float top = p.renormalize ? lanes_max<W>(in ? mine : -INFINITY) : 0.f;
    mine = p.sigmoid ? sigmoid_over(mine, top) : top == -INFINITY ? 0.f : exp_below(mine, top);
  }
  float total = 1.f;
  if (p.renormalize) {
    total = lanes_sum<W>(in ? mine : 0.f);
    if (total == 0.f) total = 1.f;  // every chosen one's score is zero: so are the weights
  }
  if (in && exists) {
    const long long at = (long long)t * p.top_k + sub;
    p.ids[at] = masked ? -1 : id;
    p.weights[at] = masked ? 0.f : nan ? __uint_as_float(0x7FC00000u) : p.scale * (mine / total);
  }
}

// Eight lanes a token where its groups and experts to choose fit them and its experts their
// slots: a warp's instructions serve four tokens.  With the arrangement 16384 x 96 with a bias and 6
// groups takes 22 to 26 us, with 32 lanes 6 more; 32768 x 8 7.0 against 12, its gradient 3.9 against 10.6.  Bound by
// instructions; one token that is decided in 64 bits makes a launch 4 us longer, of 256 experts 10.
template <int W, int kPer>
__global__ void __launch_bounds__(32 * kRouteWarps, kPer >= 8 ? 6 : 8)
    route_kernel(const __grid_constant__ RouteParams p) {
  __shared__ double scratch[kRouteWarps][32 * kPer];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_launch_dependents();
  griddep_wait();
  const int t0 = (blockIdx.x * kRouteWarps + warp) * (32 / W);
  if (t0 < p.T) route_tokens<W, kPer>(p, t0, lane, scratch[warp]);
}

// The pairs in the order of their experts.  Ids outside 0 .. E-1 have no row.  Nothing is
// kept between launches or has to be cleared, and no order depends on timing.
struct ArrangeParams {
  const int* ids;
  int *rows, *pairs, *offsets;
  int n, E, per;  // per: pairs of a warp, whole groups of 32 (arrange_kernel: of 128)
};

constexpr int kArrangeWarps = 32, kArrangeThreads = 32 * kArrangeWarps;

// Few pairs: one CTA.  A warp takes consecutive pairs, 32 at a time, and counts them by expert
// in its own counters.  Sums over warps, then over experts turn the counters into the rows
// that the warp's next pairs take; a second walk over the ids hands them out.

// The lanes whose ids are equal to this lane's, from a ballot for each of their low `bits`
// bits (match_any walks over the distinct values).
__device__ __forceinline__ uint32_t lanes_alike(int id, int bits) {
  uint32_t same = kAll;
  for (int b = 0; b < bits; ++b) {
    const uint32_t set = __ballot_sync(kAll, (id >> b) & 1);
    same &= (id >> b) & 1 ? set : ~set;
  }
  return same;
}

struct ArrangeShared {
  int counts[kArrangeWarps][kMaxExperts];
  int sums[kArrangeWarps];
};

// All threads of the CTA.
__device__ __forceinline__ void arrange_pairs(const ArrangeParams& p, ArrangeShared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int first = warp * p.per;
  const int mine = p.n > first ? (p.n - first < p.per ? p.n - first : p.per) : 0;
  int* counts = sh.counts[warp];
  for (int e = lane; e < p.E; e += 32) counts[e] = 0;
  __syncwarp();
  const uint32_t lower = (1u << lane) - 1;
  const int bits = 32 - __clz(p.E);  // of 0 .. E; an id of none has all of them set, as no expert does
  for (int pass = 0; pass < 2; ++pass) {
    for (int g = 0; g < mine; g += 32) {
      const int i = first + g + lane;
      int id = g + lane < mine ? p.ids[i] : -1;
      if ((unsigned)id >= (unsigned)p.E) id = -1;
      const uint32_t same = lanes_alike(id, bits);
      const bool leads = id >= 0 && (same & lower) == 0;
      if (pass == 1) {
        int row = -1;
        if (id >= 0) {
          row = counts[id] + __popc(same & lower);
          p.pairs[row] = i;
        }
        if (g + lane < mine) p.rows[i] = row;
        __syncwarp();
      }
      if (leads) counts[id] += __popc(same);
      __syncwarp();
    }
    if (pass == 1) break;
    __syncthreads();
    int total = 0;
    if (tid < p.E) {
#pragma unroll 8
      for (int w = 0; w < kArrangeWarps; ++w) total += sh.counts[w][tid];
    }
    int sum = total;  // with the experts before
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(kAll, sum, d);
      if (lane >= d) sum += up;
    }
    if (lane == 31) sh.sums[warp] = sum;
    __syncthreads();
    if (tid < p.E) {
      for (int w = 0; w < warp; ++w) sum += sh.sums[w];
      int row = sum - total;
      p.offsets[tid] = row;
      if (tid == p.E - 1) p.offsets[p.E] = sum;
#pragma unroll 8
      for (int w = 0; w < kArrangeWarps; ++w) {
        const int c = sh.counts[w][tid];
        sh.counts[w][tid] = row;
        row += c;
      }
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kArrangeThreads) arrange_once_kernel(const __grid_constant__ ArrangeParams p) {
  __shared__ ArrangeShared sh;
  griddep_launch_dependents();
  griddep_wait();
  arrange_pairs(p, sh);
}

// More pairs: every cluster counts all of them, its 8 CTAs a part each, and hands out the rows
// of one group of 32 of each warp, as many clusters as a warp has groups.  Only that group's
// lanes are ranked by ballots, the others add to their warp's counters: with ballots for all,
// 98304 pairs and 96 experts took 13.5 us, without 7.3 (6.4 since).
constexpr int kShareCtas = 8, kShareGroups = 32;

__global__ void __launch_bounds__(kArrangeThreads) arrange_share_kernel(const __grid_constant__ ArrangeParams p) {
  __shared__ int counts[kArrangeWarps][kMaxExperts + 1];  // a column's 32 words lie in 32 banks
  __shared__ int totals[kMaxExperts], rows[kMaxExperts], sums[kMaxExperts / 32];
  const int cta = (int)cluster_ctarank(), cluster = blockIdx.x / kShareCtas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int e = lane; e < p.E; e += 32) counts[warp][e] = 0;
  __syncwarp();
  griddep_launch_dependents();
  griddep_wait();
  const int first = (cta * kArrangeWarps + warp) * p.per, groups = p.per / 32;
  const uint32_t lower = (1u << lane) - 1;
  const int bits = 32 - __clz(p.E);
  int mine = -1, rank = 0;
  for (int g0 = 0; g0 < groups; g0 += 4) {
    int ids[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = first + (g0 + k) * 32 + lane;
      ids[k] = g0 + k < groups && i < p.n ? p.ids[i] : -1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int id = (unsigned)ids[k] < (unsigned)p.E ? ids[k] : -1;
      if (g0 + k == cluster) {
        __syncwarp();
        mine = id;
        rank = (id >= 0 ? counts[warp][id] : 0) + __popc(lanes_alike(id, bits) & lower);
        __syncwarp();
      }
      if (id >= 0) atomicAdd(&counts[warp][id], 1);
    }
  }
  __syncthreads();
  for (int e = warp; e < p.E; e += kArrangeWarps) {  // the warps before, of this CTA
    const int count = counts[lane][e];
    int sum = count;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(kAll, sum, d);
      if (lane >= d) sum += up;
    }
    counts[lane][e] = sum - count;
    if (lane == 31) totals[e] = sum;
  }
  cluster_sync_shared();
  int total = 0, before = 0;
  if (tid < p.E) {
    int of[kShareCtas];
#pragma unroll
    for (int c = 0; c < kShareCtas; ++c)
      asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(of[c]) : "r"(mapa_shared(smem_u32(&totals[tid]), c)) : "memory");
#pragma unroll
    for (int c = 0; c < kShareCtas; ++c) {
      total += of[c];
      before += c < cta ? of[c] : 0;
    }
  }
  int sum = total;  // with the experts before
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(kAll, sum, d);
    if (lane >= d) sum += up;
  }
  if (lane == 31 && warp < kMaxExperts / 32) sums[warp] = sum;
  __syncthreads();
  if (tid < p.E) {
    for (int w = 0; w < warp; ++w) sum += sums[w];
    rows[tid] = sum - total + before;
    if (blockIdx.x == 0) {
      p.offsets[tid] = sum - total;
      if (tid == p.E - 1) p.offsets[p.E] = sum;
    }
  }
  __syncthreads();
  const int i = first + cluster * 32 + lane;
  if (i < p.n) {
    int row = -1;
    if (mine >= 0) {
      row = rows[mine] + counts[warp][mine] + rank;
      p.pairs[row] = i;
    }
    p.rows[i] = row;
  }
  cluster_sync_shared();  // the totals have been read
}

// Many pairs: a cluster for each expert, whose CTAs share the ids.  Each counts the pairs of the
// experts before, which gives the expert's first row, and ranks the expert's own by ballots.  A
// warp takes 128 pairs at a time, four to a lane.  Its ballots stay in shared memory for the second
// pass where they fit (393216 pairs a CTA); else the ids are read again.
constexpr int kArrangeWords = 384;  // of ballots for a warp

__global__ void __launch_bounds__(kArrangeThreads) arrange_kernel(const __grid_constant__ ArrangeParams p) {
  extern __shared__ __align__(16) uint32_t ballots[];  // [32][per / 32]
  __shared__ int mine[32], before[32];
  __shared__ __align__(8) int totals[2];
  const int ctas = (int)cluster_size(), cta = (int)cluster_ctarank(), e = blockIdx.x / ctas;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_launch_dependents();
  griddep_wait();
  const long long first = ((long long)cta * kArrangeWarps + warp) * p.per;
  const bool kept = p.per / 32 <= kArrangeWords;
  uint32_t* words = ballots + warp * (p.per / 32);
  const long long left = p.n - first;
  const int whole = left <= 0 ? 0 : (int)((left < p.per ? left : p.per) / 128);
  const int groups = left <= 0 ? 0 : (int)(((left < p.per ? left : p.per) + 127) / 128);
  auto whole_ids = [&](int g) { return *reinterpret_cast<const int4*>(p.ids + first + g * 128 + lane * 4); };
  auto last_ids = [&](int g) {  // behind the last one: none
    const long long i = first + g * 128 + lane * 4;
    return make_int4(i < p.n ? p.ids[i] : -1, i + 1 < p.n ? p.ids[i + 1] : -1, i + 2 < p.n ? p.ids[i + 2] : -1,
                     i + 3 < p.n ? p.ids[i + 3] : -1);
  };
  // f(g, ids) for the warp's groups, four groups' ids on their way at a time
  auto walk = [&](auto&& f) {
    int g = 0;
    for (; g + 4 <= whole; g += 4) {
      int4 v[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) v[b] = whole_ids(g + b);
#pragma unroll
      for (int b = 0; b < 4; ++b) f(g + b, v[b]);
    }
    for (; g < groups; ++g) f(g, g < whole ? whole_ids(g) : last_ids(g));
  };
  int own = 0, less = 0;
  walk([&](int g, int4 v) {
    const uint32_t hits[4] = {__ballot_sync(kAll, v.x == e), __ballot_sync(kAll, v.y == e), __ballot_sync(kAll, v.z == e),
                              __ballot_sync(kAll, v.w == e)};
    own += __popc(hits[0]) + __popc(hits[1]) + __popc(hits[2]) + __popc(hits[3]);
    less += ((unsigned)v.x < (unsigned)e) + ((unsigned)v.y < (unsigned)e) + ((unsigned)v.z < (unsigned)e) +
            ((unsigned)v.w < (unsigned)e);
    if (kept && lane == 0) *reinterpret_cast<uint4*>(words + 4 * g) = make_uint4(hits[0], hits[1], hits[2], hits[3]);
    if (e == 0) {  // pairs without an expert
      const int x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const long long i = first + g * 128 + lane * 4 + k;
        if (i < p.n && (unsigned)x[k] >= (unsigned)p.E) p.rows[i] = -1;
      }
    }
  });
  less = __reduce_add_sync(kAll, less);
  if (lane == 0) {
    mine[warp] = own;
    before[warp] = less;
  }
  __syncthreads();
  if (warp == 0) {
    const int a = __reduce_add_sync(kAll, mine[lane]), b = __reduce_add_sync(kAll, before[lane]);
    if (lane == 0) {
      totals[0] = a;
      totals[1] = b;
    }
  }
  cluster_sync_shared();
  int start = 0, row = 0, count = 0;
  for (int c = 0; c < ctas; ++c) {
    int a, b;
    asm volatile("ld.shared::cluster.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(mapa_shared(smem_u32(totals), c)) : "memory");
    start += b;
    count += a;
    if (c < cta) row += a;
  }
  if (cta == 0 && threadIdx.x == 0) {
    p.offsets[e] = start;
    if (e == p.E - 1) p.offsets[p.E] = start + count;
  }
  row += start + __reduce_add_sync(kAll, lane < warp ? mine[lane] : 0);
  const uint32_t lower = (1u << lane) - 1;
  auto place = [&](int g, const uint32_t (&hits)[4]) {
    // pairs are in the order of lanes, then of a lane's four
    int at = row + __popc(hits[0] & lower) + __popc(hits[1] & lower) + __popc(hits[2] & lower) + __popc(hits[3] & lower);
    row += __popc(hits[0]) + __popc(hits[1]) + __popc(hits[2]) + __popc(hits[3]);
    const int i = (int)(first + g * 128 + lane * 4);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if ((hits[k] >> lane) & 1u) {
        p.rows[i + k] = at;
        p.pairs[at] = i + k;
        ++at;
      }
  };
  if (kept && p.E >= 32) {
    // a group has few of the expert's pairs: a lane for each group
    __syncwarp();
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const int g = g0 + lane;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (g < groups) w = *reinterpret_cast<const uint4*>(words + 4 * g);
      const int count = __popc(w.x) + __popc(w.y) + __popc(w.z) + __popc(w.w);
      int sum = count;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(kAll, sum, d);
        if (lane >= d) sum += up;
      }
      int at = row + sum - count;
      row += __shfl_sync(kAll, sum, 31);
      for (uint32_t some = w.x | w.y | w.z | w.w; some; some &= some - 1) {
        const int l = __ffs(some) - 1, i = (int)(first + g * 128 + l * 4);
        const uint32_t hits[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if ((hits[k] >> l) & 1u) {
            p.rows[i + k] = at;
            p.pairs[at] = i + k;
            ++at;
          }
      }
    }
  } else if (kept) {
    __syncwarp();
    for (int g = 0; g < groups; ++g) {
      const uint4 w = *reinterpret_cast<const uint4*>(words + 4 * g);
      const uint32_t hits[4] = {w.x, w.y, w.z, w.w};
      if (w.x | w.y | w.z | w.w) place(g, hits);
    }
  } else {
    walk([&](int g, int4 v) {
      const uint32_t hits[4] = {__ballot_sync(kAll, v.x == e), __ballot_sync(kAll, v.y == e),
                                __ballot_sync(kAll, v.z == e), __ballot_sync(kAll, v.w == e)};
      place(g, hits);
    });
  }
  cluster_sync_shared();  // the totals have been read
}

// Few tokens: both in one launch, by one CTA.
constexpr int kRouteOnceWarps = 32;
template <int kPer>
__global__ void __launch_bounds__(32 * kRouteOnceWarps) route_once_kernel(const __grid_constant__ RouteParams p,
                                                                           const __grid_constant__ ArrangeParams a) {
  extern __shared__ __align__(16) uint8_t raw[];
  double* scratch = reinterpret_cast<double*>(raw) + (threadIdx.x >> 5) * 32 * kPer;
  griddep_launch_dependents();
  griddep_wait();
  for (int t = threadIdx.x >> 5; t < p.T; t += kRouteOnceWarps) route_tokens<32, kPer>(p, t, threadIdx.x & 31, scratch);
  __syncthreads();
  arrange_pairs(a, *reinterpret_cast<ArrangeShared*>(raw));
}

struct RouteBackwardParams {
  const float* dweights;
  const void* logits;
  const int* ids;
  void* dlogits;
  int T, E, top_k, bf16, sigmoid, renormalize;
  float scale;
};

// With w_j = scale s_j / S (S = 1 unless renormalised) and g_j = scale dw_j:
//   softmax, renormalised   dl_j = g_j' u_j           u_j = s_j / S, g_j' = g_j - sum_i g_i u_i
//   softmax                 dl_e = s_e (g_e - sum_j g_j s_j), g_e = 0 for experts not chosen
//   sigmoid                 dl_j = g_j' u_j (1 - s_j)  (g_j and s_j where not renormalised), 1 - s the
//                           sigmoid of the negated logit: as a difference it has lost 17% at 15, all at 17
// The choice has no gradient.
template <int W, int kPer>
__global__ void __launch_bounds__(32 * kRouteWarps) route_backward_kernel(const RouteBackwardParams p) {
  __shared__ float shared[kRouteWarps][32 * kPer];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & (W - 1);
  griddep_launch_dependents();
  griddep_wait();
  const int t0 = (blockIdx.x * kRouteWarps + warp) * (32 / W);
  if (t0 >= p.T) return;
  const bool exists = t0 + lane / W < p.T;
  const int t = exists ? t0 + lane / W : p.T - 1;
  float* values = shared[warp] + (lane / W) * (W * kPer);
  float logit[kPer], score[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = sub + W * i;
    logit[i] = e < p.E ? load_logit(p.logits, p.bf16, (long long)t * p.E + e) : -INFINITY;
  }
  bool nan = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) nan |= logit[i] != logit[i];
  int id = -1;
  float g = 0.f;
  if (sub < p.top_k) {
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(id) : "l"(p.ids + (long long)t * p.top_k + sub) : "memory");
    if ((unsigned)id < (unsigned)p.E) g = p.scale * load_f32(p.dweights + (long long)t * p.top_k + sub);
  }
  if (!p.sigmoid && !p.renormalize) scores_of<W>(logit, false, score);
  const bool has = (unsigned)id < (unsigned)p.E;
  nan = lanes_ballot<W>(nan, lane) != 0;
  nan = lanes_ballot<W>(has, lane) != 0 && nan;  // masked tokens have no gradient
  // the chosen one's score in a softmax of all, else its logit
  const bool dense = !p.sigmoid && !p.renormalize;  // every expert has a gradient
#pragma unroll
  for (int i = 0; i < kPer; ++i) values[sub + W * i] = dense ? score[i] : logit[i];
  __syncwarp();
  const float s = has ? values[id] : dense ? 0.f : -INFINITY;
  __syncwarp();
  float u = s, rest = 1.f;
  if (p.sigmoid) {
    u = sigmoid_over(s, 0.f);
    rest = sigmoid_over(-s, 0.f);
  }
  if (p.renormalize) {
    const float top = lanes_max<W>(s);
    u = top == -INFINITY || !has ? 0.f : p.sigmoid ? sigmoid_over(s, top) : exp_below(s, top);
    const float total = lanes_sum<W>(u);
    u = total == 0.f ? 0.f : u / total;
  }
  const float mean = lanes_sum<W>(g * u);
  const float d = (p.sigmoid && !p.renormalize ? g : g - mean) * u * rest;
#pragma unroll
  for (int i = 0; i < kPer; ++i) values[sub + W * i] = dense ? -score[i] * mean : 0.f;
  __syncwarp();
  if (has) values[id] = d;
  __syncwarp();
  if (!exists) return;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = sub + W * i;
    if (e >= p.E) continue;
    const long long at = (long long)t * p.E + e;
    const float grad = nan ? __uint_as_float(0x7FC00000u) : values[e];
    if (p.bf16)
      static_cast<uint16_t*>(p.dlogits)[at] = (uint16_t)pack_bf16x2(grad, 0.f);
    else
      static_cast<float*>(p.dlogits)[at] = grad;
  }
}

// out[t] = sum_j weight[t][j] y[rows[t][j]], in fp32, in the order of j.  Bound by memory: two of
// 2048 x 6144 20 us, 6.3 TB/s.
struct CombineParams {
  const float* y;
  const float* weights;
  const int* rows;
  uint4* out;
  int vec, top_k;  // vectors of 8 columns
  long long total, pairs;
};

constexpr int kCombineThreads = 256;

__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const long long stride = (long long)gridDim.x * kCombineThreads;
  for (long long i = (long long)blockIdx.x * kCombineThreads + threadIdx.x; i < p.total; i += stride) {
    const long long t = i / p.vec;
    const int col = (int)(i - t * p.vec);
    float acc[8] = {};
    for (int j = 0; j < p.top_k; ++j) {
      const int row = p.rows[t * p.top_k + j];
      if ((unsigned long long)row >= (unsigned long long)p.pairs) continue;
      const float w = p.weights[t * p.top_k + j];
      const float* src = p.y + ((long long)row * p.vec + col) * 8;
      const uint4 a = load_v4_stream(src), b = load_v4_stream(src + 4);
      acc[0] = fmaf(w, __uint_as_float(a.x), acc[0]);
      acc[1] = fmaf(w, __uint_as_float(a.y), acc[1]);
      acc[2] = fmaf(w, __uint_as_float(a.z), acc[2]);
      acc[3] = fmaf(w, __uint_as_float(a.w), acc[3]);
      acc[4] = fmaf(w, __uint_as_float(b.x), acc[4]);
      acc[5] = fmaf(w, __uint_as_float(b.y), acc[5]);
      acc[6] = fmaf(w, __uint_as_float(b.z), acc[6]);
      acc[7] = fmaf(w, __uint_as_float(b.w), acc[7]);
    }
    p.out[i] = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                          pack_bf16x2(acc[6], acc[7]));
  }
}

// dweights[t][j] = sum_n dout[t][n] y[rows[t][j]][n]: a warp for each pair.  Bound by memory: 4096
// pairs of 6144 23 us, 5.5 TB/s.
struct DotParams {
  const uint4* dout;
  const float* y;
  const int* rows;
  float* dweights;
  int vec, top_k;
  long long pairs;
};

__global__ void __launch_bounds__(kCombineThreads) weight_grad_kernel(const DotParams p) {
  const int lane = threadIdx.x & 31;
  griddep_launch_dependents();
  griddep_wait();
  const long long pair = ((long long)blockIdx.x * kCombineThreads + threadIdx.x) >> 5;
  if (pair >= p.pairs) return;
  const int row = p.rows[pair];
  float sum[2] = {0.f, 0.f};
  if ((unsigned long long)row < (unsigned long long)p.pairs) {
    const uint4* d = p.dout + pair / p.top_k * p.vec;
    const float* y = p.y + (long long)row * p.vec * 8;
#pragma unroll 4
    for (int i = lane; i < p.vec; i += 32) {
      const uint4 g = load_v4(d + i), a = load_v4_stream(y + i * 8), b = load_v4_stream(y + i * 8 + 4);
      sum[0] = fmaf(bf16lo_to_f32(g.x), __uint_as_float(a.x), sum[0]);
      sum[1] = fmaf(bf16hi_to_f32(g.x), __uint_as_float(a.y), sum[1]);
      sum[0] = fmaf(bf16lo_to_f32(g.y), __uint_as_float(a.z), sum[0]);
      sum[1] = fmaf(bf16hi_to_f32(g.y), __uint_as_float(a.w), sum[1]);
      sum[0] = fmaf(bf16lo_to_f32(g.z), __uint_as_float(b.x), sum[0]);
      sum[1] = fmaf(bf16hi_to_f32(g.z), __uint_as_float(b.y), sum[1]);
      sum[0] = fmaf(bf16lo_to_f32(g.w), __uint_as_float(b.z), sum[0]);
      sum[1] = fmaf(bf16hi_to_f32(g.w), __uint_as_float(b.w), sum[1]);
    }
  }
  const float total = lanes_sum<32>(sum[0] + sum[1]);
  if (lane == 0) p.dweights[pair] = total;
}

// dA of an empty contraction: zero for the rows that belong to an expert.
struct ClearParams {
  uint4* out;
  const int* offsets;
  int experts, pairs, vec;  // vectors of 8 in a row
  long long total;
};

__global__ void __launch_bounds__(kCombineThreads) clear_rows_kernel(const ClearParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int used = expert_row(p.offsets, p.experts, p.pairs);
  const long long stride = (long long)gridDim.x * kCombineThreads;
  for (long long i = (long long)blockIdx.x * kCombineThreads + threadIdx.x; i < p.total; i += stride)
    if ((int)(i / p.vec % p.pairs) < used) st_global_v4(p.out + i, make_uint4(0, 0, 0, 0));
}

int check_route(const gemm_rs_route_desc* d) {
  if (!d) return GEMM_RS_ERR_INVALID_ARG;
  if (d->T < 0 || d->E < 1 || d->E > kMaxExperts || d->top_k < 1 || d->top_k > kMaxTopK || d->top_k > d->E ||
      d->T > (1ll << 30) / kMaxExperts)
    return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  if (d->groups < 1 || d->groups > kMaxGroups || d->E % d->groups || d->top_groups < 1 || d->top_groups > d->groups ||
      d->E / d->groups * d->top_groups < d->top_k || d->score < 0 || d->score > 1)
    return GEMM_RS_ERR_INVALID_ARG;
  return GEMM_RS_OK;
}

int check_pairs(int64_t T, int64_t E, int64_t top_k) {
  if (T < 0 || E < 1 || E > kMaxExperts || top_k < 1 || top_k > kMaxTopK || T > (1ll << 30) / kMaxExperts)
    return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  return GEMM_RS_OK;
}

int check_desc(const gemm_rs_moe_desc* d) {
  if (!d) return GEMM_RS_ERR_INVALID_ARG;
  const int rc = check_pairs(d->T, d->E, d->top_k);
  if (rc) return rc;
  if (d->N < 0 || d->K < 0 || d->N % 8 || d->K % 64) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  return fp8_check_sizes(d->T * d->top_k, d->E, d->N, d->K);
}

ArrangeParams arrange_params(int64_t T, int64_t E, int64_t top_k, const void* ids, void* rows, void* pairs, void* offsets,
                             int ctas, int group) {
  ArrangeParams p;
  p.ids = static_cast<const int*>(ids);
  p.rows = static_cast<int*>(rows);
  p.pairs = static_cast<int*>(pairs);
  p.offsets = static_cast<int*>(offsets);
  p.n = (int)(T * top_k);
  p.E = (int)E;
  const int warps = ctas * kArrangeWarps;
  p.per = ((p.n + warps - 1) / warps + group - 1) / group * group;
  return p;
}

int arrange(int64_t T, int64_t E, int64_t top_k, const void* ids, void* rows, void* pairs, void* offsets, cudaStream_t st,
            int sms) {
  if (T * top_k <= 32 * kArrangeWarps) {  // a group of pairs for each warp of one CTA
    const ArrangeParams p = arrange_params(T, E, top_k, ids, rows, pairs, offsets, 1, 32);
    return launch_overlapped(arrange_once_kernel, dim3(1), kArrangeThreads, 0, st, p);
  }
  // with 96 experts 24576 pairs 4.2 us against 7.4 by a cluster for each, 98304 6.4 against 10.7; with 8, 16384
  // 2.9 against 3.3 and 260000 9.2 both
  if (T * top_k <= 32 * kArrangeWarps * kShareCtas * kShareGroups) {
    const ArrangeParams p = arrange_params(T, E, top_k, ids, rows, pairs, offsets, kShareCtas, 32);
    return launch_cluster(arrange_share_kernel, p.per / 32 * kShareCtas, kShareCtas, kArrangeThreads, 0, st, p);
  }
  int ctas = 8;  // as many as run at once
  while (ctas > 1 && E * ctas > 2 * sms) ctas /= 2;
  const ArrangeParams p = arrange_params(T, E, top_k, ids, rows, pairs, offsets, ctas, 128);
  const size_t smem = p.per / 32 <= kArrangeWords ? (size_t)kArrangeWarps * (p.per / 32) * 4 : 0;
  static SmemAllowed allowed;
  if (!allowed.set(arrange_kernel, kArrangeWarps * kArrangeWords * 4)) return GEMM_RS_ERR_CUDA;
  return launch_cluster(arrange_kernel, (int)E * ctas, ctas, kArrangeThreads, smem, st, p);
}

// One CTA routes and arranges in one launch where each of its warps has a token at most: 32 tokens
// of 96 experts 5.5 us against 6.2, one 3.9 against 6.0; 16 of 256 would take 6.7 against 5.7.
constexpr int kRouteOnce = kRouteOnceWarps, kRouteOnceExperts = 128;

template <int kPer>
int route_once(const RouteParams& p, const ArrangeParams& a, cudaStream_t st) {
  constexpr size_t scratch = sizeof(double) * 32 * kPer * kRouteOnceWarps;
  constexpr size_t bytes = scratch > sizeof(ArrangeShared) ? scratch : sizeof(ArrangeShared);
  static SmemAllowed allowed;
  if (!allowed.set(route_once_kernel<kPer>, (int)bytes)) return GEMM_RS_ERR_CUDA;
  return launch_overlapped(route_once_kernel<kPer>, dim3(1), 32 * kRouteOnceWarps, bytes, st, p, a);
}

template <typename T>
T* at(void* base, size_t bytes) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(base) + bytes);
}

struct Places {
  size_t row_codes, row_scales, token_codes, token_scales, y, total;
};
Places forward_places(const gemm_rs_moe_desc& d) {
  const int64_t P = d.T * d.top_k, Kr = d.K / kWorld;
  Places w = {};
  w.row_codes = kFp8Status;
  w.row_scales = w.row_codes + align256((size_t)kWorld * P * fp8_pitch(Kr));
  w.y = w.row_scales + align256(row_scale_bytes(P, kWorld * blocks_of(Kr)));
  w.total = w.y + align256((size_t)P * d.N * 4);
  return w;
}
Places backward_places(const gemm_rs_moe_desc& d) {
  const int64_t P = d.T * d.top_k, padded = padded_rows(P, d.E);
  Places w = {};
  w.row_codes = kFp8Status;
  w.row_scales = w.row_codes + align256((size_t)P * fp8_pitch(d.N));
  w.token_codes = w.row_scales + align256(row_scale_bytes(P, blocks_of(d.N)));
  w.token_scales = w.token_codes + align256((size_t)padded * fp8_pitch(d.N));
  w.total = w.token_scales + align256(token_scale_bytes(padded, 1, d.N));
  return w;
}

int clear(void* p, size_t bytes, cudaStream_t st) {
  if (bytes == 0) return GEMM_RS_OK;
  if (!p) return GEMM_RS_ERR_INVALID_ARG;
  if (cudaMemsetAsync(p, 0, bytes, st) == cudaSuccess) return GEMM_RS_OK;
  cudaGetLastError();
  return GEMM_RS_ERR_CUDA;
}

// Eight lanes a token: one for each group and choice (and the check of the next), 16 slots.
bool eight_lanes(int E, int top_k, int groups) { return E <= 128 && top_k < 8 && groups <= 8; }

unsigned route_grid(int64_t T, bool eight) {
  const int64_t per_block = kRouteWarps * (eight ? 4 : 1);
  return (unsigned)((T + per_block - 1) / per_block);
}

}  // namespace

extern "C" int gemm_rs_moe_route(const gemm_rs_route_desc* d, const void* logits, const void* bias, const void* mask,
                                 void* ids, void* weights, void* rows, void* pairs, void* offsets, void* stream) {
  int rc = check_route(d);
  if (rc) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!offsets) return GEMM_RS_ERR_INVALID_ARG;
  if (d->T > 0 && (!logits || !ids || !weights || !rows || !pairs)) return GEMM_RS_ERR_INVALID_ARG;
  for (const void* q : {logits, bias, (const void*)ids, (const void*)weights, (const void*)rows, (const void*)pairs,
                        (const void*)offsets})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  if (d->T == 0) return clear(offsets, (size_t)(d->E + 1) * 4, st);
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  RouteParams p;
  memset(&p, 0, sizeof(p));
  p.logits = logits;
  p.bias = static_cast<const float*>(bias);
  p.mask = static_cast<const uint8_t*>(mask);
  p.ids = static_cast<int*>(ids);
  p.weights = static_cast<float*>(weights);
  p.T = (int)d->T;
  p.E = (int)d->E;
  p.top_k = d->top_k;
  p.groups = d->top_groups < d->groups ? d->groups : 1;  // all groups stay: as one
  p.top_groups = d->top_groups;
  p.group_size = p.E / p.groups;
  p.by_group = divider_of((uint32_t)p.group_size);
  p.bf16 = d->logits_bf16 != 0;
  p.sigmoid = d->score == 1;
  p.renormalize = d->renormalize != 0;
  p.scale = d->scale;
  if (d->T <= kRouteOnce && d->E <= kRouteOnceExperts) {
    const ArrangeParams a = arrange_params(d->T, d->E, d->top_k, ids, rows, pairs, offsets, 1, 32);
    return p.E <= 32    ? route_once<1>(p, a, st)
           : p.E <= 64  ? route_once<2>(p, a, st)
                        : route_once<4>(p, a, st);
  }
  const bool eight = eight_lanes(p.E, p.top_k, p.groups);
  auto kernel = eight ? (p.E <= 8    ? route_kernel<8, 1>
                         : p.E <= 16 ? route_kernel<8, 2>
                         : p.E <= 32 ? route_kernel<8, 4>
                         : p.E <= 64 ? route_kernel<8, 8>
                         : p.E <= 96 ? route_kernel<8, 12>
                                     : route_kernel<8, 16>)
                      : (p.E <= 32    ? route_kernel<32, 1>
                         : p.E <= 64  ? route_kernel<32, 2>
                         : p.E <= 128 ? route_kernel<32, 4>
                                      : route_kernel<32, 8>);
  rc = launch_overlapped(kernel, dim3(route_grid(d->T, eight)), 32 * kRouteWarps, 0, st, p);
  return rc ? rc : arrange(d->T, d->E, d->top_k, ids, rows, pairs, offsets, st, sms);
}

extern "C" int gemm_rs_moe_arrange(int64_t T, int64_t E, int64_t top_k, const void* ids, void* rows, void* pairs,
                                   void* offsets, void* stream) {
  int rc = check_pairs(T, E, top_k);
  if (rc) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!offsets || (T > 0 && (!ids || !rows || !pairs))) return GEMM_RS_ERR_INVALID_ARG;
  for (const void* q : {ids, (const void*)rows, (const void*)pairs, (const void*)offsets})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  if (T == 0) return clear(offsets, (size_t)(E + 1) * 4, st);
  int sms = 0;
  rc = current_device_sms(&sms);
  return rc ? rc : arrange(T, E, top_k, ids, rows, pairs, offsets, st, sms);
}

extern "C" int gemm_rs_moe_route_backward(const gemm_rs_route_desc* d, const void* dweights, const void* logits,
                                          const void* ids, void* dlogits, void* stream) {
  int rc = check_route(d);
  if (rc || d->T == 0) return rc;
  if (!dweights || !logits || !ids || !dlogits) return GEMM_RS_ERR_INVALID_ARG;
  for (const void* q : {dweights, logits, ids, (const void*)dlogits})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  RouteBackwardParams p;
  p.dweights = static_cast<const float*>(dweights);
  p.logits = logits;
  p.ids = static_cast<const int*>(ids);
  p.dlogits = dlogits;
  p.T = (int)d->T;
  p.E = (int)d->E;
  p.top_k = d->top_k;
  p.bf16 = d->logits_bf16 != 0;
  p.sigmoid = d->score == 1;
  p.renormalize = d->renormalize != 0;
  p.scale = d->scale;
  const bool eight = eight_lanes(p.E, p.top_k, 1);
  auto kernel = eight ? (p.E <= 8    ? route_backward_kernel<8, 1>
                         : p.E <= 16 ? route_backward_kernel<8, 2>
                         : p.E <= 32 ? route_backward_kernel<8, 4>
                         : p.E <= 64 ? route_backward_kernel<8, 8>
                         : p.E <= 96 ? route_backward_kernel<8, 12>
                                     : route_backward_kernel<8, 16>)
                      : (p.E <= 32    ? route_backward_kernel<32, 1>
                         : p.E <= 64  ? route_backward_kernel<32, 2>
                         : p.E <= 128 ? route_backward_kernel<32, 4>
                                      : route_backward_kernel<32, 8>);
  return launch_overlapped(kernel, dim3(route_grid(d->T, eight)), 32 * kRouteWarps, 0, static_cast<cudaStream_t>(stream), p);
}

extern "C" int gemm_rs_moe_checkpoint_bytes(const gemm_rs_moe_desc* d, size_t* code_bytes, size_t* scale_bytes,
                                            size_t* y_bytes) {
  const int rc = check_desc(d);
  if (rc) return rc;
  const int64_t P = d->T * d->top_k, padded = padded_rows(P, d->E), Kr = d->K / kWorld;
  if (code_bytes) *code_bytes = (size_t)kWorld * padded * fp8_pitch(Kr);
  if (scale_bytes) *scale_bytes = token_scale_bytes(padded, kWorld, Kr);
  if (y_bytes) *y_bytes = (size_t)P * d->N * 4;
  return GEMM_RS_OK;
}

extern "C" int gemm_rs_moe_workspace(const gemm_rs_moe_desc* d, size_t* bytes) {
  const int rc = check_desc(d);
  if (rc) return rc;
  const size_t f = forward_places(*d).total, b = backward_places(*d).total;
  if (bytes) *bytes = f > b ? f : b;
  return GEMM_RS_OK;
}

namespace {

int forward(Fp8Scale scale, const gemm_rs_moe_desc* d, const void* A, const void* codes, const void* scales,
            const void* weights, const void* rows, const void* offsets, void* ck_codes, void* ck_scales, void* ck_y,
            void* out, void* workspace, void* stream) {
  int rc = check_desc(d);
  if (rc) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (const void* q : {A, codes, weights, rows, offsets, (const void*)ck_codes, (const void*)ck_scales,
                        (const void*)ck_y, (const void*)out, (const void*)workspace})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  if (scale == kFp8F32 && misaligned16(scales)) return GEMM_RS_ERR_MISALIGNED;
  if (!workspace) return GEMM_RS_ERR_WORKSPACE;
  const int64_t P = d->T * d->top_k;
  const bool some = P > 0 && d->K > 0;
  if (some && ((ck_codes == nullptr) != (ck_scales == nullptr) ||
               (d->N > 0 && (ck_codes == nullptr) != (ck_y == nullptr))))
    return GEMM_RS_ERR_INVALID_ARG;
  if (!some) {
    rc = clear(workspace, sizeof(uint32_t), st);
    if (!rc && ck_y) rc = clear(ck_y, (size_t)P * d->N * 4, st);
    return rc ? rc : clear(out, (size_t)d->T * d->N * 2, st);
  }
  if (!A || !weights || !rows || !offsets || (d->N > 0 && (!codes || !scales || !out))) return GEMM_RS_ERR_INVALID_ARG;
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  const Places w = forward_places(*d);
  float* y = ck_y ? static_cast<float*>(ck_y) : at<float>(workspace, w.y);
  Fp8Quantize q;
  q.scale = scale;
  q.x = A;
  q.planes = kWorld;
  q.cols = d->K / kWorld;
  q.rows.M = P;
  q.rows.experts = (int)d->E;
  q.rows.offsets = static_cast<const int*>(offsets);
  q.row_codes = at<void>(workspace, w.row_codes);
  q.row_scales = at<void>(workspace, w.row_scales);
  q.token_codes = ck_codes;
  q.token_scales = ck_scales;
  q.status = at<uint32_t>(workspace, 0);
  rc = fp8_quantize_rows(q, st);
  if (rc || d->N == 0) return rc;
  if (fp8_few_serves(kFp8Forward, q.rows, d->N, d->K / kWorld, false, sms)) {
    Fp8Few f;
    f.scale = scale;
    f.kind = kFp8Forward;
    f.N = d->N;
    f.Kr = d->K / kWorld;
    f.rows = q.rows;
    f.rows.top_k = (int)d->top_k;
    f.a = q.row_codes;
    f.a_scale = q.row_scales;
    f.b = codes;
    f.b_scale = scales;
    f.out = out;
    f.tokens = d->T;
    f.weights = static_cast<const float*>(weights);
    f.place = static_cast<const int*>(rows);
    f.y = static_cast<float*>(ck_y);
    f.status = q.status;
    return fp8_few(f, st);
  }
  Fp8Product m;
  m.scale = scale;
  m.kind = kFp8Forward;
  m.N = d->N;
  m.Kr = d->K / kWorld;
  m.rows = q.rows;
  m.a = q.row_codes;
  m.a_scale = q.row_scales;
  m.b = codes;
  m.b_scale = scales;
  m.out = y;
  m.out_f32 = true;
  m.status = q.status;
  rc = fp8_product(m, st);
  if (rc) return rc;
  CombineParams c;
  c.y = y;
  c.weights = static_cast<const float*>(weights);
  c.rows = static_cast<const int*>(rows);
  c.out = static_cast<uint4*>(out);
  c.vec = (int)(d->N / 8);
  c.top_k = (int)d->top_k;
  c.total = d->T * c.vec;
  c.pairs = P;
  const long long blocks = (c.total + kCombineThreads - 1) / kCombineThreads;
  return launch_overlapped(combine_kernel, dim3((unsigned)(blocks < 16ll * sms ? blocks : 16ll * sms)), kCombineThreads, 0,
                           st, c);
}

int backward(Fp8Scale scale, const gemm_rs_moe_desc* d, const void* dout, const void* codes, const void* scales,
             const void* weights, const void* rows, const void* pairs, const void* offsets, const void* ck_codes,
             const void* ck_scales, const void* ck_y, void* dA, void* dW, void* dweights, void* workspace, void* stream) {
  int rc = check_desc(d);
  if (rc) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (const void* q : {dout, codes, weights, rows, pairs, offsets, ck_codes, ck_scales, ck_y, (const void*)dA,
                        (const void*)dW, (const void*)dweights, (const void*)workspace})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  if (scale == kFp8F32 && misaligned16(scales)) return GEMM_RS_ERR_MISALIGNED;
  if (!workspace) return GEMM_RS_ERR_WORKSPACE;
  const int64_t P = d->T * d->top_k;
  if (P == 0 || d->N == 0 || d->K == 0) {
    const bool some_dA = dA && P > 0 && d->K > 0;
    if (some_dA && !offsets) return GEMM_RS_ERR_INVALID_ARG;
    rc = clear(workspace, sizeof(uint32_t), st);
    if (!rc && dW) rc = clear(dW, (size_t)d->E * d->K * d->N * 2, st);
    if (!rc && dweights) rc = clear(dweights, (size_t)P * 4, st);
    if (rc || !some_dA) return rc;
    int sms = 0;
    rc = current_device_sms(&sms);
    if (rc) return rc;
    ClearParams c;
    c.out = static_cast<uint4*>(dA);
    c.offsets = static_cast<const int*>(offsets);
    c.experts = (int)d->E;
    c.pairs = (int)P;
    c.vec = (int)(d->K / kWorld / 8);
    c.total = P * (d->K / 8);
    const long long blocks = (c.total + kCombineThreads - 1) / kCombineThreads;
    return launch_overlapped(clear_rows_kernel, dim3((unsigned)(blocks < 16ll * sms ? blocks : 16ll * sms)), kCombineThreads, 0,
                             st, c);
  }
  if (!dA && !dW && !dweights) return clear(workspace, sizeof(uint32_t), st);
  if (!dout || !weights || !rows || !pairs || !offsets || (dA && (!codes || !scales)) ||
      (dW && (!ck_codes || !ck_scales)) || (dweights && !ck_y))
    return GEMM_RS_ERR_INVALID_ARG;
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  const Places w = backward_places(*d);
  if (dA || dW) {
    Fp8Quantize q;
  q.scale = scale;
    q.x = dout;
    q.planes = 1;
    q.cols = d->N;
    q.rows.M = P;
    q.rows.experts = (int)d->E;
    q.rows.offsets = static_cast<const int*>(offsets);
    q.rows.pairs = static_cast<const int*>(pairs);
    q.rows.weights = static_cast<const float*>(weights);
    q.rows.top_k = (int)d->top_k;
    if (dA) {
      q.row_codes = at<void>(workspace, w.row_codes);
      q.row_scales = at<void>(workspace, w.row_scales);
    }
    if (dW) {
      q.token_codes = at<void>(workspace, w.token_codes);
      q.token_scales = at<void>(workspace, w.token_scales);
    }
    q.status = at<uint32_t>(workspace, 0);
    const bool few = dA && fp8_few_serves(kFp8InputGrad, q.rows, d->N, d->K / kWorld, dW != nullptr, sms);
    rc = fp8_quantize_rows(q, st);
    if (rc) return rc;
    Fp8Product m;
  m.scale = scale;
    m.N = d->N;
    m.Kr = d->K / kWorld;
    m.rows = q.rows;
    m.status = q.status;
    Fp8Product g = m;
    if (few) {
      Fp8Few f;
    f.scale = scale;
      f.kind = kFp8InputGrad;
      f.N = d->N;
      f.Kr = d->K / kWorld;
      f.rows = q.rows;
      f.a = q.row_codes;
      f.a_scale = q.row_scales;
      f.b = codes;
      f.b_scale = scales;
      f.out = dA;
      f.status = q.status;
      rc = fp8_few(f, st);
      if (rc) return rc;
    } else if (dA) {
      m.kind = kFp8InputGrad;
      m.a = q.row_codes;
      m.a_scale = q.row_scales;
      m.b = codes;
      m.b_scale = scales;
      m.out = dA;
    }
    if (dW) {
      g.kind = kFp8WeightGrad;
      g.a = ck_codes;
      g.a_scale = ck_scales;
      g.b = q.token_codes;
      g.b_scale = q.token_scales;
      g.out = dW;
    }
    if (dA && dW && !few)
      rc = fp8_products(m, g, st);
    else if (dA && !few)
      rc = fp8_product(m, st);
    else if (dW)
      rc = fp8_product(g, st);
    if (rc) return rc;
  } else {
    rc = clear(workspace, sizeof(uint32_t), st);
    if (rc) return rc;
  }
  if (!dweights) return GEMM_RS_OK;
  DotParams c;
  c.dout = static_cast<const uint4*>(dout);
  c.y = static_cast<const float*>(ck_y);
  c.rows = static_cast<const int*>(rows);
  c.dweights = static_cast<float*>(dweights);
  c.vec = (int)(d->N / 8);
  c.top_k = (int)d->top_k;
  c.pairs = P;
  const long long blocks = (P * 32 + kCombineThreads - 1) / kCombineThreads;
  return launch_overlapped(weight_grad_kernel, dim3((unsigned)blocks), kCombineThreads, 0, st, c);
}

}  // namespace

extern "C" int gemm_rs_moe_forward(const gemm_rs_moe_desc* d, const void* A, const void* codes, const void* scales,
                                   const void* weights, const void* rows, const void* offsets, void* ck_codes,
                                   void* ck_scales, void* ck_y, void* out, void* workspace, void* stream) {
  return forward(kFp8F32, d, A, codes, scales, weights, rows, offsets, ck_codes, ck_scales, ck_y, out, workspace, stream);
}
extern "C" int gemm_rs_moe_forward_e8m0(const gemm_rs_moe_desc* d, const void* A, const void* codes, const void* scales,
                                        const void* weights, const void* rows, const void* offsets, void* ck_codes,
                                        void* ck_scales, void* ck_y, void* out, void* workspace, void* stream) {
  return forward(kFp8E8m0, d, A, codes, scales, weights, rows, offsets, ck_codes, ck_scales, ck_y, out, workspace, stream);
}
extern "C" int gemm_rs_moe_backward(const gemm_rs_moe_desc* d, const void* dout, const void* codes, const void* scales,
                                    const void* weights, const void* rows, const void* pairs, const void* offsets,
                                    const void* ck_codes, const void* ck_scales, const void* ck_y, void* dA, void* dW,
                                    void* dweights, void* workspace, void* stream) {
  return backward(kFp8F32, d, dout, codes, scales, weights, rows, pairs, offsets, ck_codes, ck_scales, ck_y, dA, dW, dweights,
                  workspace, stream);
}
extern "C" int gemm_rs_moe_backward_e8m0(const gemm_rs_moe_desc* d, const void* dout, const void* codes,
                                         const void* scales, const void* weights, const void* rows, const void* pairs,
                                         const void* offsets, const void* ck_codes, const void* ck_scales,
                                         const void* ck_y, void* dA, void* dW, void* dweights, void* workspace,
                                         void* stream) {
  return backward(kFp8E8m0, d, dout, codes, scales, weights, rows, pairs, offsets, ck_codes, ck_scales, ck_y, dA, dW,
                  dweights, workspace, stream);
}
