// The router's selection with its per-expert statistics, the balance loss, and
// the gradient of both back to the logits.
//
//   score   s_e = softmax(x)_e, or sigmoid(x_e);
//   select  the k experts of largest x_e (with a bias: of largest
//           sigmoid(x_e) + bias_e), ties to the lower index; -inf never;
//   gate    scale * s_j, or renormalised scale * s_j / sum of the selected;
//   stats   counts[e] = pairs on e, prob_sum[e] = sum over tokens of p_te with
//           p the scores of a row summing to one;
//   loss    alpha * E * sum_e counts[e] / (N k) * prob_sum[e] / N.
//
// Three forms, by the rows and experts at hand (route_plan, route_bwd_plan):
//   wide    a wavefront per row, lane l its experts l, l + 64, ...: every load
//           and store is one run of lanes, a lane meets the same experts in
//           every row (their probability sums and loss gradients stay in
//           registers), and the k results sit in the first k lanes;
//   narrow  the same with 16 lanes per row, four rows to a wavefront, joined by
//           DPP operands alone;
//   single  a thread per row, its logits in registers, for many rows of few
//           experts.
// What bounds them (MI355X, kernels back to back, statistics and loss apart):
// 32768 x 384 top-8 takes 15.5 us for 52.4 MB (3.4 TB/s; at the rate of a copy,
// 5.1 TB/s, 10.2 us) and 14.6 in bfloat16 for half of the bytes: issue, 165
// vector and 138 scalar instructions a row in both. 262144 x 64 top-6 single
// takes 22.2 us for 79.7 MB (3.6 TB/s): vector issue too, 16 us of it, with 198
// scalar registers (a comparison's mask per expert) in lanes of vector ones.
// The backward streams: 32768 x 384 24.4 us for 102.8 MB (4.2 TB/s), 262144 x 64
// 33.6 us for 146.8 MB (4.4 TB/s); in bfloat16 19.5 and 25.5, issue bound. Below
// some thousand rows a launch costs 2.5 to 4 us whatever it does.
#include "codecs.hpp"
#include "internal.hpp"
#include "lanes.hpp"

namespace nvfp4moe {

namespace {

constexpr int kWaves = 8;                  // wavefronts of a backward workgroup
constexpr int kMaxWaves = 16;              // of a forward one (4, 8 or 16: route_waves)
constexpr int kNarrowK = 16;               // slots of the forms with less than a wavefront per row
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float load1(const void* p, bool bf16, int64_t i) {
  return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// The element at a byte offset from a row's start. The offset is kept opaque in
// 32 bits: the row's address stays in scalar registers and the load adds them,
// where a 64-bit sum per load would take a vector instruction.
template <class T>
__device__ __forceinline__ T read_at(const void* row, uint32_t byte) {
  asm volatile("" : "+v"(byte));
  return *reinterpret_cast<const T*>(static_cast<const char*>(row) + byte);
}
template <bool BF>
__device__ __forceinline__ float load_at(const void* row, uint32_t byte) {
  if constexpr (BF) return bf16_to_f32(read_at<uint16_t>(row, byte));
  else return read_at<float>(row, byte);
}
template <class T>
__device__ __forceinline__ void store_at(T* row, uint32_t i, T v) {
  uint32_t byte = i * (uint32_t)sizeof(T);
  asm volatile("" : "+v"(byte));
  *reinterpret_cast<T*>(reinterpret_cast<char*>(row) + byte) = v;
}

template <bool BF>
__device__ __forceinline__ const void* row_of(const void* p, int64_t i) {
  return static_cast<const char*>(p) + i * (BF ? 2 : 4);
}

// A value joined over the group of L lanes, in every lane: four DPP steps make
// rows of 16 uniform, the row swaps join them.
template <int L, class T, class Op>
__device__ __forceinline__ T group_join(T v, Op op) {
  v = op(v, across<0>(v));
  v = op(v, across<1>(v));
  v = op(v, across<2>(v));
  v = op(v, across<3>(v));
  if constexpr (L == 64) {
    if constexpr (sizeof(T) == 4) {
      v = join_rows(v, op);
    } else {
      v = op(v, __shfl_xor(v, 16, 64));
      v = op(v, __shfl_xor(v, 32, 64));
    }
  }
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  return group_join<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
  return group_join<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ double group_max(double v) {
  return group_join<L>(v, [](double a, double b) { return fmax(a, b); });
}
template <int L>
__device__ __forceinline__ int group_min(int v) {
  return group_join<L>(v, [](int a, int b) { return a < b ? a : b; });
}

// exp(x) for x <= 0 by the hardware's 2^x: the rounded product x * log2(e)
// costs a relative 2^-24 |x|, the instruction one unit in the last place.
__device__ __forceinline__ float exp_neg(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}

// sigmoid(x) and 1 - sigmoid(x), both from z = exp(-|x|) so that neither
// cancels: 1 / (1 + z) and z / (1 + z), the first for the sign of x.
__device__ __forceinline__ void sigmoid(float x, float& s, float& rest) {
  const float z = exp_neg(-fabsf(x));
  const float r = __builtin_amdgcn_rcpf(1.0f + z);
  s = x >= 0.0f ? r : z * r;
  rest = x >= 0.0f ? z * r : r;
}
__device__ __forceinline__ float sigmoid(float x) {
  float s, rest;
  sigmoid(x, s, rest);
  return s;
}

// 1 / d within half a unit of its last place (the instruction's is one off), 0
// for 0: what a row's probabilities are multiplied by.
__device__ __forceinline__ float inverse(float d) {
  const float r = __builtin_amdgcn_rcpf(d);
  return d > 0.0f ? __fmaf_rn(__fmaf_rn(-d, r, 1.0f), r, r) : 0.0f;
}

// n / d, r the instruction's 1 / d: the product mended by its exact remainder.
// The quotient of a number by itself is 1, so that one expert's share of
// itself, and with it the gradient of a row that has a single one, leaves no
// rounding behind: n * r leaves 2^-24 of the gradients that should cancel.
__device__ __forceinline__ float quotient(float n, float d, float r) {
  const float q = n * r;
  return __fmaf_rn(__fmaf_rn(-q, d, n), r, q);
}
// 1 / d for quotient(), 0 for 0.
__device__ __forceinline__ float estimate(float d) {
  return d > 0.0f ? __builtin_amdgcn_rcpf(d) : 0.0f;
}

// Backward sums over sigmoid scores are formed scaled by this, an exact step, so
// that the reciprocal of a sum near 2^-126 stays in range.
constexpr float kScaleUp = 0x1p64f;

// The key experts compete with where a bias is given. 64 bits: two scores that
// differ by less than a float32 step are told apart, and the choice does not
// hang on how a float32 exponential rounds.
__device__ __forceinline__ double biased_key(float x, float bias) {
  return 1.0 / (1.0 + exp(-(double)x)) + (double)bias;
}

// Keys of experts nearer than this in float32 are told apart in 64 bits: twice
// the error of a float32 key (sigmoid 7 * 2^-24 of a value below 1, the sum
// 2^-24 of the key) with room to spare.
__device__ __forceinline__ float key_margin(float key) {
  return 0x1p-19f + 0x1p-21f * fabsf(key);
}

// k rounds of taking the group's largest remaining key, the lowest expert
// first among equals. Lane j of the group ends with the j-th expert (or -1)
// in id and its logit in sx. CHECK (float32 keys of a biased selection): one
// round more, and whether two successive keys of any row were too near.
template <int L, int NV, bool CHECK, typename Key>
__device__ __forceinline__ bool select_rounds(Key (&key)[NV], const float (&x)[NV], int k, int l,
                                              int& id, float& sx) {
  const Key none = (Key)kNegInf;
  constexpr int far = 0x7FFFFFFF;
  id = -1;
  sx = kNegInf;
  bool near = false;
  Key before = none;
  for (int j = 0; j < (CHECK ? k + 1 : k); ++j) {
    Key best = none;
#pragma unroll
    for (int i = 0; i < NV; ++i) best = key[i] > best ? key[i] : best;
    best = group_max<L>(best);
    if (!__any(best > none)) break;        // no group of the wavefront has one left
    if constexpr (CHECK) {
      near = near || (j > 0 && best > none && before - best <= key_margin(before));
      before = best;
      if (j == k) break;
    }
    int at = far;
#pragma unroll
    for (int i = NV - 1; i >= 0; --i) at = key[i] == best ? i * L + l : at;
    at = best > none ? group_min<L>(at) : far;
    float v = kNegInf;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (at == i * L + l) {
        key[i] = none;
        v = x[i];
      }
    v = group_max<L>(v);
    if (l == j && at != far) {
      id = at;
      sx = v;
    }
  }
  return CHECK && __any(near);
}

// float32 -> uint32 of the same order (-0 below +0), and back.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = f2u(x);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return u2f(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// A value that at least k of the wavefront's 64 values reach and few more do
// (or the lowest one above -inf): the largest of each group of 64 / 2^n lanes
// with 2^n >= k groups, of those the least; then a few bisections between it
// and the maximum, each one comparison and a count of the ballot.
__device__ __forceinline__ float k_reached(float v, int k) {
  const uint32_t u = ordered(v + 0.0f);          // + 0: -0 is +0, as comparisons have it
  const int level = k <= 8 ? 3 : k <= 16 ? 2 : k <= 32 ? 1 : 0;
  uint32_t hi = u, lo = u;
#define NVFP4MOE_STEP(S)                          \
  do {                                            \
    hi = max(hi, across<S>(hi));                  \
    if (S < level) lo = hi;                       \
    else lo = min(lo, across<S>(lo));             \
  } while (0)
  NVFP4MOE_STEP(0);
  NVFP4MOE_STEP(1);
  NVFP4MOE_STEP(2);
  NVFP4MOE_STEP(3);
#undef NVFP4MOE_STEP
  const auto at = [](uint32_t x, int lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
  };
  uint32_t top = max(max(at(hi, 0), at(hi, 16)), max(at(hi, 32), at(hi, 48)));
  uint32_t low = min(min(at(lo, 0), at(lo, 16)), min(at(lo, 32), at(lo, 48)));
  low = max(low, ordered(kNegInf) + 1u);
  // enough is a few more than k: a candidate costs less than another step (and
  // a step with low and top met changes neither)
  for (int step = 0; step < 8; ++step) {
    const uint32_t mid = low + ((top - low + 1u) >> 1);
    const int more = (int)__popcll(__ballot(u >= mid)) - k;
    low = more >= 0 ? mid : low;
    top = more >= 0 ? top : mid - 1u;
    if ((uint32_t)more <= 2u) break;
  }
  return unordered(low);
}

// LDS of a wavefront's selection: its candidates in expert order, then its slots.
template <bool BIAS>
struct Candidates {
  alignas(16) float key[128];                  // the upper halves: what is no candidate
  int e[128];
  float x[BIAS ? 128 : 1];                     // without a bias the key is the logit
};

// The float32 keys of a lane's experts.
template <bool BIAS, int NV>
__device__ __forceinline__ void keys32(const float (&x)[NV], const float* bias, float (&key)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    key[i] = x[i];
    if constexpr (BIAS) {
      key[i] = x[i] > kNegInf ? sigmoid(x[i]) + bias[i] : kNegInf;
    }
  }
}

// The 64-bit keys, one after the other: a rare path, few registers.
template <int NV>
__device__ __forceinline__ void keys64(const float (&x)[NV], const float* bias, double (&key)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    key[i] = x[i] > kNegInf ? biased_key(x[i], bias[i]) : (double)kNegInf;
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The k largest keys of a row held by the wavefront: lanes keep what reaches a
// value that at least k lanes reach (a dozen candidates of 384 experts,
// compacted in expert order through LDS, one per lane) and each candidate
// counts those ahead of it; its count is its slot. Lane j ends with slot j's
// expert and logit. With a bias the cut and the order are by float32 keys, the
// cut less a margin; where two of the first k + 1 are nearer than that margin
// (a row in some hundreds) the candidates are ordered by 64-bit keys instead.
// More than 64 candidates (rows of equal logits, k near 64) go through
// select_rounds.
template <bool BIAS, int NV>
__device__ __forceinline__ void select(const float (&x)[NV], const float* bias_g,
                                       const float* bias, int k, int lane, Candidates<BIAS>& list,
                                       int& id, float& sx) {
  float key[NV], best = kNegInf;
  keys32<BIAS, NV>(x, bias, key);
#pragma unroll
  for (int i = 0; i < NV; ++i) best = fmaxf(best, key[i]);
  float cut = k_reached(best, k);
  if constexpr (BIAS) cut = fmaxf(cut - key_margin(cut), -3.402823466e38f);
  int n = 0;
  uint64_t hit[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    hit[i] = __ballot(key[i] >= cut);         // the cut is above -inf
    n += __popcll(hit[i]);
  }
  id = -1;
  sx = kNegInf;
  if (n > 64) {
    if constexpr (BIAS) {
      double key64[NV];
      keys64<NV>(x, bias, key64);
      select_rounds<64, NV, false>(key64, x, k, lane, id, sx);
    } else {
      select_rounds<64, NV, false>(key, x, k, lane, id, sx);
    }
    return;
  }
  int base = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = base + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(hit[i] >> 32),
                                                         __builtin_amdgcn_mbcnt_lo((uint32_t)hit[i], 0));
    const int to = key[i] >= cut ? at : 64 + lane;
    list.key[to] = key[i];
    list.e[to] = i * 64 + lane;
    if constexpr (BIAS) list.x[to] = x[i];
    base += __popcll(hit[i]);
  }
  // Each candidate counts the keys ahead of it, equal ones of lower experts
  // among them. Up to 16 candidates: lane 16 q + c compares candidate c with
  // candidates 4 q .. 4 q + 3 (one 16-byte read), the row swaps add the quarters.
  int rank = 0;
  const int c = n <= 16 ? lane & 15 : lane;
  if (n <= 16) {
    if (lane >= n && lane < 16) list.key[lane] = kNegInf;
    wave_lds_fence();
    const int q = lane >> 4;
    const float mine = list.key[c];
    const float4 other = *reinterpret_cast<const float4*>(&list.key[4 * q]);
    const float o[4] = {other.x, other.y, other.z, other.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      rank += (int)(o[i] > mine) | ((int)(o[i] == mine) & (int)(4 * q + i < c));
    rank = join_rows(rank, [](int u, int v) { return u + v; });
  } else {
    wave_lds_fence();
    // one unsigned comparison: the key, then the earlier place in the list
    const uint32_t u = ordered((lane < n ? list.key[lane] : kNegInf) + 0.0f);
    const uint64_t mine = ((uint64_t)u << 32) | (uint32_t)(63 - lane);
    for (int j = 0; j < n; ++j) {
      const uint64_t other =
          ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)u, j) << 32) | (uint32_t)(63 - j);
      rank += other > mine;
    }
  }
  const bool holds = lane < n;                 // (c is the lane there)
  const float mykey = list.key[c];
  const int myexpert = list.e[c];
  float myx = mykey;
  if constexpr (BIAS) myx = list.x[c];
  wave_lds_fence();
  if constexpr (BIAS) {
    if (holds) list.key[rank] = mykey;
    wave_lds_fence();
    const bool near = lane < k && lane + 1 < n &&
                      list.key[lane] - list.key[lane + 1] <= key_margin(list.key[lane]);
    wave_lds_fence();
    if (__any(near)) {
      const double key64 = holds ? biased_key(myx, bias_g[myexpert]) : (double)kNegInf;
      const uint64_t bits = __double_as_longlong(key64);
      rank = 0;
      for (int j = 0; j < n; ++j) {
        const double other = __longlong_as_double(
            (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(bits >> 32), j) << 32) |
                      (uint32_t)__builtin_amdgcn_readlane((int)bits, j)));
        rank += other > key64 || (other == key64 && j < lane);
      }
    }
  }
  if (holds && rank < k) {
    list.e[rank] = myexpert;
    list.key[rank] = myx;
  }
  wave_lds_fence();
  const bool slot = lane < k && lane < n;
  const int e = list.e[lane];
  const float v = list.key[lane];
  id = slot ? e : -1;
  sx = slot ? v : kNegInf;
  wave_lds_fence();
}

// Rows whose probabilities a lane adds up in 32 bits before they go to a sum in
// 64 (in LDS), so that the error of the statistics does not grow with the rows:
// in 32 bits throughout, 4.2 million equal rows of 20 experts were off by 26
// units of 2^-24. Joins and comparison together cost 1% (32768 x 384 with
// statistics and loss 25.0 -> 25.3 us, a million rows of 64 114.0 -> 115.2).
constexpr int kHeldRows = 16;

// One workgroup's share of an expert's statistics: a sum in 64 bits, rounded once.
struct alignas(8) RoutePart {
  float prob;
  int32_t count;
};

struct RouteArgs {
  const void* logits;
  int64_t T;
  int E, k;
  const float* bias;
  const uint8_t* token_mask;
  bool renorm;
  float scale;
  int32_t* topk_ids;
  float* gate;
  RoutePart* parts;      // [grid, E + 1], the last one's count the tokens
  int64_t* counts;       // of a workgroup that is the only one: the sums themselves
  float* prob_sum;
  bool deep;             // a lane may take kHeldRows rows or more
};

// A workgroup's statistics of expert e (e = E: its tokens) on their way out.
__device__ __forceinline__ void leave_stats(const RouteArgs& a, int e, double prob, int32_t count) {
  if (a.parts) {
    a.parts[(int64_t)blockIdx.x * (a.E + 1) + e] = RoutePart{(float)prob, count};
  } else {
    if (e < a.E) a.prob_sum[e] = (float)prob;
    a.counts[e] = count;
  }
}

// Eight wavefronts a SIMD where the registers allow it (32768 x 384 top-8 15.5
// us against 16.8 without the attribute, 14.7 and 16.9 in bfloat16, 25.5 and 28.4
// with statistics and loss; the biased form, with its 64-bit path, 28.9 with eight
// and 21.1 with four). Workgroups of 16 wavefronts hold every form to 128
// registers: biased with 16 experts a lane 39 of them (73 with statistics) live
// in scratch (32768 x 1000 94 us). Of the scalar registers 16 (32) are kept in
// lanes of vector ones at 6 experts a lane.
template <bool BF, bool SIG, bool BIAS, bool STATS, int L, int NV>
__global__ __launch_bounds__(64 * kMaxWaves)
__attribute__((amdgpu_waves_per_eu(!BIAS && NV <= 6 ? 8 : NV <= 8 ? 4 : 2))) void k_route(RouteArgs a) {
  constexpr int R = 64 / L;                // rows of a wavefront
  // the lanes' probability sums, each lane its own NV: in 64 bits where a lane
  // takes kHeldRows rows or more, else the 32-bit ones on their way to the join
  extern __shared__ double sh_prob[];
  __shared__ int32_t sh_count[STATS ? NV * L + 1 : 1];
  __shared__ Candidates<BIAS> list[L == 64 ? kMaxWaves : 1];
  static_assert((STATS ? kMaxWaves * 64 * NV * sizeof(double) + 4 * (NV * L + 1) : 0) + sizeof(list) <=
                    160 * 1024,
                "LDS of a compute unit");
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & (L - 1), g = L == 64 ? 0 : lane / L;
  const int E = a.E, k = a.k, waves = blockDim.x >> 6;
  const bool renorm = a.renorm;
  const uint32_t T = (uint32_t)a.T;         // rows: below 2^31, like T k
  float bias[BIAS ? NV : 1];
  if constexpr (BIAS) {
#pragma unroll
    for (int i = 0; i < NV; ++i) bias[i] = i * L + l < E ? a.bias[i * L + l] : 0.0f;
  }
  float psum[STATS ? NV : 1];
  int held = 0;                            // rows in psum
  const int own = (w * R + g) * NV * L + l;
  if constexpr (STATS) {
#pragma unroll
    for (int i = 0; i < NV; ++i) psum[i] = 0.0f;
    if (a.deep) {
#pragma unroll
      for (int i = 0; i < NV; ++i) sh_prob[own + i * L] = 0.0;
    }
    for (int e = threadIdx.x; e <= E; e += 64 * waves) sh_count[e] = 0;
    __syncthreads();
  }
  // A row's logits, loaded one row ahead of their use. Every lane loads (past
  // the experts or the rows: the last one again), so that no branch waits.
  uint32_t off[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) off[i] = (uint32_t)(i * L + l < E ? i * L + l : E - 1) * (BF ? 2 : 4);
  // without a mask any byte is loaded (of the logits) and not looked at
  const bool masked = a.token_mask != nullptr;
  const uint8_t* mask_bytes = masked ? a.token_mask : static_cast<const uint8_t*>(a.logits);
  const auto load = [&](uint32_t t, float (&v)[NV], uint32_t& mask) {
    const uint32_t row = t < T ? t : T - 1;
    mask = mask_bytes[row];
    const void* p = row_of<BF>(a.logits, (uint64_t)row * (uint32_t)E);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = load_at<BF>(p, off[i]);
  };
  const uint32_t stride = gridDim.x * waves * R;
  uint32_t t0 = (blockIdx.x * waves + w) * R;
  float next[NV];
  uint32_t next_mask;
  load(t0 + g, next, next_mask);
  for (; t0 < T; t0 += stride) {
    const uint32_t t = t0 + g;
    bool on = t < T && (!masked || next_mask != 0);
    float x[NV];
    if constexpr (L == 64) {
      on = !masked || __builtin_amdgcn_readfirstlane(next_mask) != 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) x[i] = next[i];
      if (E != NV * L) {
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = i * L + l < E ? x[i] : kNegInf;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) x[i] = on && i * L + l < E ? next[i] : kNegInf;
    }
    load(t + stride, next, next_mask);
    if (L == 64 && !on) {                    // padding: the wavefront has nothing to select
      if (l < k) {
        store_at(a.topk_ids + (uint64_t)t * (uint32_t)k, l, -1);
        store_at(a.gate + (uint64_t)t * (uint32_t)k, l, 0.0f);
      }
      continue;
    }
    int id;
    float sx;
    if constexpr (L == 64) {
      select<BIAS, NV>(x, a.bias, bias, k, lane, list[w], id, sx);
    } else {
      float key[NV];
      keys32<BIAS, NV>(x, bias, key);
      if (select_rounds<L, NV, BIAS>(key, x, k, l, id, sx)) {
        if constexpr (BIAS) {
          double key64[NV];
          keys64<NV>(x, bias, key64);
          select_rounds<L, NV, false>(key64, x, k, l, id, sx);
        }
      }
    }
    // the row has an expert: its first slot is taken
    const bool live = L == 64 ? __builtin_amdgcn_readfirstlane(id) >= 0 : group_max<L>((float)id) >= 0.0f;
    // without a bias the first slot's logit is the row's largest
    float first = 0.0f;
    if constexpr (!SIG) {
      first = L == 64 ? u2f(__builtin_amdgcn_readfirstlane(f2u(sx))) : group_max<L>(sx);
      first = live ? first : 0.0f;
    }
    // scores; the row's probabilities where they are needed
    float top = 0.0f, total = 0.0f, p[NV];
    if (STATS || (!SIG && !renorm)) {
      if constexpr (!SIG) top = first;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if constexpr (SIG) p[i] = sigmoid(x[i]);
        else p[i] = exp_neg(x[i] - top);
        total += p[i];
      }
      total = group_sum<L>(total);
    }
    if constexpr (STATS) {
      const float r = live ? inverse(total) : 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) psum[i] = __fmaf_rn(p[i], r, psum[i]);
      if (++held == kHeldRows) {
        held = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          sh_prob[own + i * L] += (double)psum[i];
          psum[i] = 0.0f;
        }
      }
      if (l < k && id >= 0) atomicAdd(&sh_count[id], 1);
      if (l == 0 && live) atomicAdd(&sh_count[E], 1);
    }
    // gates of the selected, one per lane
    float gate = 0.0f;
    if constexpr (SIG) {
      gate = sigmoid(sx);                  // 0 in empty slots, whose logit is -inf
    } else if (renorm) {
      gate = exp_neg(sx - first);
    } else {
      gate = quotient(exp_neg(sx - top), total, estimate(total));
    }
    if (renorm) {
      // up to 16 slots lie in the first 16 lanes, whose sum is all that they need
      const float sum = L == 64 && k <= 16 ? group_sum<16>(gate) : group_sum<L>(gate);
      gate = quotient(gate, sum, estimate(sum));
    }
    if (l < k && t < T) {
      store_at(a.topk_ids + (uint64_t)t * (uint32_t)k, l, id);
      store_at(a.gate + (uint64_t)t * (uint32_t)k, l, gate * a.scale);
    }
  }
  if constexpr (STATS) {
    const auto join = [&](auto* sums) {
      __syncthreads();
      for (int e = threadIdx.x; e <= E; e += 64 * waves) {
        double s = 0.0;
        if (e < E) {
          for (int v = 0; v < waves * R; ++v) s += (double)sums[v * NV * L + e];
        }
        leave_stats(a, e, s, sh_count[e]);
      }
    };
    if (a.deep) {
#pragma unroll
      for (int i = 0; i < NV; ++i) sh_prob[own + i * L] += (double)psum[i];
      join(sh_prob);
    } else {
      float* few = reinterpret_cast<float*>(sh_prob);
#pragma unroll
      for (int i = 0; i < NV; ++i) few[own + i * L] = psum[i];
      join(few);
    }
  }
}

// ---- one thread per row (few experts): the row in its registers, no traffic
// between lanes but for the statistics.

constexpr int kRowThreads = 256;
// The largest workgroup: 16 wavefronts where one may have to take every row.
constexpr int row_threads(int NE) { return NE <= 8 ? 1024 : kRowThreads; }

// The row's E <= NE logits, -inf behind them. vec: rows are whole 16-byte pieces.
template <bool BF, int NE>
__device__ __forceinline__ void load_own_row(const void* logits, int64_t t, int E, bool vec,
                                             float (&v)[NE]) {
  const void* row = row_of<BF>(logits, t * E);
  if (vec) {
    const uint4* q = static_cast<const uint4*>(row);
    constexpr int per = BF ? 8 : 4;
#pragma unroll
    for (int i = 0; i < NE / per; ++i) {
      const uint4 u = q[i];
      if constexpr (BF) {
        v[8 * i + 0] = u2f(u.x << 16); v[8 * i + 1] = u2f(u.x & 0xFFFF0000u);
        v[8 * i + 2] = u2f(u.y << 16); v[8 * i + 3] = u2f(u.y & 0xFFFF0000u);
        v[8 * i + 4] = u2f(u.z << 16); v[8 * i + 5] = u2f(u.z & 0xFFFF0000u);
        v[8 * i + 6] = u2f(u.w << 16); v[8 * i + 7] = u2f(u.w & 0xFFFF0000u);
      } else {
        v[4 * i + 0] = u2f(u.x); v[4 * i + 1] = u2f(u.y);
        v[4 * i + 2] = u2f(u.z); v[4 * i + 3] = u2f(u.w);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < NE; ++e) v[e] = load1(row, BF, e < E ? e : E - 1);
#pragma unroll
    for (int e = 0; e < NE; ++e) v[e] = e < E ? v[e] : kNegInf;
  }
}

typedef float f32x4_t __attribute__((ext_vector_type(4)));

// One row per thread. The statistics' sums over rows are matrix products: the
// wavefront's values for expert e are the 16 x 4 operand, the other one is 1 in
// column e (mod 16), so that expert's sums land in that column of the
// accumulator (four registers for 16 experts), four rows to an element at a
// time; every kHeldRows of them it is added to sums in 64 bits. The matrix
// instruction reads every lane: lanes past the rows hold zeros.
template <bool BF, bool SIG, bool BIAS, bool STATS, int NE>
__global__ __launch_bounds__(row_threads(NE)) void k_route_rows(RouteArgs a, bool vec) {
  constexpr int most = row_threads(NE), NA = (NE + 15) / 16, slots = NE < kNarrowK ? NE : kNarrowK;
  __shared__ float chosen[slots][most];             // the selected logits of each row
  __shared__ double sh_prob[STATS ? most / 64 * NA * 16 : 1];    // each wavefront its own
  __shared__ int32_t sh_count[STATS ? NE + 1 : 1];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int E = a.E, k = a.k, threads = blockDim.x;
  const bool renorm = a.renorm;
  f32x4_t acc[STATS ? NA : 1];
  float column[STATS ? 16 : 1];
  int held = 0;                                     // rows in an element of acc
  // a lane's accumulator: four rows of column (lane mod 16)
  const auto put_by = [&]() {
    held = 0;
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      float s = (acc[i][0] + acc[i][1]) + (acc[i][2] + acc[i][3]);
      s += __shfl_xor(s, 16, 64);
      s += __shfl_xor(s, 32, 64);
      if (lane < 16) sh_prob[(w * NA + i) * 16 + lane] += (double)s;
      acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
  };
  if constexpr (STATS) {
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if (lane < 16) sh_prob[(w * NA + i) * 16 + lane] = 0.0;
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) column[c] = (lane & 15) == c ? 1.0f : 0.0f;
    for (int e = tid; e <= NE; e += threads) sh_count[e] = 0;
    __syncthreads();
  }
  for (int64_t t0 = (int64_t)blockIdx.x * threads; t0 < a.T;
       t0 += (int64_t)gridDim.x * threads) {
    const int64_t t = t0 + tid;
    const int64_t row = t < a.T ? t : a.T - 1;
    const bool in = t < a.T;
    float x[NE];
    load_own_row<BF, NE>(a.logits, row, E, vec, x);
    if (!in || (a.token_mask && a.token_mask[row] == 0)) {
#pragma unroll
      for (int e = 0; e < NE; ++e) x[e] = kNegInf;
    }
    float top = kNegInf;
#pragma unroll
    for (int e = 0; e < NE; ++e) top = fmaxf(top, x[e]);
    const bool open = top > kNegInf;
    top = open ? top : 0.0f;
    const auto score = [&](float v) {
      if constexpr (SIG) return sigmoid(v);   // 0 for -inf
      else return exp_neg(v - top);
    };
    float total = 0.0f;
    if (STATS || (!SIG && !renorm)) {
#pragma unroll
      for (int e = 0; e < NE; ++e) total += score(x[e]);
    }
    if constexpr (STATS) {
      // the row counts where it selects: where an open expert's bias is above -inf
      bool counts = open;
      if constexpr (BIAS) {
        counts = false;
#pragma unroll
        for (int e = 0; e < NE; ++e)
          counts = counts || (x[e] > kNegInf && a.bias[e < E ? e : E - 1] > kNegInf);
      }
      const float r = counts ? inverse(total) : 0.0f;
#pragma unroll
      for (int e = 0; e < NE; ++e)
        acc[e / 16] = __builtin_amdgcn_mfma_f32_16x16x4f32(score(x[e]) * r, column[e % 16],
                                                           acc[e / 16], 0, 0, 0);
      if (counts) atomicAdd(&sh_count[NE], 1);
      held += 4;
      if (held == kHeldRows) put_by();
    }
    // k rounds of the largest remaining key, the lowest expert among equals
    float sum = 0.0f;
    double key[BIAS ? NE : 1];
    if constexpr (BIAS) {
#pragma unroll
      for (int e = 0; e < NE; ++e)
        key[e] = x[e] > kNegInf ? biased_key(x[e], a.bias[e < E ? e : E - 1]) : (double)kNegInf;
    }
    for (int j = 0; j < k; ++j) {
      int at = -1;
      float v = kNegInf;
      if constexpr (BIAS) {
        double best = (double)kNegInf;
#pragma unroll
        for (int e = 0; e < NE; ++e) best = key[e] > best ? key[e] : best;
        if (best > (double)kNegInf) {
#pragma unroll
          for (int e = NE - 1; e >= 0; --e) at = key[e] == best ? e : at;
        }
#pragma unroll
        for (int e = 0; e < NE; ++e)
          if (e == at) {
            key[e] = (double)kNegInf;
            v = x[e];
          }
      } else {
#pragma unroll
        for (int e = 0; e < NE; ++e) v = fmaxf(v, x[e]);
        if (v > kNegInf) {
#pragma unroll
          for (int e = NE - 1; e >= 0; --e) at = x[e] == v ? e : at;
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) x[e] = e == at ? kNegInf : x[e];
      }
      chosen[j][tid] = v;
      if (in) a.topk_ids[t * k + j] = at;
      sum += score(v);                     // 0 in empty slots, whose logit is -inf
      if constexpr (STATS) {
        if (at >= 0) atomicAdd(&sh_count[at], 1);
      }
    }
    const float den = renorm ? sum : SIG ? 1.0f : total;
    const float r = estimate(den);
    for (int j = 0; j < k; ++j) {
      float g = score(chosen[j][tid]);
      if (!SIG || renorm) g = quotient(g, den, r);
      if (in) a.gate[t * k + j] = g * a.scale;
    }
  }
  if constexpr (STATS) {
    put_by();
    __syncthreads();
    for (int e = tid; e <= E; e += threads) {
      double s = 0.0;
      if (e < E) {
        for (int v = 0; v < threads / 64; ++v) s += sh_prob[v * NA * 16 + e];
      }
      leave_stats(a, e, s, sh_count[e < E ? e : NE]);
    }
  }
}

// Column sums of the workgroups' partials, in a fixed order: 16 columns per
// workgroup, 64 threads down each, eight loads of a thread in flight.
__global__ __launch_bounds__(1024) void k_route_stats(const RoutePart* __restrict__ parts, int n,
                                                      int E, int64_t* __restrict__ counts,
                                                      float* __restrict__ prob_sum) {
  __shared__ double sp[1024];
  __shared__ int64_t sc[1024];
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int e = blockIdx.x * 16 + col;
  const int at = e <= E ? e : E;
  double p = 0.0;
  int64_t c = 0;
  for (int g0 = row; g0 < n; g0 += 64 * 8) {
    RoutePart v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {            // past the end: the last row again, not added
      const int g = g0 + 64 * j < n ? g0 + 64 * j : n - 1;
      v[j] = parts[(int64_t)g * (E + 1) + at];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (g0 + 64 * j < n) {
        p += (double)v[j].prob;
        c += v[j].count;
      }
  }
  sp[threadIdx.x] = p;
  sc[threadIdx.x] = c;
  __syncthreads();
  for (int d = 32; d >= 1; d >>= 1) {
    if (row < d) {
      sp[threadIdx.x] += sp[threadIdx.x + 16 * d];
      sc[threadIdx.x] += sc[threadIdx.x + 16 * d];
    }
    __syncthreads();
  }
  if (row == 0 && e <= E) {
    if (e < E) prob_sum[e] = (float)sp[col];
    counts[e] = sc[col];
  }
}

__global__ __launch_bounds__(256) void k_balance_loss(const int64_t* __restrict__ counts,
                                                      const float* __restrict__ prob_sum, int E,
                                                      int k, float alpha,
                                                      float* __restrict__ loss) {
  __shared__ double sh[256];
  double s = 0.0;
  for (int e = threadIdx.x; e < E; e += 256) s += (double)counts[e] * (double)prob_sum[e];
  sh[threadIdx.x] = s;
  __syncthreads();
  for (int d = 128; d >= 1; d >>= 1) {
    if ((int)threadIdx.x < d) sh[threadIdx.x] += sh[threadIdx.x + d];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const double n = (double)counts[E];
    *loss = n > 0.0 ? (float)((double)alpha * E * sh[0] / (n * n * k)) : 0.0f;
  }
}

struct RouteBwdArgs {
  const void* logits;
  int64_t T;
  int E, k;
  const int32_t* topk_ids;
  const float* dgate;          // or nullptr
  float scale;
  const int64_t* counts;       // or nullptr: no balance loss
  float alpha;
  const float* dloss;          // or nullptr: 1
  void* dlogits;
};

// The selected experts' part of a row's gradient is computed one slot per lane
// and reaches the lanes that own the experts through LDS. With s the scores, u
// the gradient of the selected ones, a the loss's of p:
//   softmax            dx = p (u + a - sum p (u + a));
//   renormalised       q = s over its sum: the slots add q (u - sum q u), the
//                      loss p (a - sum p a);
//   sigmoid            dx = (1 - s) (s u + p (a - sum p a)), p = s over the row's
//                      sum; renormalised q (u - sum q u) in the place of s u, q
//                      = s over the selected's (quotients of at most 1: no 1 / s
//                      leaves the range).
template <bool BF, bool SIG, bool RENORM, bool BAL, int L, int NV>
__global__ __launch_bounds__(64 * kWaves) void k_route_bwd(RouteBwdArgs a) {
  constexpr int R = 64 / L;
  __shared__ float sh_all[kWaves * R][NV * L];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & (L - 1), g = L == 64 ? 0 : lane / L;
  float* sh = sh_all[w * R + g];
  const int E = a.E, k = a.k;
  const uint32_t T = (uint32_t)a.T;         // rows: below 2^31, like T k
  float coef[BAL ? NV : 1];
  if constexpr (BAL) {
    const double n = (double)a.counts[E];
    const double c = n > 0.0 ? (double)a.alpha * E / (n * n * k) * (a.dloss ? (double)*a.dloss : 1.0)
                             : 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      coef[i] = i * L + l < E ? (float)(c * (double)a.counts[i * L + l]) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) sh[i * L + l] = 0.0f;
  // a row's operands, loaded one row ahead of their use (as in k_route)
  uint32_t off[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) off[i] = (uint32_t)(i * L + l < E ? i * L + l : E - 1) * (BF ? 2 : 4);
  const int slot = l < k ? l : k - 1;
  // without dgate the ids are read in its place and not looked at
  const void* dgate = a.dgate ? static_cast<const void*>(a.dgate) : a.topk_ids;
  const auto load = [&](uint32_t t, float (&v)[NV], int& id, float& dg) {
    const uint32_t row = t < T ? t : T - 1;
    const uint64_t first = (uint64_t)row * (uint32_t)k * 4;
    id = read_at<int32_t>(reinterpret_cast<const char*>(a.topk_ids) + first, slot * 4);
    dg = read_at<float>(static_cast<const char*>(dgate) + first, slot * 4);
    const void* p = row_of<BF>(a.logits, (uint64_t)row * (uint32_t)E);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = load_at<BF>(p, off[i]);
  };
  const uint32_t stride = gridDim.x * kWaves * R;
  uint32_t t0 = (blockIdx.x * kWaves + w) * R;
  float next[NV], next_dg;
  int next_id;
  load(t0 + g, next, next_id, next_dg);
  for (; t0 < T; t0 += stride) {
    const uint32_t t = t0 + g;
    const int id = l < k && t < T && next_id >= 0 && next_id < E ? next_id : -1;
    const float dg = id >= 0 && a.dgate ? next_dg * a.scale : 0.0f;
    float x[NV], d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = i * L + l < E ? next[i] : kNegInf;
    load(t + stride, next, next_id, next_dg);
    const bool live = group_max<L>((float)id) >= 0.0f;
    // the selected logits: out of the lanes that hold the row
    float sx = kNegInf;
    if constexpr (RENORM) {
      wave_lds_fence();
#pragma unroll
      for (int i = 0; i < NV; ++i) sh[i * L + l] = x[i];
      wave_lds_fence();
      if (id >= 0) sx = sh[id];
      wave_lds_fence();
#pragma unroll
      for (int i = 0; i < NV; ++i) sh[i * L + l] = 0.0f;
    }
    // per slot
    float u = dg;
    if constexpr (RENORM) {
      float q;
      if constexpr (SIG) {
        q = sigmoid(sx) * kScaleUp;        // 0 in empty slots, whose logit is -inf
      } else {
        const float m = group_max<L>(sx);
        q = exp_neg(sx - (m > kNegInf ? m : 0.0f));
      }
      const float sum = group_sum<L>(q);
      q = quotient(q, sum, estimate(sum));
      u = (u - group_sum<L>(q * u)) * q;
    }
    wave_lds_fence();
    if (id >= 0) atomicAdd(&sh[id], u);
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = sh[i * L + l];
    wave_lds_fence();
    if (id >= 0) sh[id] = 0.0f;
    // per expert
    if constexpr (SIG) {
      float s[NV], rest[NV], total = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        sigmoid(x[i], s[i], rest[i]);
        if constexpr (!RENORM) d[i] *= s[i];
        if constexpr (BAL) {
          s[i] *= kScaleUp;
          total += s[i];
        }
      }
      if constexpr (BAL) {
        total = group_sum<L>(total);
        const float r = estimate(total);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          s[i] = quotient(s[i], total, r);
          dot += s[i] * coef[i];
        }
        dot = group_sum<L>(dot);
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] += (coef[i] - dot) * s[i];
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) d[i] *= rest[i];
    } else if constexpr (BAL || !RENORM) {
      float top = kNegInf, total = 0.0f, dot = 0.0f, p[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) top = fmaxf(top, x[i]);
      top = group_max<L>(top);
      top = top > kNegInf ? top : 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        p[i] = exp_neg(x[i] - top);
        float v = RENORM ? 0.0f : d[i];
        if constexpr (BAL) v += coef[i];
        total += p[i];
        dot += p[i] * v;
      }
      total = group_sum<L>(total);
      dot = group_sum<L>(dot);
      const float r = inverse(total), mean = quotient(dot, total, r);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float v = RENORM ? 0.0f : d[i];
        if constexpr (BAL) v += coef[i];
        const float dp = p[i] * r * (v - mean);
        d[i] = RENORM ? d[i] + dp : dp;
      }
    }
    const uint64_t at = (uint64_t)t * (uint32_t)E;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = i * L + l;
      if (e < E && t < T) {
        const float y = live ? d[i] : 0.0f;
        if constexpr (BF) store_at(static_cast<uint16_t*>(a.dlogits) + at, e, (uint16_t)pk_bf16(y, 0.0f));
        else store_at(static_cast<float*>(a.dlogits) + at, e, y);
      }
    }
  }
}

template <bool BF, bool SIG, bool RENORM, bool BAL, int NE>
__global__ __launch_bounds__(kRowThreads) void k_route_bwd_rows(RouteBwdArgs a, bool vec) {
  const int E = a.E, k = a.k;
  float coef[BAL ? NE : 1];
  if constexpr (BAL) {
    const double n = (double)a.counts[E];
    const double c = n > 0.0 ? (double)a.alpha * E / (n * n * k) * (a.dloss ? (double)*a.dloss : 1.0)
                             : 0.0;
#pragma unroll
    for (int e = 0; e < NE; ++e) coef[e] = e < E ? (float)(c * (double)a.counts[e]) : 0.0f;
  }
  for (int64_t t = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; t < a.T;
       t += (int64_t)gridDim.x * kRowThreads) {
    float x[NE], d[NE];
    load_own_row<BF, NE>(a.logits, t, E, vec, x);
#pragma unroll
    for (int e = 0; e < NE; ++e) d[e] = 0.0f;
    bool live = false;
    float top = kNegInf, sum = 0.0f, dot = 0.0f;
    if constexpr (!SIG) {
#pragma unroll
      for (int e = 0; e < NE; ++e) top = fmaxf(top, x[e]);
      top = top > kNegInf ? top : 0.0f;
    }
    // the selected: first the renormalisation's sums, then each slot's part
    const auto slot = [&](int j, int& id, float& u, float& q) {
      id = a.topk_ids[t * k + j];
      id = id >= 0 && id < E ? id : -1;
      u = id >= 0 && a.dgate ? a.dgate[t * k + j] * a.scale : 0.0f;
      if constexpr (RENORM) {
        float v = kNegInf;
#pragma unroll
        for (int e = 0; e < NE; ++e) v = e == id ? x[e] : v;
        if constexpr (SIG) q = sigmoid(v) * kScaleUp;
        else q = exp_neg(v - top);
      }
    };
    if constexpr (RENORM) {
      for (int j = 0; j < k; ++j) {
        int id;
        float u, q;
        slot(j, id, u, q);
        sum += q;
        if constexpr (!SIG) dot += q * u;
      }
    }
    const float r = RENORM ? estimate(sum) : 0.0f;
    if constexpr (RENORM && !SIG) dot = quotient(dot, sum, r);
    if constexpr (RENORM && SIG) {         // scaled scores: quotients first, to stay in range
      for (int j = 0; j < k; ++j) {
        int id;
        float u, q;
        slot(j, id, u, q);
        dot += quotient(q, sum, r) * u;
      }
    }
    for (int j = 0; j < k; ++j) {
      int id;
      float u, q;
      slot(j, id, u, q);
      if constexpr (RENORM) u = (u - dot) * quotient(q, sum, r);
      live = live || id >= 0;
#pragma unroll
      for (int e = 0; e < NE; ++e) d[e] += e == id ? u : 0.0f;
    }
    // per expert
    if constexpr (SIG) {
      float s[NE], rest[NE], total = 0.0f;
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        sigmoid(x[e], s[e], rest[e]);
        if constexpr (!RENORM) d[e] *= s[e];
        if constexpr (BAL) {
          s[e] *= kScaleUp;
          total += s[e];
        }
      }
      if constexpr (BAL) {
        const float rt = estimate(total);
        float all = 0.0f;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          s[e] = quotient(s[e], total, rt);
          all += s[e] * coef[e];
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) d[e] += (coef[e] - all) * s[e];
      }
#pragma unroll
      for (int e = 0; e < NE; ++e) d[e] *= rest[e];
    } else if constexpr (BAL || !RENORM) {
      float total = 0.0f, all = 0.0f, p[NE];
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        p[e] = exp_neg(x[e] - top);
        float v = RENORM ? 0.0f : d[e];
        if constexpr (BAL) v += coef[e];
        total += p[e];
        all += p[e] * v;
      }
      const float rt = inverse(total), mean = quotient(all, total, rt);
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        float v = RENORM ? 0.0f : d[e];
        if constexpr (BAL) v += coef[e];
        const float dp = p[e] * rt * (v - mean);
        d[e] = RENORM ? d[e] + dp : dp;
      }
    }
#pragma unroll
    for (int e = 0; e < NE; ++e) d[e] = live ? d[e] : 0.0f;
    if (vec) {
      constexpr int per = BF ? 8 : 4;
      uint4* q = static_cast<uint4*>(const_cast<void*>(row_of<BF>(a.dlogits, t * E)));
#pragma unroll
      for (int i = 0; i < NE / per; ++i) {
        if constexpr (BF)
          q[i] = make_uint4(pk_bf16(d[8 * i], d[8 * i + 1]), pk_bf16(d[8 * i + 2], d[8 * i + 3]),
                            pk_bf16(d[8 * i + 4], d[8 * i + 5]), pk_bf16(d[8 * i + 6], d[8 * i + 7]));
        else
          q[i] = make_uint4(f2u(d[4 * i]), f2u(d[4 * i + 1]), f2u(d[4 * i + 2]), f2u(d[4 * i + 3]));
      }
    } else {
#pragma unroll
      for (int e = 0; e < NE; ++e)
        if (e < E) {
          if constexpr (BF) static_cast<uint16_t*>(a.dlogits)[t * E + e] = (uint16_t)pk_bf16(d[e], 0.0f);
          else static_cast<float*>(a.dlogits)[t * E + e] = d[e];
        }
    }
  }
}

// Whether rows go to groups of 16 lanes: a round of the selection there serves
// four rows, but every slot takes one, where the wide form's cost hardly grows
// with k. Narrow against wide: 32768 x 64 top-6 8.3 and 12.7 us, top-16 16.6
// and 19.6; 131072 x 128 top-2 18.1 and 44.1, top-4 27.2 and 43.7, top-8 45.6 and
// 42.8, top-16 82.6 and 66.3; backward 131072 x 128 33.9 and 45.7, 32768 rows
// 12.6 and 14.3. The rule does not look at few rows, which pay up to 1 us for it
// (512 x 64 top-6 3.6 and 2.8, backward 3.5 and 2.9, biased 4.9 and 2.9; top-2
// 2.7 and 2.8, 32 experts top-8 3.4 and 4.1) in a call of 7 us of the host's
// time; the two meet at some 4096 rows.
bool narrow(int64_t T, int E, int k, bool biased, bool backward) {
  if (k > kNarrowK || E > 128) return false;
  return E <= 64 || (backward ? T >= 32768 : !biased && k <= 4);
}

// Whether rows go to single threads: rows enough to fill the device, few enough
// experts for the registers. Single against narrow, at the bound and at 262144
// rows: 8 experts top-2 2.5 and 2.7 us (8192 rows), 3.7 and 18.9; 64 experts
// top-6 11.7 and 14.4 (65536 rows), 22.2 and 49.7; 8 experts backward 4.2 and
// 4.5 (32768 rows), 9.1 and 17.2; biased 4.0 and 4.5, 7.7 and 20.4.
bool single(int64_t T, int E, int k, bool biased, bool backward) {
  if (k > kNarrowK || E > (biased || backward ? 8 : 64)) return false;
  return T >= (biased || backward ? 32768 : 1024 * E);
}

bool whole_rows(const void* p, int E, bool bf16) {
  return (E == 8 || E == 16 || E == 32 || E == 64) &&   // the row kernels' sizes
         (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// Experts per lane, rounded up to a form that is built.
int lanes_experts(int E) {
  const int nv = (E + 63) / 64;
  return nv <= 1 ? 1 : nv <= 2 ? 2 : nv <= 4 ? 4 : nv <= 6 ? 6 : nv <= 8 ? 8 : 16;
}

// Wavefronts of a forward workgroup: few while the rows do not fill the device
// (512 x 384 biased: 3.7 us with 4, 4.5 with 16), many when they do, for fewer
// statistics partials (32768 x 384 with statistics and loss: 36.7 us with 4, 28.0
// with 8, 25.7 with 16; without them 15.5, 15.5 and 15.3).
int route_waves(int64_t T, int rows_per_wave) {
  const int64_t need = (T + rows_per_wave - 1) / rows_per_wave;
  return need <= 1024 ? 4 : need <= 2048 ? 8 : kMaxWaves;
}

// How a launch takes its rows.
enum RouteForm { kSingle, kNarrow, kWide };       // a thread, 16 lanes, a wavefront per row
struct RoutePlan {
  RouteForm form;
  unsigned grid, threads;
  // A lane of the wide and narrow forms takes kHeldRows rows or more.
  bool deep(int64_t T) const {
    const int64_t at_once = (int64_t)grid * (threads / 64) * (form == kNarrow ? 4 : 1);
    return (T + at_once - 1) / at_once >= kHeldRows;
  }
};

// Few enough rows for one workgroup, which then leaves the statistics
// themselves: no partials and a launch fewer, of 3.3 us of the host's time
// (with the loss, kernels alone: 16 x 384 8.9 -> 6.5 us, 512 x 8 7.2 -> 5.3,
// 1024 x 8 7.6 -> 6.3).
// More rounds of one workgroup lose: 128 x 64 would take 11.2 us for 8.5, 4096 x
// 8 12.5 for 8.0.
bool alone_any(int64_t T, int E) { return T <= kMaxWaves || (E <= 8 && T <= 1024); }

RoutePlan route_plan(int64_t T, int E, int k, bool biased, bool stats) {
  if (stats && E <= 8 && alone_any(T, E))
    return RoutePlan{kSingle, 1, (unsigned)(T < 1024 ? (T + 63) / 64 * 64 : 1024)};
  RoutePlan p{kWide, 0, 0};
  int64_t rows = 0;
  if (single(T, E, k, biased, false)) {
    p.form = kSingle;
    p.threads = kRowThreads;
    rows = kRowThreads;
  } else {
    const int per_wave = narrow(T, E, k, biased, false) ? 4 : 1;
    if (per_wave == 4) p.form = kNarrow;
    const int waves = route_waves(T, per_wave);
    if (stats && T <= kMaxWaves * per_wave)       // one round of one workgroup
      return RoutePlan{p.form, 1, 64u * (unsigned)((T + per_wave - 1) / per_wave)};
    p.threads = 64u * waves;
    rows = waves * per_wave;
  }
  const int64_t need = (T + rows - 1) / rows;
  int64_t most = (int64_t)device_cu_count() * 2048 / p.threads;   // 32 wavefronts a compute unit
  if (stats && most > kMaxRouteParts) most = kMaxRouteParts;
  p.grid = (unsigned)(need < most ? need : most);
  return p;
}

RoutePlan route_bwd_plan(int64_t T, int E, int k) {
  RoutePlan p{kWide, 0, 64 * kWaves};
  int64_t rows = kWaves;
  if (single(T, E, k, false, true)) {
    p = RoutePlan{kSingle, 0, kRowThreads};
    rows = kRowThreads;
  } else if (narrow(T, E, k, false, true)) {
    p.form = kNarrow;
    rows = 4 * kWaves;
  }
  const int64_t need = (T + rows - 1) / rows;
  const int64_t most = (int64_t)device_cu_count() * 2048 / p.threads;
  p.grid = (unsigned)(need < most ? need : most);
  return p;
}

template <bool BF, bool SIG, bool BIAS, bool STATS>
void route_nv(const RouteArgs& a, const RoutePlan& at, hipStream_t s) {
  const size_t word = !STATS ? 0 : a.deep ? sizeof(double) : sizeof(float);
#define NVFP4MOE_ROUTE(L, NV) \
  k_route<BF, SIG, BIAS, STATS, L, NV><<<at.grid, at.threads, at.threads * NV * word, s>>>(a)
  if (at.form == kSingle) {
#define NVFP4MOE_ROWS(NE) \
  k_route_rows<BF, SIG, BIAS, STATS, NE><<<at.grid, at.threads, 0, s>>>(a, whole_rows(a.logits, a.E, BF))
    if constexpr (BIAS) {
      NVFP4MOE_ROWS(8);
    } else {
      if (a.E <= 8) NVFP4MOE_ROWS(8);
      else if (a.E <= 16) NVFP4MOE_ROWS(16);
      else if (a.E <= 32) NVFP4MOE_ROWS(32);
      else NVFP4MOE_ROWS(64);
    }
#undef NVFP4MOE_ROWS
    return;
  }
  if (at.form == kNarrow) {
    if (a.E <= 16) NVFP4MOE_ROUTE(16, 1);
    else if (a.E <= 32) NVFP4MOE_ROUTE(16, 2);
    else if (BIAS || a.E <= 64) NVFP4MOE_ROUTE(16, 4);
    else if constexpr (!BIAS) NVFP4MOE_ROUTE(16, 8);
    return;
  }
  switch (lanes_experts(a.E)) {
    case 1: NVFP4MOE_ROUTE(64, 1); break;
    case 2: NVFP4MOE_ROUTE(64, 2); break;
    case 4: NVFP4MOE_ROUTE(64, 4); break;
    case 6: NVFP4MOE_ROUTE(64, 6); break;
    case 8: NVFP4MOE_ROUTE(64, 8); break;
    default: NVFP4MOE_ROUTE(64, 16); break;
  }
#undef NVFP4MOE_ROUTE
}

template <bool BF>
void route_form(const RouteArgs& a, bool sigmoid, bool stats, const RoutePlan& at, hipStream_t s) {
  if (!sigmoid) {
    if (stats) route_nv<BF, false, false, true>(a, at, s);
    else route_nv<BF, false, false, false>(a, at, s);
  } else if (a.bias) {
    if (stats) route_nv<BF, true, true, true>(a, at, s);
    else route_nv<BF, true, true, false>(a, at, s);
  } else {
    if (stats) route_nv<BF, true, false, true>(a, at, s);
    else route_nv<BF, true, false, false>(a, at, s);
  }
}

template <bool BF, bool SIG, bool RENORM, bool BAL>
void bwd_nv(const RouteBwdArgs& a, const RoutePlan& at, hipStream_t s) {
#define NVFP4MOE_BWD(L, NV) k_route_bwd<BF, SIG, RENORM, BAL, L, NV><<<at.grid, at.threads, 0, s>>>(a)
  if (at.form == kSingle) {
    const bool vec = whole_rows(a.logits, a.E, BF) && whole_rows(a.dlogits, a.E, BF);
#define NVFP4MOE_ROWS(NE) \
  k_route_bwd_rows<BF, SIG, RENORM, BAL, NE><<<at.grid, at.threads, 0, s>>>(a, vec)
    NVFP4MOE_ROWS(8);
#undef NVFP4MOE_ROWS
    return;
  }
  if (at.form == kNarrow) {
    if (a.E <= 16) NVFP4MOE_BWD(16, 1);
    else if (a.E <= 32) NVFP4MOE_BWD(16, 2);
    else if (a.E <= 64) NVFP4MOE_BWD(16, 4);
    else NVFP4MOE_BWD(16, 8);
    return;
  }
  switch (lanes_experts(a.E)) {
    case 1: NVFP4MOE_BWD(64, 1); break;
    case 2: NVFP4MOE_BWD(64, 2); break;
    case 4: NVFP4MOE_BWD(64, 4); break;
    case 6: NVFP4MOE_BWD(64, 6); break;
    case 8: NVFP4MOE_BWD(64, 8); break;
    default: NVFP4MOE_BWD(64, 16); break;
  }
#undef NVFP4MOE_BWD
}

template <bool BF, bool SIG>
void bwd_form(const RouteBwdArgs& a, bool renorm, const RoutePlan& at, hipStream_t s) {
  if (renorm) {
    if (a.counts) bwd_nv<BF, SIG, true, true>(a, at, s);
    else bwd_nv<BF, SIG, true, false>(a, at, s);
  } else {
    if (a.counts) bwd_nv<BF, SIG, false, true>(a, at, s);
    else bwd_nv<BF, SIG, false, false>(a, at, s);
  }
}

}  // namespace

size_t route_workspace_bytes(int64_t T, int E) {
  if (alone_any(T, E)) return 0;
  const int64_t need = (T + 3) / 4;               // workgroups have at least 4 rows
  const int64_t parts = need < kMaxRouteParts ? need : kMaxRouteParts;
  return (size_t)(parts * ((int64_t)E + 1) * sizeof(RoutePart));
}

hipError_t launch_route(const void* logits, bool bf16, int64_t T, int E, int k, bool sigmoid,
                        bool renorm, float scale, const float* bias, const uint8_t* token_mask,
                        int32_t* topk_ids, float* gate, int64_t* counts, float* prob_sum,
                        void* workspace, hipStream_t stream) {
  const bool stats = counts != nullptr;
  RoutePart* parts = nullptr;
  unsigned grid = 0;
  if (T > 0) {
    const RoutePlan at = route_plan(T, E, k, bias != nullptr, stats);
    grid = at.grid;
    if (stats && grid > 1) parts = static_cast<RoutePart*>(workspace);
    const RouteArgs a{logits, T, E, k, bias, token_mask, renorm, scale, topk_ids, gate, parts,
                      counts, prob_sum, stats && at.deep(T)};
    if (bf16) route_form<true>(a, sigmoid, stats, at, stream);
    else route_form<false>(a, sigmoid, stats, at, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (stats && (parts || T == 0))
    k_route_stats<<<(unsigned)(E / 16 + 1), 1024, 0, stream>>>(parts, (int)grid, E, counts,
                                                               prob_sum);
  return hipGetLastError();
}

hipError_t launch_balance_loss(const int64_t* counts, const float* prob_sum, int E, int k,
                               float alpha, float* loss, hipStream_t stream) {
  k_balance_loss<<<1, 256, 0, stream>>>(counts, prob_sum, E, k, alpha, loss);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const void* logits, bool bf16, int64_t T, int E, int k, bool sigmoid,
                            bool renorm, float scale, const int32_t* topk_ids, const float* dgate,
                            const int64_t* counts, float alpha, const float* dloss, void* dlogits,
                            hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const RouteBwdArgs a{logits, T, E, k, topk_ids, dgate, scale, counts, alpha, dloss, dlogits};
  const RoutePlan at = route_bwd_plan(T, E, k);
  if (bf16) {
    if (sigmoid) bwd_form<true, true>(a, renorm, at, stream);
    else bwd_form<true, false>(a, renorm, at, stream);
  } else {
    if (sigmoid) bwd_form<false, true>(a, renorm, at, stream);
    else bwd_form<false, false>(a, renorm, at, stream);
  }
  return hipGetLastError();
}

}  // namespace nvfp4moe
