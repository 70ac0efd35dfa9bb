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
// One wavefront takes a row, lane l its experts l, l + 64, ...: every load and
// store is one run of lanes, a lane meets the same experts in every row (their
// probability sums and loss gradients stay in registers), and the k results
// sit in the first k lanes.
#include "codecs.hpp"
#include "internal.hpp"

namespace nvfp4moe {

namespace {

constexpr int kWaves = 4;                  // rows in flight per workgroup
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float load1(const void* p, bool bf16, int64_t i) {
  return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}

// Orders the LDS accesses of one wavefront's lanes before and after it (the
// hardware runs them in order; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// exp(x) for x <= 0 by the hardware's 2^x: the rounded product x * log2(e)
// costs a relative 2^-24 |x|, the instruction one unit in the last place.
__device__ __forceinline__ float exp_neg(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}

// sigmoid(x) and its derivative s (1 - s), both from z = exp(-|x|) so that
// neither cancels: s = 1 / (1 + z) or z / (1 + z), s' = z / (1 + z)^2.
__device__ __forceinline__ void sigmoid(float x, float& s, float& ds) {
  const float z = exp_neg(-fabsf(x));
  const float r = __builtin_amdgcn_rcpf(1.0f + z);
  s = x >= 0.0f ? r : z * r;
  ds = z * r * r;
}

// The key experts compete with where a bias is given. 64 bits: two scores that
// differ by less than a float32 step are told apart, and the choice does not
// hang on how a float32 exponential rounds.
__device__ __forceinline__ double biased_key(float x, float bias) {
  return 1.0 / (1.0 + exp(-(double)x)) + (double)bias;
}

// k rounds of taking the largest remaining key, the lowest expert first among
// equals. Lane j ends with the j-th expert (or -1) in id.
template <int NV, typename Key>
__device__ __forceinline__ void select_rounds(Key (&key)[NV], int k, int lane, int& id) {
  const Key none = (Key)kNegInf;
  id = -1;
  for (int j = 0; j < k; ++j) {
    Key best = none;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i * 64 + lane;
      }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const Key o = __shfl_xor(best, off, 64);
      const int oat = __shfl_xor(at, off, 64);
      if (o > best || (o == best && oat < at)) {
        best = o;
        at = oat;
      }
    }
    if (!(best > none)) return;            // the same for the whole wavefront
    if (lane == j) id = at;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (at == i * 64 + lane) key[i] = none;
  }
}

struct RouteArgs {
  const void* logits;
  int64_t T;
  int E, k;
  const float* bias;
  const uint8_t* token_mask;
  float scale;
  int32_t* topk_ids;
  float* gate;
  float* part_prob;      // [grid, E] probability sums of each workgroup's rows
  int32_t* part_count;   // [grid, E + 1]
};

template <bool BF, bool SIG, bool RENORM, bool BIAS, bool STATS, int NV>
__global__ __launch_bounds__(64 * kWaves) void k_route(RouteArgs a) {
  __shared__ float sh_prob[STATS ? kWaves * NV * 64 : 1];
  __shared__ int32_t sh_count[STATS ? NV * 64 + 1 : 1];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int E = a.E, k = a.k;
  float bias[BIAS ? NV : 1];
  if constexpr (BIAS) {
#pragma unroll
    for (int i = 0; i < NV; ++i) bias[i] = i * 64 + lane < E ? a.bias[i * 64 + lane] : 0.0f;
  }
  float psum[STATS ? NV : 1];
  if constexpr (STATS) {
#pragma unroll
    for (int i = 0; i < NV; ++i) psum[i] = 0.0f;
    for (int e = threadIdx.x; e <= E; e += 64 * kWaves) sh_count[e] = 0;
    __syncthreads();
  }
  for (int64_t t = (int64_t)blockIdx.x * kWaves + w; t < a.T; t += (int64_t)gridDim.x * kWaves) {
    const bool on = a.token_mask == nullptr || a.token_mask[t] != 0;
    float x[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = i * 64 + lane;
      x[i] = on && e < E ? load1(a.logits, BF, t * E + e) : kNegInf;
    }
    int id;
    if constexpr (BIAS) {
      double key[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i)
        key[i] = x[i] > kNegInf ? biased_key(x[i], bias[i]) : (double)kNegInf;
      select_rounds<NV>(key, k, lane, id);
    } else {
      float key[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = x[i];
      select_rounds<NV>(key, k, lane, id);
    }
    const bool live = __builtin_amdgcn_readfirstlane(id) >= 0;
    // scores; the row's probabilities where they are needed
    float top = kNegInf, total = 0.0f, p[NV];
    if constexpr (STATS || (!SIG && !RENORM)) {
      if (live) {
        if constexpr (!SIG) {
#pragma unroll
          for (int i = 0; i < NV; ++i) top = fmaxf(top, x[i]);
          top = wave_max(top);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if constexpr (SIG) {
            float ds;
            sigmoid(x[i], p[i], ds);
          } else {
            p[i] = exp_neg(x[i] - top);
          }
          total += p[i];
        }
        total = wave_sum(total);
      }
    }
    if constexpr (STATS) {
      if (live && total > 0.0f) {
        const float r = 1.0f / total;
#pragma unroll
        for (int i = 0; i < NV; ++i) psum[i] += p[i] * r;
      }
      if (lane < k && id >= 0) atomicAdd(&sh_count[id], 1);
      if (lane == 0 && live) atomicAdd(&sh_count[E], 1);
    }
    // gates of the selected, one per lane
    const float sx = id >= 0 ? load1(a.logits, BF, t * E + id) : kNegInf;
    float g = 0.0f;
    if (live) {
      if constexpr (SIG) {
        float ds;
        if (id >= 0) sigmoid(sx, g, ds);
      } else if constexpr (RENORM) {
        g = exp_neg(sx - wave_max(sx));
      } else {
        g = exp_neg(sx - top) / total;
      }
      if constexpr (RENORM) {
        const float sum = wave_sum(g);
        g = sum > 0.0f ? g / sum : 0.0f;
      }
    }
    if (lane < k) {
      a.topk_ids[t * k + lane] = id;
      a.gate[t * k + lane] = g * a.scale;
    }
  }
  if constexpr (STATS) {
#pragma unroll
    for (int i = 0; i < NV; ++i) sh_prob[w * NV * 64 + i * 64 + lane] = psum[i];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 64 * kWaves) {
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) s += sh_prob[v * NV * 64 + e];
      a.part_prob[(int64_t)blockIdx.x * E + e] = s;
    }
    for (int e = threadIdx.x; e <= E; e += 64 * kWaves)
      a.part_count[(int64_t)blockIdx.x * (E + 1) + e] = sh_count[e];
  }
}

// Column sums of the workgroups' partials, in a fixed order: 16 columns per
// workgroup, 16 threads down each.
__global__ __launch_bounds__(256) void k_route_stats(const float* __restrict__ part_prob,
                                                     const int32_t* __restrict__ part_count,
                                                     int parts, int E,
                                                     int64_t* __restrict__ counts,
                                                     float* __restrict__ prob_sum) {
  __shared__ double sp[256];
  __shared__ int64_t sc[256];
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int e = blockIdx.x * 16 + col;
  double p = 0.0;
  int64_t c = 0;
  for (int g = row; g < parts; g += 16) {
    if (e < E) p += (double)part_prob[(int64_t)g * E + e];
    if (e <= E) c += part_count[(int64_t)g * (E + 1) + e];
  }
  sp[threadIdx.x] = p;
  sc[threadIdx.x] = c;
  __syncthreads();
  if (row == 0 && e <= E) {
    for (int r = 1; r < 16; ++r) {
      p += sp[16 * r + col];
      c += sc[16 * r + col];
    }
    if (e < E) prob_sum[e] = (float)p;
    counts[e] = c;
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

// The selected experts' part of a row's gradient is computed one slot per
// lane and reaches the lanes that own the experts through LDS.
template <bool BF, bool SIG, bool RENORM, bool BAL, int NV>
__global__ __launch_bounds__(64 * kWaves) void k_route_bwd(RouteBwdArgs a) {
  __shared__ float sh[kWaves][NV * 64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int E = a.E, k = a.k;
  float coef[BAL ? NV : 1];
  if constexpr (BAL) {
    const double n = (double)a.counts[E];
    const double c = n > 0.0 ? (double)a.alpha * E / (n * n * k) * (a.dloss ? (double)*a.dloss : 1.0)
                             : 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      coef[i] = i * 64 + lane < E ? (float)(c * (double)a.counts[i * 64 + lane]) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) sh[w][i * 64 + lane] = 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * kWaves + w; t < a.T; t += (int64_t)gridDim.x * kWaves) {
    int id = lane < k ? a.topk_ids[t * k + lane] : -1;
    if (id >= E) id = -1;
    const float dg = id >= 0 && a.dgate ? a.dgate[t * k + lane] * a.scale : 0.0f;
    float x[NV], d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = i * 64 + lane;
      x[i] = e < E ? load1(a.logits, BF, t * E + e) : kNegInf;
    }
    const float sx = id >= 0 ? load1(a.logits, BF, t * E + id) : kNegInf;
    const bool live = __any(id >= 0);
    if (!live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) d[i] = 0.0f;
    } else {
      // per slot
      float u = dg;
      if constexpr (RENORM) {
        float q = 0.0f;
        if constexpr (SIG) {
          float ds;
          if (id >= 0) sigmoid(sx, q, ds);
        } else {
          q = exp_neg(sx - wave_max(sx));
        }
        const float sum = wave_sum(q), dot = wave_sum(q * u);
        const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
        u = id >= 0 ? (u - dot * r) * r : 0.0f;
        if constexpr (!SIG) u *= q;
      }
      if (id >= 0) atomicAdd(&sh[w][id], u);
      wave_lds_fence();
#pragma unroll
      for (int i = 0; i < NV; ++i) d[i] = sh[w][i * 64 + lane];
      wave_lds_fence();
      if (id >= 0) sh[w][id] = 0.0f;
      // per expert
      if constexpr (SIG) {
        float s[NV], ds[NV], total = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          sigmoid(x[i], s[i], ds[i]);
          if constexpr (BAL) {
            total += s[i];
            dot += s[i] * coef[i];
          }
        }
        if constexpr (BAL) {
          total = wave_sum(total);
          dot = wave_sum(dot);
          const float r = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
          for (int i = 0; i < NV; ++i) d[i] += (coef[i] - dot * r) * r;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] *= ds[i];
      } else if constexpr (BAL || !RENORM) {
        float top = kNegInf, total = 0.0f, dot = 0.0f, p[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) top = fmaxf(top, x[i]);
        top = wave_max(top);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          p[i] = exp_neg(x[i] - top);
          float v = RENORM ? 0.0f : d[i];
          if constexpr (BAL) v += coef[i];
          total += p[i];
          dot += p[i] * v;
        }
        total = wave_sum(total);
        dot = wave_sum(dot);
        const float r = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float v = RENORM ? 0.0f : d[i];
          if constexpr (BAL) v += coef[i];
          const float dp = p[i] * r * (v - dot * r);
          d[i] = RENORM ? d[i] + dp : dp;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = i * 64 + lane;
      if (e < E) {
        if constexpr (BF) static_cast<uint16_t*>(a.dlogits)[t * E + e] = (uint16_t)pk_bf16(d[i], 0.0f);
        else static_cast<float*>(a.dlogits)[t * E + e] = d[i];
      }
    }
  }
}

// Experts per lane, rounded up to a form that is built.
int lanes_experts(int E) {
  const int nv = (E + 63) / 64;
  return nv <= 1 ? 1 : nv <= 2 ? 2 : nv <= 4 ? 4 : nv <= 6 ? 6 : nv <= 8 ? 8 : 16;
}

int64_t route_grid(int64_t T, int per_cu) {
  const int64_t need = (T + kWaves - 1) / kWaves, most = (int64_t)device_cu_count() * per_cu;
  return need < most ? need : most;
}

constexpr int kStatsPerCu = 4;             // workgroups per CU that leave a partial

template <bool BF, bool SIG, bool RENORM, bool BIAS, bool STATS>
void route_nv(const RouteArgs& a, unsigned grid, hipStream_t s) {
  switch (lanes_experts(a.E)) {
    case 1: k_route<BF, SIG, RENORM, BIAS, STATS, 1><<<grid, 64 * kWaves, 0, s>>>(a); break;
    case 2: k_route<BF, SIG, RENORM, BIAS, STATS, 2><<<grid, 64 * kWaves, 0, s>>>(a); break;
    case 4: k_route<BF, SIG, RENORM, BIAS, STATS, 4><<<grid, 64 * kWaves, 0, s>>>(a); break;
    case 6: k_route<BF, SIG, RENORM, BIAS, STATS, 6><<<grid, 64 * kWaves, 0, s>>>(a); break;
    case 8: k_route<BF, SIG, RENORM, BIAS, STATS, 8><<<grid, 64 * kWaves, 0, s>>>(a); break;
    default: k_route<BF, SIG, RENORM, BIAS, STATS, 16><<<grid, 64 * kWaves, 0, s>>>(a); break;
  }
}

template <bool BF, bool SIG, bool RENORM>
void route_form(const RouteArgs& a, bool stats, unsigned grid, hipStream_t s) {
  if constexpr (SIG) {
    if (a.bias) {
      if (stats) route_nv<BF, SIG, RENORM, true, true>(a, grid, s);
      else route_nv<BF, SIG, RENORM, true, false>(a, grid, s);
      return;
    }
  }
  if (stats) route_nv<BF, SIG, RENORM, false, true>(a, grid, s);
  else route_nv<BF, SIG, RENORM, false, false>(a, grid, s);
}

template <bool BF, bool SIG, bool RENORM, bool BAL>
void bwd_nv(const RouteBwdArgs& a, unsigned grid, hipStream_t s) {
  switch (lanes_experts(a.E)) {
    case 1: k_route_bwd<BF, SIG, RENORM, BAL, 1><<<grid, 64 * kWaves, 0, s>>>(a); break;
    case 2: k_route_bwd<BF, SIG, RENORM, BAL, 2><<<grid, 64 * kWaves, 0, s>>>(a); break;
    case 4: k_route_bwd<BF, SIG, RENORM, BAL, 4><<<grid, 64 * kWaves, 0, s>>>(a); break;
    case 6: k_route_bwd<BF, SIG, RENORM, BAL, 6><<<grid, 64 * kWaves, 0, s>>>(a); break;
    case 8: k_route_bwd<BF, SIG, RENORM, BAL, 8><<<grid, 64 * kWaves, 0, s>>>(a); break;
    default: k_route_bwd<BF, SIG, RENORM, BAL, 16><<<grid, 64 * kWaves, 0, s>>>(a); break;
  }
}

}  // namespace

size_t route_workspace_bytes(int64_t T, int E) {
  const int64_t need = (T + kWaves - 1) / kWaves;
  const int64_t parts = need < kMaxRouteParts ? need : kMaxRouteParts;
  return (size_t)(parts * (2 * (int64_t)E + 1) * 4);
}

hipError_t launch_route(const void* logits, bool bf16, int64_t T, int E, int k, bool sigmoid,
                        bool renorm, float scale, const float* bias, const uint8_t* token_mask,
                        int32_t* topk_ids, float* gate, int64_t* counts, float* prob_sum,
                        void* workspace, hipStream_t stream) {
  const bool stats = counts != nullptr;
  int64_t grid = route_grid(T, stats ? kStatsPerCu : 8);
  if (stats && grid > kMaxRouteParts) grid = kMaxRouteParts;
  RouteArgs a{logits, T, E, k, bias, token_mask, scale, topk_ids, gate, nullptr, nullptr};
  if (stats) {
    a.part_prob = static_cast<float*>(workspace);
    a.part_count = reinterpret_cast<int32_t*>(a.part_prob + grid * E);
  }
  if (grid > 0) {
    const unsigned g = (unsigned)grid;
    if (bf16) {
      if (sigmoid) {
        if (renorm) route_form<true, true, true>(a, stats, g, stream);
        else route_form<true, true, false>(a, stats, g, stream);
      } else {
        if (renorm) route_form<true, false, true>(a, stats, g, stream);
        else route_form<true, false, false>(a, stats, g, stream);
      }
    } else {
      if (sigmoid) {
        if (renorm) route_form<false, true, true>(a, stats, g, stream);
        else route_form<false, true, false>(a, stats, g, stream);
      } else {
        if (renorm) route_form<false, false, true>(a, stats, g, stream);
        else route_form<false, false, false>(a, stats, g, stream);
      }
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (stats)
    k_route_stats<<<(unsigned)(E / 16 + 1), 256, 0, stream>>>(a.part_prob, a.part_count, (int)grid,
                                                              E, counts, prob_sum);
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
  const unsigned g = (unsigned)route_grid(T, 8);
#define NVFP4MOE_BWD(BF, SIG, REN)                                   \
  do {                                                               \
    if (counts) bwd_nv<BF, SIG, REN, true>(a, g, stream);            \
    else bwd_nv<BF, SIG, REN, false>(a, g, stream);                  \
  } while (0)
  if (bf16) {
    if (sigmoid) {
      if (renorm) NVFP4MOE_BWD(true, true, true); else NVFP4MOE_BWD(true, true, false);
    } else {
      if (renorm) NVFP4MOE_BWD(true, false, true); else NVFP4MOE_BWD(true, false, false);
    }
  } else {
    if (sigmoid) {
      if (renorm) NVFP4MOE_BWD(false, true, true); else NVFP4MOE_BWD(false, true, false);
    } else {
      if (renorm) NVFP4MOE_BWD(false, false, true); else NVFP4MOE_BWD(false, false, false);
    }
  }
#undef NVFP4MOE_BWD
  return hipGetLastError();
}

}  // namespace nvfp4moe
