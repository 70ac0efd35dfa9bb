// The whole expert layer for a few tokens: selection and gates, up-projection,
// activation, down-projection and the weighted sum, in two kernels.
//
//   (ids, gate)[t]  as moe_route
//   h[t, j]   = act(W1[e] x[t]), or act(W1a[e] x[t]) * (W1b[e] x[t]) with e = ids[t, j]
//   out[t]    = sum_j gate[t, j] W2[e] h[t, j]   over the pairs whose expert is local
//
// Weights are 4-bit (MXFP4 or NVFP4) and dequantized in registers; every
// dequantized element (up to 6 significant bits) is exact in bfloat16, so the
// products run on v_mfma_f32_16x16x32_bf16 with the weight rows as A and the
// tokens as B. The activations are not quantized. h is carried between the
// kernels as two bfloat16 parts (value and remainder, 16 bits together), each
// with a product of its own: one part would cost half the output's last bit.
//
// What bounds it is the weights' bytes: with up to 64 tokens each selected
// expert's weights are read once.
//
// k_tokens_up: every workgroup repeats the selection (a wavefront per token;
// reading a result of another launch would cost more), lists the pairs of each
// local expert, then takes (expert, 16 rows of W1) units; its wavefronts split
// the contraction and join through LDS.
// k_tokens_down: a workgroup takes 16 rows of W2 for every selected expert; its
// wavefronts split (expert, contraction) and join once at the end. A column of
// B is a token, so pairs of one token in several experts add up in the
// accumulators; gates and W2's outer scales were multiplied into h before.
#include "codecs.hpp"
#include "internal.hpp"

namespace nvfp4moe {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

constexpr int kThreads = 1024;
constexpr int kWavesT = kThreads / 64;
constexpr int kMaxExperts = 1024;
constexpr float kNegInfT = -__builtin_huge_valf();

// Workspace: what k_tokens_up leaves for k_tokens_down.
struct TokensTable {
  int n_active;                              // selected local experts
  int expert[kTokensMaxPairs];               // each one's local index, ascending
  int16_t pair[kTokensMaxPairs][kTokensMaxT];  // its pair of token t, or -1
};
constexpr size_t kTableBytes = (sizeof(TokensTable) + 255) / 256 * 256;

// ------------------------------------------------------------- wavefront reductions

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d, 64));
  return v;
}
__device__ __forceinline__ uint32_t wave_min_u32(uint32_t v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = min(v, (uint32_t)__shfl_xor((int)v, d, 64));
  return v;
}
__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Order-preserving bits of a number that can be selected; 0 for NaN and -inf.
__device__ __forceinline__ uint64_t order_key(double v) {
  if (!(v > -__builtin_huge_val())) return 0;
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v > kNegInfT)) return 0;
  const uint32_t b = f2u(v);
  return b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float logit(const TokensArgs& a, int64_t i) {
  return a.logits_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[i])
                       : static_cast<const float*>(a.logits)[i];
}

// One token's experts and gates, by one wavefront: lane j < k gets slot j's.
// Lane l looks at experts l, l + 64, ...; k rounds of a maximum, the lower
// index first among equals. BIAS: by sigmoid(x) + bias in 64 bits.
template <int NE, bool BIAS>
__device__ __forceinline__ void select(const TokensArgs& a, int t, int& id, float& gate) {
  const int lane = threadIdx.x & 63;
  const bool real = !a.token_mask || a.token_mask[t];
  float x[NE];
  uint32_t hi[NE], lo[BIAS ? NE : 1];
  float top = kNegInfT;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 64 * i;
    x[i] = real && e < a.E ? logit(a, (int64_t)t * a.E + e) : kNegInfT;
    top = fmaxf(top, x[i]);
    if constexpr (BIAS) {
      uint64_t key = 0;
      if (x[i] > kNegInfT) key = order_key(1.0 / (1.0 + exp(-(double)x[i])) + (double)a.bias[e]);
      hi[i] = (uint32_t)(key >> 32);
      lo[i] = (uint32_t)key;
    } else {
      hi[i] = order_key(x[i]);
    }
  }
  float denom = 0.0f;
  if (!a.sigmoid) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
#pragma unroll
    for (int i = 0; i < NE; ++i) denom += x[i] > kNegInfT ? expf(x[i] - top) : 0.0f;
    denom = wave_sum_f32(denom);
  }
  id = -1;
  for (int j = 0; j < a.k; ++j) {
    uint32_t bh = hi[0], bl = BIAS ? lo[0] : 0;
    int bi = lane;
#pragma unroll
    for (int i = 1; i < NE; ++i) {
      bool more = hi[i] > bh;
      if constexpr (BIAS) more = more || (hi[i] == bh && lo[i] > bl);
      bh = more ? hi[i] : bh;
      if constexpr (BIAS) bl = more ? lo[i] : bl;
      bi = more ? lane + 64 * i : bi;
    }
    const uint32_t mh = wave_max_u32(bh);
    if (mh == 0) break;                      // no expert left
    bool best = bh == mh;
    if constexpr (BIAS) {
      const uint32_t ml = wave_max_u32(best ? bl : 0u);
      best = best && bl == ml;
    }
    const int e = (int)wave_min_u32(best ? (uint32_t)bi : 0xFFFFu);
    if (lane == j) id = e;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (lane + 64 * i == e) hi[i] = 0;
    if constexpr (BIAS) {
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (lane + 64 * i == e) lo[i] = 0;
    }
  }
  float s = 0.0f;
  if (id >= 0) {
    const float v = logit(a, (int64_t)t * a.E + id);
    s = a.sigmoid ? 1.0f / (1.0f + expf(-v)) : expf(v - top) / denom;
    s = s < 0x1p-126f ? 0.0f : s;
  }
  if (a.renorm) {
    const float total = wave_sum_f32(s);
    s = total > 0.0f ? s / total : 0.0f;
  }
  gate = a.scale * s;
}

// 32 codes (16 bytes, one row's elements 32 g .. 32 g + 31 of a 128-element
// chunk) to four bfloat16 fragments. MXFP4: one scale byte, folded into the
// conversion. NVFP4: two E4M3 scales of 16, the products exact.
template <bool NV>
__device__ __forceinline__ void dequant(const u32x4v w, uint32_t s, bf16x8 (&f)[4]) {
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    uint32_t p[4];
    if constexpr (NV) {
      const float sc = __builtin_amdgcn_cvt_f32_fp8((int)(m < 2 ? s & 0xFFu : s >> 8), 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float u, v;
        e2m1x2_to_f32(w[m], i, u, v);
        p[i] = pk_bf16(__fmul_rn(u, sc), __fmul_rn(v, sc));
      }
    } else {
      const float sc = u2f(s << 23);
      p[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[m], sc, 0));
      p[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[m], sc, 1));
      p[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[m], sc, 2));
      p[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[m], sc, 3));
    }
    f[m] = __builtin_bit_cast(bf16x8, u32x4v{p[0], p[1], p[2], p[3]});
  }
}

// The scales of lane group g's 32 elements in chunk c of a row.
template <bool NV>
__device__ __forceinline__ uint32_t load_scale(const uint8_t* row, int64_t c, int g) {
  if constexpr (NV) return *reinterpret_cast<const uint16_t*>(row + c * 8 + 2 * g);
  else return row[c * 4 + g];
}

__device__ __forceinline__ float activate(float v, int act) {
  if (act == 2) return v / (1.0f + expf(-v));
  if (act == 1) {
    v = fmaxf(v, 0.0f);
    return v * v;
  }
  return v;
}

template <int NE, bool BIAS, bool NV, bool GATED>
__global__ __launch_bounds__(kThreads) void k_tokens_up(TokensArgs a) {
  __shared__ int ids[kTokensMaxPairs];
  __shared__ float gates[kTokensMaxPairs];
  __shared__ int cnt[kMaxExperts];
  __shared__ int act_e[kTokensMaxPairs], act_n[kTokensMaxPairs], act_0[kTokensMaxPairs];
  __shared__ int where[kMaxExperts];
  __shared__ int16_t list[kTokensMaxPairs];
  __shared__ int wave_a[kWavesT], wave_n[kWavesT];
  __shared__ float red[kWavesT][GATED ? 2 : 1][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int pairs = a.T * a.k;

  for (int t = wave; t < a.T; t += kWavesT) {
    int id;
    float gate;
    select<NE, BIAS>(a, t, id, gate);
    if (lane < a.k) {
      ids[t * a.k + lane] = id;
      gates[t * a.k + lane] = gate;
      if (blockIdx.x == 0) {
        a.topk_ids[t * a.k + lane] = id;
        a.gate[t * a.k + lane] = gate;
      }
    }
  }
  if (tid < a.n_local) cnt[tid] = 0;
  __syncthreads();
  // the pairs of each local expert; the order inside an expert is arbitrary
  // (a pair is a column of its own: no result depends on it)
  int le = -1, pos = 0;
  if (tid < pairs) {
    le = ids[tid] - a.e0;
    if (ids[tid] < 0 || le < 0 || le >= a.n_local) le = -1;
    if (le >= 0) pos = atomicAdd(&cnt[le], 1);
  }
  __syncthreads();
  const int c = tid < a.n_local ? cnt[tid] : 0;
  const uint64_t some = __ballot(c > 0);
  int incl = c;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(incl, d, 64);
    if (lane >= d) incl += u;
  }
  if (lane == 63) {
    wave_a[wave] = __popcll(some);
    wave_n[wave] = incl;
  }
  __syncthreads();
  int na = 0, a0 = 0, n0 = 0;
#pragma unroll
  for (int i = 0; i < kWavesT; ++i) {
    a0 += i < wave ? wave_a[i] : 0;
    n0 += i < wave ? wave_n[i] : 0;
    na += wave_a[i];
  }
  if (c > 0) {
    const int at = a0 + __popcll(some & ~(~0ull << lane));
    act_e[at] = tid;
    act_n[at] = c;
    act_0[at] = n0 + incl - c;
    where[tid] = at;
  }
  __syncthreads();
  if (le >= 0) list[act_0[where[le]] + pos] = (int16_t)tid;
  __syncthreads();

  // the table of the second kernel, a part from each workgroup
  TokensTable* tab = reinterpret_cast<TokensTable*>(a.ws);
  if (blockIdx.x == 0 && tid == 0) tab->n_active = na;
  for (int i = (int)blockIdx.x + (int)gridDim.x * wave; i < na; i += (int)gridDim.x * kWavesT) {
    int p = -1;
    for (int j = 0; j < act_n[i]; ++j) {
      const int q = list[act_0[i] + j];
      if (q / a.k == lane) p = q;
    }
    tab->pair[i][lane] = (int16_t)p;
    if (lane == 0) tab->expert[i] = act_e[i];
  }

  const int slices = (int)(a.F / 16);
  const int64_t units = (int64_t)na * slices;
  const int r = lane & 15, g = lane >> 4;
  const int64_t K = a.K, F = a.F;
  const int chunks = (int)(K / 128);
  constexpr int M = GATED ? 2 : 1;
  const int64_t srow = K / (NV ? 16 : 32);
  uint16_t* hhi = reinterpret_cast<uint16_t*>(a.ws + kTableBytes);
  uint16_t* hlo = hhi + (int64_t)pairs * F;
  const int64_t u1 = units * ((int64_t)blockIdx.x + 1) / gridDim.x;
  for (int64_t u = units * (int64_t)blockIdx.x / gridDim.x; u < u1; ++u) {
    const int ai = (int)(u / slices), sl = (int)(u % slices);
    const int e = act_e[ai], n = act_n[ai], first = act_0[ai];
    for (int t0 = 0; t0 < n; t0 += 16) {
      const int p = list[first + (t0 + r < n ? t0 + r : n - 1)];
      const uint16_t* xr = static_cast<const uint16_t*>(a.x) + (int64_t)(p / a.k) * K;
      f32x4 acc[M];
#pragma unroll
      for (int m = 0; m < M; ++m) acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int ch = wave; ch < chunks; ch += kWavesT) {
        bf16x8 b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          b[q] = *reinterpret_cast<const bf16x8*>(xr + ch * 128 + 32 * g + 8 * q);
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const int64_t row = (int64_t)e * (M * F) + m * F + sl * 16 + r;
          const u32x4v w = *reinterpret_cast<const u32x4v*>(a.w1_codes + row * (K / 2) + ch * 64 + 16 * g);
          bf16x8 f[4];
          dequant<NV>(w, load_scale<NV>(a.w1_scales + row * srow, ch, g), f);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[q], b[q], acc[m], 0, 0, 0);
        }
      }
#pragma unroll
      for (int m = 0; m < M; ++m) *reinterpret_cast<f32x4*>(&red[wave][m][lane * 4]) = acc[m];
      __syncthreads();
      if (wave == 0) {
        f32x4 v[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          v[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < kWavesT; ++i) v[m] += *reinterpret_cast<const f32x4*>(&red[i][m][lane * 4]);
        }
        if (t0 + r < n) {
          const float o1 = NV ? a.w1_outer[e] : 1.0f;
          const float go = gates[p] * (NV ? a.w2_outer[e] : 1.0f);
          float h[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            h[i] = activate(v[0][i] * o1, a.act);
            if constexpr (GATED) h[i] *= v[M - 1][i] * o1;
            h[i] *= go;
          }
          const uint32_t h01 = pk_bf16(h[0], h[1]), h23 = pk_bf16(h[2], h[3]);
          lo[0] = h[0] - u2f(h01 << 16);
          lo[1] = h[1] - u2f(h01 & 0xFFFF0000u);
          lo[2] = h[2] - u2f(h23 << 16);
          lo[3] = h[3] - u2f(h23 & 0xFFFF0000u);
          const int64_t at = (int64_t)p * F + sl * 16 + 4 * g;
          *reinterpret_cast<uint2*>(hhi + at) = make_uint2(h01, h23);
          *reinterpret_cast<uint2*>(hlo + at) = make_uint2(pk_bf16(lo[0], lo[1]), pk_bf16(lo[2], lo[3]));
        }
      }
      __syncthreads();
    }
  }
}

template <bool NV>
__global__ __launch_bounds__(kThreads) void k_tokens_down(TokensArgs a) {
  __shared__ int16_t pair[kTokensMaxPairs][kTokensMaxT];
  __shared__ int expert[kTokensMaxPairs];
  __shared__ float red[kWavesT][256];
  const TokensTable* tab = reinterpret_cast<const TokensTable*>(a.ws);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int na = tab->n_active;
  for (int i = tid; i < na; i += kThreads) expert[i] = tab->expert[i];
  for (int i = tid; i < na * kTokensMaxT / 8; i += kThreads)
    reinterpret_cast<uint4*>(pair)[i] = reinterpret_cast<const uint4*>(tab->pair)[i];
  __syncthreads();
  const int64_t K = a.K, F = a.F;
  const int chunks = (int)(F / 128);
  const int64_t srow = F / (NV ? 16 : 32);
  const uint16_t* hhi = reinterpret_cast<const uint16_t*>(a.ws + kTableBytes);
  const uint16_t* hlo = hhi + (int64_t)a.T * a.k * F;
  const int64_t c0 = (int64_t)blockIdx.x * 16;
  const int nt = (a.T + 15) / 16;
  f32x4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = wave; j < na * chunks; j += kWavesT) {
    const int ai = j / chunks, ch = j % chunks;
    const int64_t row = (int64_t)expert[ai] * K + c0 + r;
    const u32x4v w = *reinterpret_cast<const u32x4v*>(a.w2_codes + row * (F / 2) + ch * 64 + 16 * g);
    bf16x8 f[4];
    dequant<NV>(w, load_scale<NV>(a.w2_scales + row * srow, ch, g), f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= nt) break;
      const int p = pair[ai][16 * i + r];
      if (__ballot(p >= 0) == 0) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        u32x4v bh = {0, 0, 0, 0}, bl = {0, 0, 0, 0};
        if (p >= 0) {
          const int64_t at = (int64_t)p * F + ch * 128 + 32 * g + 8 * q;
          bh = *reinterpret_cast<const u32x4v*>(hhi + at);
          bl = *reinterpret_cast<const u32x4v*>(hlo + at);
        }
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[q], __builtin_bit_cast(bf16x8, bl), acc[i], 0, 0, 0);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[q], __builtin_bit_cast(bf16x8, bh), acc[i], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= nt) break;
    *reinterpret_cast<f32x4*>(&red[wave][lane * 4]) = acc[i];
    __syncthreads();
    if (wave == 0) {
      f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int q = 0; q < kWavesT; ++q) v += *reinterpret_cast<const f32x4*>(&red[q][lane * 4]);
      const int t = 16 * i + r;
      if (t < a.T) {
        const int64_t at = (int64_t)t * K + c0 + 4 * g;
        if (a.out_bf16)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
              make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
        else
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = v;
      }
    }
    __syncthreads();
  }
}

template <int NE, bool BIAS>
void up(const TokensArgs& a, unsigned grid, hipStream_t stream) {
  const bool nv = a.w1_outer != nullptr;
  auto k = nv ? (a.gated ? k_tokens_up<NE, BIAS, true, true> : k_tokens_up<NE, BIAS, true, false>)
              : (a.gated ? k_tokens_up<NE, BIAS, false, true> : k_tokens_up<NE, BIAS, false, false>);
  k<<<grid, kThreads, 0, stream>>>(a);
}

}  // namespace

size_t tokens_workspace_bytes(int64_t T, int k, int64_t F) {
  return kTableBytes + (size_t)(T * k * F) * 4;
}

hipError_t launch_ffn_tokens(const TokensArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  const int64_t most = a.T * a.k < a.n_local ? a.T * a.k : a.n_local;   // experts selected at most
  int64_t grid = most * (a.F / 16);
  if (grid > device_cu_count()) grid = device_cu_count();
  const bool bias = a.bias != nullptr;
  if (a.E <= 64) bias ? up<1, true>(a, grid, stream) : up<1, false>(a, grid, stream);
  else if (a.E <= 384) bias ? up<6, true>(a, grid, stream) : up<6, false>(a, grid, stream);
  else bias ? up<16, true>(a, grid, stream) : up<16, false>(a, grid, stream);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned cols = (unsigned)(a.K / 16);
  if (a.w1_outer) k_tokens_down<true><<<cols, kThreads, 0, stream>>>(a);
  else k_tokens_down<false><<<cols, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4moe
