// The whole expert layer for a few tokens: selection and gates, up-projection,
// activation, down-projection and the weighted sum.
//
//   (ids, gate)[t]  as moe_route
//   h[t, j]   = act(W1[e] x[t]), or act(W1a[e] x[t]) * (W1b[e] x[t]) with e = ids[t, j]
//   out[t]    = sum_j gate[t, j] W2[e] h[t, j]   over the pairs whose expert is local
//
// Weights are 4-bit (MXFP4 or NVFP4) and dequantized in registers; every
// dequantized element (up to 6 significant bits) is exact in bfloat16, so the
// products run on v_mfma_f32_16x16x32_bf16 with the weight rows as A and the
// tokens as B. The activations are not quantized. h (with the gate and W2's outer
// scale in it) is carried between the products as three bfloat16 parts of eight
// bits, which together are the float32 value, each with products of its own. y, a
// row of W2 h per pair, is float32.
//
// Launches: the router's own; up; down; the sum of a token's rows. For a few tokens
// of few experts every workgroup of the first product repeats the selection
// instead, a wavefront to a token.
//
// What bounds it is the weights' bytes in flight: each selected expert's weights
// are read once (a list of pairs at a time), the operations are few. So a
// wavefront holds one piece of its job, 64 rows of 128 or 256 elements, in registers
// while the job's next is on its way (the first piece of its next job is asked for
// with the last of this one, but the join of the sums waits for it: the registers
// are loaded under branches, and what joins behind a branch is copied there), and
// what else has to be read comes in few requests:
// the scales 32 bytes of a row at a time, the columns (tokens or h) a line at a
// time, both by DMA to the wavefront's own LDS (a byte of scale and a fragment of
// column a lane, straight to registers, took as many requests as the weights: 7
// tokens gated 143 us; through registers and LDS 89, where the join of a
// register's two values behind a branch waited for it; by DMA 85.5). Jobs go round
// a grid of one workgroup per compute unit; a job's contraction is split over as
// many wavefronts as gives the fewest steps, joined through LDS.
//
// Measured (MI355X): one token, 8 of 48 experts, 4096 -> 1536 -> 4096, NVFP4, 57
// MB: 31 us, of it up 16.5 (1.7 launch, 3 selection and lists), down 12.8 (the lists
// come a dword a lane, four times one after the other), sum 3.9; 7 tokens, 6 of 48
// experts, gated 4096 -> 2 x 2048 -> 4096, MXFP4, 390 MB: 87 us, 4.5 TB/s; 64 tokens,
// 48 of 384 experts, NVFP4, 240 MB: 69.5 us, 3.5 TB/s (its conversions, four vector
// instructions to two elements, are busy for half of it, the joins of jobs wait for
// the next one's weights, and the rounds of jobs do not come out even); 64 tokens x
// 8 on 48 experts (lists of 16), MXFP4, 118 us, 2.7 TB/s. h in two parts, 16 bits of
// it, measured 30.1, 85.5, 68.2 and 110 us and left float32 results 2.5e-6 from 64
// bits; with three 2.1e-7. Not kept: the last workgroup
// to finish 64 columns adds their rows in the down launch (64 tokens 127 us for
// 72, 7 tokens 96 for 89: every job waits for its rows to reach memory).
#include "codecs.hpp"
#include "internal.hpp"
#include "lanes.hpp"

namespace nvfp4moe {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512;
constexpr int kWavesT = kThreads / 64;
constexpr int kMaxExperts = 1024;
// Where every workgroup of the first product selects by itself; else a launch
// before it does. By itself it saves the launch and pays for rows and experts. The
// layer (1024 -> 512 -> 1024) in a graph, by itself against with the launch: an
// expert a lane, 1 to 8 tokens of 48 experts 19.6 to 20.7 us against 21.5 to 22.4, 16
// tokens 23.2 against 23.0 (with a bias 25.6 against 24.4; of 8 experts, called one
// by one, 20.6 against 21.8), 32 tokens of a larger layer 102 against 98. Six
// experts a lane (384), 1 to 8 tokens 20.6 to 21.8 against 20.5 to 22.4 (called one
// by one 21.0 to 22.2 against 21.8 to 22.8), 12 tokens 24.0 against 21.8, 16 24.5
// against 21.6; with a bias, whose keys take 64 bits, 21.8 to 29.9 against 21.0 to
// 21.9. Sixteen a lane (1024) 21.9 to 30.0 against 21.2 to 22.6.
__host__ __device__ inline bool selects_here(const TokensArgs& a) {
  return a.E <= 64 ? a.T <= 16 : a.E <= 384 && !a.bias && a.T <= 8;
}
constexpr float kNegInfT = -__builtin_huge_valf();
constexpr int kParts = 3;                    // bfloat16 parts of a value of h

// The pairs of the selected local experts in lists of up to COLS, an expert's
// lists next to each other: in LDS, and in the workspace for the second product.
struct Lists {
  int count;
  int16_t expert[kTokensMaxPairs];           // local index, ascending
  int16_t lead[kTokensMaxPairs], lists[kTokensMaxPairs];   // the expert's first list, and how many
  int16_t first[kTokensMaxPairs], n[kTokensMaxPairs];
  int16_t pair[kTokensMaxPairs];             // t k + slot, list by list
  int16_t token[kTokensMaxPairs];            // t
};
constexpr size_t kListBytes = (sizeof(Lists) + 255) / 256 * 256;

// ------------------------------------------------------------- wavefront reductions

template <class T, class Op>
__device__ __forceinline__ T wave_join(T v, Op op) {
  v = op(v, across<0>(v));
  v = op(v, across<1>(v));
  v = op(v, across<2>(v));
  v = op(v, across<3>(v));
  return join_rows(v, op);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  return wave_join(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ uint32_t wave_min(uint32_t v) {
  return wave_join(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_join(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_join(v, [](float a, float b) { return a + b; });
}

// Order-preserving bits of a number that can be selected; 0 for NaN and -inf.
__device__ __forceinline__ uint64_t order_key(double v) {
  if (!(v > -__builtin_huge_val())) return 0;
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v > kNegInfT)) return 0;
  const uint32_t b = f2u(v + 0.0f);        // + 0: -0 is +0, as comparisons have it
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
    top = wave_max(top);
    if (!a.renorm) {
#pragma unroll
      for (int i = 0; i < NE; ++i) denom += x[i] != kNegInfT ? expf(x[i] - top) : 0.0f;
      denom = wave_sum(denom);
    }
  }
  id = -1;
  float v = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    uint32_t bh = hi[0], bl = BIAS ? lo[0] : 0;
    int bi = lane;
    float bx = x[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) {
      bool more = hi[i] > bh;
      if constexpr (BIAS) more = more || (hi[i] == bh && lo[i] > bl);
      bh = more ? hi[i] : bh;
      if constexpr (BIAS) bl = more ? lo[i] : bl;
      bi = more ? lane + 64 * i : bi;
      bx = more ? x[i] : bx;
    }
    const uint32_t mh = wave_max(bh);
    if (mh == 0) break;                      // no expert left
    bool best = bh == mh;
    if constexpr (BIAS) {
      const uint32_t ml = wave_max(best ? bl : 0u);
      best = best && bl == ml;
    }
    uint64_t who = __ballot(best);
    if (who & (who - 1)) {                   // equals: the lowest index
      const int e = (int)wave_min(best ? (uint32_t)bi : 0xFFFFu);
      who = __ballot(best && bi == e);
    }
    const int from = __builtin_ctzll(who);
    const int e = __builtin_amdgcn_readlane(bi, from);
    const float ex = u2f(__builtin_amdgcn_readlane(f2u(bx), from));
    if (lane == j) {
      id = e;
      v = ex;
    }
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
    // renormalised, the softmax's own sum cancels
    s = a.sigmoid ? 1.0f / (1.0f + expf(-v)) : a.renorm ? expf(v - top) : expf(v - top) / denom;
    s = s < 0x1p-126f ? 0.0f : s;
  }
  if (a.renorm) {
    const float total = wave_sum(s);
    s = total == 0.0f ? 0.0f : s / total;
  }
  gate = a.scale * s;
}

// Fragment m of a row's elements 32 g .. 32 g + 31 of a 128-element chunk: their
// 8 m .. 8 m + 7. MXFP4: one scale byte, folded into the conversion. NVFP4: two
// E4M3 scales of 16, the products exact.
template <bool NV>
__device__ __forceinline__ bf16x8 dequant(const u32x4v w, uint32_t s, int m) {
  uint32_t p[4];
  if constexpr (NV) {
    const float sc = m < 2 ? __builtin_amdgcn_cvt_f32_fp8((int)s, 0)
                           : __builtin_amdgcn_cvt_f32_fp8((int)s, 1);
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
  return __builtin_bit_cast(bf16x8, u32x4v{p[0], p[1], p[2], p[3]});
}

__device__ __forceinline__ float activate(float v, int act) {
  if (act == 2) return v / (1.0f + expf(-v));
  if (act == 1) {
    v = v < 0.0f ? 0.0f : v;                 // NaN stays
    return v * v;
  }
  return v;
}

// select() for each token, a wavefront at a time.
template <int NE, bool BIAS>
__device__ __forceinline__ void select_all(const TokensArgs& a, int* ids, float* gates) {
  const int lane = threadIdx.x & 63;
  for (int t = threadIdx.x >> 6; t < a.T; t += kWavesT) {
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
}

// The experts and gates of all tokens (selected here, or read where a launch
// before has them) and the lists of pairs, by a whole workgroup.
template <int COLS>
__device__ __forceinline__ void route(const TokensArgs& a, Lists& l, float* gates) {
  __shared__ int ids[kTokensMaxPairs];
  __shared__ uint32_t members[2][kMaxExperts];               // an expert's tokens, a bit each
  __shared__ int16_t where[kMaxExperts];
  __shared__ int waves[kWavesT];
  static_assert(2 * kThreads >= kMaxExperts && kThreads >= kTokensMaxPairs && kTokensMaxT <= 64,
                "one pass of the threads, a bit for each token");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < kMaxExperts; i += kThreads) members[0][i] = members[1][i] = 0;
  if (!selects_here(a)) {
    if (tid < a.T * a.k) {
      ids[tid] = a.topk_ids[tid];
      gates[tid] = a.gate[tid];
    }
  } else if (a.bias) {
    select_all<1, true>(a, ids, gates);
  } else if (a.E <= 64) {
    select_all<1, false>(a, ids, gates);
  } else {
    select_all<6, false>(a, ids, gates);
  }
  __syncthreads();
  // A token selects an expert at most once: a pair's place in its expert's lists
  // is the number of earlier tokens there, the same in every workgroup.
  const int t = tid / a.k;
  int le = -1;
  if (tid < a.T * a.k) {
    le = ids[tid] - a.e0;
    if (ids[tid] < 0 || le < 0 || le >= a.n_local) le = -1;
    if (le >= 0) atomicOr(&members[t >> 5][le], 1u << (t & 31));
  }
  __syncthreads();
  // thread t: experts 2 t and 2 t + 1; lists and pairs before them in one scan
  auto size = [&](int e) { return __popc(members[0][e]) + __popc(members[1][e]); };
  const int c0 = size(2 * tid), c1 = size(2 * tid + 1);
  const int own = ((c0 + COLS - 1) / COLS + (c1 + COLS - 1) / COLS) << 16 | (c0 + c1);
  int incl = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(incl, d, 64);
    if (lane >= d) incl += u;
  }
  if (lane == 63) waves[wave] = incl;
  __syncthreads();
  int before = incl - own, all = 0;
#pragma unroll
  for (int i = 0; i < kWavesT; ++i) {
    before += i < wave ? waves[i] : 0;
    all += waves[i];
  }
  auto list = [&](int e, int c) {
    const int lead = before >> 16, lists = (c + COLS - 1) / COLS, first = before & 0xFFFF;
    for (int i = 0; i < lists; ++i) {
      l.expert[lead + i] = (int16_t)e;
      l.lead[lead + i] = (int16_t)lead;
      l.lists[lead + i] = (int16_t)lists;
      l.n[lead + i] = (int16_t)min(c - i * COLS, COLS);
      l.first[lead + i] = (int16_t)(first + i * COLS);
    }
    if (c > 0) where[e] = (int16_t)first;
    before += lists << 16 | c;
  };
  list(2 * tid, c0);
  list(2 * tid + 1, c1);
  if (tid == 0) l.count = all >> 16;
  __syncthreads();
  if (le >= 0) {
    const uint32_t m0 = members[0][le], m1 = members[1][le], below = (1u << (t & 31)) - 1;
    const int at = where[le] + (t < 32 ? __popc(m0 & below) : __popc(m0) + __popc(m1 & below));
    l.pair[at] = (int16_t)tid;
    l.token[at] = (int16_t)t;
  }
  __syncthreads();
}

typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* p, uint32_t bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uint64_t)hi << 32 | lo), (short)0,
                                           (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

enum Kind { kUp, kUpGated, kDown };
constexpr int RS = 4;                        // slices of 16 rows in a job (gated: half of each matrix)

// A grid-wide list of jobs, (list of pairs, 16 RF rows of its product): W1 x
// with the activation to h, or W2 h to y.
template <bool NV, Kind KIND, int COLS>
__global__ __launch_bounds__(kThreads) void k_tokens_product(TokensArgs a) {
  constexpr bool DOWN = KIND == kDown, GATED = KIND == kUpGated;
  constexpr int RF = GATED ? RS / 2 : RS;                    // slices of the product
  constexpr int CH = DOWN && COLS > 8 ? 1 : 2;                 // 128-element chunks of a piece
  constexpr int PL = DOWN ? kParts : 1;                      // parts of the other operand
  // Lists of 8 leave half of the matrix unit's 16 columns free: there the first two
  // parts go side by side, the third beside zeros, and the join adds the halves.
  constexpr bool FOLD = DOWN && COLS == 8;
  constexpr int OPS = FOLD ? 2 : PL;                         // operands of a fragment
  constexpr int SB = NV ? 16 : 32;                           // elements of a scale
  // A wavefront's own LDS, filled by DMA. Scales: of its rows, 32 bytes of each at
  // a time (one by one they would take as many requests as the codes). Columns: a
  // piece of all of them, 16-byte part c of column r at c ^ (r & 7).
  constexpr int SChunks = 32 * SB / 128, SQ = RS / 2;
  constexpr int SSteps = SChunks / CH;                       // steps that a block of scales lasts
  constexpr int CBytes = CH * PL * 256, XQ = COLS * CBytes / 1024;
  constexpr int CLanes = CBytes / 16;                        // lanes that hold a column
  static_assert(CH <= 2 && 64 % (16 * CH) == 0 && CLanes % (16 * CH) == 0, "a lane's chunk is the same in all loads");
  struct Own {
    uint8_t scales[RS * 16 * 32];
    uint8_t columns[COLS * CBytes];
  };
  __shared__ Lists l;
  __shared__ float gates[DOWN ? 1 : kTokensMaxPairs];
  __shared__ __attribute__((aligned(16))) Own owns[kWavesT];
  __shared__ f32x4 red[kWavesT][RS][64];
  __shared__ __attribute__((aligned(16))) uint8_t zeros[FOLD ? CH * 256 : 16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int words = (int)(sizeof(Lists) / 4);
  if constexpr (DOWN) {
    if (FOLD && tid < CH * 64) reinterpret_cast<int*>(zeros)[tid] = 0;
    for (int i = tid; i < words; i += kThreads)
      reinterpret_cast<int*>(&l)[i] = reinterpret_cast<const int*>(a.ws)[i];
    __syncthreads();
  } else {
    route<COLS>(a, l, gates);
    if (blockIdx.x == 0)
      for (int i = tid; i < words; i += kThreads)
        reinterpret_cast<int*>(a.ws)[i] = reinterpret_cast<int*>(&l)[i];
  }

  const int r = lane & 15, g = lane >> 4;
  const int64_t L = DOWN ? a.F : a.K, R = DOWN ? a.K : a.F;   // contraction, rows of the product
  const int64_t rows_e = GATED ? 2 * R : R;
  const uint8_t* codes = DOWN ? a.w2_codes : a.w1_codes;
  const uint8_t* scales = DOWN ? a.w2_scales : a.w1_scales;
  uint16_t* h = reinterpret_cast<uint16_t*>(a.ws + kListBytes);    // a plane [T k, F] for each part
  const int64_t plane = (int64_t)a.T * a.k * a.F;
  float* y = reinterpret_cast<float*>(h + kParts * plane);

  const int chunks = (int)(L / 128), groups = (int)(R / (16 * RF)), jobs = l.count * groups;
  if (jobs == 0) return;
  // S = 2^lg wavefronts share a job's contraction, per chunks each in steps of
  // CH; the workgroup has kWavesT / S jobs at once. The split of the fewest
  // steps over all rounds, a round's join counted as half of one.
  int lg = 0;
  float least = __builtin_huge_valf();
  for (int i = 0; 1 << i <= kWavesT && (i == 0 || 1 << (i - 1) < chunks); ++i) {
    const int st = (((chunks + (1 << i) - 1) >> i) + CH - 1) / CH;
    const float turns = ceilf((float)jobs * (1 << i) * __builtin_amdgcn_rcpf((float)(kWavesT * (int)gridDim.x)));
    const float cost = turns * (float)(2 * st + 1);
    if (cost <= least) {
      least = cost;
      lg = i;
    }
  }
  const int jobs_at_once = kWavesT >> lg, mine = wave >> lg;
  const int per = (chunks + (1 << lg) - 1) >> lg, steps = (per + CH - 1) / CH;
  const int c_first = (wave & ((1 << lg) - 1)) * per, c_end = min(c_first + per, chunks);
  const int rounds = (jobs + jobs_at_once - 1) / jobs_at_once;
  const int c_last = c_end > c_first ? c_end - 1 : chunks - 1;     // a step of fewer chunks reads its own again

  Own& own = owns[wave];
  // a job's list and rows; the lists of an expert take turns at the same rows
  auto decode = [&](int j, int& ai, int& group) {
    ai = j / groups;
    group = j % groups;
    const int n = l.lists[ai];
    if (n > 1) {
      const int lead = l.lead[ai], u = j - lead * groups;
      ai = lead + u % n;
      group = u / n;
    }
  };
  u32x4v w[RS][CH];
  // The job that loads are for: uniform bases, and 32 bits of offset a lane.
  const uint32_t w_lane = r * (uint32_t)(L / 2) + 16 * g;
  uint32_t x_lane[XQ];
  int64_t row0 = 0;
  int n_next = 0;
  const uint32_t x_plane = (uint32_t)(DOWN ? a.T * a.k : a.T) * (uint32_t)(2 * L), x_bytes = PL * x_plane;
  auto take = [&](int q) {
    int ai, group;
    decode(min(q * jobs_at_once + mine, jobs - 1), ai, group);
    row0 = uniform(l.expert[ai]) * rows_e + uniform(group) * (16 * RF);
    n_next = uniform(l.n[ai]);
    const int first = uniform(l.first[ai]);
#pragma unroll
    for (int i = 0; i < XQ; ++i) {
      if (i * 64 / CLanes >= n_next) break;
      const int u = i * 64 + lane, col = u / CLanes, at = first + min(col, n_next - 1);
      const int part = (u % CLanes) ^ (col & 7);             // of PL planes, in each a run of 256 bytes a chunk
      x_lane[i] = (uint32_t)(DOWN ? l.pair[at] : l.token[at]) * (uint32_t)(2 * L) + part % 16 * 16 +
                  (uint32_t)(part / (CH * 16)) * x_plane;
    }
  };
  // Its piece of step st. The columns and scales before the codes: loads return
  // in order.
  auto load = [&](int st) {
    const int c0 = min(c_first + st * CH, chunks - 1);
    const auto xr = resource(DOWN ? static_cast<const void*>(h) : a.x, x_bytes);
    // runs of chunks take turns, 16 lanes each; one behind the row's end reads the last again
    const uint32_t x_at = c0 * 256 + (CH > 1 && lane / 16 % 2 && c0 + 1 < chunks ? 256 : 0);
#pragma unroll
    for (int i = 0; i < XQ; ++i) {
      if (i * 64 / CLanes >= n_next) break;
      const uint32_t at = x_lane[i] + x_at;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (lds_void*)(own.columns + i * 1024), 16, at, 0, 0, 0);
    }
    if (st % SSteps == 0) {
      // 16 bytes a lane; what the last rows' reach past the array is not read
      const int64_t at = row0 * (L / SB) + c0 * (128 / SB);
#pragma unroll
      for (int u = 0; u < SQ; ++u) {
        const int64_t base = at + (GATED ? u * R : 32 * u) * (L / SB);
        const int64_t left = (int64_t)a.n_local * rows_e * (L / SB) - base;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            resource(scales + base, (uint32_t)min(left, (int64_t)0x7FFFFFFF)), (lds_void*)(own.scales + u * 1024), 16,
            (lane / 2) * (int)(L / SB) + lane % 2 * 16, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < RS; ++i) {
      const uint8_t* row = codes + (row0 + (GATED ? i / RF * R + 16 * (i % RF) : 16 * i)) * (L / 2);
#pragma unroll
      for (int x = 0; x < CH; ++x)
        w[i][x] = *reinterpret_cast<const u32x4v*>(row + min(c0 + x, c_last) * 64 + w_lane);
    }
  };
  if ((int)blockIdx.x < rounds) {
    take((int)blockIdx.x);
    load(0);
  }
  for (int q = (int)blockIdx.x; q < rounds; q += (int)gridDim.x) {
    const int j = q * jobs_at_once + mine;
    const bool real = j < jobs;
    const int n = n_next;
    f32x4 acc[RS];
#pragma unroll
    for (int i = 0; i < RS; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int st = 0; st < steps; ++st) {
      u32x4v wc[RS][CH];
#pragma unroll
      for (int i = 0; i < RS; ++i) {
#pragma unroll
        for (int x = 0; x < CH; ++x) wc[i][x] = w[i][x];
      }
      const int c0 = c_first + st * CH;
      // the codes are here, and so is what was asked for before them
#pragma unroll
      for (int i = 0; i < RS; ++i)
#pragma unroll
        for (int x = 0; x < CH; ++x) asm volatile("" ::"v"(wc[i][x]) : "memory");
      bf16x8 b[CH][OPS][4];                  // columns past the list: some other's, they go nowhere
      const int col = min(FOLD ? r & 7 : r, n - 1);
#pragma unroll
      for (int x = 0; x < CH; ++x)
#pragma unroll
        for (int u = 0; u < OPS; ++u) {
          const uint8_t* from = own.columns + col * CBytes + u * (CH * 256);
          if constexpr (FOLD) {
            if (u == 0) from += r >= 8 ? CH * 256 : 0;
            else from = r >= 8 ? zeros : own.columns + col * CBytes + 2 * (CH * 256);
          }
#pragma unroll
          for (int m = 0; m < 4; ++m)
            b[x][u][m] = *reinterpret_cast<const bf16x8*>(from + (((x * 16 + g * 4 + m) ^ (col & 7)) << 4));
        }
      uint32_t sc[RS][CH];
#pragma unroll
      for (int i = 0; i < RS; ++i) {
#pragma unroll
        for (int x = 0; x < CH; ++x) {
          const uint8_t* from = own.scales + (16 * i + r) * 32 + (st % SSteps * CH + x) * (128 / SB);
          if constexpr (NV) sc[i][x] = *reinterpret_cast<const uint16_t*>(from + 2 * g);
          else sc[i][x] = from[g];
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // read: free for the next piece's
      if (st + 1 < steps) {
        load(st + 1);
      } else if (q + (int)gridDim.x < rounds) {
        take(q + (int)gridDim.x);
        load(0);
      }
#pragma unroll
      for (int x = 0; x < CH; ++x) {
        if (c0 + x >= c_end || !real) continue;              // loaded to no use
#pragma unroll
        for (int i = 0; i < RS; ++i)
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const bf16x8 f = dequant<NV>(wc[i][x], sc[i][x], m);
#pragma unroll
            for (int u = 0; u < OPS; ++u)
              acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, b[x][u][m], acc[i], 0, 0, 0);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < RS; ++i) red[wave][i][lane] = acc[i];
    __syncthreads();
    // item: four rows of a slice, one column
    for (int it = tid; it < jobs_at_once * RF * 64; it += kThreads) {
      const int li = it & 63, s = it / 64 % RF, jm = it / 64 / RF;
      const int jj = q * jobs_at_once + jm;
      if (jj >= jobs) continue;
      int aj, gj;
      decode(jj, aj, gj);
      const int col = li & 15;
      if (col >= l.n[aj]) continue;
      f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f}, u = v;
      for (int i = 0; i < 1 << lg; ++i) {
        v += red[(jm << lg) + i][s][li];
        if constexpr (FOLD) v += red[(jm << lg) + i][s][li + 8];
        if constexpr (GATED) u += red[(jm << lg) + i][RF + s][li];
      }
      const int e = l.expert[aj], p = l.pair[l.first[aj] + col];
      const int64_t at = p * R + gj * (16 * RF) + 16 * s + 4 * (li >> 4);
      if constexpr (DOWN) {
        *reinterpret_cast<f32x4*>(y + at) = v;
      } else {
        const float o1 = NV ? a.w1_outer[e] : 1.0f;
        const float go = gates[p] * (NV ? a.w2_outer[e] : 1.0f);
        uint32_t part[kParts][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f = activate(v[i] * o1, a.act);
          if constexpr (GATED) f *= u[i] * o1;
          f *= go;
          // the bits cut off are exact in the next part; what is not finite has only a first one
          const bool finite = fabsf(f) < __builtin_huge_valf();
          part[0][i] = finite ? f2u(f) : pk_bf16(f, f);
#pragma unroll
          for (int j = 1; j < kParts; ++j) {
            f = finite ? f - u2f(part[j - 1][i] & 0xFFFF0000u) : 0.0f;
            part[j][i] = f2u(f);
          }
        }
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
          const uint32_t* q = part[j];
          *reinterpret_cast<uint2*>(h + j * plane + at) =
              make_uint2(q[0] >> 16 | (q[1] & 0xFFFF0000u), q[2] >> 16 | (q[3] & 0xFFFF0000u));
        }
      }
    }
    __syncthreads();
  }
}

// out[t] = the sum of y over the token's local pairs, slot by slot. A thread has
// four columns of a token.
__global__ __launch_bounds__(256) void k_tokens_sum(TokensArgs a) {
  const int t = blockIdx.y;
  const int64_t col = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (col >= a.K) return;
  const float* y = reinterpret_cast<const float*>(a.ws + kListBytes + (int64_t)a.T * a.k * a.F * (2 * kParts)) +
                   (int64_t)t * a.k * a.K + col;
  const int32_t* ids = a.topk_ids + (int64_t)t * a.k;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    f32x4 u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = min(j0 + j, a.k - 1);
      const int64_t le = (int64_t)ids[at] - a.e0;
      u[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (j0 + j < a.k && ids[at] >= 0 && le >= 0 && le < a.n_local)
        u[j] = *reinterpret_cast<const f32x4*>(y + at * a.K);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v += u[j];
  }
  const int64_t at = (int64_t)t * a.K + col;
  if (a.out_bf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
  else
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = v;
}

// Lists of 8 pairs leave the second product room for two chunks of weights in
// flight (7 tokens over 48 experts, one pair an expert, 87 us against 91 with
// lists of 16; 16 x 8 over 48 85 against 90; 40 x 8 over 48, 6.7 each, 100 against
// 107). Lists of 16 read a busy expert's weights half as often (64 x 2 over 8, 16
// each, 36 us against 44; 64 x 8 over 48, 10.7 each, 118 against 129).
template <bool NV, Kind KIND>
hipError_t product(const TokensArgs& a, unsigned grid, hipStream_t stream) {
  auto k = a.T * a.k > 7 * a.E ? k_tokens_product<NV, KIND, 16> : k_tokens_product<NV, KIND, 8>;
  k<<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

// The lists, h in bfloat16 parts, y in float32, by pair.
size_t tokens_workspace_bytes(int64_t T, int k, int64_t K, int64_t F) {
  return kListBytes + (size_t)(T * k) * (size_t)(4 * K + 2 * kParts * F);
}

hipError_t launch_ffn_tokens(const TokensArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  hipError_t e = hipSuccess;
  if (!selects_here(a))
    e = launch_route(a.logits, a.logits_bf16, a.T, a.E, a.k, a.sigmoid, a.renorm, a.scale, a.bias,
                     a.token_mask, a.topk_ids, a.gate, nullptr, nullptr, nullptr, stream);
  if (e != hipSuccess) return e;
  const bool nv = a.w1_outer != nullptr;
  const unsigned cus = (unsigned)device_cu_count();
  if (nv) e = a.gated ? product<true, kUpGated>(a, cus, stream) : product<true, kUp>(a, cus, stream);
  else e = a.gated ? product<false, kUpGated>(a, cus, stream) : product<false, kUp>(a, cus, stream);
  if (e != hipSuccess) return e;
  e = nv ? product<true, kDown>(a, cus, stream) : product<false, kDown>(a, cus, stream);
  if (e != hipSuccess) return e;
  k_tokens_sum<<<dim3((unsigned)((a.K / 4 + 255) / 256), (unsigned)a.T), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4moe
