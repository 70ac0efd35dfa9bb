// MXFP4 forward grouped GEMM on gfx950's block-scaled MFMA.
//
//   Y[r, n] = sum over blocks b of 2^(ea + eb) * sum_{k in b} e2m1_A[row, k] * e2m1_W[g, n, k]
//
// for the rows r of group g, with row = row_token[r] where the activations are
// still in token order. An MXFP4 block (32 E2M1 elements, one power of two) is
// the operand of v_mfma_scale_f32_32x32x64_f8f6f4 as it is stored: each lane
// gives 32 consecutive elements of one row (16 bytes; lanes 0-31 the first
// block of 64, lanes 32-63 the second) and their E8M0 byte. Products of E2M1
// values are multiples of 1/4 up to 36, so a block's sum is exact in the
// matrix unit, and the block sums are added in float32.
#include <type_traits>

#include "codecs.hpp"
#include "internal.hpp"
#include "tiles.hpp"

namespace nvfp4moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ i32x8 frag(const uint4 v) {
  return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// 32 rows x 128 columns per workgroup, a wavefront to 32 columns, fragments
// straight from global memory.
template <bool OUT_BF16>
__global__ __launch_bounds__(256) void k_mxfp4_small(
    const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as, int64_t a_rows,
    const int32_t* __restrict__ row_token, const uint8_t* __restrict__ bc,
    const uint8_t* __restrict__ bs, const int64_t* __restrict__ offsets, int G, int64_t N,
    int64_t K, void* __restrict__ y) {
  const int ntn = (int)(N / 128);
  const TileLoc loc = locate_tile((int)blockIdx.x, G, [&](int e) {
    return (int)((offsets[e + 1] - offsets[e] + 31) / 32) * ntn;
  });
  if (loc.g < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int half = lane >> 5, r32 = lane & 31;
  const int64_t row0 = offsets[loc.g] + (int64_t)(loc.local / ntn) * 32, row_end = offsets[loc.g + 1];
  const int64_t n0 = (int64_t)(loc.local % ntn) * 128 + wave * 32;
  int64_t ra = row0 + r32 < row_end ? row0 + r32 : row0;
  const int64_t r_out = row0 + r32;
  if (row_token) ra = row_token[ra];
  ra = ra < 0 ? 0 : (ra < a_rows ? ra : a_rows - 1);
  const int64_t rb = (int64_t)loc.g * N + n0 + r32;
  const uint8_t* pa = ac + ra * (K / 2) + 16 * half;
  const uint8_t* pb = bc + rb * (K / 2) + 16 * half;
  const uint8_t* sa = as + ra * (K / 32);
  const uint8_t* sb = bs + rb * (K / 32);
  f32x16 acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
  for (int64_t k = 0; k < K; k += 128) {
    const uint32_t xa = *reinterpret_cast<const uint32_t*>(sa + k / 32) >> (8 * half);
    const uint32_t xb = *reinterpret_cast<const uint32_t*>(sb + k / 32) >> (8 * half);
    const uint4 a0 = *reinterpret_cast<const uint4*>(pa + k / 2);
    const uint4 a1 = *reinterpret_cast<const uint4*>(pa + k / 2 + 32);
    const uint4 b0 = *reinterpret_cast<const uint4*>(pb + k / 2);
    const uint4 b1 = *reinterpret_cast<const uint4*>(pb + k / 2 + 32);
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(frag(b0), frag(a0), acc, 4, 4, 0,
                                                          (int)xb, 0, (int)xa);
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(frag(b1), frag(a1), acc, 4, 4, 2,
                                                          (int)xb, 2, (int)xa);
  }
  if (r_out >= row_end) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t at = r_out * N + n0 + 8 * q + 4 * half;
    if constexpr (OUT_BF16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) =
          make_uint2(pk_bf16(acc[4 * q], acc[4 * q + 1]), pk_bf16(acc[4 * q + 2], acc[4 * q + 3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(y) + at) =
          make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
  }
}

// ---------------------------------------------------------------------------
// Large groups: tiles of up to 256 rows x 256 columns through an LDS ring.
//
// A stage is 128 contraction elements: 64 code bytes of each row of both
// operands, by buffer loads with the LDS-destination bit (16 rows an
// instruction; 16-byte piece p of row r at position p ^ chunk_key(r)), four
// stages in the ring. The E8M0 bytes come 16 to a row, for four stages, into
// a ring of two blocks; a wavefront holds its rows' 16 bytes in registers and
// shifts a stage's four to the byte that its half of the lanes needs (the
// instruction's operand select takes byte 0 for the first 64 elements and
// byte 2 for the second).
//
// A stage is two steps of 64 elements. The fragments of a step are read from
// LDS under the products of the step before it: A in place, right after a
// fragment's last product, B into the other of two sets. One barrier a stage,
// between its steps: by then every wavefront holds the stage's last fragments,
// so its buffer takes the stage four further on.
constexpr int kBN = 256;                    // columns of a tile
constexpr int kRing = 4;                    // stages in flight
constexpr int kBufferWord3 = 0x00020000;    // raw buffer, 32-bit data format

typedef __attribute__((address_space(3))) void lds_void;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void* uniform_ptr(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<void*>(((uint64_t)hi << 32) | lo);
}

template <int N, bool LGKM>
__device__ __forceinline__ void wait_barrier() {
  if constexpr (LGKM) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
  else asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

struct Gemm {
  const uint8_t *ac, *as, *bc, *bs;
  const int32_t* row_token;
  const int64_t* offsets;
  int64_t a_rows, N, K;
  void* y;
  int G;
};

// 2 x WN wavefronts; a wavefront's row block i is 2 i + wm (so that the rows of
// a partial tile spread over all of them), its columns BN / WN from wn BN / WN.
template <int WN>
struct Ring {
  static constexpr int NW = 2 * WN;
  static constexpr int STAGE = (256 + kBN) * 64;
  static constexpr int SC = kRing * STAGE;
  static constexpr int SBLK = (256 + kBN) * 16;
  static constexpr int LDS = SC + 2 * SBLK;
  static constexpr int TN = kBN / (32 * WN);
};

template <int TM, int WN, class Store>
__device__ __forceinline__ void tile(uint8_t* lsm, const Gemm& p, int g, int64_t row0, int rows,
                                     int64_t n0, Store store) {
  using R = Ring<WN>;
  constexpr int NW = R::NW, TN = R::TN;
  constexpr int CA = (4 * TM + NW - 1) / NW, CB = 16 / NW;   // code loads of a wavefront and stage
  constexpr int NL = CA + CB, NS = 8 / NW;                   // scale loads of a block
  int tid_ = threadIdx.x;
  asm volatile("" : "+v"(tid_));            // per tile: nothing of it is held across tiles
  const int lane = tid_ & 63, wave = __builtin_amdgcn_readfirstlane(tid_ >> 6);
  const int wm = wave / WN, wn = wave % WN, half = lane >> 5, r32 = lane & 31;
  const uint32_t ldq = (uint32_t)(p.K / 2), lds_ = (uint32_t)(p.K / 32);
  const int ns = (int)(p.K / 128);
  constexpr uint32_t kAway = 0x80000000u;   // past every range: the load gives zeros

  const int64_t a_base = p.row_token ? 0 : row0;
  const int64_t b_base = (int64_t)g * p.N + n0;
  auto rsrc = [](const uint8_t* q, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(q), (short)0,
                                             (int)__builtin_amdgcn_readfirstlane((uint32_t)bytes),
                                             kBufferWord3);
  };
  const int64_t a_n = p.row_token ? p.a_rows : rows;
  const __amdgpu_buffer_rsrc_t ra = rsrc(p.ac + a_base * ldq, a_n * ldq);
  const __amdgpu_buffer_rsrc_t sa = rsrc(p.as + a_base * lds_, a_n * lds_);
  const __amdgpu_buffer_rsrc_t rb = rsrc(p.bc + b_base * ldq, (int64_t)kBN * ldq);
  const __amdgpu_buffer_rsrc_t sb = rsrc(p.bs + b_base * lds_, (int64_t)kBN * lds_);
  // the row of A that tile row r reads, or -1
  auto row_of = [&](int r) -> int64_t {
    if (r >= rows) return -1;
    if (!p.row_token) return r;
    const int64_t t = p.row_token[row0 + r];
    return t < 0 ? 0 : (t < p.a_rows ? t : p.a_rows - 1);
  };
  uint32_t oa[CA], ob[CB], os[NS];
#pragma unroll
  for (int i = 0; i < CA; ++i) {
    const int r = 16 * (NW * i + wave) + (lane >> 2);
    const int64_t t = row_of(r);
    oa[i] = t < 0 ? kAway : (uint32_t)(t * ldq) + (((lane & 3) ^ chunk_key(r)) << 4);
  }
#pragma unroll
  for (int i = 0; i < CB; ++i) {
    const int r = 16 * (NW * i + wave) + (lane >> 2);
    ob[i] = (uint32_t)r * ldq + (((lane & 3) ^ chunk_key(r)) << 4);
  }
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int q = 64 * (NW * i + wave) + lane;               // rows of A, then of B
    const int64_t t = q < 256 ? row_of(q) : 0;
    os[i] = q < 256 ? (t < 0 ? kAway : (uint32_t)(t * lds_)) : (uint32_t)(q - 256) * lds_;
  }
  auto issue = [&](int s) {
    uint8_t* st = lsm + (s & (kRing - 1)) * R::STAGE;
    const bool real = s < ns;
    const uint32_t k = real ? (uint32_t)s * 64u : 0u;
#pragma unroll
    for (int i = 0; i < CA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(st + (NW * i + wave) * 1024), 16,
                                               real ? oa[i] + k : kAway, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < CB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rb, (lds_void*)(st + 256 * 64 + (NW * i + wave) * 1024), 16, real ? ob[i] + k : kAway, 0,
          0, 0);
  };
  auto issue_scales = [&](int b) {
    uint8_t* st = lsm + R::SC + (b & 1) * R::SBLK;
    const bool real = b * 4 < ns;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int w = NW * i + wave;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(w < 4 ? sa : sb, (lds_void*)(st + w * 1024), 16,
                                               real ? os[i] + (uint32_t)b * 16u : kAway, 0, 0, 0);
    }
  };

  // fragment 0's places; fragment i of A sits 64 rows further, of B 32
  const int fa = wm * 32 + r32, fb = wn * (32 * TN) + r32;
  int pa[2], pb[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    pa[s] = fa * 64 + (((2 * s + half) ^ chunk_key(fa)) << 4);
    pb[s] = 256 * 64 + fb * 64 + (((2 * s + half) ^ chunk_key(fb)) << 4);
  }
  const int qa = R::SC + fa * 16, qb = R::SC + (256 + fb) * 16;
  u32x4 A[TM], B[2][TN], sA[TM], sB[TN];
  uint32_t ca[TM], cb[TN];
  auto read_a = [&](int i, int s, int step) {
    A[i] = *reinterpret_cast<const u32x4*>(lsm + (s & (kRing - 1)) * R::STAGE + pa[step] + i * 64 * 64);
  };
  auto read_b = [&](int set, int j, int s, int step) {
    B[set][j] = *reinterpret_cast<const u32x4*>(lsm + (s & (kRing - 1)) * R::STAGE + pb[step] + j * 32 * 64);
  };
  auto wide = [](const u32x4& v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  issue_scales(0);
#pragma unroll
  for (int s = 0; s < kRing; ++s) issue(s);
  wait_barrier<3 * NL, false>();
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    read_a(i, 0, 0);
    sA[i] = *reinterpret_cast<const u32x4*>(lsm + qa + i * 64 * 16);
  }
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    read_b(0, j, 0, 0);
    sB[j] = *reinterpret_cast<const u32x4*>(lsm + qb + j * 32 * 16);
  }

  // the products of one step, and the reads of the next one's fragments
  auto step = [&](auto at, int s_next, int scale_block) {
    constexpr int S = decltype(at)::value;                   // step of the stage
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        // columns first: a lane then holds four consecutive columns of a row
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            wide(B[S][j]), wide(A[i]), acc[i][j], 4, 4, 2 * S, (int)cb[j], 2 * S, (int)ca[i]);
      read_a(i, s_next, 1 - S);
      if (i < TN) {
        read_b(1 - S, i, s_next, 1 - S);
        if constexpr (S == 1)
          if (scale_block >= 0)
            sB[i] = *reinterpret_cast<const u32x4*>(lsm + qb + (scale_block & 1) * R::SBLK + i * 32 * 16);
      }
      if constexpr (S == 1)
        if (scale_block >= 0)
          sA[i] = *reinterpret_cast<const u32x4*>(lsm + qa + (scale_block & 1) * R::SBLK + i * 64 * 16);
    }
    if constexpr (TN > TM) {
#pragma unroll
      for (int j = TM; j < TN; ++j) {
        read_b(1 - S, j, s_next, 1 - S);
        if constexpr (S == 1)
          if (scale_block >= 0)
            sB[j] = *reinterpret_cast<const u32x4*>(lsm + qb + (scale_block & 1) * R::SBLK + j * 32 * 16);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  // Stage s = 4 b + Q. Between its steps everything but the loads of stages
  // s + 2 and s + 3 (and a scale block issued among them) has landed.
  auto stage = [&](int b, auto at) {
    constexpr int Q = decltype(at)::value;
    const int s = 4 * b + Q;
#pragma unroll
    for (int i = 0; i < TM; ++i) ca[i] = sA[i][Q] >> (8 * half);
#pragma unroll
    for (int j = 0; j < TN; ++j) cb[j] = sB[j][Q] >> (8 * half);
    step(S0{}, s, -1);
    wait_barrier<2 * NL + (Q == 1 || Q == 2 ? NS : 0), true>();
    if constexpr (Q == 0) issue_scales(b + 1);
    issue(s + kRing);
    step(S1{}, s + 1, Q == 3 ? b + 1 : -1);
  };
  const int nb = ns / 4;
  for (int b = 0; b < nb; ++b) {
    stage(b, std::integral_constant<int, 0>{});
    stage(b, std::integral_constant<int, 1>{});
    stage(b, std::integral_constant<int, 2>{});
    stage(b, std::integral_constant<int, 3>{});
  }
  const int left = ns - 4 * nb;
  if (left > 0) stage(nb, std::integral_constant<int, 0>{});
  if (left > 1) stage(nb, std::integral_constant<int, 1>{});
  if (left > 2) stage(nb, std::integral_constant<int, 2>{});
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");   // the ring is free

  store(acc, wave, lane);
}

// A tile's rows through LDS, a wavefront's 32-row blocks one at a time, written
// 16 bytes a lane along the rows.
template <typename OutT, int TM, int TN>
__device__ __forceinline__ void store_rows(uint8_t* lsm, const f32x16 (&acc)[TM][TN], int wave,
                                           int lane, int wm, int rows, OutT* y, int64_t ld) {
  constexpr int ES = sizeof(OutT), WC = 32 * TN, RS = WC * ES + 16, PPR = WC * ES / 16;
  const int half = lane >> 5, r32 = lane & 31;
  uint8_t* ep = lsm + wave * (32 * RS);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint8_t* d = ep + r32 * RS + (j * 32 + 8 * q + 4 * half) * ES;
        const f32x16& v = acc[i][j];
        if constexpr (ES == 2)
          *reinterpret_cast<uint2*>(d) = make_uint2(pk_bf16(v[4 * q], v[4 * q + 1]),
                                                    pk_bf16(v[4 * q + 2], v[4 * q + 3]));
        else
          *reinterpret_cast<float4*>(d) =
              make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      }
#pragma unroll
    for (int it = 0; it < 32 * PPR / 64; ++it) {
      const int pc = it * 64 + lane, r = pc / PPR, c = pc % PPR;
      const u32x4 v = *reinterpret_cast<const u32x4*>(ep + r * RS + c * 16);
      const int lr = (2 * i + wm) * 32 + r;
      if (lr < rows)
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(y + (int64_t)lr * ld + c * (16 / ES)));
    }
  }
}

// One workgroup per compute unit, each taking tiles v, v + gridDim.x, ...
template <bool OUT_BF16, int WN>
__global__ __launch_bounds__(128 * WN, 1) void k_mxfp4_tiles(Gemm p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lsm[];
  using R = Ring<WN>;
  using OutT = std::conditional_t<OUT_BF16, uint16_t, float>;
  int* pre = reinterpret_cast<int*>(lsm + R::LDS);
  const int ntn = (int)(p.N / kBN);
  tile_prefix(p.G, [&](int e) { return (int)((p.offsets[e + 1] - p.offsets[e] + 255) / 256) * ntn; }, pre);
  const int total = pre[p.G];
  for (int v = (int)blockIdx.x; v < total; v += (int)gridDim.x) {
    const int x = v & 7, q8 = total >> 3, r8 = total & 7;
    const int t = x * q8 + (x < r8 ? x : r8) + (v >> 3);     // contiguous tiles to an XCD
    const int g = tile_group(pre, p.G, t);
    const int64_t a0 = p.offsets[g], a1 = p.offsets[g + 1];
    int mi, ni;
    block_order(t - pre[g], (int)((a1 - a0 + 255) / 256), ntn, mi, ni);
    const int64_t row0 = a0 + (int64_t)mi * 256;
    const int rows = (int)(a1 - row0 < 256 ? a1 - row0 : 256);
    const int64_t n0 = (int64_t)ni * kBN;
    auto store = [&](const auto& acc, int wave, int lane) {
      store_rows<OutT>(lsm, acc, wave, lane, wave / WN, rows,
                       static_cast<OutT*>(p.y) + row0 * p.N + n0 + (wave % WN) * (32 * R::TN), p.N);
    };
    const int tm = (rows + 63) / 64;
    if (tm == 4) tile<4, WN>(lsm, p, g, row0, rows, n0, store);
    else if (tm == 3) tile<3, WN>(lsm, p, g, row0, rows, n0, store);
    else if (tm == 2) tile<2, WN>(lsm, p, g, row0, rows, n0, store);
    else tile<1, WN>(lsm, p, g, row0, rows, n0, store);
    __syncthreads();                        // the staging is the next tile's ring
  }
}

constexpr size_t kMaxPre = 16128;          // the tile-count scan: G <= 4000

template <bool OUT_BF16, int WN>
hipError_t tiles(const Gemm& p, int64_t most, hipStream_t stream) {
  static bool done = false;
  auto k = k_mxfp4_tiles<OUT_BF16, WN>;
  constexpr size_t lds = Ring<WN>::LDS;
  static_assert(lds + kMaxPre + 256 <= 160 * 1024, "LDS");
  if (!done) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                                       hipFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(lds + kMaxPre));
    if (e != hipSuccess) return e;
    done = true;
  }
  const int64_t grid = most < device_cu_count() ? most : device_cu_count();
  const size_t pre = ((size_t)(p.G + 1) * 4 + 15) & ~(size_t)15;
  k<<<(unsigned)grid, 128 * WN, lds + pre, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fwd_mxfp4(const uint8_t* ac, const uint8_t* as, int64_t a_rows,
                            const int32_t* row_token, const uint8_t* bc, const uint8_t* bs,
                            const int64_t* offsets, int G, int64_t m_cap, int64_t N, int64_t K,
                            void* y, bool y_bf16, hipStream_t stream) {
  const int64_t a_bytes = (row_token ? a_rows : 256) * (K / 2);
  if (N % kBN == 0 && m_cap > 128 * (int64_t)G && a_bytes < (int64_t)1 << 31) {
    const Gemm p{ac, as, bc, bs, row_token, offsets, a_rows, N, K, y, G};
    const int64_t most = ((m_cap + 255) / 256 + G) * (N / kBN);
    return y_bf16 ? tiles<true, 4>(p, most, stream) : tiles<false, 4>(p, most, stream);
  }
  const int64_t tiles = ((m_cap + 31) / 32 + G) * (N / 128);
  auto k = y_bf16 ? k_mxfp4_small<true> : k_mxfp4_small<false>;
  k<<<(unsigned)tiles, 256, 0, stream>>>(ac, as, a_rows, row_token, bc, bs, offsets, G, N, K, y);
  return hipGetLastError();
}

}  // namespace nvfp4moe
