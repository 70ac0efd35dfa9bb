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
//
// What bounds it (MI355X). Large groups: the wait for a stage, of which one at most
// is on its way. Tiles of 256 x 256 on all compute units take 1.72 us a stage (5.0
// PFLOP/s) and 6.3 us each from one to the next (whole rounds of them, contractions
// of 1024 to 8192). One group of 16384, 8192 -> 8192: 500 us (4.4 PFLOP/s), the
// matrix unit busy 71% of the cycles, at 1.76 GHz for the card's power (on zeros,
// whose products cost less, 2.25 GHz and the same cycles). 31596 rows over 48
// groups, 4096 -> 1536: 133 us (2.99 PFLOP/s), busy 42 to 50%: 27.5 us of stages a
// tile beside those 6.3, three and a half rounds in the time of four, the tiles'
// rows filled to 84%; 1536 -> 4096 165 us. Few rows to a group: the weights' bytes,
// 506 rows over 48 groups 45 us for 163 MB (3.6 TB/s; 288 tiles on 256 compute
// units), 1536 -> 4096 40 us (768 tiles, 4.1 TB/s). Short contractions: the output,
// 8 groups of about 1024 rows, 1024 -> 2048, float32, 24 us for 67 MB written after
// four stages a tile.
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

// Gathered activations of 2 GiB and more, past the 32-bit offsets of the tiles
// below: 32 rows x 128 columns per workgroup, a wavefront to 32 columns,
// fragments straight from global memory. Each fragment waits for its loads: rows
// gathered from 1050000 tokens (2.0 GiB) against tiles and 1040000, 4096 -> 1536: 506
// rows over 48 groups 57 us against 34, 8192 over 8 269 against 32, 31596 over 48
// 1088 against 131. So the tiles take all else.
template <bool OUT_BF16>
__global__ __launch_bounds__(256) void k_mxfp4_wide(
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
// A stage is 256 contraction elements: 128 code bytes (a cache line) of each
// row of both operands, by buffer loads with the LDS-destination bit (8 rows an
// instruction; 16-byte piece c of row r at position c ^ piece_key(r)), two
// stages in the ring. The E8M0 bytes come 16 to a row, for two stages, into a
// ring of two such blocks; a wavefront holds its rows' 16 bytes in registers and
// shifts a dword of them to the byte that its half of the lanes needs (the
// instruction's operand select takes byte 0 for the first 64 elements and byte 2
// for the second).
//
// A stage is four steps of 64 elements. The fragments of a step are read from
// LDS under the products of the step before it: A in place, right after a
// fragment's last product, B into the other of two sets. One barrier a stage,
// before its last step: by then every wavefront holds the stage's last
// fragments, so its buffer takes the stage after the next.
constexpr int kWN = 4, kWaves = 2 * kWN;    // 2 x 4 wavefronts of 128 x 64
constexpr int kTN = 2;
constexpr int kBN = 256;                    // columns of a tile
constexpr int kRB = 128;                    // code bytes of a row and stage
constexpr int kStage = 512 * kRB;
constexpr int kScales = 2 * kStage;         // LDS offset of the scale ring
constexpr int kScaleBlock = 512 * 16;
constexpr int kLds = kScales + 2 * kScaleBlock;
constexpr int kBufferWord3 = 0x00020000;    // raw buffer, 32-bit data format
constexpr uint32_t kAway = 0x80000000u;     // past every range: the load gives zeros

typedef __attribute__((address_space(3))) void lds_void;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Rows of 128 bytes: for one piece, 8 consecutive rows land in the 8 distinct
// 16-byte groups of 128 bytes and 16 in the 16 of 256.
__device__ __forceinline__ int piece_key(int r) { return (r & 7) ^ ((r >> 3) & 1); }

__device__ __forceinline__ void* uniform_ptr(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<void*>(((uint64_t)hi << 32) | lo);
}

template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

struct Gemm {
  const uint8_t *ac, *as, *bc, *bs;
  const int32_t* row_token;
  const int64_t* offsets;
  int64_t a_rows, N, K;
  void* y;
  int G;
};

// A tile's place: rows row0 .. row0 + rows - 1 of group g, cols (256, or 128 at
// the end of an odd N / 128) columns from n0.
struct Tile {
  int g, rows, cols;
  int64_t row0, n0;
};

// What a tile's loads need, in registers from before its first load to its
// last. A wavefront's load i fills rows 8 (kWaves i + wave) + lane / 8 of an
// operand, and a lane's piece is the same in all of them.
struct Loads {
  __amdgpu_buffer_rsrc_t ra, rb, rs;        // codes of A and B, scales of the rows it loads
  uint32_t oa[4], ob, ob2, os;              // byte offsets (B: its first and second 128 rows)
  int end;                                  // stage offsets below it are inside the row

  __device__ __forceinline__ void init(const Gemm& p, const Tile& t, int lane, int wave) {
    const uint32_t ldq = (uint32_t)(p.K / 2), lds_ = (uint32_t)(p.K / 32);
    const int64_t a_base = p.row_token ? 0 : t.row0, a_n = p.row_token ? p.a_rows : t.rows;
    const int64_t b_base = (int64_t)t.g * p.N + t.n0;
    auto rsrc = [](const uint8_t* q, int64_t bytes) {
      return __builtin_amdgcn_make_buffer_rsrc(
          uniform_ptr(q), (short)0, (int)__builtin_amdgcn_readfirstlane((uint32_t)bytes),
          kBufferWord3);
    };
    ra = rsrc(p.ac + a_base * ldq, a_n * ldq);
    rb = rsrc(p.bc + b_base * ldq, (int64_t)t.cols * ldq);
    const bool of_a = wave < kWaves / 2;    // 64 rows' scales a wavefront: A's, or B's
    rs = of_a ? rsrc(p.as + a_base * lds_, a_n * lds_)
              : rsrc(p.bs + b_base * lds_, (int64_t)t.cols * lds_);
    // the row of A that tile row r reads, or -1
    auto row_of = [&](int r) -> int64_t {
      if (r >= t.rows) return -1;
      if (!p.row_token) return r;
      const int64_t q = p.row_token[t.row0 + r];
      return q < 0 ? 0 : (q < p.a_rows ? q : p.a_rows - 1);
    };
    const int piece = (lane & 7) ^ piece_key(8 * wave + (lane >> 3));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t q = row_of(8 * (kWaves * i + wave) + (lane >> 3));
      oa[i] = q < 0 ? kAway : (uint32_t)(q * ldq) + 16u * piece;
    }
    ob = (uint32_t)(8 * wave + (lane >> 3)) * ldq + 16u * piece;
    ob2 = t.cols > 128 ? ob : kAway;
    end = (int)ldq - 16 * piece;
    const int r = 64 * (wave % kWN) + lane;
    const int64_t q = of_a ? row_of(r) : r < t.cols ? r : -1;
    os = q < 0 ? kAway : (uint32_t)(q * lds_);
  }
  // Load i of A's codes of stage s, and of B's. The range check covers the
  // vector offset alone, and the scalar one (the place in the row, B's rows)
  // stays inside the operand where that passes; elements past a row's end are
  // zeros.
  __device__ __forceinline__ void a(uint8_t* lsm, int s, int wave, int i) const {
    const uint32_t k = (uint32_t)s * (uint32_t)kRB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        ra, (lds_void*)(lsm + (s & 1) * kStage + (kWaves * i + wave) * 1024), 16,
        (int)k < end ? oa[i] : kAway, k, 0, 0);
  }
  __device__ __forceinline__ void b(uint8_t* lsm, const Gemm& p, int s, int wave, int i) const {
    const uint32_t k = (uint32_t)s * (uint32_t)kRB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rb, (lds_void*)(lsm + (s & 1) * kStage + 256 * kRB + (kWaves * i + wave) * 1024), 16,
        (int)k < end ? (i < 2 ? ob : ob2) : kAway,
        k + (uint32_t)(8 * kWaves * i) * (uint32_t)(p.K / 2), 0, 0);
  }
  // The first loads of a tile: the scales of block 0, the codes of stage 0.
  __device__ __forceinline__ void first(uint8_t* lsm, const Gemm& p, int wave) const {
    scales(lsm, p, 0, wave);
#pragma unroll
    for (int i = 0; i < 4; ++i) a(lsm, 0, wave, i);
#pragma unroll
    for (int i = 0; i < 4; ++i) b(lsm, p, 0, wave, i);
  }
  // The scales of stages 2 b and 2 b + 1 (those behind the row's end are another
  // row's, and are not used).
  __device__ __forceinline__ void scales(uint8_t* lsm, const Gemm& p, int b, int wave) const {
    const bool real = b * 512 < p.K;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rs, (lds_void*)(lsm + kScales + (b & 1) * kScaleBlock + wave * 1024), 16,
        real ? os + 16u * (uint32_t)b : kAway, 0, 0, 0);
  }
};

// The products of a tile of 64 TM rows whose first stage is in LDS and whose
// second stage's loads of A are on their way. A
// wavefront's row block i is block 2 i + wm of the tile (so that the rows of a
// partial tile spread over all of them), its columns the 64 from 64 wn.
template <int TM>
__device__ __forceinline__ void products(uint8_t* lsm, const Gemm& p, const Loads& ld, int lane,
                                         int wave, f32x16 (&acc)[4][kTN]) {
  constexpr int TN = kTN;
  const int wm = wave / kWN, wn = wave % kWN, half = lane >> 5, r32 = lane & 31;
  const int ns = (int)((p.K + 255) / 256);
  // fragment 0's places; fragment i of A sits 64 rows further, of B 32
  const int fa = wm * 32 + r32, fb = wn * (32 * TN) + r32;
  int pa[4], pb[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    pa[s] = fa * kRB + (((2 * s + half) ^ piece_key(fa)) << 4);
    pb[s] = 256 * kRB + fb * kRB + (((2 * s + half) ^ piece_key(fb)) << 4);
  }
  const int qa = kScales + fa * 16, qb = kScales + (256 + fb) * 16;
  u32x4 A[TM], B[2][TN], sA[TM], sB[TN];
  uint32_t ca[TM], cb[TN];
  auto read_a = [&](int i, int s, int step) {
    A[i] = *reinterpret_cast<const u32x4*>(lsm + (s & 1) * kStage + pa[step] + i * 64 * kRB);
  };
  auto read_b = [&](int set, int j, int s, int step) {
    B[set][j] = *reinterpret_cast<const u32x4*>(lsm + (s & 1) * kStage + pb[step] + j * 32 * kRB);
  };
  auto read_sa = [&](int i, int b) {
    sA[i] = *reinterpret_cast<const u32x4*>(lsm + qa + (b & 1) * kScaleBlock + i * 64 * 16);
  };
  auto read_sb = [&](int j, int b) {
    sB[j] = *reinterpret_cast<const u32x4*>(lsm + qb + (b & 1) * kScaleBlock + j * 32 * 16);
  };
  auto wide = [](const u32x4& v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
  };
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    read_a(i, 0, 0);
    read_sa(i, 0);
  }
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    read_b(0, j, 0, 0);
    read_sb(j, 0);
  }

  // The products of step T of a stage, and the reads of the next step's
  // fragments (of the next stage after the last step, and of the next scale
  // block after that block's last stage). load(i) follows the products of row
  // block i.
  auto step = [&](auto at, int s_next, int scale_block, auto load) {
    constexpr int T = decltype(at)::value, S = T & 1, NX = (T + 1) % 4;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      __builtin_amdgcn_sched_barrier(0);    // reads and loads stay where they are written
#pragma unroll
      for (int j = 0; j < TN; ++j)
        // columns first: a lane then holds four consecutive columns of a row
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            wide(B[S][j]), wide(A[i]), acc[i][j], 4, 4, 2 * S, (int)cb[j], 2 * S, (int)ca[i]);
      load(i);
      read_a(i, s_next, NX);
      if (i < TN) read_b(1 - S, i, s_next, NX);
      if constexpr (T == 3)
        if (scale_block >= 0) {
          read_sa(i, scale_block);
          if (i < TN) read_sb(i, scale_block);
        }
    }
#pragma unroll
    for (int j = TM; j < TN; ++j) {
      read_b(1 - S, j, s_next, NX);
      if constexpr (T == 3)
        if (scale_block >= 0) read_sb(j, scale_block);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // Stage 2 b + Q. The loads into the buffer of the stage before it, free since
  // that stage's barrier, follow its products one by one: A's in that stage's
  // last step, B's in this one's first (eight at once hold up all wavefronts).
  auto stage = [&](int b, auto at) {
    constexpr int Q = decltype(at)::value;
    const int s = 2 * b + Q;
    // The scales of half a stage; of a second half behind the row's end 2^-127: the
    // bytes there may be any, and 255 (NaN) times the codes' zeros would be NaN.
    auto shift = [&](int d) {
      const uint32_t real = d % 2 == 0 || 512 * b + 128 * d < (int)p.K ? ~0u : 0u;
#pragma unroll
      for (int i = 0; i < TM; ++i) ca[i] = (sA[i][d] >> (8 * half)) & real;
#pragma unroll
      for (int j = 0; j < TN; ++j) cb[j] = (sB[j][d] >> (8 * half)) & real;
    };
    shift(2 * Q);
    step(std::integral_constant<int, 0>{}, s, -1, [&](int i) {
#pragma unroll
      for (int d = i * 4 / TM; d < (i + 1) * 4 / TM; ++d) ld.b(lsm, p, s + 1, wave, d);
    });
    step(std::integral_constant<int, 1>{}, s, -1, [](int) {});
    shift(2 * Q + 1);
    step(std::integral_constant<int, 2>{}, s, -1, [](int) {});
    wait_barrier<0>();
    if constexpr (Q == 0) ld.scales(lsm, p, b + 1, wave);
    step(std::integral_constant<int, 3>{}, s + 1, Q == 1 ? b + 1 : -1,
         [&](int i) { ld.a(lsm, s + 2, wave, i); });
  };
  const int nb = ns / 2;
  for (int b = 0; b < nb; ++b) {
    stage(b, std::integral_constant<int, 0>{});
    stage(b, std::integral_constant<int, 1>{});
  }
  if (ns & 1) stage(nb, std::integral_constant<int, 0>{});
  wait_barrier<0>();                        // the ring is free
}

// A tile's rows through LDS (the second stage's buffer), a wavefront's 32-row
// blocks one at a time, written 16 bytes a lane along the rows. Float32 rows
// take two halves of a block's columns one after the other.
template <typename OutT, int TM>
__device__ __forceinline__ void store_rows(uint8_t* lsm, const f32x16 (&acc)[4][kTN], int lane,
                                           int wave, int rows, OutT* y, int64_t ld) {
  constexpr int ES = sizeof(OutT), NC = ES == 2 ? kTN : 1;   // 32-column blocks at a time
  constexpr int WC = 32 * NC, RS = WC * ES + 16, PPR = WC * ES / 16;
  static_assert(kWaves * 32 * RS <= kStage, "the staging fits a stage's buffer");
  const int wm = wave / kWN, half = lane >> 5, r32 = lane & 31;
  uint8_t* ep = lsm + kStage + wave * (32 * RS);
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int c0 = 0; c0 < kTN; c0 += NC) {
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint8_t* d = ep + r32 * RS + (j * 32 + 8 * q + 4 * half) * ES;
          const f32x16& v = acc[i][c0 + j];
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
          __builtin_nontemporal_store(
              v, reinterpret_cast<u32x4*>(y + (int64_t)lr * ld + c0 * 32 + c * (16 / ES)));
      }
    }
}

template <typename OutT>
constexpr int kStores = 8 * sizeof(OutT);   // of a wavefront and whole tile: 128 x 64 in 16 bytes a lane

// One workgroup per compute unit. The tiles are split into eight contiguous
// ranges, one per XCD (workgroup w runs on XCD w % 8), whose workgroups take
// theirs a round at a time: those an XCD runs together share rows of both
// operands in its L2. (Lower tiles last, for an even load, measured slower: the
// weights are then read twice.) What does not fill a round goes by halves or
// quarters of its rows (by halves of the columns where there are few rows), where
// that gives no workgroup a second piece, and goes first: behind a whole tile its
// loads would wait for that tile's rows to be written, and at the end of the grid
// most of the card would be idle (8 x 1024 rows, 1024 -> 2048, one round and an
// eighth: uncut 29.5, cut and last 27.5, first 24.0 us; 506 rows over 48 groups
// 48.1 -> 44.8; 16384 x 2, 1024 -> 2048 in float32 86 -> 71; 31000 rows over 48
// groups, three and a half rounds, 134.8 -> 133; nine rounds 166 -> 163.5). The
// loads of a tile's first stage are asked for before the rows of the tile before it
// are written, which then wait for them: the compiler cannot tell the rows' staging
// from the loads' place in LDS.
template <bool OUT_BF16>
__global__ __launch_bounds__(64 * kWaves, 1) void k_mxfp4_tiles(Gemm p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lsm[];
  using OutT = std::conditional_t<OUT_BF16, uint16_t, float>;
  int* pre = reinterpret_cast<int*>(lsm + kLds);
  const int ntn = (int)((p.N + kBN - 1) / kBN);
  tile_prefix(p.G, [&](int e) { return (int)((p.offsets[e + 1] - p.offsets[e] + 255) / 256) * ntn; }, pre);
  const int total = pre[p.G];
  const int x = blockIdx.x & 7, place = blockIdx.x >> 3;
  const int wide = (int)gridDim.x >> 3;     // workgroups on this XCD
  const int first = (int)((int64_t)total * x / 8), n = (int)((int64_t)total * (x + 1) / 8) - first;
  const int whole = n / wide * wide, left = n - whole;
  const int cut = 4 * left <= wide ? 4 : 2 * left <= wide ? 2 : 1;
  // this workgroup's next tile
  int round = 0;
  bool part = place < left * cut;
  auto place_of = [&](int at, int piece, int pieces, Tile& t) {
    at += first;
    t.g = tile_group(pre, p.G, at);
    const int64_t a0 = p.offsets[t.g], a1 = p.offsets[t.g + 1];
    int mi, ni;
    block_order(at - pre[t.g], (int)((a1 - a0 + 255) / 256), ntn, mi, ni);
    t.row0 = a0 + (int64_t)mi * 256;
    t.n0 = (int64_t)ni * kBN;
    t.rows = (int)(a1 - t.row0 < 256 ? a1 - t.row0 : 256);
    t.cols = p.N - t.n0 < kBN ? 128 : kBN;
    if (pieces > 1 && t.rows <= 64) {       // two halves of the columns
      t.n0 += 128 * piece;
      t.cols = piece * 128 < t.cols ? 128 : 0;
    } else if (pieces > 1) {                // of the rows
      const int most = 256 / pieces, from = piece * most;
      t.row0 += from;
      t.rows = t.rows - from < most ? t.rows - from : most;
    }
    return t.rows > 0 && t.cols > 0;
  };
  auto locate = [&](Tile& t) {
    if (part) {
      part = false;
      if (place_of(whole + place / cut, place % cut, cut, t)) return true;
    }
    const int at = round++ * wide + place;
    return at < whole && place_of(at, 0, 1, t);
  };
  Tile t;
  if (!locate(t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Loads ld;
  ld.init(p, t, threadIdx.x & 63, wave);
  ld.first(lsm, p, wave);
  bool stored = false;                      // a whole tile's rows since the first stage's loads
  for (;;) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));          // per tile: nothing derived from it is held across tiles
#pragma unroll
    for (int i = 0; i < 4; ++i) ld.a(lsm, 1, wave, i);
    // the first stage: all but these loads, and the stores between them (of a
    // whole tile; of a partial one some may not have been issued), which go on
    if (stored) wait_barrier<4 + kStores<OutT>>();
    else wait_barrier<4>();
    f32x16 acc[4][kTN];
    const int tm = (t.rows + 63) / 64;
    if (tm == 4) products<4>(lsm, p, ld, lane, wave, acc);
    else if (tm == 3) products<3>(lsm, p, ld, lane, wave, acc);
    else if (tm == 2) products<2>(lsm, p, ld, lane, wave, acc);
    else products<1>(lsm, p, ld, lane, wave, acc);
    const Tile done = t;
    stored = done.rows == 256 && done.cols == kBN;
    const bool more = locate(t);
    if (more) {
      ld.init(p, t, lane, wave);
      ld.first(lsm, p, wave);
    }
    OutT* y = static_cast<OutT*>(p.y) + done.row0 * p.N + done.n0 + (wave % kWN) * (32 * kTN);
    if ((wave % kWN) * (32 * kTN) >= done.cols) {
    } else if (tm == 4) store_rows<OutT, 4>(lsm, acc, lane, wave, done.rows, y, p.N);
    else if (tm == 3) store_rows<OutT, 3>(lsm, acc, lane, wave, done.rows, y, p.N);
    else if (tm == 2) store_rows<OutT, 2>(lsm, acc, lane, wave, done.rows, y, p.N);
    else store_rows<OutT, 1>(lsm, acc, lane, wave, done.rows, y, p.N);
    if (!more) return;
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // the staging is read
  }
}

constexpr size_t kMaxPre = 16128;          // the tile-count scan: G <= 4000

template <bool OUT_BF16>
hipError_t tiles(const Gemm& p, int64_t most, hipStream_t stream) {
  static bool done = false;
  auto k = k_mxfp4_tiles<OUT_BF16>;
  static_assert(kLds + kMaxPre + 256 <= 160 * 1024, "LDS");
  if (!done) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                                       hipFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(kLds + kMaxPre));
    if (e != hipSuccess) return e;
    done = true;
  }
  // a multiple of eight workgroups: every XCD's range has some
  const int64_t cus = device_cu_count() / 8 * 8, upto = (most + 7) / 8 * 8;
  const int64_t grid = upto < cus ? upto : cus;
  const size_t pre = ((size_t)(p.G + 1) * 4 + 15) & ~(size_t)15;
  k<<<(unsigned)grid, 64 * kWaves, kLds + pre, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

// The tiles address the rows they gather by 32 bits, in place a tile's own rows.
bool fwd_mxfp4_wide(bool gathers, int64_t a_rows, int64_t K) {
  return (gathers ? a_rows : 256) * (K / 2) >= (int64_t)1 << 31;
}

hipError_t launch_fwd_mxfp4(const uint8_t* ac, const uint8_t* as, int64_t a_rows,
                            const int32_t* row_token, const uint8_t* bc, const uint8_t* bs,
                            const int64_t* offsets, int G, int64_t m_cap, int64_t N, int64_t K,
                            void* y, bool y_bf16, hipStream_t stream) {
  if (!fwd_mxfp4_wide(row_token != nullptr, a_rows, K)) {
    const Gemm p{ac, as, bc, bs, row_token, offsets, a_rows, N, K, y, G};
    const int64_t most = ((m_cap + 255) / 256 + G) * ((N + kBN - 1) / kBN);
    return y_bf16 ? tiles<true>(p, most, stream) : tiles<false>(p, most, stream);
  }
  const int64_t tiles = ((m_cap + 31) / 32 + G) * (N / 128);
  auto k = y_bf16 ? k_mxfp4_wide<true> : k_mxfp4_wide<false>;
  k<<<(unsigned)tiles, 256, 0, stream>>>(ac, as, a_rows, row_token, bc, bs, offsets, G, N, K, y);
  return hipGetLastError();
}

}  // namespace nvfp4moe
