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

}  // namespace

hipError_t launch_fwd_mxfp4(const uint8_t* ac, const uint8_t* as, int64_t a_rows,
                            const int32_t* row_token, const uint8_t* bc, const uint8_t* bs,
                            const int64_t* offsets, int G, int64_t m_cap, int64_t N, int64_t K,
                            void* y, bool y_bf16, hipStream_t stream) {
  const int64_t tiles = ((m_cap + 31) / 32 + G) * (N / 128);
  auto k = y_bf16 ? k_mxfp4_small<true> : k_mxfp4_small<false>;
  k<<<(unsigned)tiles, 256, 0, stream>>>(ac, as, a_rows, row_token, bc, bs, offsets, G, N, K, y);
  return hipGetLastError();
}

}  // namespace nvfp4moe
