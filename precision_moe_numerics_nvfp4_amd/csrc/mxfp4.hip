// MXFP4 quantization of rows, and MXFP4 / MXFP8 back to values.
//
// MXFP4 (OCP Microscaling): E2M1 elements with one E8M0 power of two per 32
// consecutive elements of a row. Block exponent: the smallest e with
// max|x_block| <= 6 * 2^e (the rule of the MXFP8 quantizers with E2M1's largest
// value: no element saturates), codes E2M1_RNE(x * 2^-e). The product is exact
// but for results far below half of the smallest code, so the codes do not
// depend on the precision they are computed in.
//
// A row is a whole number of blocks, so the tensor is one run of blocks: four
// lanes to a block, eight consecutive elements each (16 bytes of bfloat16).
#include "codecs.hpp"
#include "internal.hpp"

namespace nvfp4moe {

namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// E8M0 code c = e + 127 of the smallest e with amax <= 6 * 2^e, from amax's
// bits: adding 0x3FFFFF carries into the exponent field exactly when the
// mantissa exceeds 0.5 (6 = 1.5 * 2^2), so c is that field minus 2. Zero and
// subnormal amax give c = 0; finite amax gives c <= 253.
__device__ __forceinline__ uint32_t e8m0_code_e2m1(uint32_t amax_bits) {
  const uint32_t t = (amax_bits + 0x3FFFFFu) >> 23;
  return (t > 2u ? t : 2u) - 2u;
}

// Eight consecutive elements as raw words.
template <bool BF16>
struct Eight {
  static constexpr int W = BF16 ? 4 : 8;
  uint32_t w[W];
};

template <bool BF16>
__device__ __forceinline__ void load8(const void* x, int64_t chunk, Eight<BF16>& r) {
  const uint4* p = static_cast<const uint4*>(x) + chunk * (BF16 ? 1 : 2);
#pragma unroll
  for (int i = 0; i < Eight<BF16>::W / 4; ++i) {
    const uint4 a = ld_stream16(p + i);
    r.w[4 * i] = a.x; r.w[4 * i + 1] = a.y; r.w[4 * i + 2] = a.z; r.w[4 * i + 3] = a.w;
  }
}

// float32 bits of the largest magnitude of the eight.
template <bool BF16>
__device__ __forceinline__ uint32_t amax8(const Eight<BF16>& r) {
  if constexpr (BF16) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    auto mag = [](uint32_t w) { return __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu); };
    const u16x2 m = __builtin_elementwise_max(
        __builtin_elementwise_max(mag(r.w[0]), mag(r.w[1])),
        __builtin_elementwise_max(mag(r.w[2]), mag(r.w[3])));
    return (uint32_t)max(m.x, m.y) << 16;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, r.w[i] & 0x7FFFFFFFu);
    return m;
  }
}

// The eight codes under the block scale `scale` (a float32 whose exponent field
// is the E8M0 code): the scaled conversions round x / scale to nearest, ties to
// the even code, sign kept.
template <bool BF16>
__device__ __forceinline__ uint32_t codes8(const Eight<BF16>& r, float scale) {
  uint32_t w = 0;
  if constexpr (BF16) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    auto v = [&](int i) { return __builtin_bit_cast(bf16x2, r.w[i]); };
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, v(0), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, v(1), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, v(2), scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, v(3), scale, 3);
  } else {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, u2f(r.w[0]), u2f(r.w[1]), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, u2f(r.w[2]), u2f(r.w[3]), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, u2f(r.w[4]), u2f(r.w[5]), scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, u2f(r.w[6]), u2f(r.w[7]), scale, 3);
  }
  return w;
}

// A workgroup's wavefronts take runs of 64 U chunks of eight elements, all loads
// first. The bytes bound it: 262144 x 2048 bfloat16 205 us (1.36 GB, 6.6 TB/s),
// 8002 x 1536 float32 of a buffer of 40009 rows 12 us (56 MB, 4.7 TB/s); U = 2
// (bfloat16) and 1 measured 1 to 3% slower.
template <bool BF16>
__global__ __launch_bounds__(256) void k_mxfp4_quantize(const void* __restrict__ x, int64_t chunks,
                                                        int64_t row_chunks,
                                                        const int64_t* __restrict__ n_live,
                                                        uint32_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
  constexpr int U = BF16 ? 4 : 2;
  if (n_live) {
    const int64_t live = *n_live * row_chunks;
    chunks = live < chunks ? live : chunks;
  }
  const int64_t c0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * (64 * U) + (threadIdx.x & 63);
  Eight<BF16> v[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c0 + 64 * u < chunks) load8<BF16>(x, c0 + 64 * u, v[u]);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = c0 + 64 * u;
    if (c >= chunks) break;              // a block's four lanes are all in or all out
    const uint32_t e = e8m0_code_e2m1(quad_max_bits(amax8<BF16>(v[u])));
    codes[c] = codes8<BF16>(v[u], u2f(e << 23));
    if ((c & 3) == 0) scales[c >> 2] = (uint8_t)e;
  }
}

// 2^(c - 127): a normal float32 but for c = 0 (2^-127).
__device__ __forceinline__ float e8m0_value(uint32_t c) {
  return u2f(c ? c << 23 : 0x00400000u);
}

// Values of E4M3 (MX8) or E2M1 elements, 16 bytes of them a lane and store, so
// that a wavefront's stores are whole lines: N elements, eight of bfloat16 or
// four of float32. The values go past the caches. 40009 x 1536 to float32 (279
// MB): eight elements in two stores 32 bytes apart 64 us, whole lines 56, past
// the caches too 42 (6.6 TB/s).
template <bool MX8, bool BF16>
__global__ __launch_bounds__(256) void k_mx_dequantize(const uint8_t* __restrict__ q,
                                                       const uint8_t* __restrict__ e8,
                                                       int64_t chunks, u32x4_t* __restrict__ out) {
  constexpr int U = 2, N = BF16 ? 8 : 4, QB = MX8 ? N : N / 2;      // bytes of N elements
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const int64_t c0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * (64 * U) + (threadIdx.x & 63);
  u32x2_t w[U];
  uint32_t s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = c0 + 64 * u < chunks ? c0 + 64 * u : chunks - 1;
    if constexpr (QB == 8) w[u] = reinterpret_cast<const u32x2_t*>(q)[c];
    else if constexpr (QB == 4) w[u].x = reinterpret_cast<const uint32_t*>(q)[c];
    else w[u].x = reinterpret_cast<const uint16_t*>(q)[c];
    s[u] = e8[c / (32 / N)];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = c0 + 64 * u;
    if (c >= chunks) break;
    const float scale = e8m0_value(s[u]);
    float v[N];
    if constexpr (MX8) {
#pragma unroll
      for (int h = 0; h < N / 4; ++h) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u][h], false);
        const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u][h], true);
        v[4 * h] = a.x; v[4 * h + 1] = a.y; v[4 * h + 2] = b.x; v[4 * h + 3] = b.y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < N / 2; ++j) e2m1x2_to_f32(w[u].x, j, v[2 * j], v[2 * j + 1]);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = __fmul_rn(v[j], scale);
    u32x4_t o;
    if constexpr (BF16)
      o = u32x4_t{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7])};
    else
      o = u32x4_t{f2u(v[0]), f2u(v[1]), f2u(v[2]), f2u(v[3])};
    __builtin_nontemporal_store(o, out + c);
  }
}

inline unsigned blocks_of(int64_t chunks, int per) { return (unsigned)((chunks + per - 1) / per); }

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, bool bf16, int64_t rows, int64_t cols,
                                 const int64_t* n_live, uint8_t* codes, uint8_t* scales,
                                 hipStream_t stream) {
  const int64_t row_chunks = cols / 8, chunks = rows * row_chunks;
  if (chunks == 0) return hipSuccess;
  uint32_t* q = reinterpret_cast<uint32_t*>(codes);
  if (bf16)
    k_mxfp4_quantize<true><<<blocks_of(chunks, 1024), 256, 0, stream>>>(x, chunks, row_chunks,
                                                                        n_live, q, scales);
  else
    k_mxfp4_quantize<false><<<blocks_of(chunks, 512), 256, 0, stream>>>(x, chunks, row_chunks,
                                                                        n_live, q, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(bool mx8, const uint8_t* q, const uint8_t* e8, int64_t rows,
                                int64_t cols, void* out, bool out_bf16, hipStream_t stream) {
  const int n = out_bf16 ? 8 : 4;            // elements of a chunk
  const int64_t chunks = rows * cols / n;
  auto k = mx8 ? (out_bf16 ? k_mx_dequantize<true, true> : k_mx_dequantize<true, false>)
               : (out_bf16 ? k_mx_dequantize<false, true> : k_mx_dequantize<false, false>);
  // A launch holds less than 2^32 threads, of two chunks each: 2^35 float32 values
  // would take that many. (Four chunks a thread fit, and measured 3 to 8% slower.)
  constexpr int64_t kMost = (int64_t)1 << 31;
  for (int64_t at = 0; at < chunks; at += kMost) {
    const int64_t now = chunks - at < kMost ? chunks - at : kMost;
    k<<<blocks_of(now, 512), 256, 0, stream>>>(q + at * n / (mx8 ? 1 : 2), e8 + at * n / 32, now,
                                               static_cast<u32x4_t*>(out) + at);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace nvfp4moe
