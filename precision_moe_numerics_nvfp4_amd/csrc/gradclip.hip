// The global norm of a list of gradients and their clipping by it.
//
//   sumsq = sum over tensors and elements of g^2 (64-bit products and sums: no
//           overflow or lost small terms whatever the gradients' scale);
//   out   = g * min(1, max_norm / (sqrt(sumsq) + 1e-6)).
//
// Both passes stream: the tensors are cut into chunks of 16384 elements, each
// workgroup takes a contiguous run of chunks of the whole list, so a list of
// many small tensors and one of a few large ones both fill the device. The
// list travels in the kernel arguments (no copy to the device, nothing to keep
// alive), up to kTable tensors a launch.
#include "codecs.hpp"
#include "internal.hpp"

namespace nvfp4moe {

namespace {

constexpr int kTable = 96;              // tensors per launch: 2.9 KB of arguments
constexpr int kChunkElems = 16384;
constexpr int kThreads = 256;
constexpr int kMaxParts = 2048;         // workgroups, so partial sums, per launch

struct GradTable {
  const void* in[kTable];
  void* out[kTable];
  int64_t numel[kTable];
  uint32_t first[kTable + 1];           // the tensor's first chunk; [n]: all chunks
  uint8_t bf16[kTable];
  int n;
};

// Sum over the 256 threads of the workgroup, in a fixed order (thread 0 has it).
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double sh[kThreads / 64];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) s += sh[i];
  return s;
}

// The tensor that chunk c lies in: the last one whose first chunk is not past c.
__device__ __forceinline__ int table_find(const GradTable& t, uint32_t c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double sq(float v, double acc) {
  const double d = (double)v;
  return __fma_rn(d, d, acc);
}

__global__ __launch_bounds__(kThreads) void k_grad_sumsq(GradTable t, uint32_t per,
                                                         double* __restrict__ parts) {
  const uint32_t all = t.first[t.n];
  const uint32_t c0 = blockIdx.x * per, c1 = c0 + per < all ? c0 + per : all;
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  int j = table_find(t, c0);
  for (uint32_t c = c0; c < c1; ++c) {
    while (t.first[j + 1] <= c) ++j;
    const int64_t at = (int64_t)(c - t.first[j]) * kChunkElems;
    const int64_t left = t.numel[j] - at;
    const int len = left < kChunkElems ? (int)left : kChunkElems;
    const bool wide = (reinterpret_cast<uintptr_t>(t.in[j]) & 15u) == 0;
    if (t.bf16[j]) {
      const uint16_t* p = static_cast<const uint16_t*>(t.in[j]) + at;
      int done = 0;
      if (wide) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
        const int nq = len / 8;
        for (int i = threadIdx.x; i < nq; i += kThreads) {
          const uint4 v = q[i];
          acc[0] = sq(u2f(v.x << 16), acc[0]);
          acc[1] = sq(u2f(v.x & 0xFFFF0000u), acc[1]);
          acc[2] = sq(u2f(v.y << 16), acc[2]);
          acc[3] = sq(u2f(v.y & 0xFFFF0000u), acc[3]);
          acc[0] = sq(u2f(v.z << 16), acc[0]);
          acc[1] = sq(u2f(v.z & 0xFFFF0000u), acc[1]);
          acc[2] = sq(u2f(v.w << 16), acc[2]);
          acc[3] = sq(u2f(v.w & 0xFFFF0000u), acc[3]);
        }
        done = nq * 8;
      }
      for (int i = done + threadIdx.x; i < len; i += kThreads) acc[0] = sq(bf16_to_f32(p[i]), acc[0]);
    } else {
      const float* p = static_cast<const float*>(t.in[j]) + at;
      int done = 0;
      if (wide) {
        const float4* q = reinterpret_cast<const float4*>(p);
        const int nq = len / 4;
        for (int i = threadIdx.x; i < nq; i += kThreads) {
          const float4 v = q[i];
          acc[0] = sq(v.x, acc[0]);
          acc[1] = sq(v.y, acc[1]);
          acc[2] = sq(v.z, acc[2]);
          acc[3] = sq(v.w, acc[3]);
        }
        done = nq * 4;
      }
      for (int i = done + threadIdx.x; i < len; i += kThreads) acc[0] = sq(p[i], acc[0]);
    }
  }
  const double s = block_sum((acc[0] + acc[1]) + (acc[2] + acc[3]));
  if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void k_grad_join(const double* __restrict__ parts, int n,
                                                        double* __restrict__ sumsq) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += parts[i];
  s = block_sum(s);
  if (threadIdx.x == 0) *sumsq = s;
}

__global__ __launch_bounds__(kThreads) void k_grad_clip(GradTable t, uint32_t per,
                                                        const double* __restrict__ sumsq,
                                                        float max_norm, float* __restrict__ norm) {
  const double root = sqrt(*sumsq);
  const double share = (double)max_norm / (root + 1e-6);
  const float coef = share >= 1.0 ? 1.0f : (float)share;     // a NaN norm stays NaN
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)root;
  if (t.n == 0) return;
  const uint32_t all = t.first[t.n];
  const uint32_t c0 = blockIdx.x * per, c1 = c0 + per < all ? c0 + per : all;
  int j = table_find(t, c0);
  for (uint32_t c = c0; c < c1; ++c) {
    while (t.first[j + 1] <= c) ++j;
    if (coef == 1.0f && t.out[j] == t.in[j]) continue;        // in place and within the bound
    const int64_t at = (int64_t)(c - t.first[j]) * kChunkElems;
    const int64_t left = t.numel[j] - at;
    const int len = left < kChunkElems ? (int)left : kChunkElems;
    const bool wide = ((reinterpret_cast<uintptr_t>(t.in[j]) |
                        reinterpret_cast<uintptr_t>(t.out[j])) & 15u) == 0;
    if (t.bf16[j]) {
      const uint16_t* p = static_cast<const uint16_t*>(t.in[j]) + at;
      uint16_t* o = static_cast<uint16_t*>(t.out[j]) + at;
      int done = 0;
      if (wide) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
        uint4* r = reinterpret_cast<uint4*>(o);
        const int nq = len / 8;
        for (int i = threadIdx.x; i < nq; i += kThreads) {
          const uint4 v = q[i];
          uint4 y;
          y.x = pk_bf16(u2f(v.x << 16) * coef, u2f(v.x & 0xFFFF0000u) * coef);
          y.y = pk_bf16(u2f(v.y << 16) * coef, u2f(v.y & 0xFFFF0000u) * coef);
          y.z = pk_bf16(u2f(v.z << 16) * coef, u2f(v.z & 0xFFFF0000u) * coef);
          y.w = pk_bf16(u2f(v.w << 16) * coef, u2f(v.w & 0xFFFF0000u) * coef);
          r[i] = y;
        }
        done = nq * 8;
      }
      for (int i = done + threadIdx.x; i < len; i += kThreads)
        o[i] = (uint16_t)pk_bf16(bf16_to_f32(p[i]) * coef, 0.0f);
    } else {
      const float* p = static_cast<const float*>(t.in[j]) + at;
      float* o = static_cast<float*>(t.out[j]) + at;
      int done = 0;
      if (wide) {
        const float4* q = reinterpret_cast<const float4*>(p);
        float4* r = reinterpret_cast<float4*>(o);
        const int nq = len / 4;
        for (int i = threadIdx.x; i < nq; i += kThreads) {
          float4 v = q[i];
          v.x *= coef; v.y *= coef; v.z *= coef; v.w *= coef;
          r[i] = v;
        }
        done = nq * 4;
      }
      for (int i = done + threadIdx.x; i < len; i += kThreads) o[i] = p[i] * coef;
    }
  }
}

// Tensors [at, at + ...) of the list, empty ones left out; returns the first
// one that the next launch takes.
int fill_table(GradTable& t, int at, const void* const* grads, void* const* outs,
               const int* dtypes, const int64_t* numels, int n) {
  uint32_t chunks = 0;                  // below 2^31: the C ABI bounds the elements and tensors
  t.n = 0;
  for (; at < n && t.n < kTable; ++at) {
    if (numels[at] == 0) continue;
    t.in[t.n] = grads[at];
    t.out[t.n] = outs ? outs[at] : nullptr;
    t.numel[t.n] = numels[at];
    t.bf16[t.n] = dtypes[at] == 1;
    t.first[t.n] = chunks;
    chunks += (uint32_t)((numels[at] + kChunkElems - 1) / kChunkElems);
    ++t.n;
  }
  t.first[t.n] = chunks;
  return at;
}

uint32_t per_workgroup(uint32_t chunks, int64_t most) {
  return (uint32_t)((chunks + most - 1) / most);
}

}  // namespace

size_t grad_workspace_bytes(int n) {
  return (size_t)(n / kTable + 2) * kMaxParts * sizeof(double);
}

hipError_t launch_grad_sumsq(const void* const* grads, const int* dtypes, const int64_t* numels,
                             int n, double* sumsq, void* workspace, hipStream_t stream) {
  double* parts = static_cast<double*>(workspace);
  int used = 0;
  for (int at = 0; at < n;) {
    GradTable t;
    at = fill_table(t, at, grads, nullptr, dtypes, numels, n);
    if (t.n == 0) break;
    const uint32_t chunks = t.first[t.n];
    const uint32_t per = per_workgroup(chunks, kMaxParts);
    const unsigned grid = (chunks + per - 1) / per;
    k_grad_sumsq<<<grid, kThreads, 0, stream>>>(t, per, parts + used);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    used += (int)grid;
  }
  k_grad_join<<<1, kThreads, 0, stream>>>(parts, used, sumsq);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const void* const* grads, void* const* outs, const int* dtypes,
                            const int64_t* numels, int n, const double* sumsq, float max_norm,
                            float* norm, hipStream_t stream) {
  int at = 0;
  do {
    GradTable t;
    at = fill_table(t, at, grads, outs, dtypes, numels, n);
    if (t.n == 0 && norm == nullptr) break;
    const uint32_t chunks = t.n ? t.first[t.n] : 0;
    const uint32_t per = chunks ? per_workgroup(chunks, kMaxParts) : 1;
    const unsigned grid = chunks ? (chunks + per - 1) / per : 1;
    k_grad_clip<<<grid, kThreads, 0, stream>>>(t, per, sumsq, max_norm, norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    norm = nullptr;                       // the first launch writes it
  } while (at < n);
  return hipSuccess;
}

}  // namespace nvfp4moe
