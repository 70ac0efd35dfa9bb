// The global norm of a list of gradients and their clipping by it.
//
//   sumsq = sum over tensors and elements of g^2 (64-bit products and sums: no
//           overflow or lost small terms whatever the gradients' scale);
//   out   = g * min(1, max_norm / (sqrt(sumsq) + 1e-6)), g for an infinite max_norm.
//
// Both passes stream: the tensors are cut into chunks, each workgroup takes a
// contiguous run of chunks of the whole list, so a list of many small tensors
// and one of a few large ones both fill the device. The list travels in the
// kernel arguments (no copy to the device, nothing to keep alive): up to 280
// tensors a launch for the sum, 180 for the scaling, within 4 KiB.
//
// Memory bounds large lists (604M float32 elements: the sum 406 us, 6.0 TB/s,
// the scaling 892 us, 5.4 TB/s, in place or into copies; a copy reaches 5.1; in
// place within the bound 19 us, nothing read), launches the short ones (1.6M
// elements: 3.7 + 2.2 + 4.7 us of kernels).
#include "codecs.hpp"
#include "internal.hpp"

namespace nvfp4moe {

namespace {

constexpr int kSumTable = 280, kClipTable = 180;    // tensors per launch, at most
constexpr int kShortTable = 16;                     // of a short list: 0.4 KB of arguments, not 4
constexpr int kThreads = 256;
constexpr int kMaxParts = 2048;                     // workgroups, so partial sums, per launch
constexpr int kAloneChunks = 8;                     // a list that one workgroup sums
// Chunk sizes, 2^shift elements: the largest one streams with the least
// overhead, smaller ones spread a short list over the compute units.
constexpr int kMinShift = 11, kMaxShift = 14;

template <int N, bool OUT>
struct GradTable {
  const void* in[N];
  void* out[OUT ? N : 1];
  uint32_t first[N + 1];                // the tensor's first chunk; [n]: all chunks
  uint16_t last[N];                     // elements of its last chunk less one; bit 15: bfloat16
  int n, shift;
};

// A run of one tensor's elements.
struct Chunk {
  int j;
  int64_t at;
  int len;
  bool bf16;
};

// Chunk c of the list; j: a tensor at or before it.
template <class Table>
__device__ __forceinline__ Chunk chunk(const Table& t, uint32_t c, int j) {
  while (t.first[j + 1] <= c) ++j;
  const int size = 1 << t.shift;
  const uint32_t last = t.last[j];
  return Chunk{j, (int64_t)(c - t.first[j]) << t.shift,
               c + 1 == t.first[j + 1] ? (int)(last & 0x7FFFu) + 1 : size, (last & 0x8000u) != 0};
}

// The tensor that chunk c lies in: the last one whose first chunk is not past c.
template <class Table>
__device__ __forceinline__ int table_find(const Table& t, uint32_t c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Sum over the 256 threads of the workgroup, in a fixed order (every thread has it).
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

__device__ __forceinline__ double sq(float v, double acc) {
  const double d = (double)v;
  return __fma_rn(d, d, acc);
}

template <bool BF>
__device__ __forceinline__ float element(const void* p, int i) {
  if constexpr (BF) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

template <bool BF>
__device__ __forceinline__ void sq16(const uint4& v, double (&acc)[4]) {
  if constexpr (BF) {
    acc[0] = sq(u2f(v.x << 16), acc[0]);
    acc[1] = sq(u2f(v.x & 0xFFFF0000u), acc[1]);
    acc[2] = sq(u2f(v.y << 16), acc[2]);
    acc[3] = sq(u2f(v.y & 0xFFFF0000u), acc[3]);
    acc[0] = sq(u2f(v.z << 16), acc[0]);
    acc[1] = sq(u2f(v.z & 0xFFFF0000u), acc[1]);
    acc[2] = sq(u2f(v.w << 16), acc[2]);
    acc[3] = sq(u2f(v.w & 0xFFFF0000u), acc[3]);
  } else {
    acc[0] = sq(u2f(v.x), acc[0]);
    acc[1] = sq(u2f(v.y), acc[1]);
    acc[2] = sq(u2f(v.z), acc[2]);
    acc[3] = sq(u2f(v.w), acc[3]);
  }
}

template <bool BF>
__device__ __forceinline__ uint4 scale16(const uint4& v, float c) {
  if constexpr (BF)
    return make_uint4(pk_bf16(u2f(v.x << 16) * c, u2f(v.x & 0xFFFF0000u) * c),
                      pk_bf16(u2f(v.y << 16) * c, u2f(v.y & 0xFFFF0000u) * c),
                      pk_bf16(u2f(v.z << 16) * c, u2f(v.z & 0xFFFF0000u) * c),
                      pk_bf16(u2f(v.w << 16) * c, u2f(v.w & 0xFFFF0000u) * c));
  else
    return make_uint4(f2u(u2f(v.x) * c), f2u(u2f(v.y) * c), f2u(u2f(v.z) * c), f2u(u2f(v.w) * c));
}

// Elements before the first 16-byte boundary, at most len.
template <bool BF>
__device__ __forceinline__ int head_of(const void* p, int len) {
  const int h = (int)((16u - ((uint32_t)reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / (BF ? 2 : 4);
  return h < len ? h : len;
}

constexpr int kFlight = 4;              // 16-byte loads of a thread in flight

template <bool BF>
__device__ __forceinline__ void sum_run(const void* base, int len, double (&acc)[4]) {
  constexpr int per = BF ? 8 : 4;       // elements of 16 bytes
  const int tid = threadIdx.x, head = head_of<BF>(base, len);
  const int nq = (len - head) / per, tail = head + nq * per;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + head * (BF ? 2 : 4));
  int i = tid;
  for (; i + (kFlight - 1) * kThreads < nq; i += kFlight * kThreads) {
    uint4 v[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) v[u] = q[i + u * kThreads];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) sq16<BF>(v[u], acc);
  }
  for (; i < nq; i += kThreads) sq16<BF>(q[i], acc);
  if (tid < head) acc[0] = sq(element<BF>(base, tid), acc[0]);
  if (tid < len - tail) acc[1] = sq(element<BF>(base, tail + tid), acc[1]);
}

template <bool BF>
__device__ __forceinline__ void scale_run(const void* base, void* out, int len, float c) {
  constexpr int per = BF ? 8 : 4;
  const int tid = threadIdx.x;
  const auto put = [&](int i) {
    const float y = element<BF>(base, i) * c;
    if constexpr (BF) static_cast<uint16_t*>(out)[i] = (uint16_t)pk_bf16(y, 0.0f);
    else static_cast<float*>(out)[i] = y;
  };
  // No common 16-byte grid: element by element (64M float32 125 us, where both
  // start one element off the grid 120 and on it 102; bfloat16 53, 57 and 48).
  if (((reinterpret_cast<uintptr_t>(base) ^ reinterpret_cast<uintptr_t>(out)) & 15u) != 0) {
    for (int i = tid; i < len; i += kThreads) put(i);
    return;
  }
  const int head = head_of<BF>(base, len);
  const int nq = (len - head) / per, tail = head + nq * per;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + head * (BF ? 2 : 4));
  uint4* r = reinterpret_cast<uint4*>(static_cast<char*>(out) + head * (BF ? 2 : 4));
  int i = tid;
  for (; i + (kFlight - 1) * kThreads < nq; i += kFlight * kThreads) {
    uint4 v[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) v[u] = ld_stream16(q + i + u * kThreads);
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const uint4 y = scale16<BF>(v[u], c);
      __builtin_nontemporal_store(u32x4_t{y.x, y.y, y.z, y.w},
                                  reinterpret_cast<u32x4_t*>(r + i + u * kThreads));
    }
  }
  for (; i < nq; i += kThreads) r[i] = scale16<BF>(q[i], c);
  if (tid < head) put(tid);
  if (tid < len - tail) put(tail + tid);
}

template <int N>
__global__ __launch_bounds__(kThreads) void k_grad_sumsq(GradTable<N, false> t, uint32_t per,
                                                         double* __restrict__ parts) {
  const uint32_t all = t.first[t.n];
  const uint32_t c0 = blockIdx.x * per, c1 = c0 + per < all ? c0 + per : all;
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  int j = table_find(t, c0);
  for (uint32_t c = c0; c < c1; ++c) {
    const Chunk k = chunk(t, c, j);
    j = k.j;
    if (k.bf16) sum_run<true>(static_cast<const uint16_t*>(t.in[j]) + k.at, k.len, acc);
    else sum_run<false>(static_cast<const float*>(t.in[j]) + k.at, k.len, acc);
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

// Each workgroup goes through its run backwards: what the sum read last is still
// in the 256 MB Infinity Cache (604M float32 elements: 1314 -> 1295 us for both
// passes; non-temporal loads and stores, against plain ones, 1362 -> 1295).
template <int N>
__global__ __launch_bounds__(kThreads) void k_grad_clip(GradTable<N, true> t, uint32_t per,
                                                        const double* __restrict__ sumsq,
                                                        float max_norm, float* __restrict__ norm) {
  const double root = sqrt(*sumsq);
  const double share = (double)max_norm / (root + 1e-6);
  // no bound leaves the gradients as they are, infinite ones too; a NaN norm stays NaN
  const bool whole = share >= 1.0 || (max_norm == __builtin_huge_valf() && root == root);
  const float coef = whole ? 1.0f : (float)share;
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)root;
  if (t.n == 0) return;
  const uint32_t all = t.first[t.n];
  const uint32_t c0 = blockIdx.x * per, c1 = c0 + per < all ? c0 + per : all;
  int j = table_find(t, c1 - 1);
  for (uint32_t c = c1; c-- > c0;) {
    while (t.first[j] > c) --j;
    const Chunk k = chunk(t, c, j);
    if (coef == 1.0f && t.out[j] == t.in[j]) continue;        // in place and within the bound
    if (k.bf16)
      scale_run<true>(static_cast<const uint16_t*>(t.in[j]) + k.at,
                      static_cast<uint16_t*>(t.out[j]) + k.at, k.len, coef);
    else
      scale_run<false>(static_cast<const float*>(t.in[j]) + k.at,
                       static_cast<float*>(t.out[j]) + k.at, k.len, coef);
  }
}

// The chunk size for a list: the smallest whose chunks, two per workgroup,
// still fill kMaxParts workgroups.
int chunk_shift(const int64_t* numels, int n) {
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += numels[i];
  int shift = kMinShift;
  while (shift < kMaxShift && (total >> shift) > 2 * kMaxParts) ++shift;
  return shift;
}

// Tensors [at, ...) of the list, empty ones left out, into one launch's table;
// returns the first one that the next launch takes. Chunks stay below 2^32:
// the C ABI bounds elements and tensors.
template <int N, bool OUT>
int fill_table(GradTable<N, OUT>& t, int shift, int at, const void* const* grads,
               void* const* outs, const int* dtypes, const int64_t* numels, int n) {
  uint32_t chunks = 0;
  t.n = 0;
  t.shift = shift;
  for (; at < n && t.n < N; ++at) {
    if (numels[at] == 0) continue;
    const int64_t whole = (numels[at] - 1) >> shift;           // chunks before the last
    t.in[t.n] = grads[at];
    if constexpr (OUT) t.out[t.n] = outs[at];
    t.first[t.n] = chunks;
    t.last[t.n] = (uint16_t)((numels[at] - 1 - (whole << shift)) | (dtypes[at] == 1 ? 0x8000 : 0));
    chunks += (uint32_t)whole + 1;
    ++t.n;
  }
  t.first[t.n] = chunks;
  return at;
}

uint32_t per_workgroup(uint32_t chunks) { return (chunks + kMaxParts - 1) / kMaxParts; }

int64_t chunks_of(const int64_t* numels, int n, int shift) {
  int64_t all = 0;
  for (int i = 0; i < n; ++i) all += (numels[i] + ((int64_t)1 << shift) - 1) >> shift;
  return all;
}

// A list of a few chunks: one workgroup leaves the sum itself (no partials, and
// a launch fewer of 3.3 us of the host's time).
bool alone(int64_t chunks, int n) { return chunks > 0 && chunks <= kAloneChunks && n <= kShortTable; }

template <int N>
hipError_t sumsq_launches(const void* const* grads, const int* dtypes, const int64_t* numels, int n,
                          int shift, double* sumsq, double* parts, hipStream_t stream) {
  int used = 0;
  for (int at = 0; at < n;) {
    GradTable<N, false> t;
    at = fill_table(t, shift, at, grads, nullptr, dtypes, numels, n);
    if (t.n == 0) break;
    const uint32_t chunks = t.first[t.n];
    if (!parts) {
      k_grad_sumsq<N><<<1, kThreads, 0, stream>>>(t, chunks, sumsq);
      return hipGetLastError();
    }
    const uint32_t per = per_workgroup(chunks);
    const unsigned grid = (chunks + per - 1) / per;
    k_grad_sumsq<N><<<grid, kThreads, 0, stream>>>(t, per, parts + used);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    used += (int)grid;
  }
  k_grad_join<<<1, kThreads, 0, stream>>>(parts, used, sumsq);
  return hipGetLastError();
}

template <int N>
hipError_t clip_launches(const void* const* grads, void* const* outs, const int* dtypes,
                         const int64_t* numels, int n, int shift, const double* sumsq,
                         float max_norm, float* norm, hipStream_t stream) {
  int at = 0;
  do {
    GradTable<N, true> t;
    at = fill_table(t, shift, at, grads, outs, dtypes, numels, n);
    if (t.n == 0 && norm == nullptr) break;
    const uint32_t chunks = t.first[t.n];
    const uint32_t per = chunks ? per_workgroup(chunks) : 1;
    const unsigned grid = chunks ? (chunks + per - 1) / per : 1;
    k_grad_clip<N><<<grid, kThreads, 0, stream>>>(t, per, sumsq, max_norm, norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    norm = nullptr;                       // the first launch writes it
  } while (at < n);
  return hipSuccess;
}

}  // namespace

size_t grad_workspace_bytes(const int64_t* numels, int n) {
  const int64_t chunks = chunks_of(numels, n, chunk_shift(numels, n));
  if (alone(chunks, n)) return 0;
  const int64_t most = (int64_t)(n / kSumTable + 1) * kMaxParts;
  return (size_t)((chunks < most ? chunks : most) + 1) * sizeof(double);
}

hipError_t launch_grad_sumsq(const void* const* grads, const int* dtypes, const int64_t* numels,
                             int n, double* sumsq, void* workspace, hipStream_t stream) {
  const int shift = chunk_shift(numels, n);
  double* parts = alone(chunks_of(numels, n, shift), n) ? nullptr : static_cast<double*>(workspace);
  if (n <= kShortTable)
    return sumsq_launches<kShortTable>(grads, dtypes, numels, n, shift, sumsq, parts, stream);
  return sumsq_launches<kSumTable>(grads, dtypes, numels, n, shift, sumsq, parts, stream);
}

hipError_t launch_grad_clip(const void* const* grads, void* const* outs, const int* dtypes,
                            const int64_t* numels, int n, const double* sumsq, float max_norm,
                            float* norm, hipStream_t stream) {
  const int shift = chunk_shift(numels, n);
  if (n <= kShortTable)
    return clip_launches<kShortTable>(grads, outs, dtypes, numels, n, shift, sumsq, max_norm, norm,
                                      stream);
  return clip_launches<kClipTable>(grads, outs, dtypes, numels, n, shift, sumsq, max_norm, norm,
                                   stream);
}

}  // namespace nvfp4moe
