// Global 2-norm of a list of gradients, and the gradients scaled to it, for gfx950.
//
//   s = sum over all tensors of g^2 (binary64),  norm = sqrt(s),
//   c = RN32(min(1, max_norm / (norm + 1e-6))),  g' = RN32(g c), rounded once more for 16 bits
//
// (the rounding to binary32 moves a 16-bit result by at most 2^-24 of its value besides its own
// half step; one rounding of the 32- to 35-bit product would take binary64 or a correction step).
//
// Both passes are bound by memory.  The tensors' addresses travel in the kernel arguments
// (kPerLaunch tensors per launch), so a call needs no table in device memory, no copy from
// the host and no synchronization, and can be captured.  A block takes one chunk of
// kChunk elements of one tensor.  The sum of squares keeps one binary64 partial per block
// (workspace), added in a fixed order: the result does not depend on the schedule.
#include "device_common.h"
#include "intlora_internal.h"

namespace intlora {
namespace {

enum { D_BF16 = 0, D_FP16 = 1, D_FP32 = 2 };

constexpr int kPerLaunch = 112;     // 112 x 32 bytes of entries: under the 4 KB of kernel arguments
constexpr int kChunk = 16384;       // elements per block
constexpr int kThreads = 256;
constexpr int kSmallChunks = 16;    // at most so many chunks are summed by one block
constexpr int64_t kMaxTensors = 65536;

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

struct Entry {
  const void* src;
  void* dst;
  int64_t numel;
  int32_t chunk0;  // first chunk of the tensor within the launch
  int32_t dtype;
};

struct Table {
  int32_t count, chunks;
  int64_t partial0;  // index of the launch's first partial sum
  Entry t[kPerLaunch];
};
static_assert(sizeof(Table) + 64 <= 4096, "kernel arguments are limited to 4 KB");

// The entry that chunk c belongs to (entries have ascending chunk0): the lanes look at all
// entries at once, where a binary search would be seven dependent loads.
__device__ __forceinline__ int find_entry(const Table& t, int c) {
  const int lane = threadIdx.x & 63;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kPerLaunch; i += 64)
    n += __builtin_popcountll(
        __builtin_amdgcn_ballot_w64(i + lane < t.count && t.t[i + lane < kPerLaunch ? i + lane : 0].chunk0 <= c));
  return n - 1;
}

template <int D>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if (D == D_FP32) return static_cast<const float*>(p)[i];
  if (D == D_FP16) return (float)static_cast<const _Float16*>(p)[i];
  return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}

// The 16 bytes of a vector as floats: 4 (fp32) or 8.
template <int D>
__device__ __forceinline__ void widen(u4 r, float* v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (D == D_FP32) {
      v[e] = __uint_as_float(r[e]);
    } else if (D == D_FP16) {
      const uint32_t bits = (uint32_t)r[e];
      const h2 x = __builtin_bit_cast(h2, bits);
      v[2 * e] = (float)x.x;
      v[2 * e + 1] = (float)x.y;
    } else {
      v[2 * e] = __uint_as_float(r[e] << 16);
      v[2 * e + 1] = __uint_as_float(r[e] & 0xFFFF0000u);
    }
  }
}

template <int D>
__device__ __forceinline__ double sum_chunk(const void* src, int64_t i0, int64_t i1) {
  constexpr int V = D == D_FP32 ? 4 : 8;
  const int tid = threadIdx.x & (kThreads - 1);
  double s = 0.0;
  const int64_t full = i0 + (i1 - i0) / V * V;
  const u4* p = reinterpret_cast<const u4*>(static_cast<const uint8_t*>(src) + i0 * (D == D_FP32 ? 4 : 2));
  const int nv = (int)((full - i0) / V);
  for (int b = tid; b < nv; b += 8 * kThreads) {
    u4 r[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) r[u] = b + u * kThreads < nv ? p[b + u * kThreads] : u4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      float v[V];
      widen<D>(r[u], v);
#pragma unroll
      for (int e = 0; e < V; ++e) s = fma((double)v[e], (double)v[e], s);
    }
  }
  const int64_t i = full + tid;
  if (i < i1) {
    const double v = (double)load1<D>(src, i);
    s = fma(v, v, s);
  }
  return s;
}

__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
  return s;
}

// 168 M elements of fp32 in 448 tensors: 4 launches of 37 us, 4.5 TB/s (part of it from the
// last-level cache); the scaling pass 62 us each, 5.4 TB/s read and written.
__global__ void __launch_bounds__(kThreads) k_grad_sumsq(const Table t, double* __restrict__ partial) {
  __shared__ double w[4];
  const int c = blockIdx.x;
  const Entry& e = t.t[find_entry(t, c)];
  const int64_t i0 = (int64_t)(c - e.chunk0) * kChunk;
  const int64_t i1 = i0 + kChunk < e.numel ? i0 + kChunk : e.numel;
  double s;
  if (e.dtype == D_FP32)
    s = sum_chunk<D_FP32>(e.src, i0, i1);
  else if (e.dtype == D_FP16)
    s = sum_chunk<D_FP16>(e.src, i0, i1);
  else
    s = sum_chunk<D_BF16>(e.src, i0, i1);
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) partial[t.partial0 + c] = (w[0] + w[1]) + (w[2] + w[3]);
}

// Small lists: one block takes all chunks, in order, and writes the sum itself, one launch less
// (a call on 8 chunks 13.2 us, on 16 16.0, on 17, in two launches, 16.2; alone this kernel takes 6.0
// us for 12 tensors of 56 k elements, the other two 4.2 and 1.8).
__global__ void __launch_bounds__(1024) k_grad_sumsq_small(const Table t, double* __restrict__ sumsq) {
  __shared__ double w[16];
  const int sub = threadIdx.x >> 8;  // four chunks at a time
  double s = 0.0;
  for (int c = sub; c < t.chunks; c += 4) {
    const Entry& e = t.t[__builtin_amdgcn_readfirstlane(find_entry(t, c))];
    const int64_t i0 = (int64_t)(c - e.chunk0) * kChunk;
    const int64_t i1 = i0 + kChunk < e.numel ? i0 + kChunk : e.numel;
    if (e.dtype == D_FP32)
      s += sum_chunk<D_FP32>(e.src, i0, i1);
    else if (e.dtype == D_FP16)
      s += sum_chunk<D_FP16>(e.src, i0, i1);
    else
      s += sum_chunk<D_BF16>(e.src, i0, i1);
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double r = 0.0;
    for (int k = 0; k < 16; ++k) r += w[k];
    sumsq[0] = r;
  }
}

__global__ void __launch_bounds__(1024) k_grad_total(const double* __restrict__ partial, int64_t n,
                                                     double* __restrict__ sumsq) {
  __shared__ double w[16];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 8 * 1024) {  // eight loads in flight
    double v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = i + u * 1024 < n ? partial[i + u * 1024] : 0.0;
#pragma unroll
    for (int u = 0; u < 8; ++u) s += v[u];
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double r = 0.0;
    for (int k = 0; k < 16; ++k) r += w[k];
    sumsq[0] = r;
  }
}

template <int D>
__device__ __forceinline__ void clip_chunk(const void* src, void* dst, int64_t i0, int64_t i1, float c) {
  constexpr int V = D == D_FP32 ? 4 : 8;
  constexpr int EB = D == D_FP32 ? 4 : 2;
  const int tid = threadIdx.x;
  const int nv = (int)((i1 - i0) / V);
  const u4* p = reinterpret_cast<const u4*>(static_cast<const uint8_t*>(src) + i0 * EB);
  u4* o = reinterpret_cast<u4*>(static_cast<uint8_t*>(dst) + i0 * EB);
  for (int b = tid; b < nv; b += 8 * kThreads) {
    u4 r[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (b + u * kThreads < nv) r[u] = p[b + u * kThreads];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (b + u * kThreads >= nv) break;
      float v[V];
      widen<D>(r[u], v);
      u4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (D == D_FP32)
          y[e] = __float_as_uint(v[e] * c);
        else if (D == D_FP16)
          y[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){v[2 * e] * c, v[2 * e + 1] * c}, h2));
        else
          y[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){v[2 * e] * c, v[2 * e + 1] * c}, bf2));
      }
      o[b + u * kThreads] = y;
    }
  }
  const int64_t i = i0 + (int64_t)nv * V + tid;
  if (i < i1) {
    const float y = load1<D>(src, i) * c;
    if (D == D_FP32)
      static_cast<float*>(dst)[i] = y;
    else if (D == D_FP16)
      static_cast<_Float16*>(dst)[i] = (_Float16)y;
    else
      static_cast<__bf16*>(dst)[i] = (__bf16)y;
  }
}

__global__ void __launch_bounds__(kThreads) k_grad_clip(const Table t, const double* __restrict__ sumsq,
                                                        double max_norm, float* __restrict__ norm_out) {
  const double norm = sqrt(sumsq[0]);
  const double q = max_norm / (norm + 1e-6);
  const float coef = q < 1.0 ? (float)q : (q != q ? (float)q : 1.0f);  // a NaN norm passes on
  if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) norm_out[0] = (float)norm;
  if (t.chunks == 0) return;
  // last chunk first: what the sum of squares read last is still in the last-level cache
  const int c = t.chunks - 1 - (int)blockIdx.x;
  const Entry& e = t.t[find_entry(t, c)];
  if (coef == 1.0f && e.src == e.dst) return;  // nothing to change in place
  const int64_t i0 = (int64_t)(c - e.chunk0) * kChunk;
  const int64_t i1 = i0 + kChunk < e.numel ? i0 + kChunk : e.numel;
  if (e.dtype == D_FP32)
    clip_chunk<D_FP32>(e.src, e.dst, i0, i1, coef);
  else if (e.dtype == D_FP16)
    clip_chunk<D_FP16>(e.src, e.dst, i0, i1, coef);
  else
    clip_chunk<D_BF16>(e.src, e.dst, i0, i1, coef);
}

int64_t chunks_of(int64_t numel) { return (numel + kChunk - 1) / kChunk; }

// Fills a table from tensor `i` on (empty tensors are left out); returns the next tensor.
int64_t fill(Table& t, int64_t i, int64_t count, const void* const* src, void* const* dst, const int64_t* numel,
             const int32_t* dtype) {
  t.count = 0;
  t.chunks = 0;
  for (; i < count && t.count < kPerLaunch; ++i) {
    if (numel[i] == 0) continue;
    const int64_t c = chunks_of(numel[i]);
    if (t.count > 0 && t.chunks + c > 0x7FFFFFFF) break;
    Entry& e = t.t[t.count++];
    e.src = src[i];
    e.dst = dst ? dst[i] : nullptr;
    e.numel = numel[i];
    e.chunk0 = t.chunks;
    e.dtype = dtype[i];
    t.chunks += (int32_t)c;
  }
  return i;
}

}  // namespace

size_t grad_ws_bytes(int64_t count, const int64_t* numel) {
  int64_t c = 0;
  for (int64_t i = 0; i < count; ++i) c += chunks_of(numel[i]);
  return (size_t)(c < 2 ? 2 : c) * 8;
}

hipError_t launch_grad_sumsq(int64_t count, const void* const* src, const int64_t* numel, const int32_t* dtype,
                             double* sumsq, void* ws, hipStream_t st) {
  Table t;
  double* partial = static_cast<double*>(ws);
  int64_t done = 0;
  for (int64_t i = 0; i < count;) {
    i = fill(t, i, count, src, nullptr, numel, dtype);
    if (t.count == 0) break;
    t.partial0 = done;
    if (done == 0 && i == count && t.chunks <= kSmallChunks) {
      k_grad_sumsq_small<<<1, 1024, 0, st>>>(t, sumsq);
      return hipGetLastError();
    }
    k_grad_sumsq<<<dim3((unsigned)t.chunks), kThreads, 0, st>>>(t, partial);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    done += t.chunks;
  }
  k_grad_total<<<1, 1024, 0, st>>>(partial, done, sumsq);
  return hipGetLastError();
}

hipError_t launch_grad_clip(int64_t count, const void* const* src, void* const* dst, const int64_t* numel,
                            const int32_t* dtype, const double* sumsq, double max_norm, float* norm, hipStream_t st) {
  Table t;
  t.partial0 = 0;
  // where the launches' tensors begin; the last ones first (see k_grad_clip)
  static_assert(kMaxTensors / kPerLaunch < 640, "launches of the longest list");
  int64_t begin[640];
  int launches = 0;
  for (int64_t i = 0; i < count;) {
    begin[launches] = i;
    i = fill(t, i, count, src, dst, numel, dtype);
    if (t.count > 0) ++launches;
  }
  if (launches == 0) {
    t.count = t.chunks = 0;
    if (norm == nullptr) return hipSuccess;
    k_grad_clip<<<1, kThreads, 0, st>>>(t, sumsq, max_norm, norm);
    return hipGetLastError();
  }
  for (int k = launches - 1; k >= 0; --k) {
    fill(t, begin[k], count, src, dst, numel, dtype);
    k_grad_clip<<<dim3((unsigned)t.chunks), kThreads, 0, st>>>(t, sumsq, max_norm, k == 0 ? norm : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace intlora
