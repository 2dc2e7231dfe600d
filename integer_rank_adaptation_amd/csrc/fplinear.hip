// Floating-point linear layers for gfx950: the 8-bit layer with one power-of-two scale per
// block of 128, and products grouped by expert (8-bit, bf16, fp16) with their gradients: the
// quantizers, and the launches of the products in gemm_tile.h.
#include "gemm_tile.h"

namespace intlora {

namespace {

// ------------------------------------------------------------------------ quantizers
// Scale exponent of a block whose largest magnitude has the binary32 bits `top`: the least
// e >= -127 with top 2^-e <= 448 = 1.75 x 2^8, so the exponent of `top` less 8, one more
// when its significand is above 1.75; 0 for an empty block.  Returned as the E8M0 byte
// e + 127; 255 (NaN) for a block that holds a NaN or an infinity.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return 255u;
  if (top == 0) return 127u;
  const int f = (int)(top >> 23);
  const int e = f - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // subnormals land below -127
  return (uint32_t)((e < -127 ? -127 : e) + 127);
}

// 2^-e for that byte (a normal binary32 for every e in [-127, 120]).
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Four values to e4m3 codes, x 2^-e exact, one rounding (half to even).
__device__ __forceinline__ uint32_t cvt4(float a, float b, float c, float d) {
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return (uint32_t)r;
}

// Eight elements of type TI.
template <int TI>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if (TI == T_FP32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = s[0], b = s[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const v4i r = *reinterpret_cast<const v4i*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (TI == T_BF16) {
        v[2 * e] = __uint_as_float((uint32_t)r[e] << 16);
        v[2 * e + 1] = __uint_as_float((uint32_t)r[e] & 0xFFFF0000u);
      } else {
        const uint32_t bits = (uint32_t)r[e];
        const h2 x = __builtin_bit_cast(h2, bits);
        v[2 * e] = (float)x.x;
        v[2 * e + 1] = (float)x.y;
      }
    }
  }
}

__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
    m = b > m ? b : m;
  }
  return m;
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], uint32_t byte) {
  if (byte == 255u) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float s = inv_scale(byte);
  return make_uint2(cvt4(v[0] * s, v[1] * s, v[2] * s, v[3] * s), cvt4(v[4] * s, v[5] * s, v[6] * s, v[7] * s));
}

// Activations: 16 lanes take one block of 1 x 128 (8 elements each); the largest magnitude
// goes round the 16 lanes as integer bits, so a NaN wins.  Bound by memory: 8192 x 14336 bf16
// 64 us, 5.5 TB/s (two or four blocks per 16 lanes with their loads together: the same or
// slower, and 0.3 to 1.4 us more at 64 x 4096).
template <int TI>
__global__ void __launch_bounds__(256) k_fp8_act(uint32_t units, uint32_t n, uint32_t nb, uint32_t lds,
                                                 const void* __restrict__ X, uint8_t* __restrict__ xq,
                                                 uint8_t* __restrict__ sx) {
  const uint32_t l = threadIdx.x & 15;
  const uint32_t u = blockIdx.x * 16 + (threadIdx.x >> 4);
  if (u >= units) return;  // whole groups of 16 lanes leave together
  const uint32_t row = u / nb, b = u - row * nb, k = 128 * b + 8 * l;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (k < n) load8<TI>(X, (int64_t)row * n + k, v);
  uint32_t m = amax8(v);
#pragma unroll
  for (int s = 8; s; s >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)m, s, 16);
    m = o > m ? o : m;
  }
  const uint32_t byte = scale_byte(m);
  if (k < n) *reinterpret_cast<uint2*>(xq + (int64_t)row * n + k) = codes8(v, byte);
  if (l == 0 || (b == nb - 1 && b + l < lds))  // and the bytes that pad the row
    sx[(int64_t)row * lds + b + l] = (uint8_t)(l == 0 ? byte : 127u);
}

// Weights: one block of 128 x 128 per workgroup, and, when asked for, the same codes
// transposed (through LDS) for the input gradient's product.  Bound by memory: 14336 x 4096 bf16
// 35 us, 5.0 TB/s; with the transpose 44 us, 5.3 TB/s.
template <int TI>
__global__ void __launch_bounds__(256) k_fp8_weight(int d, int n, int lds, int lds_t, const void* __restrict__ W,
                                                    uint8_t* __restrict__ wq, uint8_t* __restrict__ sw,
                                                    uint8_t* __restrict__ wt, uint8_t* __restrict__ swt) {
  __shared__ uint32_t top[4];
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * 132];
  const int tid = threadIdx.x, l = tid & 15, r0 = tid >> 4;
  const int64_t e = blockIdx.z;
  const int i0 = blockIdx.y * 128, k0 = blockIdx.x * 128, k = k0 + 8 * l;
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int i = i0 + r0 + 16 * q;
#pragma unroll
    for (int c = 0; c < 8; ++c) v[q][c] = 0.f;
    if (i < d && k < n) load8<TI>(W, (e * d + i) * n + k, v[q]);
    const uint32_t o = amax8(v[q]);
    m = o > m ? o : m;
  }
#pragma unroll
  for (int s = 32; s; s >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)m, s);
    m = o > m ? o : m;
  }
  if ((tid & 63) == 0) top[tid >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) m = top[w] > m ? top[w] : m;
  const uint32_t byte = scale_byte(m);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int r = r0 + 16 * q;
    const uint2 c = codes8(v[q], byte);
    if (i0 + r < d && k < n) *reinterpret_cast<uint2*>(wq + (e * d + i0 + r) * n + k) = c;
    if (wt != nullptr) {
      *reinterpret_cast<uint32_t*>(tile + r * 132 + 8 * l) = c.x;
      *reinterpret_cast<uint32_t*>(tile + r * 132 + 8 * l + 4) = c.y;
    }
  }
  const int nb = gridDim.x, db = gridDim.y;
  if (tid < 4) {  // this block's scale, and in the last block of a row the bytes that pad it
    const int b = (int)blockIdx.x + tid;
    if (tid == 0 || ((int)blockIdx.x == nb - 1 && b < lds))
      sw[(e * db + blockIdx.y) * lds + b] = (uint8_t)(tid == 0 ? byte : 127u);
    if (wt != nullptr) {
      const int bt = (int)blockIdx.y + tid;
      if (tid == 0 || ((int)blockIdx.y == db - 1 && bt < lds_t))
        swt[(e * nb + blockIdx.x) * lds_t + bt] = (uint8_t)(tid == 0 ? byte : 127u);
    }
  }
  if (wt == nullptr) return;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 8; ++q) {  // row k0 + c of the transpose: 8 codes per lane
    const int c = r0 + 16 * q;
    if (k0 + c >= n || i0 + 8 * l >= d) continue;
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int x = 0; x < 8; ++x) o[x >> 2] |= (uint32_t)tile[(8 * l + x) * 132 + c] << (8 * (x & 3));
    *reinterpret_cast<uint2*>(wt + (e * n + k0 + c) * d + i0 + 8 * l) = make_uint2(o[0], o[1]);
  }
}

}  // namespace

int fp8_scale_stride(int64_t n) { return (int)(4 * ((n + 511) / 512)); }

hipError_t launch_fp8_quant_act(int64_t M, int64_t n, int dtype, const void* X, uint8_t* xq, uint8_t* sx,
                                hipStream_t st) {
  const uint32_t nb = (uint32_t)((n + 127) / 128), lds = (uint32_t)fp8_scale_stride(n);
  // A grid holds less than 2^32 work-items, so less than 2^28 blocks of 16 each: rows past those
  // take another launch (from 2^28 rows of up to 128 columns on).
  const int64_t most = ((int64_t(1) << 28) - 16) / nb, eb = dtype == T_FP32 ? 4 : 2;
  for (int64_t row = 0; row < M; row += most) {
    const uint32_t units = (uint32_t)((M - row < most ? M - row : most) * nb);
    const dim3 grid((units + 15) / 16);
    const uint8_t* x = static_cast<const uint8_t*>(X) + row * n * eb;
    uint8_t *q = xq + row * n, *s = sx + row * lds;
    if (dtype == T_FP32)
      k_fp8_act<T_FP32><<<grid, 256, 0, st>>>(units, (uint32_t)n, nb, lds, x, q, s);
    else if (dtype == T_FP16)
      k_fp8_act<T_FP16><<<grid, 256, 0, st>>>(units, (uint32_t)n, nb, lds, x, q, s);
    else
      k_fp8_act<T_BF16><<<grid, 256, 0, st>>>(units, (uint32_t)n, nb, lds, x, q, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_fp8_quant_weight(int64_t E, int64_t d, int64_t n, int dtype, const void* W, uint8_t* wq,
                                   uint8_t* sw, uint8_t* wt, uint8_t* swt, hipStream_t st) {
  const int lds = fp8_scale_stride(n), lds_t = fp8_scale_stride(d);
  const dim3 grid((unsigned)((n + 127) / 128), (unsigned)((d + 127) / 128), (unsigned)E);
  if (dtype == T_FP32)
    k_fp8_weight<T_FP32><<<grid, 256, 0, st>>>((int)d, (int)n, lds, lds_t, W, wq, sw, wt, swt);
  else if (dtype == T_FP16)
    k_fp8_weight<T_FP16><<<grid, 256, 0, st>>>((int)d, (int)n, lds, lds_t, W, wq, sw, wt, swt);
  else
    k_fp8_weight<T_BF16><<<grid, 256, 0, st>>>((int)d, (int)n, lds, lds_t, W, wq, sw, wt, swt);
  return hipGetLastError();
}

hipError_t launch_fp8_linear(int64_t M, int64_t E, int64_t d, int64_t n, const uint8_t* xq, const uint8_t* sx,
                             const int64_t* offsets, const uint8_t* wq, const uint8_t* sw, uint16_t* Y,
                             hipStream_t st) {
  GemmArgs a{};
  a.A = xq;
  a.B = wq;
  a.C = Y;
  a.sa = sx;
  a.sb = sw;
  a.offsets = offsets;
  a.T = (int)M;
  a.E = (int)E;
  a.cols = (int)d;
  a.kdim = (int)n;
  a.lds = fp8_scale_stride(n);
  return run_gemm<T_FP8, L_NT, T_BF16>(a, st);
}

hipError_t launch_grouped(int direction, int64_t M, int64_t E, int64_t d, int64_t n, int dtype, int out_dtype,
                          const void* tokens, const int64_t* offsets, const void* other, void* out, hipStream_t st) {
  GemmArgs a{};
  a.A = static_cast<const uint8_t*>(tokens);
  a.B = static_cast<const uint8_t*>(other);
  a.C = out;
  a.offsets = offsets;
  a.T = (int)M;
  a.E = (int)E;
  if (direction == kGroupedFwd) {
    a.cols = (int)d;
    a.kdim = (int)n;
    return dtype == T_BF16 ? run_gemm<T_BF16, L_NT, T_BF16>(a, st) : run_gemm<T_FP16, L_NT, T_FP16>(a, st);
  }
  if (direction == kGroupedDx) {
    a.cols = (int)n;
    a.kdim = (int)d;
    return dtype == T_BF16 ? run_gemm<T_BF16, L_NN, T_BF16>(a, st) : run_gemm<T_FP16, L_NN, T_FP16>(a, st);
  }
  a.rows = (int)d;
  a.cols = (int)n;
  if (out_dtype == T_FP32)
    return dtype == T_BF16 ? run_gemm<T_BF16, L_TN, T_FP32>(a, st) : run_gemm<T_FP16, L_TN, T_FP32>(a, st);
  return dtype == T_BF16 ? run_gemm<T_BF16, L_TN, T_BF16>(a, st) : run_gemm<T_FP16, L_TN, T_FP16>(a, st);
}

}  // namespace intlora
