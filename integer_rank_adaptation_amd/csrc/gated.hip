// Gated feed-forward layers and activations saved in 8 bits, for gfx950: the launches of the gated
// products in gemm_tile.h, the gated product's backward, and what reads e4m3 codes in a backward
// pass.
//
//   H = act(G) U,  [G | U] = X_e W_e^T;   dG = dH U act'(G),  dU = dH act(G).
#include "gemm_tile.h"

namespace intlora {

namespace {

// 2^(byte - 127); NaN for the byte 255.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// Four codes of a word as numbers.
__device__ __forceinline__ void codes4(uint32_t w, float s, float* v) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  v[0] = a[0] * s, v[1] = a[1] * s, v[2] = b[0] * s, v[3] = b[1] * s;
}

// A number past fp16's range is the largest of its sign (the code of 65504 is 65536); NaN stays.
template <int TO>
__device__ __forceinline__ float saturate(float v) {
  return TO != T_FP16 || v != v ? v : __builtin_amdgcn_fmed3f(v, -65504.f, 65504.f);
}

// Codes [rows, n] and scale bytes [rows, lds] back to numbers: a product of a code and a power of
// two, exact in binary32, rounded once for a 16-bit type.  16 codes per lane, so that every lane
// loads 16 bytes and a lane's codes have one scale.  Bound by memory: 8192 x 4096 to bf16 22 us
// (101 MB, 4.5 TB/s).
template <int TO>
__global__ void __launch_bounds__(256) k_fp8_restore(uint32_t units, uint32_t per_row, uint32_t lds,
                                                     const uint8_t* __restrict__ q, const uint8_t* __restrict__ sq,
                                                     uint8_t* __restrict__ X) {
  const uint32_t u = blockIdx.x * 256 + threadIdx.x;
  if (u >= units) return;
  const uint32_t row = u / per_row, c = u - row * per_row;
  const u4i w = *reinterpret_cast<const u4i*>(q + (int64_t)u * 16);
  const float s = scale_of(sq[(int64_t)row * lds + (c >> 3)]);
  float v[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) codes4(w[i], s, v + 4 * i);
  if (TO == T_FP32) {
    float4* x = reinterpret_cast<float4*>(X + (int64_t)u * 64);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    u4i* x = reinterpret_cast<u4i*>(X + (int64_t)u * 32);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u4i o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = saturate<TO>(v[8 * i + 2 * e]), b = saturate<TO>(v[8 * i + 2 * e + 1]);
        o[e] = pack2<TO == T_FP32 ? T_BF16 : TO>(a, b);
      }
      x[i] = o;
    }
  }
}

template <int TY>
__device__ __forceinline__ void unpack8(u4i r, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (TY == T_BF16) {
      v[2 * e] = __uint_as_float(r[e] << 16);
      v[2 * e + 1] = __uint_as_float(r[e] & 0xFFFF0000u);
    } else {
      const uint32_t bits = r[e];
      const h2 x = __builtin_bit_cast(h2, bits);
      v[2 * e] = (float)x.x;
      v[2 * e + 1] = (float)x.y;
    }
  }
}
template <int TY>
__device__ __forceinline__ u4i pack8(const float (&v)[8]) {
  return u4i{pack2<TY>(v[0], v[1]), pack2<TY>(v[2], v[3]), pack2<TY>(v[4], v[5]), pack2<TY>(v[6], v[7])};
}

// [dG | dU] (and H) of dH and [G | U], the latter in 16 bits or as codes, in binary32 and rounded
// once.  One pass over what is read and written; 8 columns per lane, so that 16-bit rows are loaded
// and stored 16 bytes a lane, and the 8 codes of a lane have one scale.  Bound by memory: 4096 x
// 14336 from codes, with H, 98 us (587 MB, 6.0 TB/s); 8192 x 2048 in 16 bits, without H, 26 us (168
// MB, 6.5 TB/s, part of it still in the last-level cache).
template <int TY, int ACT, bool CODES>
__global__ void __launch_bounds__(256) k_gated_dgu(uint32_t units, uint32_t per_row, uint32_t f, uint32_t lds,
                                                   const uint8_t* __restrict__ dH, const uint8_t* __restrict__ GU,
                                                   const uint8_t* __restrict__ sGU, uint8_t* __restrict__ dGU,
                                                   uint8_t* __restrict__ H) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= units) return;
  const uint32_t row = i / per_row, c = (i - row * per_row) * 8;
  const int64_t at = (int64_t)row * 2 * f + c;  // of the gate's numbers; the up's f further
  float d[8], g[8], u[8];
  unpack8<TY>(*reinterpret_cast<const u4i*>(dH + (int64_t)i * 16), d);
  if (CODES) {
    const uint2 a = *reinterpret_cast<const uint2*>(GU + at), b = *reinterpret_cast<const uint2*>(GU + at + f);
    const uint8_t* sc = sGU + (int64_t)row * lds;
    const float sa = scale_of(sc[c >> 7]), sb = scale_of(sc[(f + c) >> 7]);
    codes4(a.x, sa, g);
    codes4(a.y, sa, g + 4);
    codes4(b.x, sb, u);
    codes4(b.y, sb, u + 4);
  } else {
    unpack8<TY>(*reinterpret_cast<const u4i*>(GU + 2 * at), g);
    unpack8<TY>(*reinterpret_cast<const u4i*>(GU + 2 * (at + f)), u);
  }
  float h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 s = act_slope(ACT, g[e]);
    const float a = g[e] * s.x;
    h[e] = a * u[e];
    g[e] = d[e] * u[e] * s.y;
    u[e] = d[e] * a;
  }
  *reinterpret_cast<u4i*>(dGU + 2 * at) = pack8<TY>(g);
  *reinterpret_cast<u4i*>(dGU + 2 * (at + f)) = pack8<TY>(u);
  if (H) *reinterpret_cast<u4i*>(H + (int64_t)i * 16) = pack8<TY>(h);
}

template <int TY>
void dgu(int act, bool codes, uint32_t units, uint32_t f, uint32_t lds, const uint8_t* dH, const uint8_t* GU,
         const uint8_t* sGU, uint8_t* dGU, uint8_t* H, hipStream_t st) {
  const dim3 grid((units + 255) / 256);
  auto k = act == ACT_SILU ? (codes ? k_gated_dgu<TY, ACT_SILU, true> : k_gated_dgu<TY, ACT_SILU, false>)
                           : (codes ? k_gated_dgu<TY, ACT_GELU, true> : k_gated_dgu<TY, ACT_GELU, false>);
  k<<<grid, 256, 0, st>>>(units, f / 8, f, lds, dH, GU, sGU, dGU, H);
}

}  // namespace

hipError_t launch_gated(int64_t M, int64_t E, int64_t f, int64_t n, int dtype, int act, const void* X,
                        const int64_t* offsets, const void* W, void* H, void* GU, hipStream_t st) {
  GemmArgs a{};
  a.A = static_cast<const uint8_t*>(X);
  a.B = static_cast<const uint8_t*>(W);
  a.C = H;
  a.C2 = GU;
  a.act = act;
  a.offsets = offsets;
  a.T = (int)M;
  a.E = (int)E;
  a.cols = (int)f;
  a.kdim = (int)n;
  if (GU) return dtype == T_BF16 ? run_gemm<T_BF16, L_NT, T_BF16, 2>(a, st) : run_gemm<T_FP16, L_NT, T_FP16, 2>(a, st);
  return dtype == T_BF16 ? run_gemm<T_BF16, L_NT, T_BF16, 1>(a, st) : run_gemm<T_FP16, L_NT, T_FP16, 1>(a, st);
}

hipError_t launch_gated_dgu(int64_t M, int64_t f, int dtype, int act, const void* dH, const void* GU, const uint8_t* sGU,
                            void* dGU, void* H, hipStream_t st) {
  const uint8_t *d = static_cast<const uint8_t*>(dH), *s = static_cast<const uint8_t*>(GU);
  uint8_t *o = static_cast<uint8_t*>(dGU), *h = static_cast<uint8_t*>(H);
  const uint32_t units = (uint32_t)(M * (f / 8)), lds = (uint32_t)fp8_scale_stride(2 * f);
  if (dtype == T_BF16)
    dgu<T_BF16>(act, sGU != nullptr, units, (uint32_t)f, lds, d, s, sGU, o, h, st);
  else
    dgu<T_FP16>(act, sGU != nullptr, units, (uint32_t)f, lds, d, s, sGU, o, h, st);
  return hipGetLastError();
}

hipError_t launch_fp8_restore(int64_t M, int64_t n, int dtype, const uint8_t* xq, const uint8_t* sx, void* X,
                              hipStream_t st) {
  const uint32_t per_row = (uint32_t)(n / 16), units = (uint32_t)(M * per_row), lds = (uint32_t)fp8_scale_stride(n);
  const dim3 grid((units + 255) / 256);
  uint8_t* x = static_cast<uint8_t*>(X);
  if (dtype == T_FP32)
    k_fp8_restore<T_FP32><<<grid, 256, 0, st>>>(units, per_row, lds, xq, sx, x);
  else if (dtype == T_FP16)
    k_fp8_restore<T_FP16><<<grid, 256, 0, st>>>(units, per_row, lds, xq, sx, x);
  else
    k_fp8_restore<T_BF16><<<grid, 256, 0, st>>>(units, per_row, lds, xq, sx, x);
  return hipGetLastError();
}

}  // namespace intlora
