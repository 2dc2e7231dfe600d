// Low-rank adapters of many requests beside a shared layer, for gfx950.
//
// Token row t belongs to adapter a = index[t] (none outside [0, L)):
//   h_t = B_a x_t,  Y_t = base_t + s_a A_a h_t           A: L x d x r, B: L x r x n
// and backwards, with dh_t = A_a^T dY_t:
//   dX_t = base_t + s_a B_a^T dh_t,  dA_a = sum_t s_a dY_t h_t^T,  dB_a = sum_t s_a dh_t x_t^T.
// k_down forms h (and dh, on A transposed), k_up the outputs (and dX, on B transposed), k_sums the
// factors' gradients.  h stays in binary32; where it meets 16-bit weights on the matrix cores it
// goes as a sum of two 16-bit numbers (16 or more significant bits, against the outputs' 8 or
// 11), and in the sums over tokens, whose results may be binary32, as a sum of three (24 bits).
#include "device_common.h"
#include "intlora_internal.h"

namespace intlora {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t u4i __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v4s* lds_v4s_t;

enum { T_BF16 = 0, T_FP16 = 1, T_FP32 = 2 };

constexpr uint32_t kOOB = 0x80000000u;  // a buffer offset past every record: the lane reads zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t r, uint32_t offset) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0));
}

template <int TY>
__device__ __forceinline__ v4f mfma(v4i rows, v4i cols, v4f c) {
  if (TY == T_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, rows), __builtin_bit_cast(bf8, cols), c, 0, 0,
                                                   0);
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, rows), __builtin_bit_cast(h8, cols), c, 0, 0, 0);
}

// Two floats to 16 bits each (round to nearest even), and back.
template <int TY>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if (TY == T_FP16) return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){x, y}, h2));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){x, y}, bf2));
}
template <int TY>
__device__ __forceinline__ f2 unpack2(uint32_t v) {
  if (TY == T_FP16) return __builtin_convertvector(__builtin_bit_cast(h2, v), f2);
  return f2{__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u)};
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

// The bf16 number at or next to v towards zero (v itself where it is not finite): the rest v - top
// is exact.
__device__ __forceinline__ float top_bf16(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }

// ---- the adapters of a tile of 16 TT token rows
// Lane l holds the adapters of tokens 16 tt + l % 16 (-1: none).
template <int TT>
struct Tile {
  int id[TT];
  __device__ __forceinline__ void read(const int32_t* __restrict__ index, int64_t t0, int64_t M, int L) {
    const int fr = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int64_t t = t0 + 16 * i + fr;
      const int a = t < M ? index[t] : -1;
      id[i] = a >= 0 && a < L ? a : -1;
    }
  }
  // The first adapter of the tile that is above -1; -1 when none is left.
  __device__ __forceinline__ int first() const {
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const uint64_t m = __builtin_amdgcn_ballot_w64(id[i] >= 0);
      if (m) return __builtin_amdgcn_readlane(id[i], __builtin_ctzll(m));
    }
    return -1;
  }
  // The adapter of token `slot` (of the first 16) if no earlier one of these has the same, else -1.
  __device__ __forceinline__ int leader(int slot) const {
    const int a = __builtin_amdgcn_readlane(id[0], slot);
    const uint64_t m = __builtin_amdgcn_ballot_w64(id[0] == a);
    return a >= 0 && (int)__builtin_ctzll(m) == slot ? a : -1;
  }
};

struct DownArgs {
  const uint8_t* X;  // M x n
  const uint8_t* W;  // L x r x n
  const int32_t* index;
  float* H;          // splits x M x rp
  int64_t M;
  int L, n, r, rp;
  int splits, per;   // columns per split (a multiple of 64)
  int slots;         // 0: a wave takes all adapters of its tile in turn; else one wave per token of a tile of 16
};

// h = W_a x.  A wave computes 16 TT tokens x 16 RT ranks over one split of the columns; lane l
// holds token l % 16 and ranks 4 (l / 16) + 0 .. 3 of a tile.  Rows of other adapters read as zeros
// and are not written.
template <int TY, int TT, int RT>
__global__ void __launch_bounds__(256) k_down(const DownArgs p) {
  const int lane = threadIdx.x & 63, fr = lane & 15, q = lane >> 4;
  const int groups = (p.rp + 16 * RT - 1) / (16 * RT);
  const int per_tile = p.splits * groups * (p.slots ? p.slots : 1);
  const int64_t unit = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tile = unit / per_tile;
  int rest = (int)(unit - tile * per_tile);
  const int64_t t0 = tile * 16 * TT;
  if (t0 >= p.M) return;
  const int split = rest % p.splits;
  rest /= p.splits;
  const int g0 = rest % groups * 16 * RT;
  const int slot = rest / groups;
  Tile<TT> tl;
  tl.read(p.index, t0, p.M, p.L);
  const int rows = p.M - t0 < 16 * TT ? (int)(p.M - t0) : 16 * TT;
  const uint32_t ld = (uint32_t)p.n * 2;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.X + t0 * ld, (int64_t)rows * ld);
  const int k0 = split * p.per, k1 = k0 + p.per < p.n ? k0 + p.per : p.n;
  for (int a = p.slots ? tl.leader(slot) : tl.first(); a >= 0; a = tl.first()) {
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.W + (int64_t)a * p.r * ld, (int64_t)p.r * ld);
    uint32_t ox[TT], ow[RT];
#pragma unroll
    for (int i = 0; i < TT; ++i) ox[i] = tl.id[i] == a ? (16 * i + fr) * ld : kOOB;
#pragma unroll
    for (int j = 0; j < RT; ++j) ow[j] = g0 + 16 * j + fr < p.r ? (g0 + 16 * j + fr) * ld : kOOB;
    v4f acc[TT][RT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    constexpr int U = TT * RT > 4 ? 2 : 4;
    for (int k = k0; k < k1; k += 32 * U) {
      v4i x[U][TT], w[U][RT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = k + 32 * u + 8 * q;
        const uint32_t o = c < k1 ? 2u * c : kOOB;
#pragma unroll
        for (int i = 0; i < TT; ++i) x[u][i] = load16(rx, (ox[i] | o) & kOOB ? kOOB : ox[i] + o);
#pragma unroll
        for (int j = 0; j < RT; ++j) w[u][j] = load16(rw, (ow[j] | o) & kOOB ? kOOB : ow[j] + o);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[i][j] = mfma<TY>(w[u][j], x[u][i], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      if (tl.id[i] != a) continue;
      float* h = p.H + (split * p.M + t0 + 16 * i + fr) * p.rp + g0 + 4 * q;
#pragma unroll
      for (int j = 0; j < RT; ++j)
        if (g0 + 16 * j < p.rp) *reinterpret_cast<v4f*>(h + 16 * j) = acc[i][j];
      tl.id[i] = -1;
    }
    if (p.slots) return;
  }
}

struct UpArgs {
  const float* H;       // splits x M x rp
  const uint8_t* W;     // L x d rows of ld elements, r of them used
  const int32_t* index;
  const float* scale;   // [L]
  const uint8_t* base;  // M x d, or NULL: zeros
  uint8_t* Y;           // M x d (may be base)
  int64_t M;
  int L, d, r, ld, rp, splits;
  int ranks;            // numbers of a row of H that count
  int slots;            // as k_down
  int chunk;            // output columns of a wave (a multiple of 64)
};

// Eight numbers of a weight row from number k on; zeros past the row's r.
template <bool WIDE>
__device__ __forceinline__ v4i row8(const uint16_t* __restrict__ row, int k, int r) {
  if (WIDE) return k < r ? *reinterpret_cast<const v4i*>(row + k) : v4i{0, 0, 0, 0};
  uint32_t v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t lo = k + 2 * e < r ? row[k + 2 * e] : 0, hi = k + 2 * e + 1 < r ? row[k + 2 * e + 1] : 0;
    v[e] = lo | hi << 16;
  }
  return v4i{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
}

// Y = base + s_a W_a h.  A wave takes 16 TT tokens and 64 columns at a time.  Row m of the matrix
// instruction's tile u is column 16 (m / 4) + 4 u + m % 4, so lane l ends up with columns
// 16 (l / 16) + 0 .. 15 of token l % 16: whole 128-byte pieces of a row are read and written.
// KT: steps of 32 of the rank.
template <int TY, int TT, int KT, bool WIDE>
__global__ void __launch_bounds__(256) k_up(const UpArgs p) {
  const int lane = threadIdx.x & 63, fr = lane & 15, q = lane >> 4;
  const int chunks = (p.d + p.chunk - 1) / p.chunk, slots = p.slots ? p.slots : 1;
  const int64_t tiles = (p.M + 16 * TT - 1) / (16 * TT);
  // the four waves of a block: neighbouring tiles (or tokens of a tile), the same columns
  const int64_t unit = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t block = unit / (tiles * slots);
  if (block >= chunks) return;
  const int64_t in = unit - block * tiles * slots, tile = in / slots;
  const int64_t t0 = tile * 16 * TT;
  Tile<TT> tl, all;
  tl.read(p.index, t0, p.M, p.L);
  all = tl;
  const int c0 = (int)block * p.chunk, c1 = c0 + p.chunk < p.d ? c0 + p.chunk : p.d;
  for (int a = p.slots ? tl.leader((int)(in - tile * slots)) : tl.first(); a >= 0; a = tl.first()) {
    const float s = p.scale[a];
    v4i hi[TT][KT], lo[TT][KT];
    float back[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      float v[KT][8];
      const bool mine = tl.id[i] == a;
#pragma unroll
      for (int c = 0; c < KT; ++c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] = 0.f;
        const int k = 32 * c + 8 * q;
        if (!mine || k >= p.rp) continue;
        const float* h = p.H + (t0 + 16 * i + fr) * p.rp + k;
        for (int z = 0; z < p.splits; ++z, h += p.M * p.rp) {
          const float4 x = *reinterpret_cast<const float4*>(h), y = *reinterpret_cast<const float4*>(h + 4);
          v[c][0] += x.x, v[c][1] += x.y, v[c][2] += x.z, v[c][3] += x.w;
          v[c][4] += y.x, v[c][5] += y.y, v[c][6] += y.z, v[c][7] += y.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] = k + e < p.ranks ? v[c][e] * s : 0.f;  // (an infinite x leaves NaN past them)
      }
      // fp16: a power of two per token brings its largest finite |h| into [1/2, 1)
      back[i] = 1.f;
      if (TY == T_FP16) {
        float m = 0.f;
#pragma unroll
        for (int c = 0; c < KT; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, finite(v[c][e]) ? fabsf(v[c][e]) : 0.f);
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        if (m > 0.f) {
          int e = (int)(__float_as_uint(m) >> 23) - 126;  // m < 2^e (subnormals: e = -126)
          e = e < -100 ? -100 : e > 126 ? 126 : e;
          back[i] = __uint_as_float((uint32_t)(e + 127) << 23);
          const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
          for (int c = 0; c < KT; ++c)
#pragma unroll
            for (int x = 0; x < 8; ++x) v[c][x] *= f;
        }
      }
#pragma unroll
      for (int c = 0; c < KT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = v[c][2 * e], y = v[c][2 * e + 1];
          uint32_t t, b;
          if (TY == T_FP16) {
            t = pack2<T_FP16>(x, y);
            const f2 w = unpack2<T_FP16>(t);
            b = pack2<T_FP16>(finite(w.x) ? x - w.x : 0.f, finite(w.y) ? y - w.y : 0.f);
          } else {
            const float tx = top_bf16(x), ty = top_bf16(y);
            t = pack2<T_BF16>(tx, ty);
            b = pack2<T_BF16>(finite(x) ? x - tx : 0.f, finite(y) ? y - ty : 0.f);
          }
          hi[i][c][e] = (int)t;
          lo[i][c][e] = (int)b;
        }
    }
    const uint16_t* W = reinterpret_cast<const uint16_t*>(p.W) + (int64_t)a * p.d * p.ld;
    for (int n0 = c0; n0 < c1; n0 += 64) {
      v4f acc[TT][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = n0 + 16 * (fr >> 2) + 4 * u + (fr & 3);
        v4i w[KT];
#pragma unroll
        for (int c = 0; c < KT; ++c)
          w[c] = row8<WIDE>(W + (int64_t)row * p.ld, row < p.d ? 32 * c + 8 * q : p.r, p.r);
#pragma unroll
        for (int i = 0; i < TT; ++i) {
          acc[i][u] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < KT; ++c) {
            acc[i][u] = mfma<TY>(w[c], lo[i][c], acc[i][u]);
            acc[i][u] = mfma<TY>(w[c], hi[i][c], acc[i][u]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const int64_t at = (t0 + 16 * i + fr) * p.d;
#pragma unroll
        for (int g = 0; g < 2; ++g) {  // eight columns
          const int col = n0 + 16 * q + 8 * g;
          if (tl.id[i] != a || col >= p.d) continue;
          u4i b = u4i{0, 0, 0, 0};
          if (p.base) b = *reinterpret_cast<const u4i*>(p.base + 2 * (at + col));
          u4i y;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f2 f = unpack2<TY>(b[e]);
            const v4f& t = acc[i][2 * g + e / 2];
            y[e] = pack2<TY>(f.x + t[2 * (e & 1)] * back[i], f.y + t[2 * (e & 1) + 1] * back[i]);
          }
          *reinterpret_cast<u4i*>(p.Y + 2 * (at + col)) = y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i)
      if (tl.id[i] == a) tl.id[i] = -1;
    if (p.slots) break;
  }
  // Rows without an adapter: the base's (nothing to do in place).
  if (p.base == p.Y || (p.slots && in - tile * slots != 0)) return;
  for (int n0 = c0; n0 < c1; n0 += 64)
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int64_t t = t0 + 16 * i + fr;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int col = n0 + 16 * q + 8 * g;
        if (all.id[i] >= 0 || t >= p.M || col >= p.d) continue;
        u4i b = u4i{0, 0, 0, 0};
        if (p.base) b = *reinterpret_cast<const u4i*>(p.base + 2 * (t * p.d + col));
        *reinterpret_cast<u4i*>(p.Y + 2 * (t * p.d + col)) = b;
      }
    }
}

// out[a] (cols x ldo) = in[a] (rows x cols) transposed, zeros from column `rows` on.
__global__ void __launch_bounds__(256) k_turn(const uint16_t* __restrict__ in, uint16_t* __restrict__ out, int rows,
                                              int cols, int ldo) {
  __shared__ uint16_t t[32][34];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t c0 = (int64_t)blockIdx.x * 32, r0 = (int64_t)blockIdx.y * 32;
  in += (int64_t)blockIdx.z * rows * cols;
  out += (int64_t)blockIdx.z * cols * ldo;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + y + 8 * i, c = c0 + x;
    t[y + 8 * i][x] = r < rows && c < cols ? in[r * cols + c] : 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = c0 + y + 8 * i, c = r0 + x;
    if (r < cols && c < ldo) out[r * ldo + c] = t[x][y + 8 * i];
  }
}

struct SumArgs {
  const uint8_t* P;      // M x F token rows (dY or X)
  const float* H;        // splits x M x rp (h or dh)
  const int32_t* index;
  const float* scale;
  void* out;             // L x F x r (ranks in the lanes) or L x r x F
  int64_t M;
  int L, F, r, rp, splits;
  int64_t per;           // tokens of a part
  int64_t numel;         // of `out`: parts lie one after the other
};

// sum over an adapter's tokens of P_t h_t^T s_a.  A block takes 64 columns of P and all ranks: it
// collects its adapter's tokens in order, 32 at a time, and each wave adds 16 columns x 16 RT ranks.
// Both operands have the contraction (tokens) in rows and leave LDS through the transposing reads.
// h goes as three bf16 numbers; fp16 rows of P as two (exact).
template <int TY, int TO, int RT, bool RANK_LANES>
__global__ void __launch_bounds__(256) k_sums(const SumArgs p) {
  constexpr int PP = TY == T_FP16 ? 2 : 1;
  constexpr int PS = 64 + 8, HS = 16 * RT + 8;  // row strides (16-bit numbers)
  __shared__ __attribute__((aligned(16))) uint16_t lp[PP][32 * PS];
  __shared__ __attribute__((aligned(16))) uint16_t lh[3][32 * HS];
  __shared__ int list[256 + 32];
  __shared__ int counts[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, fr = lane & 15, q = lane >> 4;
  const int a = blockIdx.y, f0 = blockIdx.x * 64;
  const float s = p.scale[a];
  const int64_t tb = blockIdx.z * p.per, te = tb + p.per < p.M ? tb + p.per : p.M;
  v4f acc[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};

  auto batch = [&](int64_t base, int from, int n) {  // tokens base + list[from .. from + n), n <= 32
    __syncthreads();
    {
      const int row = tid >> 3, c = (tid & 7) * 8;
      u4i v = u4i{0, 0, 0, 0};
      if (row < n && f0 + c < p.F) v = *reinterpret_cast<const u4i*>(p.P + 2 * ((base + list[from + row]) * p.F + f0 + c));
      if (TY == T_FP16) {
        u4i t, b;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f2 x = unpack2<T_FP16>(v[e]);
          const f2 y = f2{top_bf16(x.x), top_bf16(x.y)};
          t[e] = pack2<T_BF16>(y.x, y.y);
          b[e] = pack2<T_BF16>(finite(x.x) ? x.x - y.x : 0.f, finite(x.y) ? x.y - y.y : 0.f);
        }
        *reinterpret_cast<u4i*>(&lp[0][row * PS + c]) = t;
        *reinterpret_cast<u4i*>(&lp[PP - 1][row * PS + c]) = b;
      } else {
        *reinterpret_cast<u4i*>(&lp[0][row * PS + c]) = v;
      }
    }
    for (int i = tid; i < 32 * 4 * RT; i += 256) {
      const int row = i / (4 * RT), c = i % (4 * RT) * 4;
      float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < n && c < p.rp) {
        const float* src = p.H + (base + list[from + row]) * p.rp + c;
        for (int z = 0; z < p.splits; ++z, src += p.M * p.rp) {
          const float4 x = *reinterpret_cast<const float4*>(src);
          h.x += x.x, h.y += x.y, h.z += x.z, h.w += x.w;
        }
        h.x *= s, h.y *= s, h.z *= s, h.w *= s;
      }
      float v[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        float t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          t[e] = top_bf16(v[e]);
          v[e] = finite(v[e]) ? v[e] - t[e] : 0.f;
        }
        *reinterpret_cast<uint2*>(&lh[k][row * HS + c]) = make_uint2(pack2<T_BF16>(t[0], t[1]), pack2<T_BF16>(t[2], t[3]));
      }
    }
    __syncthreads();
    auto frag = [&](const uint16_t* m, int stride, int col) {  // rows 8 q .. 8 q + 7 of column col + fr
      const uint16_t* at = m + (8 * q + (fr >> 2)) * stride + col + 4 * (fr & 3);
      const int2 x = __builtin_bit_cast(int2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t)at));
      const int2 y = __builtin_bit_cast(int2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t)(at + 4 * stride)));
      return v4i{x.x, x.y, y.x, y.y};
    };
    v4i pf[PP];
#pragma unroll
    for (int k = 0; k < PP; ++k) pf[k] = frag(lp[k], PS, 16 * wave);
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int k = 2; k >= 0; --k) {
        const v4i h = frag(lh[k], HS, 16 * j);
#pragma unroll
        for (int z = PP - 1; z >= 0; --z)
          acc[j] = RANK_LANES ? mfma<T_BF16>(pf[z], h, acc[j]) : mfma<T_BF16>(h, pf[z], acc[j]);
      }
  };

  int have = 0;  // collected, not yet added (positions in the list relative to tb)
  for (int64_t t = tb; t < te; t += 256) {
    const bool hit = t + tid < te && p.index[t + tid] == a;
    const uint64_t m = __builtin_amdgcn_ballot_w64(hit);
    __syncthreads();
    if (lane == 0) counts[wave] = __builtin_popcountll(m);
    __syncthreads();
    int at = have, all = have;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) at += counts[w];
      all += counts[w];
    }
    if (hit) list[at + __builtin_popcountll(m & ((1ull << lane) - 1))] = (int)(t - tb) + tid;
    int from = 0;
    for (; all - from >= 32; from += 32) batch(tb, from, 32);
    have = all - from;
    __syncthreads();
    const int keep = tid < have ? list[from + tid] : 0;
    __syncthreads();
    if (tid < have) list[tid] = keep;
  }
  if (have > 0) batch(tb, 0, have);

  // lane l: column (rank) l % 16 of the tile, rows 4 (l / 16) + 0 .. 3
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int f = f0 + 16 * wave + (RANK_LANES ? 4 * q + e : fr), k = 16 * j + (RANK_LANES ? fr : 4 * q + e);
      if (f >= p.F || k >= p.r) continue;
      const int64_t at = blockIdx.z * p.numel + (RANK_LANES ? ((int64_t)a * p.F + f) * p.r + k : ((int64_t)a * p.r + k) * p.F + f);
      if (TO == T_FP32)
        static_cast<float*>(p.out)[at] = acc[j][e];
      else
        static_cast<uint16_t*>(p.out)[at] = (uint16_t)pack2<TO>(acc[j][e], 0.f);
    }
}

// out = the parts added in order; numel a multiple of 4.
template <int TO>
__global__ void __launch_bounds__(256) k_parts(const float* __restrict__ in, void* __restrict__ out, int64_t numel,
                                               int parts) {
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < numel; i += (int64_t)gridDim.x * 1024) {
    float4 s = *reinterpret_cast<const float4*>(in + i);
    for (int z = 1; z < parts; ++z) {
      const float4 x = *reinterpret_cast<const float4*>(in + z * numel + i);
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    if (TO == T_FP32)
      *reinterpret_cast<float4*>(static_cast<float*>(out) + i) = s;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + i) = make_uint2(pack2<TO>(s.x, s.y), pack2<TO>(s.z, s.w));
  }
}

constexpr int64_t kSlotRows = 1024;  // up to here one wave per token of a tile

int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }
int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// Splits of a k_down call over n columns, and the columns of each.
struct Splits {
  int count, per;
};
Splits down_splits(int64_t M, int64_t n, int64_t r) {
  const int64_t tiles = (r + 15) / 16;
  const int64_t waves = M <= kSlotRows ? M * tiles : (M + 31) / 32 * ((tiles + 3) / 4);
  int64_t s = waves > 0 ? (2048 + waves - 1) / waves : 1;
  const int64_t most = (n + 255) / 256;
  s = s > 16 ? 16 : s;
  s = s > most ? most : s;
  const int64_t per = ((n + s - 1) / s + 63) / 64 * 64;
  return {(int)((n + per - 1) / per), (int)per};
}

// Parts of the tokens of a k_sums call.
struct Parts {
  int count;
  int64_t per;
};
Parts sum_parts(int64_t M, int64_t L, int64_t F) {
  const int64_t blocks = L * ((F + 63) / 64);
  int64_t z = blocks >= 512 ? 1 : (512 + blocks - 1) / blocks;
  const int64_t most = (M + 511) / 512;
  z = z > 32 ? 32 : z;
  z = z > most ? (most < 1 ? 1 : most) : z;
  const int64_t per = M < 1 ? 256 : ((M + z - 1) / z + 255) / 256 * 256;
  const int64_t c = (M + per - 1) / per;
  return {(int)(c < 1 ? 1 : c), per};
}

template <int TY>
hipError_t down(DownArgs a, const Splits& s, hipStream_t st) {
  a.splits = s.count;
  a.per = s.per;
  const int rt = a.rp / 16;
  a.slots = a.M <= kSlotRows ? (a.M < 16 ? (int)a.M : 16) : 0;
  const int tt = a.slots ? 1 : 2, per_wave = a.slots ? 1 : (rt >= 4 ? 4 : rt == 1 ? 1 : 2);
  const int64_t units = (a.M + 16 * tt - 1) / (16 * tt) * s.count * ((rt + per_wave - 1) / per_wave) * (a.slots ? a.slots : 1);
  const dim3 grid((unsigned)((units + 3) / 4));
  if (a.slots)
    k_down<TY, 1, 1><<<grid, 256, 0, st>>>(a);
  else if (per_wave == 1)
    k_down<TY, 2, 1><<<grid, 256, 0, st>>>(a);
  else if (per_wave == 2)
    k_down<TY, 2, 2><<<grid, 256, 0, st>>>(a);
  else
    k_down<TY, 2, 4><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

template <int TY, int TT, bool WIDE>
void up_kt(const UpArgs& a, dim3 grid, hipStream_t st) {
  if (a.r <= 32)
    k_up<TY, TT, 1, WIDE><<<grid, 256, 0, st>>>(a);
  else if (a.r <= 64)
    k_up<TY, TT, 2, WIDE><<<grid, 256, 0, st>>>(a);
  else
    k_up<TY, TT, 4, WIDE><<<grid, 256, 0, st>>>(a);
}

template <int TY>
hipError_t up(UpArgs a, hipStream_t st) {
  a.slots = a.M <= kSlotRows ? (a.M < 16 ? (int)a.M : 16) : 0;
  const int tt = a.slots ? 1 : 2;
  const int64_t tiles = (a.M + 16 * tt - 1) / (16 * tt) * (a.slots ? a.slots : 1);
  int64_t chunk = 512;
  while (chunk > 64 && tiles * ((a.d + chunk - 1) / chunk) < 2048) chunk /= 2;
  a.chunk = (int)chunk;
  const dim3 grid((unsigned)((tiles * ((a.d + chunk - 1) / chunk) + 3) / 4));
  const bool wide = a.r % 8 == 0 && a.ld % 8 == 0;
  if (a.slots)
    wide ? up_kt<TY, 1, true>(a, grid, st) : up_kt<TY, 1, false>(a, grid, st);
  else
    wide ? up_kt<TY, 2, true>(a, grid, st) : up_kt<TY, 2, false>(a, grid, st);
  return hipGetLastError();
}

template <int TY, int TO, bool RANK_LANES>
void sums_rt(const SumArgs& a, dim3 grid, hipStream_t st) {
  if (a.rp <= 16)
    k_sums<TY, TO, 1, RANK_LANES><<<grid, 256, 0, st>>>(a);
  else if (a.rp <= 32)
    k_sums<TY, TO, 2, RANK_LANES><<<grid, 256, 0, st>>>(a);
  else if (a.rp <= 64)
    k_sums<TY, TO, 4, RANK_LANES><<<grid, 256, 0, st>>>(a);
  else
    k_sums<TY, TO, 8, RANK_LANES><<<grid, 256, 0, st>>>(a);
}

template <int TY, bool RANK_LANES>
hipError_t sums(SumArgs a, const Parts& z, int out_dtype, void* out, float* ws, hipStream_t st) {
  a.per = z.per;
  a.numel = (int64_t)a.L * a.F * a.r;
  a.out = z.count > 1 ? ws : out;
  const dim3 grid((unsigned)((a.F + 63) / 64), (unsigned)a.L, (unsigned)z.count);
  if (z.count > 1 || out_dtype == T_FP32)
    sums_rt<TY, T_FP32, RANK_LANES>(a, grid, st);
  else
    sums_rt<TY, TY, RANK_LANES>(a, grid, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || z.count == 1) return e;
  const int64_t want = (a.numel / 4 + 255) / 256;
  const unsigned blocks = (unsigned)(want < 2048 ? want : 2048);
  if (out_dtype == T_FP32)
    k_parts<T_FP32><<<blocks, 256, 0, st>>>(ws, out, a.numel, z.count);
  else
    k_parts<TY><<<blocks, 256, 0, st>>>(ws, out, a.numel, z.count);
  return hipGetLastError();
}

// The workspace: h, and for the gradients dh, A and B transposed, and the parts of the sums.
struct Ws {
  int64_t h, dh, at, bt, parts, bytes;
};
Ws carve(int64_t M, int64_t L, int64_t d, int64_t n, int64_t r, bool grads) {
  Ws w{};
  const int64_t rp = round16(r);
  int64_t at = up256(4 * M * rp * down_splits(M, n, r).count);
  if (grads) {
    w.dh = at;
    at += up256(4 * M * rp * down_splits(M, d, r).count);
    w.at = at;
    at += up256(2 * L * r * d);
    w.bt = at;
    at += up256(2 * L * n * rp);
    w.parts = at;
    const int64_t za = sum_parts(M, L, d).count, zb = sum_parts(M, L, n).count;
    const int64_t pa = za > 1 ? 4 * za * L * d * r : 0, pb = zb > 1 ? 4 * zb * L * n * r : 0;
    at += up256(pa > pb ? pa : pb);
  }
  w.bytes = at;
  return w;
}

template <int TY>
hipError_t fwd(const AdapterArgs& p, uint8_t* ws, hipStream_t st) {
  const Splits s = down_splits(p.M, p.n, p.r);
  const int rp = (int)round16(p.r);
  DownArgs x{};
  x.X = static_cast<const uint8_t*>(p.X);
  x.W = static_cast<const uint8_t*>(p.B);
  x.index = p.index;
  x.H = reinterpret_cast<float*>(ws);
  x.M = p.M;
  x.L = (int)p.L;
  x.n = (int)p.n;
  x.r = (int)p.r;
  x.rp = rp;
  hipError_t e = down<TY>(x, s, st);
  if (e != hipSuccess) return e;
  UpArgs y{};
  y.H = x.H;
  y.W = static_cast<const uint8_t*>(p.A);
  y.index = p.index;
  y.scale = p.scale;
  y.base = static_cast<const uint8_t*>(p.base);
  y.Y = static_cast<uint8_t*>(p.Y);
  y.M = p.M;
  y.L = (int)p.L;
  y.d = (int)p.d;
  y.r = y.ld = (int)p.r;
  y.rp = rp;
  y.ranks = (int)p.r;
  y.splits = s.count;
  return up<TY>(y, st);
}

template <int TY>
hipError_t bwd(const AdapterArgs& p, uint8_t* ws, hipStream_t st) {
  const Ws w = carve(p.M, p.L, p.d, p.n, p.r, true);
  const int rp = (int)round16(p.r);
  const int L = (int)p.L, d = (int)p.d, n = (int)p.n, r = (int)p.r;
  float *h = reinterpret_cast<float*>(ws), *dh = reinterpret_cast<float*>(ws + w.dh),
        *parts = reinterpret_cast<float*>(ws + w.parts);
  uint16_t *at = reinterpret_cast<uint16_t*>(ws + w.at), *bt = reinterpret_cast<uint16_t*>(ws + w.bt);
  hipError_t e;
  const Splits sh = down_splits(p.M, n, r), sd = down_splits(p.M, d, r);
  if (p.M > 0) {
    k_turn<<<dim3((r + 31) / 32, (d + 31) / 32, L), 256, 0, st>>>(static_cast<const uint16_t*>(p.A), at, d, r, d);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    DownArgs x{};
    x.index = p.index;
    x.M = p.M;
    x.L = L;
    x.r = r;
    x.rp = rp;
    x.X = static_cast<const uint8_t*>(p.X);
    x.W = static_cast<const uint8_t*>(p.B);
    x.H = h;
    x.n = n;
    if ((e = down<TY>(x, sh, st)) != hipSuccess) return e;
    x.X = static_cast<const uint8_t*>(p.dY);
    x.W = reinterpret_cast<const uint8_t*>(at);
    x.H = dh;
    x.n = d;
    if ((e = down<TY>(x, sd, st)) != hipSuccess) return e;
    if (p.Y) {
      k_turn<<<dim3((n + 31) / 32, (rp + 31) / 32, L), 256, 0, st>>>(static_cast<const uint16_t*>(p.B), bt, r, n, rp);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      UpArgs y{};
      y.H = dh;
      y.W = reinterpret_cast<const uint8_t*>(bt);
      y.index = p.index;
      y.scale = p.scale;
      y.base = static_cast<const uint8_t*>(p.base);
      y.Y = static_cast<uint8_t*>(p.Y);
      y.M = p.M;
      y.L = L;
      y.d = n;
      y.r = y.ld = y.rp = rp;  // (the padding is zeros on both sides)
      y.ranks = r;
      y.splits = sd.count;
      if ((e = up<TY>(y, st)) != hipSuccess) return e;
    }
  }
  SumArgs q{};
  q.index = p.index;
  q.scale = p.scale;
  q.M = p.M;
  q.L = L;
  q.r = r;
  q.rp = rp;
  q.P = static_cast<const uint8_t*>(p.dY);
  q.H = h;
  q.F = d;
  q.splits = sh.count;
  if ((e = sums<TY, true>(q, sum_parts(p.M, L, d), p.out_dtype, p.dA, parts, st)) != hipSuccess) return e;
  q.P = static_cast<const uint8_t*>(p.X);
  q.H = dh;
  q.F = n;
  q.splits = sd.count;
  return sums<TY, false>(q, sum_parts(p.M, L, n), p.out_dtype, p.dB, parts, st);
}

}  // namespace

// Blocks of the largest launch: a grid holds less than 2^32 work-items.
bool adapters_fit(int64_t M, int64_t d, int64_t n, int64_t r) {
  const int64_t tiles = M <= kSlotRows ? M + 15 : (M + 31) / 32, widest = d > n ? d : n;
  const int64_t ups = tiles * ((widest + 63) / 64 < 32 ? (widest + 63) / 64 : (widest + 511) / 512 + 32);
  const int64_t downs = tiles * ((r + 15) / 16) * 16;
  return (ups > downs ? ups : downs) / 4 < (int64_t(1) << 24) - 1;
}

size_t adapters_ws_bytes(int64_t M, int64_t L, int64_t d, int64_t n, int64_t r, bool grads) {
  return (size_t)carve(M, L, d, n, r, grads).bytes;
}

hipError_t launch_adapters(const AdapterArgs& p, void* ws, hipStream_t st) {
  return p.dtype == T_BF16 ? fwd<T_BF16>(p, static_cast<uint8_t*>(ws), st) : fwd<T_FP16>(p, static_cast<uint8_t*>(ws), st);
}

hipError_t launch_adapters_grad(const AdapterArgs& p, void* ws, hipStream_t st) {
  return p.dtype == T_BF16 ? bwd<T_BF16>(p, static_cast<uint8_t*>(ws), st) : bwd<T_FP16>(p, static_cast<uint8_t*>(ws), st);
}

}  // namespace intlora
