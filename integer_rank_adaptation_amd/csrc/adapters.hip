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

// h = W_a x of one or two problems (h and dh: blockIdx.y).
struct Down {
  const uint8_t* X;  // M x n
  const uint8_t* W;  // L x r x n
  float* H;          // splits x M x rp
  int n, splits;
};
struct DownArgs {
  Down of[2];
  const int32_t* index;
  int64_t M;
  int L, r, rp;
  int slots;  // 0: a block takes all adapters of its tile in turn; else one block per token of a tile of 16
};

// A block computes 16 TT tokens x 16 RT ranks over one split of the columns: its eight waves take
// runs of 64 columns in turn, and their sums meet in LDS, where each wave adds the eight parts of
// a tile in order.  Lane l holds token l % 16 and ranks 4 (l / 16) + 0 .. 3 of a tile.  Rows of
// other adapters read as zeros and are not written.
constexpr int kDownWaves = 8;

template <int TY, int TT, int RT>
__global__ void __launch_bounds__(64 * kDownWaves) k_down(const DownArgs p) {
  constexpr int PASS = TT * RT > 8 ? 8 / TT : RT;  // rank tiles whose sums LDS holds at a time
  __shared__ __attribute__((aligned(16))) float sums[kDownWaves][TT * PASS][256];
  const Down& of = p.of[blockIdx.y];
  const int lane = threadIdx.x & 63, fr = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = (p.rp + 16 * RT - 1) / (16 * RT);
  const uint32_t per_tile = of.splits * groups * (p.slots ? p.slots : 1);
  const int64_t tile = blockIdx.x / per_tile, t0 = tile * 16 * TT;
  if (t0 >= p.M) return;
  int rest = (int)(blockIdx.x - tile * per_tile);
  const int split = rest % of.splits;
  rest /= of.splits;
  const int g0 = rest % groups * 16 * RT, slot = rest / groups;
  Tile<TT> tl;
  tl.read(p.index, t0, p.M, p.L);
  const int rows = p.M - t0 < 16 * TT ? (int)(p.M - t0) : 16 * TT;
  const uint32_t ld = (uint32_t)of.n * 2;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(of.X + t0 * ld, (int64_t)rows * ld);
  const int first = 64 * (wave + kDownWaves * split), step = 64 * kDownWaves * of.splits;
  for (int a = p.slots ? tl.leader(slot) : tl.first(); a >= 0; a = tl.first()) {
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(of.W + (int64_t)a * p.r * ld, (int64_t)p.r * ld);
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
    // Two runs are in flight at a time (lane q: 16 bytes each at 8 q and 32 + 8 q of a run).  Runs past
    // the last read zeros.
    struct Run {
      v4i x[2][TT], w[2][RT];
    };
    auto load = [&](int k, Run& f) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = k + 32 * u + 8 * q;
        const uint32_t o = c < of.n ? 2u * c : kOOB;
#pragma unroll
        for (int i = 0; i < TT; ++i) f.x[u][i] = load16(rx, (ox[i] | o) & kOOB ? kOOB : ox[i] + o);
#pragma unroll
        for (int j = 0; j < RT; ++j) f.w[u][j] = load16(rw, (ow[j] | o) & kOOB ? kOOB : ow[j] + o);
      }
    };
    auto add = [&](const Run& f) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[i][j] = mfma<TY>(f.w[u][j], f.x[u][i], acc[i][j]);
    };
    Run f0, f1;
    load(first, f0);
    for (int k = first; k < of.n; k += 2 * step) {
      load(k + step, f1);
      add(f0);
      load(k + 2 * step, f0);
      add(f1);
    }
#pragma unroll
    for (int g = 0; g < RT; g += PASS) {
      if (g0 + 16 * g >= p.rp) break;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int j = 0; j < PASS; ++j) *reinterpret_cast<v4f*>(&sums[wave][i * PASS + j][4 * lane]) = acc[i][g + j];
      __syncthreads();
#pragma unroll
      for (int y = 0; y < TT * PASS; y += kDownWaves) {
        const int z = y + wave, i = z / PASS, j = z % PASS;  // this wave's tile
        if (z >= TT * PASS) break;
        v4f s = *reinterpret_cast<const v4f*>(&sums[0][z][4 * lane]);
#pragma unroll
        for (int w = 1; w < kDownWaves; ++w) s += *reinterpret_cast<const v4f*>(&sums[w][z][4 * lane]);
        const int id = TT == 1 || i == 0 ? tl.id[0] : tl.id[TT - 1];
        if (id == a && g0 + 16 * (g + j) < p.rp)
          *reinterpret_cast<v4f*>(of.H + (split * p.M + t0 + 16 * i + fr) * p.rp + g0 + 16 * (g + j) + 4 * q) = s;
      }
    }
    if (p.slots) return;
#pragma unroll
    for (int i = 0; i < TT; ++i)
      if (tl.id[i] == a) tl.id[i] = -1;
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
  int chunk;            // output columns of a wave (a multiple of 32)
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

// Y = base + s_a W_a h.  A wave takes 16 TT tokens and 32 columns at a time.  Row m of the matrix
// instruction's tile u is column 8 (m / 4) + 4 u + m % 4, so lane l ends up with columns
// 8 (l / 16) + 0 .. 7 of token l % 16, and a row is read and written in whole runs of 64 bytes.  The
// next columns' weights are loaded while these are at work, the first ones before h is there.
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
    const uint16_t* W = reinterpret_cast<const uint16_t*>(p.W) + (int64_t)a * p.d * p.ld;
    struct Cols {
      v4i w[2][KT];
    };
    auto load = [&](int n0, Cols& f) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = n0 + 8 * (fr >> 2) + 4 * u + (fr & 3);
#pragma unroll
        for (int c = 0; c < KT; ++c)
          f.w[u][c] = row8<WIDE>(W + (int64_t)row * p.ld, row < p.d ? 32 * c + 8 * q : p.r, p.r);
      }
    };
    Cols cur;
    load(c0, cur);
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
#pragma unroll 4
        for (int z = 0; z < p.splits; ++z) {
          const float4 *o = reinterpret_cast<const float4*>(h + z * p.M * p.rp), x = o[0], y = o[1];
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
    for (int n0 = c0; n0 < c1; n0 += 32) {
      const int col = n0 + 8 * q;
      u4i b[TT];
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        b[i] = u4i{0, 0, 0, 0};
        if (p.base && tl.id[i] == a && col < p.d)
          b[i] = *reinterpret_cast<const u4i*>(p.base + 2 * ((t0 + 16 * i + fr) * p.d + col));
      }
      Cols next;
      load(n0 + 32 < c1 ? n0 + 32 : p.d, next);
      v4f acc[TT][2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < TT; ++i) {
          acc[i][u] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < KT; ++c) {
            acc[i][u] = mfma<TY>(cur.w[u][c], lo[i][c], acc[i][u]);
            acc[i][u] = mfma<TY>(cur.w[u][c], hi[i][c], acc[i][u]);
          }
        }
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        if (tl.id[i] != a || col >= p.d) continue;
        u4i y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f2 f = unpack2<TY>(b[i][e]);
          const v4f& t = acc[i][e / 2];
          y[e] = pack2<TY>(f.x + t[2 * (e & 1)] * back[i], f.y + t[2 * (e & 1) + 1] * back[i]);
        }
        *reinterpret_cast<u4i*>(p.Y + 2 * ((t0 + 16 * i + fr) * p.d + col)) = y;
      }
      cur = next;
    }
    if (p.slots) break;
#pragma unroll
    for (int i = 0; i < TT; ++i)
      if (tl.id[i] == a) tl.id[i] = -1;
  }
  // Rows without an adapter: the base's (nothing to do in place).
  if (p.base == p.Y || (p.slots && in - tile * slots != 0)) return;
  for (int col = c0 + 8 * q; col < c1; col += 32)
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int64_t t = t0 + 16 * i + fr;
      if (all.id[i] >= 0 || t >= p.M) continue;
      u4i b = u4i{0, 0, 0, 0};
      if (p.base) b = *reinterpret_cast<const u4i*>(p.base + 2 * (t * p.d + col));
      *reinterpret_cast<u4i*>(p.Y + 2 * (t * p.d + col)) = b;
    }
}

// out[a] (cols x ldo) = in[a] (rows x cols) transposed, zeros from column `rows` on, of both factors.
struct Turn {
  const uint16_t* in;
  uint16_t* out;
  int rows, cols, ldo, tiles_x, tiles;  // tiles of 32 x 32: along the columns, in all
};
struct TurnArgs {
  Turn of[2];
};
__global__ void __launch_bounds__(256) k_turn(const TurnArgs p) {
  __shared__ uint16_t t[32][34];
  const bool second = (int)blockIdx.x >= p.of[0].tiles;
  const Turn& w = p.of[second];
  const int tile = blockIdx.x - (second ? p.of[0].tiles : 0);
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t c0 = (int64_t)(tile % w.tiles_x) * 32, r0 = (int64_t)(tile / w.tiles_x) * 32;
  const uint16_t* in = w.in + (int64_t)blockIdx.y * w.rows * w.cols;
  uint16_t* out = w.out + (int64_t)blockIdx.y * w.cols * w.ldo;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + y + 8 * i, c = c0 + x;
    t[y + 8 * i][x] = r < w.rows && c < w.cols ? in[r * w.cols + c] : 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = c0 + y + 8 * i, c = r0 + x;
    if (r < w.cols && c < w.ldo) out[r * w.ldo + c] = t[x][y + 8 * i];
  }
}

struct Sum {
  const uint8_t* P;  // M x F token rows (dY or X)
  const float* H;    // splits x M x rp (h or dh)
  void* out;         // L x F x r (dA) or L x r x F (dB)
  int F, splits;
};
struct SumArgs {
  Sum of[2];             // dA, dB
  const int32_t* index;
  const float* scale;
  int64_t M;
  int L, r, rp;
  int blocks0;           // blocks of 64 columns of the first one
  int64_t per;           // tokens of a part
  int64_t numel[2];      // of the outputs: parts lie one after the other
};

// sum over an adapter's tokens of P_t h_t^T s_a.  A block takes 64 columns of P and all ranks: it
// lists its adapter's tokens (of 2048 rows at a time, in order) and adds them T at a time, each
// wave 16 columns x 16 RT ranks; the next ones are loaded meanwhile.  Both operands have the
// contraction (tokens) in rows and leave LDS through the transposing reads.  h goes as three bf16
// numbers; fp16 rows of P as two (exact).
template <int TY, int RT>
struct SumLds {
  static constexpr int PP = TY == T_FP16 ? 2 : 1, T = RT == 8 ? 32 : 64;
  static constexpr int PS = 64 + 8, HS = 16 * RT + 8;  // row strides (16-bit numbers)
  static constexpr int kScan = 2048;
  uint16_t p[PP][T * PS];
  uint16_t h[3][T * HS];
  int list[kScan + T];
  int counts[4];
};

template <int TY, int TO, int RT, bool RANK_LANES>
__device__ __forceinline__ void sum_block(const SumArgs& p, const Sum& of, int64_t numel, int block, SumLds<TY, RT>& L) {
  using S = SumLds<TY, RT>;
  constexpr int PP = S::PP, T = S::T, PS = S::PS, HS = S::HS;
  constexpr int NP = T / 32, NH = T * RT / 64;  // 16-byte loads of a thread
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, fr = lane & 15, q = lane >> 4;
  const int a = blockIdx.y, f0 = block * 64;
  const float s = p.scale[a];
  const int64_t tb = blockIdx.z * p.per, te = tb + p.per < p.M ? tb + p.per : p.M;
  v4f acc[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
  u4i pv[NP];
  float4 hv[NH];

  // tokens tb + list[from .. from + n), n <= T: rows past n are zeros
  auto fetch = [&](int from, int n) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int row = (tid >> 3) + 32 * i, c = (tid & 7) * 8;
      pv[i] = u4i{0, 0, 0, 0};
      if (row < n && f0 + c < of.F)
        pv[i] = *reinterpret_cast<const u4i*>(of.P + 2 * ((tb + L.list[from + row]) * of.F + f0 + c));
    }
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const int at = tid + 256 * i, row = at / (4 * RT), c = at % (4 * RT) * 4;
      hv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < n && c < p.rp) {
        const float* src = of.H + (tb + L.list[from + row]) * p.rp + c;
        for (int z = 0; z < of.splits; ++z) {
          const float4 x = *reinterpret_cast<const float4*>(src + z * p.M * p.rp);
          hv[i].x += x.x, hv[i].y += x.y, hv[i].z += x.z, hv[i].w += x.w;
        }
      }
    }
  };
  auto store = [&]() {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int at = ((tid >> 3) + 32 * i) * PS + (tid & 7) * 8;
      if (TY == T_FP16) {
        u4i t, b;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f2 x = unpack2<T_FP16>(pv[i][e]);
          const f2 y = f2{top_bf16(x.x), top_bf16(x.y)};
          t[e] = pack2<T_BF16>(y.x, y.y);
          b[e] = pack2<T_BF16>(finite(x.x) ? x.x - y.x : 0.f, finite(x.y) ? x.y - y.y : 0.f);
        }
        *reinterpret_cast<u4i*>(&L.p[0][at]) = t;
        *reinterpret_cast<u4i*>(&L.p[PP - 1][at]) = b;
      } else {
        *reinterpret_cast<u4i*>(&L.p[0][at]) = pv[i];
      }
    }
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const int at = tid + 256 * i, row = at / (4 * RT), c = at % (4 * RT) * 4;
      float v[4] = {hv[i].x * s, hv[i].y * s, hv[i].z * s, hv[i].w * s};
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        float t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          t[e] = top_bf16(v[e]);
          v[e] = finite(v[e]) ? v[e] - t[e] : 0.f;
        }
        *reinterpret_cast<uint2*>(&L.h[k][row * HS + c]) = make_uint2(pack2<T_BF16>(t[0], t[1]), pack2<T_BF16>(t[2], t[3]));
      }
    }
  };
  auto frag = [&](const uint16_t* m, int stride, int row, int col) {  // rows row + 8 q + 0 .. 7 of column col + fr
    const uint16_t* at = m + (row + 8 * q + (fr >> 2)) * stride + col + 4 * (fr & 3);
    const int2 x = __builtin_bit_cast(int2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t)at));
    const int2 y = __builtin_bit_cast(int2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t)(at + 4 * stride)));
    return v4i{x.x, x.y, y.x, y.y};
  };
  auto add = [&]() {
#pragma unroll
    for (int t = 0; t < T; t += 32) {
      v4i pf[PP];
#pragma unroll
      for (int k = 0; k < PP; ++k) pf[k] = frag(L.p[k], PS, t, 16 * wave);
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int k = 2; k >= 0; --k) {
          const v4i h = frag(L.h[k], HS, t, 16 * j);
#pragma unroll
          for (int z = PP - 1; z >= 0; --z)
            acc[j] = RANK_LANES ? mfma<T_BF16>(pf[z], h, acc[j]) : mfma<T_BF16>(h, pf[z], acc[j]);
        }
    }
  };
  auto run = [&](int n) {  // whole lots of T tokens of the list, or (n < T) its last ones
    fetch(0, n);
    for (int from = 0;;) {
      __syncthreads();
      store();
      __syncthreads();
      from += T;
      const bool more = from + T <= n;
      if (more) fetch(from, T);
      add();
      if (!more) break;
    }
  };

  int have = 0;  // listed, not yet added
  for (int64_t t = tb; t < te; t += S::kScan) {
    // eight rows in a row for each thread
    const int64_t mine = t + 8 * tid;
    uint32_t hits = 0;
    if (mine + 8 <= te) {
      const int4 x = *reinterpret_cast<const int4*>(p.index + mine), y = *reinterpret_cast<const int4*>(p.index + mine + 4);
      hits = (x.x == a) | (x.y == a) << 1 | (x.z == a) << 2 | (x.w == a) << 3 | (y.x == a) << 4 | (y.y == a) << 5 |
             (y.z == a) << 6 | (y.w == a) << 7;
    } else {
      for (int e = 0; e < 8; ++e)
        if (mine + e < te && p.index[mine + e] == a) hits |= 1u << e;
    }
    int at = __builtin_popcount(hits);
    const int n = at;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
      const int o = __shfl_up(at, k);
      if (lane >= k) at += o;
    }
    __syncthreads();
    if (lane == 63) L.counts[wave] = at;
    __syncthreads();
    int all = have;
    at += have - n;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < wave) at += L.counts[w];
      all += L.counts[w];
    }
    for (uint32_t m = hits; m; m &= m - 1) L.list[at++] = (int)(mine - tb) + __builtin_ctz(m);
    __syncthreads();
    const int whole = all / T * T;
    if (whole) run(whole);
    have = all - whole;
    __syncthreads();
    const int keep = tid < have ? L.list[whole + tid] : 0;
    __syncthreads();
    if (tid < have) L.list[tid] = keep;
  }
  __syncthreads();
  if (have > 0) run(have);

  // lane l: column (rank) l % 16 of the tile, rows 4 (l / 16) + 0 .. 3
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int f = f0 + 16 * wave + (RANK_LANES ? 4 * q + e : fr), k = 16 * j + (RANK_LANES ? fr : 4 * q + e);
      if (f >= of.F || k >= p.r) continue;
      const int64_t at = blockIdx.z * numel + (RANK_LANES ? ((int64_t)a * of.F + f) * p.r + k : ((int64_t)a * p.r + k) * of.F + f);
      if (TO == T_FP32)
        static_cast<float*>(of.out)[at] = acc[j][e];
      else
        static_cast<uint16_t*>(of.out)[at] = (uint16_t)pack2<TO>(acc[j][e], 0.f);
    }
}

template <int TY, int TO, int RT>
__global__ void __launch_bounds__(256) k_sums(const SumArgs p) {
  __shared__ __attribute__((aligned(16))) SumLds<TY, RT> lds;
  const int b = blockIdx.x;
  if (b < p.blocks0)
    sum_block<TY, TO, RT, true>(p, p.of[0], p.numel[0], b, lds);
  else
    sum_block<TY, TO, RT, false>(p, p.of[1], p.numel[1], b - p.blocks0, lds);
}

// out = the parts added in order, of both gradients; numbers of elements multiples of 4.
struct PartsArgs {
  const float* in[2];
  void* out[2];
  int64_t numel[2];
};
template <int TO>
__global__ void __launch_bounds__(256) k_parts(const PartsArgs p, int parts) {
  const int64_t all = p.numel[0] + p.numel[1];
  for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; at < all; at += (int64_t)gridDim.x * 1024) {
    const int b = at >= p.numel[0];
    const int64_t i = at - (b ? p.numel[0] : 0);
    const float* in = p.in[b] + i;
    float4 s = *reinterpret_cast<const float4*>(in);
    for (int z = 1; z < parts; ++z) {
      const float4 x = *reinterpret_cast<const float4*>(in + z * p.numel[b]);
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    if (TO == T_FP32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out[b]) + i) = s;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out[b]) + i) = make_uint2(pack2<TO>(s.x, s.y), pack2<TO>(s.z, s.w));
  }
}

constexpr int64_t kSlotRows = 1024;  // up to here one block (wave) per token of a tile

int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }
int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// Splits of k_down over n columns: where its blocks are fewer than the compute units, down to two
// runs of 64 columns for each wave.
int down_splits(int64_t M, int64_t n, int64_t r) {
  const int64_t blocks = M <= kSlotRows ? M * ((r + 15) / 16) : (M + 31) / 32;
  const int64_t most = n / (2 * 64 * kDownWaves);
  int64_t s = blocks > 0 ? 256 / blocks : 1;
  s = s > most ? most : s;
  return (int)(s > 8 ? 8 : s < 1 ? 1 : s);
}

// Parts of the tokens of k_sums, each a multiple of 8 rows.
struct Parts {
  int count;
  int64_t per;
};
Parts sum_parts(int64_t M, int64_t L, int64_t d, int64_t n) {
  const int64_t blocks = L * ((d + 63) / 64 + (n + 63) / 64);
  int64_t z = (256 + blocks - 1) / blocks;
  const int64_t most = (M + 511) / 512;
  z = z > most ? most : z;
  z = z < 1 ? 1 : z;
  int64_t per = ((M + z - 1) / z + 7) / 8 * 8;
  per = per < 8 ? 8 : per;
  const int64_t c = (M + per - 1) / per;
  return {(int)(c < 1 ? 1 : c), per};
}

template <int TY>
hipError_t down(DownArgs a, int problems, hipStream_t st) {
  const int rt = a.rp / 16;
  a.slots = a.M <= kSlotRows ? (a.M < 16 ? (int)a.M : 16) : 0;
  const int tt = a.slots ? 1 : 2, per = a.slots ? 1 : rt > 4 ? 8 : rt > 2 ? 4 : rt;
  int64_t blocks = 0;
  for (int i = 0; i < problems; ++i) {
    const int64_t b = (a.M + 16 * tt - 1) / (16 * tt) * a.of[i].splits * ((rt + per - 1) / per) * (a.slots ? a.slots : 1);
    blocks = b > blocks ? b : blocks;
  }
  const dim3 grid((unsigned)blocks, (unsigned)problems);
  const int threads = 64 * kDownWaves;
  if (a.slots)
    k_down<TY, 1, 1><<<grid, threads, 0, st>>>(a);
  else if (per == 1)
    k_down<TY, 2, 1><<<grid, threads, 0, st>>>(a);
  else if (per == 2)
    k_down<TY, 2, 2><<<grid, threads, 0, st>>>(a);
  else if (per == 4)
    k_down<TY, 2, 4><<<grid, threads, 0, st>>>(a);
  else
    k_down<TY, 2, 8><<<grid, threads, 0, st>>>(a);
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

// Columns of a wave: at least 2048 waves where there are columns for them.
int64_t up_chunk(int64_t tiles, int64_t d) {
  int64_t chunk = 512;
  while (chunk > 64 && tiles * ((d + chunk - 1) / chunk) < 2048) chunk /= 2;
  return chunk;
}

template <int TY>
hipError_t up(UpArgs a, hipStream_t st) {
  a.slots = a.M <= kSlotRows ? (a.M < 16 ? (int)a.M : 16) : 0;
  const int tt = a.slots ? 1 : 2;
  const int64_t tiles = (a.M + 16 * tt - 1) / (16 * tt) * (a.slots ? a.slots : 1), chunk = up_chunk(tiles, a.d);
  a.chunk = (int)chunk;
  const dim3 grid((unsigned)((tiles * ((a.d + chunk - 1) / chunk) + 3) / 4));
  const bool wide = a.r % 8 == 0 && a.ld % 8 == 0;
  if (a.slots)
    wide ? up_kt<TY, 1, true>(a, grid, st) : up_kt<TY, 1, false>(a, grid, st);
  else
    wide ? up_kt<TY, 2, true>(a, grid, st) : up_kt<TY, 2, false>(a, grid, st);
  return hipGetLastError();
}

template <int TY, int TO>
void sums_rt(const SumArgs& a, dim3 grid, hipStream_t st) {
  if (a.rp <= 16)
    k_sums<TY, TO, 1><<<grid, 256, 0, st>>>(a);
  else if (a.rp <= 32)
    k_sums<TY, TO, 2><<<grid, 256, 0, st>>>(a);
  else if (a.rp <= 64)
    k_sums<TY, TO, 4><<<grid, 256, 0, st>>>(a);
  else
    k_sums<TY, TO, 8><<<grid, 256, 0, st>>>(a);
}

template <int TY>
hipError_t sums(SumArgs a, const Parts& z, int out_dtype, float* ws, hipStream_t st) {
  a.per = z.per;
  PartsArgs q{};
  for (int i = 0; i < 2; ++i) {
    a.numel[i] = q.numel[i] = (int64_t)a.L * a.of[i].F * a.r;
    q.out[i] = a.of[i].out;
    if (z.count > 1) a.of[i].out = ws + (i ? z.count * a.numel[0] : 0);
    q.in[i] = static_cast<const float*>(a.of[i].out);
  }
  a.blocks0 = (a.of[0].F + 63) / 64;
  const dim3 grid((unsigned)(a.blocks0 + (a.of[1].F + 63) / 64), (unsigned)a.L, (unsigned)z.count);
  if (z.count > 1 || out_dtype == T_FP32)
    sums_rt<TY, T_FP32>(a, grid, st);
  else
    sums_rt<TY, TY>(a, grid, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || z.count == 1) return e;
  const int64_t want = ((q.numel[0] + q.numel[1]) / 4 + 255) / 256;
  const unsigned blocks = (unsigned)(want < 2048 ? want : 2048);
  if (out_dtype == T_FP32)
    k_parts<T_FP32><<<blocks, 256, 0, st>>>(q, z.count);
  else
    k_parts<TY><<<blocks, 256, 0, st>>>(q, z.count);
  return hipGetLastError();
}

// The workspace: h, and for the gradients dh, A and B transposed, and the parts of the sums.
struct Ws {
  int64_t h, dh, at, bt, parts, bytes;
};
Ws carve(int64_t M, int64_t L, int64_t d, int64_t n, int64_t r, bool grads) {
  Ws w{};
  const int64_t rp = round16(r);
  int64_t at = up256(4 * M * rp * down_splits(M, n, r));
  if (grads) {
    w.dh = at;
    at += up256(4 * M * rp * down_splits(M, d, r));
    w.at = at;
    at += up256(2 * L * r * d);
    w.bt = at;
    at += up256(2 * L * n * rp);
    w.parts = at;
    const int64_t z = sum_parts(M, L, d, n).count;
    at += z > 1 ? up256(4 * z * L * r * (d + n)) : 0;
  }
  w.bytes = at;
  return w;
}

DownArgs down_args(const AdapterArgs& p) {
  DownArgs a{};
  a.index = p.index;
  a.M = p.M;
  a.L = (int)p.L;
  a.r = (int)p.r;
  a.rp = (int)round16(p.r);
  return a;
}

UpArgs up_args(const AdapterArgs& p) {
  UpArgs a{};
  a.index = p.index;
  a.scale = p.scale;
  a.base = static_cast<const uint8_t*>(p.base);
  a.Y = static_cast<uint8_t*>(p.Y);
  a.M = p.M;
  a.L = (int)p.L;
  a.rp = (int)round16(p.r);
  a.ranks = (int)p.r;
  return a;
}

template <int TY>
hipError_t fwd(const AdapterArgs& p, uint8_t* ws, hipStream_t st) {
  float* h = reinterpret_cast<float*>(ws);
  const int s = down_splits(p.M, p.n, p.r);
  DownArgs x = down_args(p);
  x.of[0] = Down{static_cast<const uint8_t*>(p.X), static_cast<const uint8_t*>(p.B), h, (int)p.n, s};
  const hipError_t e = down<TY>(x, 1, st);
  if (e != hipSuccess) return e;
  UpArgs y = up_args(p);
  y.H = h;
  y.splits = s;
  y.W = static_cast<const uint8_t*>(p.A);
  y.d = (int)p.d;
  y.r = y.ld = (int)p.r;
  return up<TY>(y, st);
}

template <int TY>
hipError_t bwd(const AdapterArgs& p, uint8_t* ws, hipStream_t st) {
  const Ws w = carve(p.M, p.L, p.d, p.n, p.r, true);
  const int rp = (int)round16(p.r), L = (int)p.L, d = (int)p.d, n = (int)p.n, r = (int)p.r;
  float *h = reinterpret_cast<float*>(ws), *dh = reinterpret_cast<float*>(ws + w.dh);
  uint16_t *at = reinterpret_cast<uint16_t*>(ws + w.at), *bt = reinterpret_cast<uint16_t*>(ws + w.bt);
  const uint8_t *X = static_cast<const uint8_t*>(p.X), *dY = static_cast<const uint8_t*>(p.dY);
  const int sh = down_splits(p.M, n, r), sd = down_splits(p.M, d, r);
  hipError_t e;
  if (p.M > 0) {
    TurnArgs t{};
    t.of[0] = Turn{static_cast<const uint16_t*>(p.A), at, d, r, d, (r + 31) / 32, (r + 31) / 32 * ((d + 31) / 32)};
    t.of[1] = Turn{static_cast<const uint16_t*>(p.B), bt, r, n, rp, (n + 31) / 32, (n + 31) / 32 * ((rp + 31) / 32)};
    k_turn<<<dim3(t.of[0].tiles + (p.Y ? t.of[1].tiles : 0), L), 256, 0, st>>>(t);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    DownArgs x = down_args(p);
    x.of[0] = Down{X, static_cast<const uint8_t*>(p.B), h, n, sh};
    x.of[1] = Down{dY, reinterpret_cast<const uint8_t*>(at), dh, d, sd};
    if ((e = down<TY>(x, 2, st)) != hipSuccess) return e;
    if (p.Y) {
      UpArgs y = up_args(p);
      y.H = dh;
      y.splits = sd;
      y.W = reinterpret_cast<const uint8_t*>(bt);
      y.d = n;
      y.r = y.ld = rp;  // (the padding is zeros on both sides)
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
  q.of[0] = Sum{dY, h, p.dA, d, sh};
  q.of[1] = Sum{X, dh, p.dB, n, sd};
  return sums<TY>(q, sum_parts(p.M, L, d, n), p.out_dtype, reinterpret_cast<float*>(ws + w.parts), st);
}

}  // namespace

// Blocks of the largest launch: a grid holds less than 2^32 work-items.
bool adapters_fit(int64_t M, int64_t d, int64_t n, int64_t r) {
  const int64_t slots = M < 16 ? (M < 1 ? 1 : M) : 16;
  const int64_t tiles = M <= kSlotRows ? (M + 15) / 16 * slots : (M + 31) / 32, widest = d > n ? d : n;
  const int64_t chunk = up_chunk(tiles, widest);
  const int64_t ups = tiles * ((widest + chunk - 1) / chunk) / 4 + 1, downs = tiles * ((r + 15) / 16) * 8;
  const int64_t turns = (d + 31) / 32 * ((r + 31) / 32) + (n + 31) / 32 * ((r + 31) / 32);
  const int64_t most = int64_t(1) << 32;
  return ups * 256 < most && (M <= kSlotRows ? downs : tiles) * 64 * kDownWaves < most && turns < (int64_t(1) << 31);
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
