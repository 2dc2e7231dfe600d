// Low-rank adapters of many requests beside a shared layer, for gfx950.
//
// Token row t belongs to adapter a = index[t] (none outside [0, L)):
//   h_t = B_a x_t,  Y_t = base_t + s_a A_a h_t           A: L x d x r, B: L x r x n
// and backwards, with dh_t = A_a^T dY_t:
//   dX_t = base_t + s_a B_a^T dh_t,  dA_a = sum_t s_a dY_t h_t^T,  dB_a = sum_t s_a dh_t x_t^T.
// k_down forms h (and dh, on A transposed), k_up the outputs (and dX, on B transposed), k_sums the
// factors' gradients.  h stays in binary32; where it meets 16-bit weights on the matrix cores it
// goes as a sum of two 16-bit numbers (16 or more significant bits, against the outputs' 8 or
// 11; of fp16 ranks below 2^-20 of the token's largest, 11 bits), and in the sums over tokens, whose
// results may be binary32, as a sum of three (24 bits).
#include "gemm_tile.h"

namespace intlora {

namespace {

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

// Two 16-bit numbers of a word.
template <int TY>
__device__ __forceinline__ f2 unpack2(uint32_t v) {
  if (TY == T_FP16) return __builtin_convertvector(__builtin_bit_cast(h2, v), f2);
  return f2{__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u)};
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

// The bf16 number at or next to v towards zero (v itself where it is not finite): the rest v - top
// is exact.
__device__ __forceinline__ float top_bf16(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }

// ---- few tokens: the adapters of a tile of 16 token rows, lane l that of token l % 16 (-1: none)
__device__ __forceinline__ int adapter_of(const int32_t* __restrict__ index, int64_t t, int64_t M, int L) {
  const int a = t < M ? index[t] : -1;
  return a >= 0 && a < L ? a : -1;
}
// The adapter of token `slot` if no earlier one of the tile has the same, else -1.
__device__ __forceinline__ int leader(int id, int slot) {
  const int a = __builtin_amdgcn_readlane(id, slot);
  const uint64_t m = __builtin_amdgcn_ballot_w64(id == a);
  // (in a scalar register for the compiler too, which would load lane by lane otherwise)
  return __builtin_amdgcn_readfirstlane(a >= 0 && (int)__builtin_ctzll(m) == slot ? a : -1);
}

// ---- more tokens: the rows of each adapter, in order
// Rows are taken `chunk` at a time (less than 2^31 bytes of any of the tensors, so that offsets
// inside fit 32 bits; one chunk as a rule).  For each chunk: order[] = its rows sorted by adapter, the ones
// without an adapter last (group L); group g has the places starts[g] .. starts[g + 1] - 1, and the
// tiles t32[g] .. of 32 places, t64[g] .. of 64, tp[g] .. of `part`.
struct Lists {
  int32_t *order, *starts, *t32, *t64, *tp;  // order: M; the others chunks x (L + 2)
  int64_t M, chunk;
  int L, part;
  __device__ __forceinline__ int rows(int c) const {
    const int64_t n = M - c * chunk;
    return (int)(n < chunk ? n : chunk);
  }
};

// For the gradients, out[a] (cols x ldo) = in[a] (rows x cols) transposed, zeros from column `rows` on, of
// both factors.
struct Turn {
  const uint16_t* in;
  uint16_t* out;
  int rows, cols, ldo, tiles_x, tiles;  // tiles of 64 x 64: along the columns, in all
};
struct ListArgs {
  const int32_t* index;
  Lists lists;
  int blocks;  // L + 1 for each chunk; the blocks behind them turn four tiles each
  Turn turn[2];
};

// A tile by 256 threads, 16 bytes at a time (rows of A that are no multiple of 8 long two numbers
// at a time, odd ones one by one): 16 adapters of 4096 x 64 and 64 x 4096 11.5 us with the lists (33 MB
// read and written; tiles of 32 x 32, a number a lane 25.5).
__device__ __forceinline__ void turn_tile(const ListArgs& p, int unit) {
  __shared__ __attribute__((aligned(16))) uint16_t tiles[4][64][66];
  auto& t = tiles[threadIdx.x >> 8];
  const int all = p.turn[0].tiles + p.turn[1].tiles, a = unit / all, in_a = unit - a * all;
  const bool live = a < p.lists.L, second = in_a >= p.turn[0].tiles;
  const Turn& w = p.turn[second];
  const int tile = in_a - (second ? p.turn[0].tiles : 0);
  const int y = threadIdx.x >> 3 & 31, x = (threadIdx.x & 7) * 8;
  const int64_t c0 = (int64_t)(tile % w.tiles_x) * 64, r0 = (int64_t)(tile / w.tiles_x) * 64;
  const uint16_t* in = w.in + (int64_t)a * w.rows * w.cols;
  uint16_t* out = w.out + (int64_t)a * w.cols * w.ldo;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t r = r0 + y + 32 * i, c = c0 + x;
    u4i v = u4i{0, 0, 0, 0};
    if (live && r < w.rows && c < w.cols) {
      const uint16_t* at = in + r * w.cols + c;
      if (w.cols % 8 == 0) {
        v = *reinterpret_cast<const u4i*>(at);
      } else if (w.cols % 2 == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + 2 * e < w.cols) v[e] = *reinterpret_cast<const uint32_t*>(at + 2 * e);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < w.cols) v[e / 2] |= (uint32_t)at[e] << 16 * (e & 1);
      }
    }
    uint32_t* to = reinterpret_cast<uint32_t*>(&t[y + 32 * i][x]);
#pragma unroll
    for (int e = 0; e < 4; ++e) to[e] = v[e];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t r = c0 + y + 32 * i, c = r0 + x;
    if (!live || r >= w.cols || c >= w.ldo) continue;
    u4i v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = t[x + 2 * e][y + 32 * i] | (uint32_t)t[x + 2 * e + 1][y + 32 * i] << 16;
    *reinterpret_cast<u4i*>(out + r * w.ldo + c) = v;  // (ldo is a multiple of 8)
  }
}

// A block for each group: it counts all rows by adapter in LDS, which gives its first place and
// tiles, and then lists its own.  Bound by latency for few adapters: 8192 rows of 16 7.2 us.  As every
// block counts all rows, the work is that of rows x adapters: 8192 rows of 512 and 4096 adapters 14 and
// 83 us, 32768 rows 30 and 192, where it is the longest kernel of the call; 641 rows of 4096 71.
constexpr int kMaxGroups = 4096 + 1;

__global__ void __launch_bounds__(1024) k_lists(const ListArgs p) {
  __shared__ int count[kMaxGroups];
  __shared__ int sums[16][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if ((int)blockIdx.x >= p.blocks) {
    turn_tile(p, ((int)blockIdx.x - p.blocks) * 4 + (tid >> 8));
    return;
  }
  const Lists& l = p.lists;
  const int groups = l.L + 1, c = blockIdx.x / groups, g = blockIdx.x - c * groups;
  const int rows = l.rows(c);
  const int32_t* index = p.index + c * l.chunk;
  for (int i = tid; i < groups; i += 1024) count[i] = 0;
  __syncthreads();
  // the groups of rows r .. r + 7 (-1 past the end)
  auto keys = [&](int r, int (&k)[8]) {
    if (r + 8 <= rows) {
      const int4 x = *reinterpret_cast<const int4*>(index + r), y = *reinterpret_cast<const int4*>(index + r + 4);
      k[0] = x.x, k[1] = x.y, k[2] = x.z, k[3] = x.w, k[4] = y.x, k[5] = y.y, k[6] = y.z, k[7] = y.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = r + e < rows ? index[r + e] : 0;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) k[e] = r + e >= rows ? -1 : k[e] >= 0 && k[e] < l.L ? k[e] : l.L;
  };
  int k[8];
  for (int r0 = 0; r0 < rows; r0 += 8192) {
    keys(r0 + 8 * tid, k);
    bool same = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) same = same && k[e] == __builtin_amdgcn_readfirstlane(k[0]);
    if (__builtin_amdgcn_ballot_w64(!same) == 0) {  // the wave's 512 rows at once
      if (lane == 0 && k[0] >= 0) atomicAdd(&count[k[0]], 512);
      continue;
    }
    int at = k[0], n = 1;  // neighbours of one group at once
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      if (k[e] == at) {
        ++n;
        continue;
      }
      if (at >= 0) atomicAdd(&count[at], n);
      at = k[e];
      n = 1;
    }
    if (at >= 0) atomicAdd(&count[at], n);
  }
  __syncthreads();
  int s[4] = {0, 0, 0, 0};  // places and tiles in front
  for (int i = tid; i < g; i += 1024) {
    const int n = count[i];
    s[0] += n;
    s[1] += (n + 31) / 32;
    s[2] += (n + 63) / 64;
    s[3] += (n + l.part - 1) / l.part;
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) {
#pragma unroll
    for (int y = 32; y; y >>= 1) s[x] += __shfl_xor(s[x], y);
    if (lane == 0) sums[wave][x] = s[x];
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    s[x] = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) s[x] += sums[w][x];
  }
  const int mine = count[g], at = c * (l.L + 2) + g;
  if (tid == 0) {
    l.starts[at] = s[0];
    l.t32[at] = s[1];
    l.t64[at] = s[2];
    l.tp[at] = s[3];
    if (g == l.L) {
      l.starts[at + 1] = s[0] + mine;
      l.t32[at + 1] = s[1] + (mine + 31) / 32;
      l.t64[at + 1] = s[2] + (mine + 63) / 64;
      l.tp[at + 1] = s[3] + (mine + l.part - 1) / l.part;
    }
  }
  if (mine == 0) return;
  int32_t* out = l.order + c * l.chunk + s[0];
  for (int r0 = 0; r0 < rows; r0 += 8192) {
    if (rows > 8192) keys(r0 + 8 * tid, k);  // (else they are still there)
    int n = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) n += k[e] == g;
    int before = n;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
      const int o = __shfl_up(before, x);
      if (lane >= x) before += o;
    }
    __syncthreads();
    if (lane == 63) sums[wave][0] = before;
    __syncthreads();
    before -= n;
    int all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      if (w < wave) before += sums[w][0];
      all += sums[w][0];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k[e] == g) out[before++] = r0 + 8 * tid + e;
    out += all;
  }
}

// The group, first place and places of a tile of SIZE places (0: `part`); rows = 0: there is no such
// tile.
struct Place {
  int group, at, rows;
};
template <int SIZE>
__device__ __forceinline__ Place find_tile(const Lists& l, int c, int tile) {
  const int32_t *t = (SIZE == 32 ? l.t32 : SIZE == 64 ? l.t64 : l.tp) + c * (l.L + 2), *starts = l.starts + c * (l.L + 2);
  const int lane = threadIdx.x & 63, last = l.L + 1;
  // the last group whose first tile is not behind this one: 64 at a time, before them every 128th
  int base = 0;
  if (last >= 64) {
    const uint64_t m = __builtin_amdgcn_ballot_w64(128 * lane <= last && t[128 * lane <= last ? 128 * lane : last] <= tile);
    base = 128 * (__builtin_popcountll(m) - 1);
  }
  int n = 0;
  for (int h = 0; h < (last >= 64 ? 2 : 1); ++h) {
    const int i = base + 64 * h + lane;
    n += __builtin_popcountll(__builtin_amdgcn_ballot_w64(i <= last && t[i <= last ? i : last] <= tile));
  }
  const int g = __builtin_amdgcn_readfirstlane(base + n - 1);
  if (g >= last) return Place{last, 0, 0};
  const int size = SIZE ? SIZE : l.part, at = starts[g] + size * (tile - t[g]), left = starts[g + 1] - at;
  return Place{g, __builtin_amdgcn_readfirstlane(at), __builtin_amdgcn_readfirstlane(left < size ? left : size)};
}

// h = W_a x of one or two problems (h and dh: blockIdx.y).
struct Down {
  const uint8_t* X;   // M x n
  const uint8_t* W;   // L x r x n
  float* H;           // splits x M x rp (NULL: not wanted)
  int n, splits;
  uint16_t* pieces;   // more tokens, one split: h scaled, in pieces, as k_split's (NULL: not wanted)
};

// The bf16 number at or next to v towards zero three times over, each of what the last one left, of
// four numbers: 24 bits in three pieces.
__device__ __forceinline__ void put_pieces(v4f v, uint16_t* out, int64_t stride) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    float t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      t[e] = top_bf16(v[e]);
      v[e] = finite(v[e]) ? v[e] - t[e] : 0.f;
    }
    *reinterpret_cast<uint2*>(out + k * stride) = make_uint2(pack2<T_BF16>(t[0], t[1]), pack2<T_BF16>(t[2], t[3]));
  }
}
struct DownArgs {
  Down of[2];
  const int32_t* index;
  const float* scale;
  Lists lists;
  int64_t M;
  int L, r, rp;
  int slots;  // few tokens: tokens of a tile of 16
};

// For few tokens: a block for each token of a tile of 16 and each 16 ranks, where the token is the
// first of its adapter in the tile: it takes all of that adapter's tokens there.  Its eight waves take
// runs of 64 columns in turn, and their sums meet in LDS, where they are added in order.  Lane l holds
// token l % 16 and ranks 4 (l / 16) + 0 .. 3.  Rows of other adapters read as zeros and are not
// written.  64 adapters of rank 64, n = 4096, a token each 10.3 us (34 MB, 3.3 TB/s; four waves a block
// 12.1).
constexpr int kDownWaves = 8;

template <int TY>
__global__ void __launch_bounds__(64 * kDownWaves) k_down_few(const DownArgs p) {
  __shared__ __attribute__((aligned(16))) float sums[kDownWaves][256];
  const Down& of = p.of[blockIdx.y];
  const int lane = threadIdx.x & 63, fr = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t groups = p.rp / 16;
  uint32_t rest = blockIdx.x;
  const int split = rest % of.splits;
  rest /= of.splits;
  const int g0 = rest % groups * 16;
  rest /= groups;
  const int64_t t0 = (int64_t)(rest / p.slots) * 16;
  if (t0 >= p.M) return;
  const int id = adapter_of(p.index, t0 + fr, p.M, p.L), a = leader(id, rest % p.slots);
  if (a < 0) return;
  const int rows = p.M - t0 < 16 ? (int)(p.M - t0) : 16;
  const uint32_t ld = (uint32_t)of.n * 2;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(of.X + t0 * ld, (int64_t)rows * ld);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(of.W + (int64_t)a * p.r * ld, (int64_t)p.r * ld);
  const uint32_t ox = id == a ? fr * ld : kOOB, ow = g0 + fr < p.r ? (g0 + fr) * ld : kOOB;
  // (lane q: 16 bytes each at 8 q and 32 + 8 q of a run; four runs in flight)
  constexpr int U = 8;
  const int first = 64 * (wave + kDownWaves * split), step = 64 * kDownWaves * of.splits;
  // The blocks of an XCD (each eighth one) start at different runs: rows are a power of two of bytes
  // apart as a rule, and blocks at the same columns would all be at the same few channels.
  const int runs = (of.n + step - 1) / step, turn = (int)((blockIdx.x >> 3) % runs);
  v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
  for (int run = 0; run < runs; run += U / 2) {
    v4i x[U], w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = run + u / 2, k = first + (i + turn < runs ? i + turn : i + turn - runs) * step;
      const int c = k + 32 * (u & 1) + 8 * q;
      const uint32_t o = i < runs && c < of.n ? 2u * c : kOOB;
      w[u] = load16(rw, (ow | o) & kOOB ? kOOB : ow + o);
      x[u] = load16(rx, (ox | o) & kOOB ? kOOB : ox + o);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) acc = mfma<TY>(w[u], x[u], acc);
  }
  *reinterpret_cast<v4f*>(&sums[wave][4 * lane]) = acc;
  __syncthreads();
  if (wave != 0 || id != a) return;
#pragma unroll
  for (int w = 1; w < kDownWaves; ++w) acc += *reinterpret_cast<const v4f*>(&sums[w][4 * lane]);
  *reinterpret_cast<v4f*>(of.H + (split * p.M + t0 + fr) * p.rp + g0 + 4 * q) = acc;
}

// For more tokens: a block computes 32 rows of one adapter x 16 RT ranks over one split of the columns.
// Stages of 256 bytes of the rows go through a ring of three LDS buffers filled by direct loads of
// 4 rows x 256 bytes (fragments straight from memory, 16 pieces of 64 bytes a load, took twice as
// long); each of the four waves takes a quarter of a stage, and their sums meet in LDS, where they are
// added in order.  Bound by the rows' way from memory (16384 x 4096, rank 16: 39 us, 3.5 TB/s) and, with
// more ranks, the factor's from L2 (rank 64 47 us, 128 69); 8192 x 4096, rank 64 26.9 us.  Tiles of 64
// rows read the factor half as often: 47 and 59 us for the same ranks at 16384 rows, 23.5 at 8192 in
// three splits, of which k_up's joining takes two back; deeper rings 33.
template <int RT_>
struct DownTile {
  static constexpr int RT = RT_, ROWS = 32 + 16 * RT, RING = 3, STAGE = ROWS * 256;
  static constexpr int LOADS = 2 + RT;  // direct loads of a wave and stage
  static constexpr int LDS = RING * STAGE;
  static_assert(4 * 2 * RT * 1024 <= LDS && LDS <= 160 * 1024, "the sums take the ring's place");
};

template <int TY, class C>
__global__ void __launch_bounds__(256) k_down(const DownArgs p) {
  constexpr int RT = C::RT;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const Down& of = p.of[blockIdx.y];
  const int lane = threadIdx.x & 63, fr = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = blockIdx.z, tile = blockIdx.x / of.splits, split = blockIdx.x - tile * of.splits;
  const Place pl = find_tile<32>(p.lists, c, tile);
  if (pl.rows <= 0 || pl.group >= p.L) return;
  const int a = pl.group;
  const int64_t first = c * p.lists.chunk;  // the chunk's first row, and first place
  const int row = (lane & 31) < pl.rows ? p.lists.order[first + pl.at + (lane & 31)] : -1;
  const int ld = of.n * 2, stages = (ld + 255) / 256;
  const int mine = stages > split ? (stages - split + of.splits - 1) / of.splits : 0;
  // (blocks of an XCD start at different stages, as in k_down_few)
  const int turn = mine > 0 ? (int)((blockIdx.x >> 3) % mine) : 0;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)lds;
  // Lane l of a load: row l / 16 of its four, whose 16-byte chunk k lies at k ^ row % 16.
  uint32_t ow[RT], ox[2];
  int cx[2], cw[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int k = 4 * (wave * RT + j) + q;
    cw[j] = 16 * (fr ^ (k & 15));
    ow[j] = k < p.r ? k * ld + cw[j] : kOOB;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = 8 * wave + 4 * i + q, r = __shfl(row, k);
    cx[i] = 16 * (fr ^ (k & 15));
    ox[i] = r >= 0 ? (uint32_t)r * ld + cx[i] : kOOB;
  }
  const uint8_t *px = of.X + first * ld, *pw = of.W + (int64_t)a * p.r * ld;
  const int bytes = p.lists.rows(c) * ld;
  auto issue = [&](int i, int place) {  // (stages past the last: loads of nothing, so that counts stay)
    const int at = i < mine ? (i + turn < mine ? i + turn : i + turn - mine) * of.splits + split : stages;
    const int k0 = at * 256, left = ld - k0;
    const rsrc_t rx = make_desc(px + k0, bytes - k0), rw = make_desc(pw + k0, p.r * ld - k0);
    const uint32_t S = lds0 + place * C::STAGE;
#pragma unroll
    for (int k = 0; k < 2; ++k) direct_load16(rx, S + (2 * wave + k) * 1024, cx[k] < left ? ox[k] : kOOB);
#pragma unroll
    for (int j = 0; j < RT; ++j) direct_load16(rw, S + 8192 + (wave * RT + j) * 1024, cw[j] < left ? ow[j] : kOOB);
  };
  v4f acc[2][RT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  issue(0, 0);
  issue(1, 1);
  int place = 0;
  const uint32_t at = fr * 256 + (((4 * wave + q) ^ fr) << 4);
  for (int i = 0; i < mine; ++i) {
    wait_loads<C::LOADS>();  // this stage has landed, and every wave is done with the one before
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
    const uint8_t* S = lds + place * C::STAGE + at;
    issue(i + 2, place == 0 ? 2 : place - 1);
    place = place == 2 ? 0 : place + 1;
    v4i x[2], w[RT];
#pragma unroll
    for (int t = 0; t < 2; ++t) x[t] = *reinterpret_cast<const v4i*>(S + t * 4096);
#pragma unroll
    for (int j = 0; j < RT; ++j) w[j] = *reinterpret_cast<const v4i*>(S + 8192 + j * 4096);
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t) acc[t][j] = mfma<TY>(w[j], x[t], acc[t][j]);
  }
  wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
  v4f* sums = reinterpret_cast<v4f*>(lds);
#pragma unroll
  for (int z = 0; z < 2 * RT; ++z) sums[(wave * 2 * RT + z) * 64 + lane] = acc[z & 1][z >> 1];
  __syncthreads();
#pragma unroll
  for (int y = 0; y < 2 * RT; y += 4) {
    const int z = y + wave;  // this wave's tile
    if (z >= 2 * RT) break;
    v4f s = sums[z * 64 + lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) s += sums[(w * 2 * RT + z) * 64 + lane];
    const int i = 16 * (z & 1) + fr, g = 16 * (z >> 1);
    if (i >= pl.rows || g >= p.rp) continue;
    const int64_t to = (first + pl.at + i) * p.rp + g + 4 * q;
    if (of.H) *reinterpret_cast<v4f*>(of.H + split * p.M * p.rp + to) = s;
    if (of.pieces) put_pieces(s * p.scale[a], of.pieces + to, p.M * p.rp);
  }
}

struct UpArgs {
  const float* H;       // splits x M x rp, by row (few tokens) or by place in the lists
  Lists lists;
  const uint8_t* W;     // L x d rows of ld elements, r of them used
  const int32_t* index;
  const float* scale;   // [L]
  const uint8_t* base;  // M x d, or NULL: zeros
  uint8_t* Y;           // M x d (may be base)
  int64_t M;
  int L, d, r, ld, rp, splits;
  int ranks;            // numbers of a row of H that count
  int slots;            // as k_down
  int chunk;            // output columns of a block (a multiple of 128)
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

// A token row's h, scaled, as the operand of the matrix cores: the sum of two 16-bit numbers each,
// and what to multiply the sums with.  Lane l: token l % 16, ranks 32 c + 8 (l / 16) + 0 .. 7.
// KT: steps of 32 of the rank.
//
// bf16 has binary32's range, and the two numbers hold 16 bits.  fp16 has not: a power of two brings the
// token's largest number into [1/2, 1), hi is what fp16 holds of each and lo 2^24 times the rest, which
// is at most 2^-12.  What lo leaves is 2^-12 of that rest, or 2^-49 where lo is subnormal itself; with
// k = -log2 of the number that is 24 bits of it while hi is normal (k <= 14), then 37 - k, so 16 up to
// k = 20, and never less than 11, fp16's own, down to k = 38.
template <int TY, int KT>
struct Low {
  v4i hi[KT], lo[KT];
  float back;

  // sum over the ranks of weights w and h; ROWS: the tokens are the matrix instruction's rows
  template <bool ROWS>
  __device__ __forceinline__ v4f times(const v4i (&w)[KT]) const {
    auto step = [&](const v4i& x, int c, v4f t) { return ROWS ? mfma<TY>(x, w[c], t) : mfma<TY>(w[c], x, t); };
    v4f t = v4f{0.f, 0.f, 0.f, 0.f};
    if (TY == T_FP16) {
#pragma unroll
      for (int c = 0; c < KT; ++c) t = step(lo[c], c, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] *= 0x1p-24f;
#pragma unroll
      for (int c = 0; c < KT; ++c) t = step(hi[c], c, t);
    } else {
#pragma unroll
      for (int c = 0; c < KT; ++c) {
        t = step(lo[c], c, t);
        t = step(hi[c], c, t);
      }
    }
    return t;
  }

  __device__ __forceinline__ void read(const UpArgs& p, int64_t t, bool mine, float s) {
    fill(p, mine, s, [&](int k, float (&v)[8]) {
      const float* h = p.H + t * p.rp + k;
#pragma unroll 4
      for (int z = 0; z < p.splits; ++z) {
        const float4 *o = reinterpret_cast<const float4*>(h + z * p.M * p.rp), x = o[0], y = o[1];
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
        v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
      }
    });
  }

  // add(k, v): adds h of ranks k .. k + 7 to v
  template <class Add>
  __device__ __forceinline__ void fill(const UpArgs& p, bool mine, float s, Add add) {
    const int q = (threadIdx.x & 63) >> 4;
    float v[KT][8];
#pragma unroll
    for (int c = 0; c < KT; ++c) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = 0.f;
      const int k = 32 * c + 8 * q;
      if (!mine || k >= p.rp) continue;
      add(k, v[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = k + e < p.ranks ? v[c][e] * s : 0.f;  // (an infinite x leaves NaN past them)
    }
    // fp16: a power of two per token brings its largest finite |h| into [1/2, 1)
    back = 1.f;
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
        back = __uint_as_float((uint32_t)(e + 127) << 23);
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
        uint32_t t2, b;
        if (TY == T_FP16) {
          t2 = pack2<T_FP16>(x, y);
          const f2 w = unpack2<T_FP16>(t2);
          b = pack2<T_FP16>(finite(w.x) ? (x - w.x) * 0x1p24f : 0.f, finite(w.y) ? (y - w.y) * 0x1p24f : 0.f);
        } else {
          const float tx = top_bf16(x), ty = top_bf16(y);
          t2 = pack2<T_BF16>(tx, ty);
          b = pack2<T_BF16>(finite(x) ? x - tx : 0.f, finite(y) ? y - ty : 0.f);
        }
        hi[c][e] = (int)t2;
        lo[c][e] = (int)b;
      }
  }
};

// Y = base + s_a W_a h.  Row m of the matrix instruction's tile u is column 8 (m / 4) + 4 u + m % 4,
// so lane l ends up with columns 8 (l / 16) + 0 .. 7 of token l % 16.
//
// For few tokens: a block for each token of a tile of 16 (as k_down_few), its four waves 32 columns
// in turn.  Bound by the factors' bytes: the next columns' weights are loaded while these are at
// work, the first ones before h is there (64 adapters of 14336 x 64, a token each 28.5 us: 121 MB, 4.2
// TB/s).
template <int TY, int KT, bool WIDE>
__global__ void __launch_bounds__(256) k_up_few(const UpArgs p) {
  const int lane = threadIdx.x & 63, fr = lane & 15, q = lane >> 4;
  const uint32_t tokens = (uint32_t)((p.M + 15) / 16) * p.slots;
  const uint32_t block = blockIdx.x / tokens, in = blockIdx.x - block * tokens;
  const int slot = in % p.slots;
  const int64_t t = (int64_t)(in / p.slots) * 16 + fr;  // this lane's token
  const int id = adapter_of(p.index, t, p.M, p.L), a = leader(id, slot);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = (int)block * p.chunk + 32 * wave, c1 = (int)block * p.chunk + p.chunk;
  // Steps of 128 columns; the blocks of an XCD start at different ones (as in k_down_few).
  const int steps = p.chunk / 128, turn = (int)((blockIdx.x >> 3) % steps);
  auto column = [&](int step) { return first + 128 * (step + turn < steps ? step + turn : step + turn - steps); };
  if (a >= 0) {
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
    load(column(0), cur);
    const bool mine = id == a;
    Low<TY, KT> h;
    h.read(p, t, mine, p.scale[a]);
    for (int step = 0; step < steps; ++step) {
      const int col = column(step) + 8 * q;
      u4i b = u4i{0, 0, 0, 0};
      if (p.base && mine && col < p.d) b = *reinterpret_cast<const u4i*>(p.base + 2 * (t * p.d + col));
      Cols next;
      load(step + 1 < steps ? column(step + 1) : p.d, next);
      __builtin_amdgcn_sched_barrier(0);
      v4f acc[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) acc[u] = h.template times<false>(cur.w[u]);
      if (mine && col < p.d) {
        u4i y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f2 f = unpack2<TY>(b[e]);
          const v4f& v = acc[e / 2];
          y[e] = pack2<TY>(f.x + v[2 * (e & 1)] * h.back, f.y + v[2 * (e & 1) + 1] * h.back);
        }
        *reinterpret_cast<u4i*>(p.Y + 2 * (t * p.d + col)) = y;
      }
      cur = next;
    }
  }
  // Rows without an adapter: the base's (nothing to do in place).
  if (p.base == p.Y || slot != 0 || id >= 0 || t >= p.M) return;
  for (int col = first + 8 * q; col < c1 && col < p.d; col += 128) {
    u4i b = u4i{0, 0, 0, 0};
    if (p.base) b = *reinterpret_cast<const u4i*>(p.base + 2 * (t * p.d + col));
    *reinterpret_cast<u4i*>(p.Y + 2 * (t * p.d + col)) = b;
  }
}

// Both steps in one launch, for few tokens and up to 16 ranks: a block for each token of a tile of 16 (as
// above) and 256 columns forms h itself, as k_down_few does, and then 32 columns each wave.  Every
// block of a token reads all of B_a, from L2 but for the first: 35 GB/s of a compute unit, so this
// pays as long as that takes less than a launch.  Bound by latency, the launch and two chains of loads:
// 4096 x 4096, rank 16, 1 token 8 us.
constexpr int kTokenCols = 256;

template <int TY, bool WIDE>
__global__ void __launch_bounds__(64 * kDownWaves) k_token(const Down of, const UpArgs p) {
  __shared__ __attribute__((aligned(16))) float sums[kDownWaves][256];
  const int lane = threadIdx.x & 63, fr = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tokens = (uint32_t)((p.M + 15) / 16) * p.slots;
  const uint32_t block = blockIdx.x / tokens, in = blockIdx.x - block * tokens;
  const int slot = in % p.slots;
  const int64_t t0 = (int64_t)(in / p.slots) * 16, t = t0 + fr;
  const int id = adapter_of(p.index, t, p.M, p.L), a = leader(id, slot);
  const int n0 = (int)block * kTokenCols + 32 * wave, col = n0 + 8 * q;
  const bool mine = id == a;
  if (a >= 0) {
    const uint16_t* W = reinterpret_cast<const uint16_t*>(p.W) + (int64_t)a * p.d * p.ld;
    v4i w[2][1];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = n0 + 8 * (fr >> 2) + 4 * u + (fr & 3);
      w[u][0] = row8<WIDE>(W + (int64_t)row * p.ld, row < p.d ? 8 * q : p.r, p.r);
    }
    u4i b = u4i{0, 0, 0, 0};
    if (p.base && mine && col < p.d) b = *reinterpret_cast<const u4i*>(p.base + 2 * (t * p.d + col));
    const float s = p.scale[a];
    const int rows = p.M - t0 < 16 ? (int)(p.M - t0) : 16;
    const uint32_t ld = (uint32_t)of.n * 2;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(of.X + t0 * ld, (int64_t)rows * ld);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(of.W + (int64_t)a * p.ranks * ld, (int64_t)p.ranks * ld);
    const uint32_t ox = mine ? fr * ld : kOOB, ow = fr < p.ranks ? fr * ld : kOOB;
    constexpr int U = 8, step = 64 * kDownWaves;
    v4f part = v4f{0.f, 0.f, 0.f, 0.f};
    for (int k = 64 * wave; k < of.n; k += U / 2 * step) {
      v4i x[U], v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = k + u / 2 * step + 32 * (u & 1) + 8 * q;
        const uint32_t o = c < of.n ? 2u * c : kOOB;
        v[u] = load16(rw, (ow | o) & kOOB ? kOOB : ow + o);
        x[u] = load16(rx, (ox | o) & kOOB ? kOOB : ox + o);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) part = mfma<TY>(v[u], x[u], part);
    }
    *reinterpret_cast<v4f*>(&sums[wave][4 * lane]) = part;
    __syncthreads();
    Low<TY, 1> h;
    h.fill(p, mine, s, [&](int k, float (&v)[8]) {  // lane l of a wave's part: token l % 16, ranks 4 (l / 16) ..
#pragma unroll
      for (int z = 0; z < kDownWaves; ++z) {
        const float* o = &sums[z][4 * (fr + 4 * k)];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] += o[e];
          v[4 + e] += o[64 + e];
        }
      }
    });
    u4i y;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const v4f acc = h.template times<false>(w[u]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const f2 f = unpack2<TY>(b[2 * u + e]);
        y[2 * u + e] = pack2<TY>(f.x + acc[2 * e] * h.back, f.y + acc[2 * e + 1] * h.back);
      }
    }
    if (mine && col < p.d) *reinterpret_cast<u4i*>(p.Y + 2 * (t * p.d + col)) = y;
  }
  // Rows without an adapter: the base's (nothing to do in place).
  if (p.base == p.Y || slot != 0 || id >= 0 || t >= p.M || col >= p.d) return;
  u4i b = u4i{0, 0, 0, 0};
  if (p.base) b = *reinterpret_cast<const u4i*>(p.base + 2 * (t * p.d + col));
  *reinterpret_cast<u4i*>(p.Y + 2 * (t * p.d + col)) = b;
}

// Rows of `chunks` 16-byte chunks in LDS, chunk c of row m at c ^ turned(m): the 16 lanes that read a
// chunk of rows 0 .. 15 at a time are on different banks (a power of two of chunks; rows of other
// lengths spread by themselves).
__device__ __forceinline__ int turned(int m, int chunks) {
  return chunks == 16 ? m : chunks == 8 ? m >> 1 : chunks == 4 ? m >> 2 : chunks == 2 ? m >> 3 : 0;
}

// For more tokens: a block takes 64 rows of one adapter, 16 each wave, and 128 columns at a time.  The
// columns' weights go through two LDS buffers filled by direct loads, for all four waves.  Here the
// tokens are the matrix instruction's rows, and row m of the weights' tile u is column 8 m + u: a
// lane ends up with columns 8 (l % 16) + 0 .. 7 of tokens 4 (l / 16) + 0 .. 3, so that rows are read and
// written in runs of 256 bytes with no step through LDS.  The next columns' rows of the base are
// loaded while these are at work.  Rows without an adapter (the last group) take the base's values.
// Bound by memory and by the last tiles: 8192 x 4096, rank 64 38 us (134 MB read and written, 3.5 TB/s;
// one adapter, without partly filled tiles, 32).  Weights straight from memory to registers took 51,
// sums turned to rows in LDS with one block to a unit 80.
template <int TY, int KT>
__global__ void __launch_bounds__(256) k_up(const UpArgs p) {
  constexpr int NL = 2 * KT, BUF = 4 * NL * 1024;  // direct loads of a wave; bytes of a buffer
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * BUF];
  const int lane = threadIdx.x & 63, fr = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int chunks = (p.d + p.chunk - 1) / p.chunk, tile = blockIdx.x / chunks, block = blockIdx.x - tile * chunks;
  const int c = blockIdx.y;
  const Place pl = find_tile<64>(p.lists, c, tile);
  if (pl.rows <= 0 || (pl.group >= p.L && p.base == p.Y)) return;
  const int a = pl.group;
  const int64_t first = c * p.lists.chunk;  // the chunk's first row, and first place
  const int at = 16 * wave + fr;            // this lane's place in the tile
  const int row = at < pl.rows ? p.lists.order[first + pl.at + at] : -1;
  const int ldo = 2 * p.d;
  uint32_t ro[4];  // of this lane's tokens of the outputs
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = __shfl(row, 4 * q + e);
    ro[e] = r >= 0 ? (uint32_t)r * ldo : kOOB;
  }
  const int64_t bytes = (int64_t)p.lists.rows(c) * ldo;
  const __amdgpu_buffer_rsrc_t ry = make_rsrc(p.Y + first * ldo, bytes);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.base ? p.base + first * ldo : p.Y, p.base ? bytes : 0);
  const int c0 = block * p.chunk, steps = p.chunk / 128, turn = (int)((blockIdx.x >> 3) % steps);
  auto column = [&](int step) { return c0 + 128 * (step + turn < steps ? step + turn : step + turn - steps); };
  auto place = [&](int e, int col) { return col < p.d && ro[e] != kOOB ? ro[e] + 2 * col : kOOB; };  // of eight columns
  struct Rows {
    v4i v[4];
  };
  auto fetch = [&](int step, Rows& b) {
    const int col = step < steps ? column(step) + 8 * fr : p.d;
#pragma unroll
    for (int e = 0; e < 4; ++e) b.v[e] = load16(rb, place(e, col));
  };
  if (a >= p.L) {
    for (int step = 0; step < steps; ++step) {
      Rows b;
      fetch(step, b);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4i, b.v[e]), ry, place(e, column(step) + 8 * fr), 0, 0);
    }
    return;
  }
  // Weights in LDS: rows of `per` chunks of 16 bytes, row 16 u + m holds column 8 m + u, its chunk k at
  // k ^ turned(m): the 16 rows of a fragment are on different banks.
  const int per = p.ld / 8;
  uint32_t wo[NL];
#pragma unroll
  for (int j = 0; j < NL; ++j) {
    const int k = 64 * (wave * NL + j) + lane, R = k / per, m = R & 15;
    wo[j] = R < 128 ? 16 * ((8 * m + (R >> 4)) * per + ((k - R * per) ^ turned(m, per))) : kOOB;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)lds + wave * NL * 1024;
  const uint8_t* W = p.W + (int64_t)a * p.d * p.ld * 2;
  auto issue = [&](int step) {
    const int col = step < steps ? column(step) : p.d;
    const int64_t left = (int64_t)(p.d - col) * p.ld * 2;
    const int bytes = col < p.d ? (int)(left < 65536 ? left : 65536) : 0;
    const rsrc_t rw = make_desc(col < p.d ? W + (int64_t)col * p.ld * 2 : W, bytes);
#pragma unroll
    for (int j = 0; j < NL; ++j) direct_load16(rw, lds0 + (step & 1) * BUF + 1024 * j, wo[j]);
  };
  Rows b0, b1;
  issue(0);
  fetch(0, b0);
  __builtin_amdgcn_sched_barrier(0);
  Low<TY, KT> h;
  float back[4];
  h.read(p, first + pl.at + at, row >= 0, p.scale[a]);
#pragma unroll
  for (int e = 0; e < 4; ++e) back[e] = TY == T_FP16 ? __shfl(h.back, 4 * q + e) : 1.f;
  auto one = [&](int step, Rows& cur, Rows& next) {
    // this step's weights have landed (newer: its rows of the base and the last step's stores)
    if (step == 0)
      wait_loads<4>();
    else
      wait_loads<8>();
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
    issue(step + 1);
    fetch(step + 1, next);
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* S = lds + (step & 1) * BUF;
    v4f acc[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      v4i w[KT];
#pragma unroll
      for (int x = 0; x < KT; ++x) {
        const int k = 4 * x + q;
        w[x] = k < per ? *reinterpret_cast<const v4i*>(S + 16 * ((16 * u + fr) * per + (k ^ turned(fr, per))))
                       : v4i{0, 0, 0, 0};
      }
      acc[u] = h.template times<true>(w);
    }
    const int col = column(step) + 8 * fr;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u4i y;
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const f2 g = unpack2<TY>((uint32_t)cur.v[e][z]);
        y[z] = pack2<TY>(g.x + acc[2 * z][e] * back[e], g.y + acc[2 * z + 1][e] * back[e]);
      }
      __builtin_amdgcn_raw_buffer_store_b128(y, ry, place(e, col), 0, 0);
    }
  };
  for (int step = 0; step < steps; step += 2) {
    one(step, b0, b1);
    if (step + 1 < steps) one(step + 1, b1, b0);
  }
  wait_loads<0>();  // the weights loaded past the last step (zeros)
}

// Rows of `ld` numbers of rows of r, zeros behind them, so that direct loads bring whole 16 bytes of
// ranks that are no multiple of 8.  Bound by the launch for all but the largest sets of adapters.
__global__ void __launch_bounds__(256) k_pad(const uint16_t* __restrict__ in, uint16_t* __restrict__ out, int64_t units,
                                             int r, int ld) {
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    const int per = ld / 8;
    const int64_t row = u / per;
    const v4i v = row8<false>(in + row * r, (int)(u - row * per) * 8, r);
    *reinterpret_cast<v4i*>(out + u * 8) = v;
  }
}

// Launches of kernels with more LDS than the default limit.
template <class K>
hipError_t allow_lds(K kernel, int bytes, int& ready_dev) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess || dev == ready_dev) return e;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) ready_dev = dev;
  return e;
}

template <int TY, class C>
hipError_t launch_down(const DownArgs& a, dim3 grid, hipStream_t st) {
  static thread_local int ready_dev = -1;
  const hipError_t e = allow_lds(&k_down<TY, C>, C::LDS, ready_dev);
  if (e != hipSuccess) return e;
  k_down<TY, C><<<grid, 256, C::LDS, st>>>(a);
  return hipGetLastError();
}

// h and dh, scaled, as three bf16 numbers each (24 bits) for k_sums: planes x M x rp, by place in the
// lists.  Rows without an adapter are left out.
struct Split {
  const float* H;  // splits x M x rp
  uint16_t* out;
  int splits;
};
struct SplitArgs {
  Split of[2];
  const int32_t* index;
  const float* scale;
  Lists lists;
  int64_t M;
  int L, rp;
  int by_row;  // H's order: rows (few tokens) or places
};
__global__ void __launch_bounds__(256) k_split(const SplitArgs p) {
  const Split& of = p.of[blockIdx.y];
  const int per = p.rp / 4;
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x, place = u / per;
  if (place >= p.M) return;
  const int64_t row = place / p.lists.chunk * p.lists.chunk + p.lists.order[place];
  const int a = p.index[row];
  if (a < 0 || a >= p.L) return;
  const float s = p.scale[a];
  const float* H = of.H + (p.by_row ? row : place) * p.rp + 4 * (u - place * per);
  float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int z = 0; z < of.splits; ++z) {
    const float4 x = *reinterpret_cast<const float4*>(H + z * p.M * p.rp);
    h.x += x.x, h.y += x.y, h.z += x.z, h.w += x.w;
  }
  put_pieces(v4f{h.x * s, h.y * s, h.z * s, h.w * s}, of.out + 4 * u, p.M * p.rp);
}

struct Sum {
  const uint8_t* P;   // M x F token rows (dY or X)
  const uint16_t* H;  // 3 x M x rp (h or dh of k_split)
  void* out;          // L x F x r (dA) or L x r x F (dB)
  int F;
};
struct SumArgs {
  Sum of[2];         // dA, dB
  Lists lists;
  int64_t M;
  int L, r, rp;
  int blocks0;   // blocks of 128 columns of the first one
  int parts;     // of a chunk at most, each with sums of its own (float); 0: a block takes all of an adapter
  int64_t each;  // numbers of a part: d r of dA's, then r n of dB's
};

// sum over an adapter's tokens of P_t h_t^T s_a.  A block takes 128 columns of P, all ranks and all of
// the adapter's rows, or one of the parts that they are cut into, T of them at a time, each wave 32
// columns x 16 RT ranks; the next ones are loaded meanwhile.  Both operands have the contraction
// (tokens) in rows and leave LDS through the transposing reads.  h is three bf16 numbers; fp16 rows of P
// become two (exact).  4099 rows of 5 adapters, 2560 and 640 columns in fp16, rank 20: 14.1 us, a chain of
// LDS writes, barriers and products per 64 rows, with three blocks to a unit (rows padded to other
// banks instead of turned, and two blocks: 18; h split here, 64 columns a block and rows cut by range
// instead of by adapter: 43).
template <int TY, int RT>
struct SumLds {
  static constexpr int PP = TY == T_FP16 ? 2 : 1, T = RT == 8 ? 32 : 64;
  static constexpr int F = 128, PS = F, HS = 16 * RT;  // row strides (16-bit numbers)
  static constexpr int kList = 512;                    // rows' numbers at a time
  uint16_t p[PP][T * PS];
  uint16_t h[3][T * HS];
  int list[kList];
};

// Where column c of a row is: the 32 bytes that half a wave reads of each of 8 rows are on different
// banks, and so are 16 lanes' writes of 16 bytes.
__device__ __forceinline__ int spread(int row, int c, int stride) {
  return c ^ 16 * (row / (128 / stride) % (stride / 16));
}

template <int TY, int TO, int RT, bool RANK_LANES>
__device__ __forceinline__ void sum_block(const SumArgs& p, const Sum& of, int block, SumLds<TY, RT>& L) {
  using S = SumLds<TY, RT>;
  constexpr int PP = S::PP, T = S::T, PS = S::PS, HS = S::HS, NT = S::F / 64;
  constexpr int NP = T / 16, NH = (6 * T * RT + 255) / 256;  // 16-byte loads of a thread
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, fr = lane & 15, q = lane >> 4;
  const int f0 = block * S::F, c0 = p.parts ? blockIdx.z : 0;
  const int chunks = p.parts ? c0 + 1 : (int)((p.M + p.lists.chunk - 1) / p.lists.chunk);
  int a = blockIdx.y;
  Place pl{};
  if (p.parts) {
    pl = find_tile<0>(p.lists, c0, blockIdx.y);
    a = pl.group;
    if (pl.rows <= 0 || a >= p.L) return;
  }
  v4f acc[NT][RT];
#pragma unroll
  for (int j = 0; j < NT * RT; ++j) acc[j / RT][j % RT] = v4f{0.f, 0.f, 0.f, 0.f};
  struct Lot {
    u4i p[NP], h[NH];
  };
  Lot lot;

  // places at + from .. at + n - 1, at most T: zeros behind them; list: their rows from `at` on
  auto fetch = [&](int64_t first, int at0, int from, int n) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int row = (tid >> 4) + 16 * i, c = (tid & 15) * 8;
      lot.p[i] = u4i{0, 0, 0, 0};
      if (from + row < n && f0 + c < of.F)
        lot.p[i] = *reinterpret_cast<const u4i*>(of.P + 2 * ((first + L.list[from + row]) * of.F + f0 + c));
    }
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const int at = tid + 256 * i, k = at / (2 * RT * T), in = at % (2 * RT * T), row = in / (2 * RT), c = in % (2 * RT) * 8;
      lot.h[i] = u4i{0, 0, 0, 0};
      if (k < 3 && from + row < n && c < p.rp)
        lot.h[i] = *reinterpret_cast<const u4i*>(of.H + (k * p.M + first + at0 + from + row) * p.rp + c);
    }
  };
  auto store = [&]() {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int row = (tid >> 4) + 16 * i, at = row * PS + spread(row, (tid & 15) * 8, PS);
      if (TY == T_FP16) {
        u4i t, b;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f2 x = unpack2<T_FP16>(lot.p[i][e]);
          const f2 y = f2{top_bf16(x.x), top_bf16(x.y)};
          t[e] = pack2<T_BF16>(y.x, y.y);
          b[e] = pack2<T_BF16>(finite(x.x) ? x.x - y.x : 0.f, finite(x.y) ? x.y - y.y : 0.f);
        }
        *reinterpret_cast<u4i*>(&L.p[0][at]) = t;
        *reinterpret_cast<u4i*>(&L.p[PP - 1][at]) = b;
      } else {
        *reinterpret_cast<u4i*>(&L.p[0][at]) = lot.p[i];
      }
    }
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const int at = tid + 256 * i, k = at / (2 * RT * T), in = at % (2 * RT * T), row = in / (2 * RT), c = in % (2 * RT) * 8;
      if (k < 3) *reinterpret_cast<u4i*>(&L.h[k][row * HS + spread(row, c, HS)]) = lot.h[i];
    }
  };
  // Rows row + 4 q + 0 .. 3 and 16 further of column col + fr: in both operands the same ones.
  auto frag = [&](const uint16_t* m, int stride, int row, int col) {
    const int R = row + 4 * q + (fr >> 2);
    const uint16_t* at = m + R * stride + spread(R, col + 4 * (fr & 3), stride);
    const int2 x = __builtin_bit_cast(int2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t)at));
    const int2 y = __builtin_bit_cast(int2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t)(at + 16 * stride)));
    return v4i{x.x, x.y, y.x, y.y};
  };
  auto add = [&]() {
#pragma unroll
    for (int t = 0; t < T; t += 32) {
      v4i pf[NT][PP];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int k = 0; k < PP; ++k) pf[i][k] = frag(L.p[k], PS, t, 32 * wave + 16 * i);
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int k = 2; k >= 0; --k) {
          const v4i h = frag(L.h[k], HS, t, 16 * j);
#pragma unroll
          for (int z = PP - 1; z >= 0; --z)
#pragma unroll
            for (int i = 0; i < NT; ++i)
              acc[i][j] = RANK_LANES ? mfma<T_BF16>(pf[i][z], h, acc[i][j]) : mfma<T_BF16>(h, pf[i][z], acc[i][j]);
        }
    }
  };
  for (int c = c0; c < chunks; ++c) {
    const int64_t first = c * p.lists.chunk;  // the chunk's first row, and first place
    const int32_t* starts = p.lists.starts + c * (p.L + 2) + a;
    const int r0 = p.parts ? pl.at : starts[0], r1 = p.parts ? pl.at + pl.rows : starts[1];
    for (int at = r0; at < r1; at += S::kList) {
      const int n = r1 - at < S::kList ? r1 - at : S::kList;
      __syncthreads();
      for (int i = tid; i < n; i += 256) L.list[i] = p.lists.order[first + at + i];
      __syncthreads();
      fetch(first, at, 0, n);
      for (int from = 0; from < n; from += T) {
        __syncthreads();
        store();
        __syncthreads();
        fetch(first, at, from + T, n);
        __builtin_amdgcn_sched_barrier(0);
        add();
      }
    }
  }

  const int64_t to = p.parts ? ((int64_t)c0 * p.parts + blockIdx.y) * p.each + (RANK_LANES ? 0 : (int64_t)p.of[0].F * p.r)
                             : (int64_t)a * of.F * p.r;
  // lane l: column (rank) l % 16 of the tile, rows 4 (l / 16) + 0 .. 3
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int f = f0 + 32 * wave + 16 * i + (RANK_LANES ? 4 * q + e : fr), k = 16 * j + (RANK_LANES ? fr : 4 * q + e);
        if (f >= of.F || k >= p.r) continue;
        const int64_t at = to + (RANK_LANES ? (int64_t)f * p.r + k : (int64_t)k * of.F + f);
        if (TO == T_FP32)
          static_cast<float*>(of.out)[at] = acc[i][j][e];
        else
          static_cast<uint16_t*>(of.out)[at] = (uint16_t)pack2<TO>(acc[i][j][e], 0.f);
      }
}

template <int TY, int TO, int RT>
__global__ void __launch_bounds__(256) k_sums(const SumArgs p) {
  __shared__ __attribute__((aligned(16))) SumLds<TY, RT> lds;
  const int b = blockIdx.x;
  if (b < p.blocks0)
    sum_block<TY, TO, RT, true>(p, p.of[0], b, lds);
  else
    sum_block<TY, TO, RT, false>(p, p.of[1], b - p.blocks0, lds);
}

// An adapter's gradients: its parts added in order.  d and n are multiples of 8.
struct PartsArgs {
  const float* in;
  void *dA, *dB;
  Lists lists;
  int chunks, parts, na;  // na = d r
  int64_t each;
};
template <int TO>
__global__ void __launch_bounds__(256) k_parts(const PartsArgs p) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int a = blockIdx.y;
  if (i >= p.each) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = 0; c < p.chunks; ++c) {
    const int32_t* t = p.lists.tp + c * (p.lists.L + 2) + a;
    const int z1 = t[1];
#pragma unroll 4
    for (int z = t[0]; z < z1; ++z) {
      const float4 x = *reinterpret_cast<const float4*>(p.in + ((int64_t)c * p.parts + z) * p.each + i);
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
  }
  const int64_t at = i < p.na ? (int64_t)a * p.na + i : a * (p.each - p.na) + i - p.na;
  void* out = i < p.na ? p.dA : p.dB;
  if (TO == T_FP32)
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = s;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack2<TO>(s.x, s.y), pack2<TO>(s.z, s.w));
}

// Few tokens take a block for each token of a tile of 16, without lists; more are listed by adapter
// first.  Without lists a row costs its adapter's bytes again, with them each adapter (of how many the
// host knows only that they are at most L and M) a tile that is filled in part, and the lists 7 us.
// us of the kernels without and with lists, 4096 x 4096: rank 16, one adapter, 128 rows 15.0 and 17.3;
// 8 adapters, 200 rows 20 and 18; 64, 256 rows 21 and 27; 512, 256 rows 22 and 58.  Rank 64: one, 64
// rows 19 and 22, 128 rows 32 and 22; 8, 64 rows 17 and 21, 128 rows 26 and 21; 64, 128 rows 28 and 33,
// 256 rows 45 and 36; 512, 256 rows 54 and 92.  14336 x 4096, rank 64: one, 48 rows 29 and 21; 64, 96
// rows 47 and 58, 256 rows 97 and 78.  640 x 640, 256 rows, one: rank 16 8.8 and 15.7, rank 64 19 and
// 19.  The gradients need lists in any case (2560 x 640, rank 20, us without the launches that both have:
// 33 rows 13.0 and 14.5, 100 rows 16.8 and 15.4, 200 rows 24 and 15; 4096 x 4096, rank 64, 200 rows 57
// and 21).  At 640 rows the rule stops, and from there to about as many rows as 2 to 4 times the
// adapters those without lists would still be faster where there are hundreds (4096 x 4096, without and
// with lists: rank 16, 512 adapters, 641 rows 37 and 92, 1024 50 and 106, 2048 91 and 94; 2048 adapters,
// 641 rows 39 and 154, 4096 204 and 270; rank 64, 512, 641 rows 110 and 147, 2048, 641 rows 129 and 237,
// 2048 rows 333 and 394, 4096 rows 622 and 464).
bool few_rows(int64_t M, int64_t L, int64_t d, int64_t n, int64_t r, bool grads) {
  if (grads) return M <= 64;
  return M <= 640 && (d + n) * (M * r - (L < M ? L : M) * (2 * r + 48)) < 3 << 23;
}

int token_slots(int64_t M) { return M < 16 ? (M < 1 ? 1 : (int)M) : 16; }

// Rows at a time: less than 2^31 bytes of the widest tensor.
int64_t list_chunk(int64_t M, int64_t d, int64_t n) {
  const int64_t most = ((int64_t(1) << 31) - 65536) / (2 * (d > n ? d : n)) / 64 * 64;
  return M < most ? (M < 1 ? 1 : M) : most;
}
int64_t list_chunks(int64_t M, int64_t d, int64_t n) {
  const int64_t c = list_chunk(M, d, n);
  return M < 1 ? 1 : (M + c - 1) / c;
}
// Tiles of `size` rows that a chunk can have.
int64_t most_tiles(int64_t M, int64_t L, int64_t d, int64_t n, int64_t size) {
  const int64_t c = list_chunk(M, d, n);
  return c / size + (L + 1 < c ? L + 1 : c);
}

int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }
int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// Splits of the columns in k_down (and k_down_few): where its blocks are fewer than the compute units,
// with at least two runs of 64 columns for each wave, or 1024 columns for a block.  Few tokens count
// every token's blocks, of which only those of the first of its adapter in a tile have work (one
// adapter, 64 rows, rank 64: 256 counted, 16 at work, and so no split).  The forward's tiles
// go for two blocks to a unit, which evens out a last tile more than units (8192 x 4096, rank
// 64, 262 tiles: 31.7 us, in two splits 27.7); in the gradients one split saves k_split's launch.
int down_splits(int64_t M, int64_t n, int64_t r, bool few, bool grads) {
  const int64_t blocks = few ? M * ((r + 15) / 16) : (M + 31) / 32;
  const int64_t most = few ? n / (2 * 64 * kDownWaves) : n / 1024;
  int64_t s = blocks > 0 ? (few || grads ? 256 : 512) / blocks : 1;
  s = s > most ? most : s;
  return (int)(s > 8 ? 8 : s < 1 ? 1 : s);
}

// Rows of a part in k_sums (a multiple of 64), 0: an adapter's rows in one go.  Where there are fewer
// blocks than two to a compute unit, the rows are cut so that about three to a unit have work.
int64_t part_rows(int64_t M, int64_t L, int64_t d, int64_t n) {
  const int64_t blocks = (d + 127) / 128 + (n + 127) / 128;
  if (L * blocks >= 512 || M < 1) return 0;
  const int64_t parts = (768 + blocks - 1) / blocks;
  const int64_t rows = ((M + parts - 1) / parts + 63) / 64 * 64;
  return rows < 128 ? 128 : rows;
}
// Parts of a chunk at most.
int64_t most_parts(int64_t M, int64_t L, int64_t d, int64_t n) {
  const int64_t rows = part_rows(M, L, d, n), c = list_chunk(M, d, n);
  return rows ? c / rows + (L < c ? L : c) : 0;
}

template <int TY>
hipError_t down(DownArgs a, int problems, bool few, hipStream_t st) {
  const int rt = a.rp / 16, splits = a.of[0].splits > a.of[1].splits ? a.of[0].splits : a.of[1].splits;
  if (few) {
    a.slots = token_slots(a.M);
    const dim3 grid((unsigned)((a.M + 15) / 16 * a.slots * rt * splits), (unsigned)problems);
    k_down_few<TY><<<grid, 64 * kDownWaves, 0, st>>>(a);
    return hipGetLastError();
  }
  const int64_t tiles = a.lists.chunk / 32 + (a.L < a.lists.chunk ? a.L : a.lists.chunk);
  const dim3 grid((unsigned)(tiles * splits), (unsigned)problems, (unsigned)((a.M + a.lists.chunk - 1) / a.lists.chunk));
  return rt == 1   ? launch_down<TY, DownTile<1>>(a, grid, st)
         : rt == 2 ? launch_down<TY, DownTile<2>>(a, grid, st)
         : rt <= 4 ? launch_down<TY, DownTile<4>>(a, grid, st)
                   : launch_down<TY, DownTile<8>>(a, grid, st);
}

template <int TY, bool WIDE>
hipError_t up_few(const UpArgs& a, dim3 grid, hipStream_t st) {
  if (a.r <= 32)
    k_up_few<TY, 1, WIDE><<<grid, 256, 0, st>>>(a);
  else if (a.r <= 64)
    k_up_few<TY, 2, WIDE><<<grid, 256, 0, st>>>(a);
  else
    k_up_few<TY, 4, WIDE><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

// Columns of a block: at least `want` blocks where there are columns for them.  tiles: without the partly
// filled ones that adapters add; for few tokens one each token, as in down_splits.
int64_t up_chunk(int64_t tiles, int64_t d, int64_t want) {
  int64_t chunk = 1024;
  while (chunk > 128 && tiles * ((d + chunk - 1) / chunk) < want) chunk /= 2;
  return chunk;
}

// Rows of the factors need to be multiples of 8 for many tokens: others are padded first.
template <int TY>
hipError_t up(UpArgs a, uint16_t* pad, bool few, hipStream_t st) {
  if (few) {
    a.slots = token_slots(a.M);
    const int64_t chunk = up_chunk(a.M, a.d, 1024);
    a.chunk = (int)chunk;
    const dim3 grid((unsigned)((a.M + 15) / 16 * a.slots * ((a.d + chunk - 1) / chunk)));
    return a.r % 8 == 0 && a.ld % 8 == 0 ? up_few<TY, true>(a, grid, st) : up_few<TY, false>(a, grid, st);
  }
  if (a.ld % 8 != 0) {
    const int ld = (a.r + 7) / 8 * 8;
    const int64_t units = (int64_t)a.L * a.d * (ld / 8), want = (units + 255) / 256;
    k_pad<<<(unsigned)(want < 8192 ? want : 8192), 256, 0, st>>>(reinterpret_cast<const uint16_t*>(a.W), pad, units, a.r, ld);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.W = reinterpret_cast<const uint8_t*>(pad);
    a.r = a.ld = ld;
  }
  const int64_t chunk = up_chunk((a.M + 63) / 64, a.d, 512), rows = a.lists.chunk;
  a.chunk = (int)chunk;
  const int64_t tiles = rows / 64 + (a.L + 1 < rows ? a.L + 1 : rows);
  const dim3 grid((unsigned)(tiles * ((a.d + chunk - 1) / chunk)), (unsigned)((a.M + rows - 1) / rows));
  if (a.r <= 32)
    k_up<TY, 1><<<grid, 256, 0, st>>>(a);
  else if (a.r <= 64)
    k_up<TY, 2><<<grid, 256, 0, st>>>(a);
  else
    k_up<TY, 4><<<grid, 256, 0, st>>>(a);
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
hipError_t sums(SumArgs a, const AdapterArgs& p, float* ws, hipStream_t st) {
  const int chunks = (int)list_chunks(p.M, p.d, p.n);
  a.parts = (int)most_parts(p.M, p.L, p.d, p.n);
  a.each = p.r * (p.d + p.n);
  a.blocks0 = (a.of[0].F + 127) / 128;
  const unsigned blocks = (unsigned)(a.blocks0 + (a.of[1].F + 127) / 128);
  if (a.parts) a.of[0].out = a.of[1].out = ws;
  const dim3 grid(blocks, (unsigned)(a.parts ? a.parts : p.L), (unsigned)(a.parts ? chunks : 1));
  if (a.parts || p.out_dtype == T_FP32)
    sums_rt<TY, T_FP32>(a, grid, st);
  else
    sums_rt<TY, TY>(a, grid, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.parts) return e;
  const PartsArgs q{ws, p.dA, p.dB, a.lists, chunks, a.parts, (int)(p.d * p.r), a.each};
  const dim3 each((unsigned)((a.each / 4 + 255) / 256), (unsigned)p.L);
  if (p.out_dtype == T_FP32)
    k_parts<T_FP32><<<each, 256, 0, st>>>(q);
  else
    k_parts<TY><<<each, 256, 0, st>>>(q);
  return hipGetLastError();
}

// One launch: one rank tile, B_a small, and no more blocks than compute units (one token, 4096 columns,
// rank 16, us of the kernels alone: n = 640 4.7, in two launches 6.6; 2560 6.7 and 7.1; 4096 7.7 and
// 7.1, but a call 9.8 and 13.9 with its host side; rank 64 with n = 640 would be 9.1 and 7.5).  Wider rows
// lose more than the host's side saves in a graph, where it does not count: n = 5120 9.0 and 7.4, 8192
// 11.8 and 7.5, 14336 18.4 and 8.1.  Blocks are counted as in down_splits.
bool in_one(int64_t M, int64_t d, int64_t n, int64_t r) {
  return r <= 16 && n <= 4096 && M * ((d + kTokenCols - 1) / kTokenCols) <= 256;
}

// The workspace: h, the lists, A padded, and for the gradients dh, both in pieces, A and B transposed,
// and the parts of the sums.
struct Ws {
  int64_t lists, pad, dh, ph, pdh, at, bt, parts, bytes;
};
Ws carve(int64_t M, int64_t L, int64_t d, int64_t n, int64_t r, bool grads) {
  Ws w{};
  const int64_t rp = round16(r);
  if (!grads && in_one(M, d, n, r)) return w;
  const bool few = few_rows(M, L, d, n, r, grads);
  int64_t at = up256(4 * M * rp * down_splits(M, n, r, few, grads));
  auto take = [&](int64_t& place, int64_t bytes) {
    place = at;
    at += up256(bytes);
  };
  if (grads || !few) take(w.lists, 4 * M + 16 * list_chunks(M, d, n) * (L + 2));
  if (!grads) {
    take(w.pad, !few && r % 8 != 0 ? 2 * L * d * ((r + 7) / 8 * 8) : 0);
  } else {
    take(w.dh, 4 * M * rp * down_splits(M, d, r, few, grads));
    take(w.ph, 6 * M * rp);
    take(w.pdh, 6 * M * rp);
    take(w.at, 2 * L * r * d);
    take(w.bt, 2 * L * n * rp);
    take(w.parts, 4 * most_parts(M, L, d, n) * list_chunks(M, d, n) * r * (d + n));
  }
  w.bytes = at;
  return w;
}

Lists lists_of(const AdapterArgs& p, uint8_t* at) {
  Lists l{};
  const int64_t tables = list_chunks(p.M, p.d, p.n) * (p.L + 2);
  l.order = reinterpret_cast<int32_t*>(at);
  l.starts = l.order + p.M;
  l.t32 = l.starts + tables;
  l.t64 = l.t32 + tables;
  l.tp = l.t64 + tables;
  const int64_t part = part_rows(p.M, p.L, p.d, p.n);
  l.part = part ? (int)part : 64;
  l.M = p.M;
  l.chunk = list_chunk(p.M, p.d, p.n);
  l.L = (int)p.L;
  return l;
}

hipError_t make_lists(const AdapterArgs& p, ListArgs a, hipStream_t st) {
  a.index = p.index;
  a.blocks = (int)((p.L + 1) * list_chunks(p.M, p.d, p.n));
  const int64_t turns = p.L * (a.turn[0].tiles + a.turn[1].tiles);
  k_lists<<<(unsigned)(a.blocks + (turns + 3) / 4), 1024, 0, st>>>(a);
  return hipGetLastError();
}

template <int TY>
hipError_t token(const Down& of, UpArgs a, hipStream_t st) {
  a.slots = token_slots(a.M);
  const dim3 grid((unsigned)((a.M + 15) / 16 * a.slots * ((a.d + kTokenCols - 1) / kTokenCols)));
  if (a.r % 8 == 0)
    k_token<TY, true><<<grid, 64 * kDownWaves, 0, st>>>(of, a);
  else
    k_token<TY, false><<<grid, 64 * kDownWaves, 0, st>>>(of, a);
  return hipGetLastError();
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
  const bool few = few_rows(p.M, p.L, p.d, p.n, p.r, false);
  const int s = down_splits(p.M, p.n, p.r, few, false);
  const Down of{static_cast<const uint8_t*>(p.X), static_cast<const uint8_t*>(p.B), h, (int)p.n, s, nullptr};
  UpArgs y = up_args(p);
  y.H = h;
  y.splits = s;
  y.W = static_cast<const uint8_t*>(p.A);
  y.d = (int)p.d;
  y.r = y.ld = (int)p.r;
  if (in_one(p.M, p.d, p.n, p.r)) return token<TY>(of, y, st);
  const Ws w = carve(p.M, p.L, p.d, p.n, p.r, false);
  DownArgs x = down_args(p);
  x.of[0] = of;
  hipError_t e;
  if (!few) {
    ListArgs l{};
    l.lists = x.lists = y.lists = lists_of(p, ws + w.lists);
    if ((e = make_lists(p, l, st)) != hipSuccess) return e;
  }
  if ((e = down<TY>(x, 1, few, st)) != hipSuccess) return e;
  return up<TY>(y, reinterpret_cast<uint16_t*>(ws + w.pad), few, st);
}

template <int TY>
hipError_t bwd(const AdapterArgs& p, uint8_t* ws, hipStream_t st) {
  const Ws w = carve(p.M, p.L, p.d, p.n, p.r, true);
  const int rp = (int)round16(p.r), L = (int)p.L, d = (int)p.d, n = (int)p.n, r = (int)p.r;
  float *h = reinterpret_cast<float*>(ws), *dh = reinterpret_cast<float*>(ws + w.dh);
  uint16_t *at = reinterpret_cast<uint16_t*>(ws + w.at), *bt = reinterpret_cast<uint16_t*>(ws + w.bt);
  const uint8_t *X = static_cast<const uint8_t*>(p.X), *dY = static_cast<const uint8_t*>(p.dY);
  const bool few = few_rows(p.M, L, d, n, r, true);
  const int sh = down_splits(p.M, n, r, few, true), sd = down_splits(p.M, d, r, few, true);
  uint16_t *ph = reinterpret_cast<uint16_t*>(ws + w.ph), *pdh = reinterpret_cast<uint16_t*>(ws + w.pdh);
  const Lists lists = lists_of(p, ws + w.lists);
  ListArgs l{};
  l.lists = lists;
  if (p.M > 0) {
    l.turn[0] = Turn{static_cast<const uint16_t*>(p.A), at, d, r, d, (r + 63) / 64, (r + 63) / 64 * ((d + 63) / 64)};
    if (p.Y)
      l.turn[1] = Turn{static_cast<const uint16_t*>(p.B), bt, r, n, rp, (n + 63) / 64, (n + 63) / 64 * ((rp + 63) / 64)};
  }
  hipError_t e = make_lists(p, l, st);  // (without a row too: the lists are then empty)
  if (e != hipSuccess) return e;
  if (p.M > 0) {
    const bool split = few || sh > 1 || sd > 1;
    DownArgs x = down_args(p);
    x.lists = lists;
    x.scale = p.scale;
    x.of[0] = Down{X, static_cast<const uint8_t*>(p.B), split ? h : nullptr, n, sh, split ? nullptr : ph};
    x.of[1] = Down{dY, reinterpret_cast<const uint8_t*>(at), split || p.Y ? dh : nullptr, d, sd, split ? nullptr : pdh};
    if ((e = down<TY>(x, 2, few, st)) != hipSuccess) return e;
    if (p.Y) {
      UpArgs y = up_args(p);
      y.lists = lists;
      y.H = dh;
      y.splits = sd;
      y.W = reinterpret_cast<const uint8_t*>(bt);
      y.d = n;
      y.r = y.ld = rp;  // (the padding is zeros on both sides)
      if ((e = up<TY>(y, nullptr, few, st)) != hipSuccess) return e;
    }
    if (split) {
      SplitArgs v{};
      v.of[0] = Split{h, ph, sh};
      v.of[1] = Split{dh, pdh, sd};
      v.index = p.index;
      v.scale = p.scale;
      v.lists = lists;
      v.M = p.M;
      v.L = L;
      v.rp = rp;
      v.by_row = few;
      k_split<<<dim3((unsigned)((p.M * (rp / 4) + 255) / 256), 2), 256, 0, st>>>(v);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  SumArgs q{};
  q.lists = lists;
  q.M = p.M;
  q.L = L;
  q.r = r;
  q.rp = rp;
  q.of[0] = Sum{dY, ph, p.dA, d};
  q.of[1] = Sum{X, pdh, p.dB, n};
  return sums<TY>(q, p, reinterpret_cast<float*>(ws + w.parts), st);
}

}  // namespace

// Whether every launch of a call holds: less than 2^32 work-items, at most 65535 blocks along y and z.
// (Few tokens are at most 640: their blocks always do.)  Transposes, pieces and parts are the gradients'
// alone.
bool adapters_fit(int64_t M, int64_t L, int64_t d, int64_t n, int64_t r, bool grads) {
  const int64_t most = int64_t(1) << 32, widest = d > n ? d : n, chunks = list_chunks(M, d, n);
  const int64_t turns = grads ? ((d + 63) / 64 + (n + 63) / 64) * ((round16(r) + 63) / 64) : 0;
  if (chunks > 65535 || (turns * L + 4) * 256 + (L + 1) * chunks * 1024 >= most) return false;
  if (grads && (most_parts(M, L, d, n) > 65535 || M * (round16(r) / 4) + 256 >= most)) return false;
  const int64_t downs = most_tiles(M, L, d, n, 32) * 8 * 2 * chunks;
  const int64_t ups = most_tiles(M, L, d, n, 64) * ((widest + 1023) / 1024 + 4) * chunks;
  return downs * 256 < most && ups * 256 < most;
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
