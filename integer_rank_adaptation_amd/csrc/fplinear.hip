// Floating-point linear layers for gfx950: the 8-bit layer with one power-of-two scale per
// block of 128, and products grouped by expert (8-bit, bf16, fp16) with their gradients.
//
// Group e owns the token rows offsets[e] .. offsets[e + 1] (one group of all rows without
// offsets).  With X [T, K], W [E, N, K], Y / dY [T, N]:
//   forward   Y_t   = X_t W_e^T     both operands have the contraction contiguous  (NT)
//   dX        dX_t  = dY_t W_e      the second operand is [contraction, columns]    (NN)
//   dW        dW_e  = dY_e^T X_e    both operands are [contraction, columns]        (TN)
// One kernel template serves all: only the way a fragment leaves LDS differs.
#include <type_traits>

#include "device_common.h"
#include "intlora_internal.h"

namespace intlora {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(3))) v4s* lds_v4s_t;

namespace {

enum { T_BF16 = 0, T_FP16 = 1, T_FP32 = 2, T_FP8 = 3 };
enum { L_NT = 0, L_NN = 1, L_TN = 2 };

constexpr uint32_t kOOB = 0x80000000u;  // a buffer offset past every record: the lane reads zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  const int64_t cap = 0x7FFFFFF0;  // lane offsets stay below 2^31: every tile and stage has a base of its own
  const int nrec = (int)(bytes < 0 ? 0 : (bytes > cap ? cap : bytes));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, nrec, 0x00020000);
}

// At most N direct loads still in flight, and every LDS read returned.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

__device__ __forceinline__ int clamp_row(int64_t o, int T) { return o < 0 ? 0 : (o > T ? T : (int)o); }

// Rows of the groups: boundary j is the largest of offsets[0 .. j], each forced into
// [0, T], and group e lies between boundaries e and e + 1.  For ascending offsets that is
// offsets[e] .. offsets[e + 1]; whatever else the array holds, no row outside [0, T) is
// touched and no row belongs to two groups.
struct Group {
  int e, row0, rows;
};

// The unit (row tile x units_per_tile) number `want` over all groups whose row count lies
// in [least, most]; each such group has ceil(rows / bm) row tiles.  False when there are
// fewer.  A wave takes 64 groups at a time, one per lane; all waves find the same.
__device__ __forceinline__ bool find_unit(const int64_t* __restrict__ offsets, int E, int T, int want, int bm,
                                          int units_per_tile, int least, int most, Group& g, int& unit) {
  const int lane = threadIdx.x & 63;
  if (offsets == nullptr) {  // one group of all rows
    g.e = 0;
    g.row0 = 0;
    g.rows = T;
    unit = want;
    return T >= least && T <= most && want < (T + bm - 1) / bm * units_per_tile;
  }
  int before = clamp_row(offsets[0], T);  // boundary in front of this chunk of groups
  int done = 0;                           // units in front of it
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int b = e < E ? clamp_row(offsets[e + 1], T) : 0;
    if (b < before) b = before;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(b, s);
      if (lane >= s && o > b) b = o;
    }
    int a = __shfl_up(b, 1);
    if (lane == 0) a = before;
    const int rows = b - a;
    const int mine = rows >= least && rows <= most ? (rows + bm - 1) / bm * units_per_tile : 0;
    int inc = mine;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(inc, s);
      if (lane >= s) inc += o;
    }
    const uint64_t hit = __builtin_amdgcn_ballot_w64(done + inc > want);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      g.e = e0 + src;
      g.row0 = __builtin_amdgcn_readlane(a, src);
      g.rows = __builtin_amdgcn_readlane(rows, src);
      unit = want - done - __builtin_amdgcn_readlane(inc - mine, src);
      return true;
    }
    done += __builtin_amdgcn_readlane(inc, 63);
    before = __builtin_amdgcn_readlane(b, 63);
  }
  return false;
}

// Rows of group e.
__device__ __forceinline__ Group group_rows(const int64_t* __restrict__ offsets, int e, int T) {
  const int lane = threadIdx.x & 63;
  int a = 0;
  for (int j = lane; j <= e; j += 64) {
    const int o = clamp_row(offsets[j], T);
    a = o > a ? o : a;
  }
#pragma unroll
  for (int s = 32; s; s >>= 1) {
    const int o = __shfl_xor(a, s);
    a = o > a ? o : a;
  }
  a = __builtin_amdgcn_readfirstlane(a);
  const int b = clamp_row(offsets[e + 1], T);
  return Group{e, a, b > a ? b - a : 0};
}

// Blocks are dealt to the 8 XCDs in turn; this renumbers each run of 256 of them so that an
// XCD works on 32 consecutive tiles, whose operands its own L2 then serves.
__device__ __forceinline__ int xcd_slot(int b, int n) {
  if ((b | 255) >= n) return b;
  return (b & ~255) | ((b & 7) << 5) | ((b & 255) >> 3);
}

// ------------------------------------------------------------------------ tiled kernel
// A block computes BM x BN outputs with 4 waves (2 x 2), each (BM / 2) x (BN / 2) in tiles
// of 32 x 32.  The contraction goes in stages of 64 bytes of a row (32 16-bit or 64 8-bit
// elements) through a ring of three LDS stages filled by direct loads.
constexpr int kStages = 3;
constexpr int kScaleBytes = 1024;  // 8-bit: 128 rows' and the weight blocks' scale dwords of a stage

template <int TY, int LAY, int BM, int BN>
struct Tile {
  static constexpr bool F8 = TY == T_FP8;
  static constexpr int EB = F8 ? 1 : 2;        // bytes per element
  static constexpr int BK = 64 / EB;           // elements per stage
  static constexpr int A_BYTES = BM * 64, B_BYTES = BN * 64;
  static constexpr int STAGE = A_BYTES + B_BYTES + (F8 ? kScaleBytes : 0);
  static constexpr int AL = A_BYTES / 4096, BL = B_BYTES / 4096;  // direct loads per wave and stage
  static constexpr int LOADS = AL + BL + (F8 ? 1 : 0);
  static constexpr int WM = BM / 2, WN = BN / 2, MT = WM / 32, NT = WN / 32;
  static constexpr int RING = kStages * STAGE;
  static constexpr bool TA = LAY == L_TN, TB = LAY != L_NT;  // operands stored [contraction, columns]
};

// LDS rows of 64 bytes: the 16-byte chunk c of row r lies at c ^ swz64(r), so that the 16
// lanes of a fragment read touch every bank once.
__device__ __forceinline__ int swz64(int row) { return (row ^ (row >> 2)) & 3; }

// Rows [contraction k][columns]: a transposing read takes 4 rows x 32 bytes per 16 lanes;
// chunk c of row k lies at c ^ 2 (k & 3), which puts the four rows on different banks.
__device__ __forceinline__ int swzT(int k) { return 2 * (k & 3); }

// Byte offset, from the operand tile's first byte, of the 16 bytes that this lane brings to
// LDS with its load q: row-contiguous operand (TR = 0, ld bytes per row, rows = outputs) or
// [contraction, columns] operand of C columns (TR = 1, rows = contraction).
template <bool TR, int C>
__device__ __forceinline__ uint32_t lane_offset(int g, int lane, uint32_t ld, int& kk) {
  if (!TR) {
    const int row = 16 * g + (lane >> 2);
    kk = 16 * ((lane & 3) ^ swz64(row));
    return (uint32_t)row * ld + kk;
  }
  constexpr int PER = C / 8;  // chunks per row
  const int row = (64 / PER) * g + lane / PER;
  kk = 0;
  return (uint32_t)row * ld + 16 * ((lane % PER) ^ swzT(row));
}

// Fragment of 16 bytes (sub-step ks of lane half h: contraction chunk 2 h + ks of the
// stage) for the 32 rows / columns from r0.
template <bool TR, int C>
__device__ __forceinline__ v4i read_frag(const uint8_t* S, int r0, int ks) {
  const int lane = threadIdx.x & 63, h = lane >> 5;
  if (!TR) {
    const int row = r0 + (lane & 31);
    return *reinterpret_cast<const v4i*>(S + row * 64 + (((2 * h + ks) ^ swz64(lane & 31)) << 4));
  }
  // two transposing reads of 4 contraction rows x 16 columns per 16 lanes: lane j points at
  // row j / 4, columns 4 (j % 4) .. + 3 and receives column j, the four rows
  const int j = lane & 15;
  const int k = 8 * (2 * h + ks) + (j >> 2);
  const int col = r0 + (lane & 16) + 4 * (j & 3);
  const uint32_t at = (uint32_t)(k * (2 * C) + (((col >> 3) ^ swzT(k)) << 4) + ((col & 7) << 1));
  const uint8_t* p = S + at;
  v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t)p);
  v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t)(p + 4 * 2 * C));
  const int2 a = __builtin_bit_cast(int2, lo), b = __builtin_bit_cast(int2, hi);
  return v4i{a.x, a.y, b.x, b.y};
}

template <int TY>
__device__ __forceinline__ v16f mfma16(v4i b, v4i a, v16f c) {
  if (TY == T_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, b), __builtin_bit_cast(bf8, a), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, b), __builtin_bit_cast(h8, a), c, 0, 0, 0);
}

// Two floats to the output's 16-bit type (round to nearest even).
template <int TO>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if (TO == T_FP16) return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){x, y}, h2));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){x, y}, bf2));
}

struct GemmArgs {
  const uint8_t* A;       // NT, NN: tokens x contraction; TN: tokens x rows
  const uint8_t* B;       // NT: E x cols x contraction; NN: E x contraction x cols; TN: tokens x cols
  void* C;                // NT, NN: tokens x cols; TN: E x rows x cols
  const uint8_t* sa;      // 8-bit: scale bytes [T, lds]
  const uint8_t* sb;      // 8-bit: scale bytes [E, ceil(cols / 128), lds]
  const int64_t* offsets;  // [E + 1], or NULL for one group of T rows
  int T, E, least, most;  // groups with rows outside [least, most] are not this launch's
  int rows, cols, kdim;   // TN: output rows; columns; contraction length (NT, NN)
  int lds;                // scale bytes per row
  int tiles;              // the launch's block count
};

template <int TY, int LAY, int TO, int BM, int BN>
__global__ void __launch_bounds__(256, 2) k_gemm(const GemmArgs p) {
  using C = Tile<TY, LAY, BM, BN>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid >> 1, wn = wid & 1;
  const int tiles_n = (p.cols + BN - 1) / BN;

  // ---- the block's tile
  Group g;
  int tm, tn;
  const int slot = xcd_slot(blockIdx.x, gridDim.x);
  if (LAY == L_TN) {
    const int tiles_m = (p.rows + BM - 1) / BM;
    const int e = slot / (tiles_m * tiles_n);
    const int in = slot - e * tiles_m * tiles_n;
    tn = in / tiles_m;
    tm = in - tn * tiles_m;
    if (p.offsets == nullptr)
      g = Group{0, 0, p.T};
    else
      g = group_rows(p.offsets, e, p.T);
  } else {
    int unit;
    if (!find_unit(p.offsets, p.E, p.T, slot, BM, tiles_n, p.least, p.most, g, unit)) return;
    // patches of 8 row tiles: the weight tile of one column is read for all of them in turn
    const int tiles_m = (g.rows + BM - 1) / BM;
    const int patch = unit / (8 * tiles_n), first = patch * 8;
    const int size = tiles_m - first < 8 ? tiles_m - first : 8;
    const int in = unit - patch * 8 * tiles_n;
    tn = in / size;
    tm = first + in - tn * size;
  }
  const int m0 = tm * BM, n0 = tn * BN;  // first output row (inside the group, or of dW) and column
  const int kdim = LAY == L_TN ? g.rows : p.kdim;
  const int KT = (kdim + C::BK - 1) / C::BK;

  // ---- operand tiles: first byte, bytes to the operand's end, bytes per stage step
  const uint32_t lda = (uint32_t)((LAY == L_TN ? p.rows : p.kdim) * C::EB);
  const uint32_t ldb = (uint32_t)((LAY == L_NT ? p.kdim : p.cols) * C::EB);
  const uint8_t *pa, *pb;
  int64_t na, nb, da, db;
  if (C::TA) {
    pa = p.A + (int64_t)g.row0 * lda + (int64_t)m0 * C::EB;
    na = (int64_t)g.rows * lda - (int64_t)m0 * C::EB;
    da = (int64_t)C::BK * lda;
  } else {
    pa = p.A + (int64_t)(g.row0 + m0) * lda;
    na = (int64_t)(g.rows - m0) * lda;
    da = 64;
  }
  if (LAY == L_NT) {
    pb = p.B + ((int64_t)g.e * p.cols + n0) * ldb;
    nb = (int64_t)(p.cols - n0) * ldb;
    db = 64;
  } else if (LAY == L_NN) {
    pb = p.B + (int64_t)g.e * p.kdim * ldb + (int64_t)n0 * C::EB;
    nb = (int64_t)p.kdim * ldb - (int64_t)n0 * C::EB;
    db = (int64_t)C::BK * ldb;
  } else {
    pb = p.B + (int64_t)g.row0 * ldb + (int64_t)n0 * C::EB;
    nb = (int64_t)g.rows * ldb - (int64_t)n0 * C::EB;
    db = (int64_t)C::BK * ldb;
  }
  // 8-bit: waves 0 and 1 bring 64 rows' scale dwords each, waves 2 and 3 the weight blocks'
  const uint8_t* ps = nullptr;
  int64_t ns = 0;
  uint32_t so = 0;
  if (C::F8) {
    if (wid < 2) {
      ps = p.sa + (int64_t)(g.row0 + m0) * p.lds;
      ns = (int64_t)(g.rows - m0) * p.lds;
      so = (uint32_t)((64 * wid + lane) * p.lds);
    } else {
      const int blocks = (p.cols + 127) >> 7;
      ps = p.sb + ((int64_t)g.e * blocks + (n0 >> 7)) * p.lds;
      ns = (int64_t)(blocks - (n0 >> 7)) * p.lds;
      so = (uint32_t)((lane & (BN / 128 - 1)) * p.lds);
    }
  }

  uint32_t oa[C::AL], ob[C::BL];
  int ka[C::AL], kb[C::BL];
#pragma unroll
  for (int q = 0; q < C::AL; ++q) oa[q] = lane_offset<C::TA, BM>(wid * C::AL + q, lane, lda, ka[q]);
#pragma unroll
  for (int q = 0; q < C::BL; ++q) ob[q] = lane_offset<C::TB, BN>(wid * C::BL + q, lane, ldb, kb[q]);

  // Direct loads of stage kt.  Rows past the operand's end and stages past KT read zeros;
  // so do the chunks past a row's end in the last stage, in both operands (what lies there
  // may be a NaN, and 0 x NaN is not 0).
  auto issue = [&](int kt, uint8_t* S) {
    const bool live = kt < KT;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(pa + (live ? kt * da : 0), live ? na - kt * da : 0);
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(pb + (live ? kt * db : 0), live ? nb - kt * db : 0);
    const int left = kdim * C::EB - kt * 64;  // bytes of a contiguous row from this stage on
#pragma unroll
    for (int q = 0; q < C::AL; ++q) {
      const uint32_t o = C::TA || ka[q] < left ? oa[q] : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(S + (wid * C::AL + q) * 1024), 16, o, 0, 0, 0);
    }
#pragma unroll
    for (int q = 0; q < C::BL; ++q) {
      const uint32_t o = C::TB || kb[q] < left ? ob[q] : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)(S + C::A_BYTES + (wid * C::BL + q) * 1024), 16, o, 0, 0,
                                               0);
    }
    if (C::F8) {  // the dword of four 128-blocks that holds this stage's scale
      const int64_t at = (int64_t)(kt >> 3) * 4;
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(ps + (live ? at : 0), live ? ns - at : 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(S + C::A_BYTES + C::B_BYTES + wid * 256), 4, so, 0, 0, 0);
    }
  };

  v16f acc[C::MT][C::NT];
#pragma unroll
  for (int i = 0; i < C::MT; ++i)
#pragma unroll
    for (int j = 0; j < C::NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  issue(0, lds);
  issue(1, lds + C::STAGE);
  int cur = 0;
  for (int kt = 0; kt < KT; ++kt) {
    // stage kt has landed (kt + 1 may be in flight); behind the barrier it is visible to all
    // waves and every wave is done with stage kt - 1, whose buffer kt + 2 takes
    wait_loads<C::LOADS>();
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
    const int nxt = cur == 0 ? 2 : cur - 1;  // (cur + 2) % 3
    issue(kt + 2, lds + nxt * C::STAGE);
    const uint8_t* S = lds + cur * C::STAGE;
    const uint8_t* SB = S + C::A_BYTES;
    v4i af[C::MT][2], bf[C::NT][2];
#pragma unroll
    for (int i = 0; i < C::MT; ++i)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) af[i][ks] = read_frag<C::TA, BM>(S, wm * C::WM + 32 * i, ks);
#pragma unroll
    for (int j = 0; j < C::NT; ++j)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) bf[j][ks] = read_frag<C::TB, BN>(SB, wn * C::WN + 32 * j, ks);
    if (C::F8) {
      const uint32_t* sc = reinterpret_cast<const uint32_t*>(S + C::A_BYTES + C::B_BYTES);
      const int sh = 8 * ((kt >> 1) & 3);
      const int sw = (int)(sc[128 + (wn * C::WN) / 128] >> sh);
      int sx[C::MT];
#pragma unroll
      for (int i = 0; i < C::MT; ++i) sx[i] = (int)(sc[wm * C::WM + 32 * i + (lane & 31)] >> sh);
#pragma unroll
      for (int i = 0; i < C::MT; ++i)
#pragma unroll
        for (int j = 0; j < C::NT; ++j) {
          const v8i a = __builtin_shufflevector(af[i][0], af[i][1], 0, 1, 2, 3, 4, 5, 6, 7);
          const v8i b = __builtin_shufflevector(bf[j][0], bf[j][1], 0, 1, 2, 3, 4, 5, 6, 7);
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc[i][j], 0, 0, 0, sw, 0, sx[i]);
        }
    } else {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
#pragma unroll
          for (int j = 0; j < C::NT; ++j) acc[i][j] = mfma16<TY>(bf[j][ks], af[i][ks], acc[i][j]);
    }
    cur = cur == 2 ? 0 : cur + 1;
  }
  wait_loads<0>();
  __syncthreads();

  // ---- epilogue: lane l holds row l % 32 of a tile and columns 8 a + 4 (l / 32) + 0 .. 3 in
  // registers 4 a .. 4 a + 3.  A wave passes 32 rows x WN columns at a time through its own
  // part of the ring and stores whole row pieces.
  constexpr int OB = TO == T_FP32 ? 4 : 2;
  constexpr int RS = C::WN * OB + 16;
  static_assert(4 * 32 * RS <= C::RING, "epilogue staging fits the ring");
  uint8_t* stg = lds + wid * 32 * RS;
  const int fr = lane & 31, h = lane >> 5;
  const int rows_left = (LAY == L_TN ? p.rows : g.rows) - m0 - wm * C::WM;
  const int c0 = n0 + wn * C::WN, cols_left = p.cols - c0;
  const int64_t out_row = (LAY == L_TN ? (int64_t)g.e * p.rows : (int64_t)g.row0) + m0 + wm * C::WM;
  uint8_t* out = static_cast<uint8_t*>(p.C) + (out_row * p.cols + c0) * OB;
  const bool whole = ((int64_t)p.cols * OB) % 16 == 0 && cols_left >= C::WN;
#pragma unroll
  for (int i = 0; i < C::MT; ++i) {
#pragma unroll
    for (int j = 0; j < C::NT; ++j)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const float y0 = acc[i][j][4 * a], y1 = acc[i][j][4 * a + 1], y2 = acc[i][j][4 * a + 2],
                    y3 = acc[i][j][4 * a + 3];
        uint8_t* at = stg + fr * RS + (32 * j + 8 * a + 4 * h) * OB;
        if (TO == T_FP32)
          *reinterpret_cast<float4*>(at) = make_float4(y0, y1, y2, y3);
        else
          *reinterpret_cast<uint2*>(at) = make_uint2(pack2<TO>(y0, y1), pack2<TO>(y2, y3));
      }
    __builtin_amdgcn_wave_barrier();
    const int live = rows_left - 32 * i < 32 ? rows_left - 32 * i : 32;
    if (whole) {
      constexpr int PER = C::WN * OB / 16;  // 16-byte pieces per row
#pragma unroll
      for (int q = 0; q < 32 * PER / 64; ++q) {
        const int id = q * 64 + lane, r = id / PER, c = id % PER;
        if (r < live)
          *reinterpret_cast<v4i*>(out + (int64_t)(32 * i + r) * p.cols * OB + 16 * c) =
              *reinterpret_cast<const v4i*>(stg + r * RS + 16 * c);
      }
    } else {
      for (int r = 0; r < live; ++r)
        for (int c = lane; c < C::WN; c += 64)
          if (c < cols_left) {
            if (TO == T_FP32)
              reinterpret_cast<float*>(out + (int64_t)(32 * i + r) * p.cols * OB)[c] =
                  reinterpret_cast<const float*>(stg + r * RS)[c];
            else
              reinterpret_cast<uint16_t*>(out + (int64_t)(32 * i + r) * p.cols * OB)[c] =
                  reinterpret_cast<const uint16_t*>(stg + r * RS)[c];
          }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int TY, int LAY, int TO, int BM, int BN>
hipError_t launch_gemm(const GemmArgs& a, hipStream_t st) {
  using C = Tile<TY, LAY, BM, BN>;
  static thread_local int ready_dev = -1;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev != ready_dev) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_gemm<TY, LAY, TO, BM, BN>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, C::RING);
    if (e != hipSuccess) return e;
    ready_dev = dev;
  }
  k_gemm<TY, LAY, TO, BM, BN><<<dim3((unsigned)a.tiles), 256, C::RING, st>>>(a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------ few rows
// Groups of few rows are bound by the weights' bytes: a block streams 16 weight rows
// straight into registers, its waves taking runs of 512 bytes of the contraction in turn,
// against 16 x TT token rows; the waves' sums meet in LDS in a fixed order.
template <int TY, int TT>
__global__ void __launch_bounds__(512, 2) k_few(const GemmArgs p) {
  constexpr bool F8 = TY == T_FP8;
  constexpr int EB = F8 ? 1 : 2;
  constexpr int TO = TY == T_FP16 ? T_FP16 : T_BF16;
  __shared__ __attribute__((aligned(16))) float part[8][TT][256];
  const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = blockDim.x >> 6;
  const int fr = lane & 15, q = lane >> 4;
  Group g;
  if (p.offsets == nullptr)
    g = Group{0, 0, p.T};
  else
    g = group_rows(p.offsets, (int)blockIdx.y, p.T);
  if (g.rows < p.least || g.rows > p.most || g.rows == 0) return;
  const int n0 = blockIdx.x * 16;
  const uint32_t ld = (uint32_t)(p.kdim * EB);
  const int runs = (int)((ld + 511) >> 9);
  const uint8_t* wb = p.B + ((int64_t)g.e * p.cols + n0) * ld;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(wb, (int64_t)(p.cols - n0 < 16 ? p.cols - n0 : 16) * ld);
  const int blocks = (p.cols + 127) >> 7;
  const uint8_t* swp = F8 ? p.sb + ((int64_t)g.e * blocks + (n0 >> 7)) * p.lds : nullptr;

  for (int t0 = 0; t0 < g.rows; t0 += 16 * TT) {
    const int64_t row0 = (int64_t)g.row0 + t0;
    const int rows = g.rows - t0 < 16 * TT ? g.rows - t0 : 16 * TT;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.A + row0 * ld, (int64_t)rows * ld);
    const __amdgpu_buffer_rsrc_t rsx = make_rsrc(F8 ? p.sa + row0 * p.lds : nullptr, F8 ? (int64_t)rows * p.lds : 0);
    v4f acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int run = wid; run < runs; run += waves) {
      v4i w[8], x[TT][8];
      uint32_t swd = 0, sxd[TT];
#pragma unroll
      for (int u = 0; u < 8; ++u) {  // chunk u: bytes 64 u + 16 q .. of the run
        const uint32_t k = (uint32_t)run * 512 + 64 * u + 16 * q;
        const uint32_t ow = k < ld ? (uint32_t)fr * ld + k : kOOB;
        w[u] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rw, ow, 0, 0));
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const uint32_t ox = k < ld ? (uint32_t)(16 * t + fr) * ld + k : kOOB;
          x[t][u] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rx, ox, 0, 0));
        }
      }
      if (F8) {
        swd = *reinterpret_cast<const uint32_t*>(swp + 4 * run);
#pragma unroll
        for (int t = 0; t < TT; ++t)
          sxd[t] = __builtin_amdgcn_raw_buffer_load_b32(rsx, (uint32_t)((16 * t + fr) * p.lds + 4 * run), 0, 0);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          if (F8) {
            const v8i a = __builtin_shufflevector(x[t][2 * u], x[t][2 * u + 1], 0, 1, 2, 3, 4, 5, 6, 7);
            const v8i b = __builtin_shufflevector(w[2 * u], w[2 * u + 1], 0, 1, 2, 3, 4, 5, 6, 7);
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, acc[t], 0, 0, 0, (int)(swd >> (8 * u)), 0,
                                                                      (int)(sxd[t] >> (8 * u)));
          } else {
#pragma unroll
            for (int v = 2 * u; v < 2 * u + 2; ++v) {
              if (TY == T_BF16)
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, w[v]),
                                                                 __builtin_bit_cast(bf8, x[t][v]), acc[t], 0, 0, 0);
              else
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, w[v]),
                                                                __builtin_bit_cast(h8, x[t][v]), acc[t], 0, 0, 0);
            }
          }
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) *reinterpret_cast<v4f*>(&part[wid][t][4 * lane]) = acc[t];
    __syncthreads();
    // lane l of a tile: token l % 16, columns 4 (l / 16) + 0 .. 3
    for (int id = tid; id < TT * 64; id += blockDim.x) {
      const int t = id >> 6, l = id & 63;
      v4f s = v4f{0.f, 0.f, 0.f, 0.f};
      for (int w = 0; w < waves; ++w) s += *reinterpret_cast<const v4f*>(&part[w][t][4 * l]);
      const int row = 16 * t + (l & 15), col = n0 + 4 * (l >> 4);
      if (row < rows) {
        uint16_t* y = static_cast<uint16_t*>(p.C) + (row0 + row) * p.cols + col;
        const uint32_t lo = pack2<TO>(s.x, s.y), hi = pack2<TO>(s.z, s.w);
        if ((p.cols & 3) == 0 && col + 4 <= p.cols) {
          *reinterpret_cast<uint2*>(y) = make_uint2(lo, hi);
        } else {
          const uint16_t v[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (col + c < p.cols) y[c] = v[c];
        }
      }
    }
    __syncthreads();
  }
}

template <int TY>
hipError_t launch_few(const GemmArgs& a, hipStream_t st) {
  const int runs = (int)(((int64_t)a.kdim * (TY == T_FP8 ? 1 : 2) + 511) / 512);
  const int waves = runs >= 8 ? 8 : runs >= 4 ? 4 : runs >= 2 ? 2 : 1;
  const dim3 grid((unsigned)((a.cols + 15) / 16), (unsigned)a.E);
  if (a.most <= 16)
    k_few<TY, 1><<<grid, 64 * waves, 0, st>>>(a);
  else
    k_few<TY, 2><<<grid, 64 * waves, 0, st>>>(a);
  return hipGetLastError();
}

// Groups of up to kFew rows go to the few-row kernel, the others to the tiled one.  Without
// the offsets (device memory) the host knows only T and E, so it launches whichever can have
// work; a group that is not a kernel's costs its blocks one look at the offsets.
constexpr int kFew = 32;

template <int TY, int LAY, int TO>
hipError_t run_gemm(GemmArgs a, hipStream_t st) {
  constexpr int BM = 128, BN = 256;
  const int64_t tn = ((int64_t)a.cols + BN - 1) / BN;
  int64_t tiles;
  if (LAY == L_TN) {
    tiles = (int64_t)a.E * (((int64_t)a.rows + BM - 1) / BM) * tn;
  } else {
    const int64_t full = (a.T + BM - 1) / BM;
    const int64_t groups = a.E < a.T ? a.E : a.T;
    tiles = (full + groups - 1) * tn;
  }
  if (tiles >= (int64_t(1) << 31) - 256) return hipErrorInvalidValue;
  a.tiles = (int)tiles;
  a.least = 1;
  a.most = 0x7FFFFFFF;
  if (LAY == L_NT) {
    const bool few = (int64_t)a.T <= (int64_t)kFew * a.E;
    if (few) {
      GemmArgs f = a;
      f.most = a.T < kFew ? a.T : kFew;
      const hipError_t e = launch_few<TY>(f, st);
      if (e != hipSuccess || a.T <= kFew) return e;
      a.least = kFew + 1;
    }
  }
  return launch_gemm<TY, LAY, TO, BM, BN>(a, st);
}

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
// goes round the 16 lanes as integer bits, so a NaN wins.
template <int TI>
__global__ void __launch_bounds__(256) k_fp8_act(int64_t units, int n, int nb, int lds, const void* __restrict__ X,
                                                 uint8_t* __restrict__ xq, uint8_t* __restrict__ sx) {
  const int64_t u = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int l = threadIdx.x & 15;
  if (u >= units) return;  // whole groups of 16 lanes leave together
  const int64_t row = u / nb;
  const int b = (int)(u - row * nb);
  const int k = 128 * b + 8 * l;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (k < n) load8<TI>(X, row * n + k, v);
  uint32_t m = amax8(v);
#pragma unroll
  for (int s = 8; s; s >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)m, s, 16);
    m = o > m ? o : m;
  }
  const uint32_t byte = scale_byte(m);
  if (k < n) *reinterpret_cast<uint2*>(xq + row * n + k) = codes8(v, byte);
  if (l == 0) sx[row * lds + b] = (uint8_t)byte;
  if (b == nb - 1 && l > 0 && b + l < lds) sx[row * lds + b + l] = 127;
}

// Weights: one block of 128 x 128 per workgroup, and, when asked for, the same codes
// transposed (through LDS) for the input gradient's product.
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
  const int nb = (int)((n + 127) / 128), lds = fp8_scale_stride(n);
  const int64_t units = M * nb;
  const dim3 grid((unsigned)((units + 15) / 16));
  if (dtype == T_FP32)
    k_fp8_act<T_FP32><<<grid, 256, 0, st>>>(units, (int)n, nb, lds, X, xq, sx);
  else if (dtype == T_FP16)
    k_fp8_act<T_FP16><<<grid, 256, 0, st>>>(units, (int)n, nb, lds, X, xq, sx);
  else
    k_fp8_act<T_BF16><<<grid, 256, 0, st>>>(units, (int)n, nb, lds, X, xq, sx);
  return hipGetLastError();
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
