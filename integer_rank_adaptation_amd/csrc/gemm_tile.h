// Products of the floating-point linear layers for gfx950, on the matrix cores: dense or grouped
// by expert, in 8 bits (one power-of-two scale per block of 128), bf16 and fp16.  Included by the
// sources that instantiate them.
//
// Group e owns the token rows offsets[e] .. offsets[e + 1] (one group of all rows without
// offsets).  With X [T, K], W [E, N, K], Y / dY [T, N]:
//   forward   Y_t   = X_t W_e^T     both operands have the contraction contiguous  (NT)
//   dX        dX_t  = dY_t W_e      the second operand is [contraction, columns]    (NN)
//   dW        dW_e  = dY_e^T X_e    both operands are [contraction, columns]        (TN)
// One kernel template serves all: only the way a fragment leaves LDS differs.
#pragma once

#include <type_traits>

#include "device_common.h"
#include "intlora_internal.h"

namespace intlora {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t u4i __attribute__((ext_vector_type(4)));
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

typedef uint32_t rsrc_t __attribute__((ext_vector_type(4)));

// Buffer descriptor of `bytes` bytes from `base` (none if negative): what lies past them
// reads zeros.  Lane offsets stay below 2^31: every tile and stage has a base of its own.
__device__ __forceinline__ rsrc_t make_desc(const void* base, int bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  // (uniform values; readfirstlane keeps them in scalar registers)
  return rsrc_t{(uint32_t)__builtin_amdgcn_readfirstlane((int)a),
                (uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32) & 0xFFFF),
                (uint32_t)__builtin_amdgcn_readfirstlane(bytes < 0 ? 0 : bytes), 0x00020000u};
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  const int64_t cap = 0x7FFFFFF0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0,
                                           (int)(bytes < 0 ? 0 : (bytes > cap ? cap : bytes)), 0x00020000);
}

// Direct load: lane l's 16 (4) bytes at `offset` of the buffer go to LDS at lds + 16 l (4 l).
// As instructions of our own and not the builtin, for which the compiler waits until every
// direct load in flight has landed before almost every LDS read; the stage loop's own waits
// order the two (with the compiler's waits the dX and dW loops took 1.5 times as long).  There
// is no output register; M0 is reserved (the compiler writes it right before each use of its
// own).  The s_nop covers the wait states between writes of M0 or the descriptor and their use.
__device__ __forceinline__ void direct_load16(const rsrc_t& r, uint32_t lds, uint32_t offset) {
  __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                   :
                   : "s"(lds), "v"(offset), "s"(r)
                   : "memory");
}
__device__ __forceinline__ void direct_load4(const rsrc_t& r, uint32_t lds, uint32_t offset) {
  __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
                   :
                   : "s"(lds), "v"(offset), "s"(r)
                   : "memory");
}

// At most N direct loads still in flight.
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// Every LDS read returned.
__device__ __forceinline__ void wait_lgkm() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }
// Both.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// At most N loads in flight, or N + MORE where `more` is not 0.  In one piece: a branch of the
// compiler's would cut the stage loop into blocks, and it would then move matrix instructions
// past the wait and spill.
template <int N, int MORE>
__device__ __forceinline__ void wait_vm_more(int more) {
  static_assert(N >= 0 && N + MORE < 64, "vmcnt is 6 bits");
  __asm__ volatile("s_cmp_lg_u32 %0, 0\n\ts_cbranch_scc1 .Lmore%=\n\ts_waitcnt vmcnt(%1)\n.Lmore%=:\n\ts_waitcnt vmcnt(%2)"
                   :
                   : "s"(__builtin_amdgcn_readfirstlane(more)), "n"(N), "n"(N + MORE)
                   : "memory", "scc");
}

__device__ __forceinline__ int clamp_row(int64_t o, int T) { return o < 0 ? 0 : (o > T ? T : (int)o); }

// Rows of the groups: boundary j is the largest of offsets[0 .. j], each forced into
// [0, T], and group e lies between boundaries e and e + 1.  For ascending offsets that is
// offsets[e] .. offsets[e + 1]; whatever else the array holds, no row outside [0, T) is
// touched and no row belongs to two groups.
struct Group {
  int e, row0, rows;
};

// Row tiles of all groups in order.  A wave looks at 64 groups at a time, one per lane, and
// keeps the chunk it looked at last (in LDS: it is needed once per tile); all waves of a
// block compute the same.
struct Groups {
  const int64_t* offsets;  // NULL: one group of all T rows
  int* at;                 // the wave's 3 x 64 words of LDS: first row, rows, running units
  int E, T, bm, per_tile;  // rows per tile; units per row tile
  int least, most;         // groups with other row counts have no tiles
  int e0, before, done;    // the chunk's first group, its first boundary, the units in front of it

  __device__ __forceinline__ int units(int n) const {
    return n >= least && n <= most ? (n + bm - 1) / bm * per_tile : 0;
  }
  __device__ __forceinline__ void chunk() {
    const int lane = threadIdx.x & 63, e = e0 + lane;
    int b = e < E ? clamp_row(offsets[e + 1], T) : 0;
    if (b < before) b = before;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(b, s);
      if (lane >= s && o > b) b = o;
    }
    int a = __shfl_up(b, 1);
    if (lane == 0) a = before;
    int inc = units(b - a);
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(inc, s);
      if (lane >= s) inc += o;
    }
    at[lane] = a;
    at[64 + lane] = b - a;
    at[128 + lane] = inc;
    __builtin_amdgcn_wave_barrier();
  }
  __device__ __forceinline__ void first() {
    e0 = 0;
    done = 0;
    before = __builtin_amdgcn_readfirstlane(clamp_row(offsets[0], T));
    chunk();
  }
  __device__ __forceinline__ bool advance() {
    if (e0 + 64 >= E) return false;
    done += __builtin_amdgcn_readfirstlane(at[128 + 63]);
    before = __builtin_amdgcn_readfirstlane(at[63] + at[64 + 63]);
    e0 += 64;
    chunk();
    return true;
  }
  // At most 64 groups, the ones of most rows first: at[] = their numbers, first rows, rows.
  __device__ __forceinline__ void sort() {
    if (offsets == nullptr) {
      at[0] = at[64] = 0;
      at[128] = T;
      __builtin_amdgcn_wave_barrier();
      return;
    }
    first();
    const int lane = threadIdx.x & 63;
    const int row0 = at[lane], rows = at[64 + lane];
    int rank = 0;
    for (int j = 0; j < E; ++j) {
      const int o = __builtin_amdgcn_readlane(rows, j);
      rank += o > rows || (o == rows && j < lane);
    }
    if (lane < E) {
      at[rank] = lane;
      at[64 + rank] = row0;
      at[128 + rank] = rows;
    }
    __builtin_amdgcn_wave_barrier();
  }
  // Number of units; leaves the last chunk in place.
  __device__ __forceinline__ int total() {
    if (offsets == nullptr) return units(T);
    first();
    while (advance()) {
    }
    return done + __builtin_amdgcn_readfirstlane(at[128 + 63]);
  }
  // The group of unit `want` (below total()), and the unit's number inside it.
  __device__ __forceinline__ Group find(int want, int& unit) {
    if (offsets == nullptr) {
      unit = want;
      return Group{0, 0, T};
    }
    if (want < done) first();
    uint64_t hit;
    while ((hit = __builtin_amdgcn_ballot_w64(done + at[128 + (threadIdx.x & 63)] > want)) == 0) {
      if (!advance()) break;
    }
    const int src = hit ? __builtin_ctzll(hit) : 63;
    const int row0 = __builtin_amdgcn_readfirstlane(at[src]), rows = __builtin_amdgcn_readfirstlane(at[64 + src]);
    unit = want - done - (__builtin_amdgcn_readfirstlane(at[128 + src]) - units(rows));
    return Group{e0 + src, row0, rows};
  }
};

// Rows of group e.
__device__ __forceinline__ Group group_rows(const int64_t* __restrict__ offsets, int e, int T) {
  if (offsets == nullptr) return Group{0, 0, T};
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
  const int b = __builtin_amdgcn_readfirstlane(clamp_row(offsets[e + 1], T));
  return Group{e, a, b > a ? b - a : 0};
}

// Blocks are dealt to the 8 XCDs in turn; this renumbers each run of 256 of them so that an
// XCD works on 32 consecutive tiles, whose operands its own L2 then serves.
__device__ __forceinline__ int xcd_slot(int b, int n) {
  if ((b | 255) >= n) return b;
  return (b & ~255) | ((b & 7) << 5) | ((b & 255) >> 3);
}

// ------------------------------------------------------------------------ tiled kernel
// A block computes BM x BN outputs at a time, each wave WM x WN of them in tiles of 32 x 32.
// The contraction goes in stages of 128 bytes of a row (64 16-bit or 128 8-bit elements)
// through a ring of ST LDS buffers filled by direct loads; a stage is two sub-steps of 64
// bytes.  With KS > 1 the block has KS such sets of waves with a ring each, which take the
// stages in turn; their sums meet in LDS.
//
// Products of many rows are bound by the matrix cores and by the loads that feed them: a stage of
// a 256 x 256 tile takes about 1.7 us, its matrix instructions alone 1.0 and its direct loads alone
// 1.1 (64 KB per compute unit through L2).  256 x 256 x 8 waves because the bytes loaded per
// product fall with the tile's side and the sums of 64 x 128 outputs are half of a wave's
// registers.  8192^3: 8 bits 433 us (2.54 PFLOP/s), bf16 forward 836, dX 867, dW 857 us (1.32,
// 1.27, 1.28 PFLOP/s); the matrix cores are busy 54 to 67 % of the time.
//
// Gated (GATE_ > 0; NT, 16 bits): the weight has 2 cols rows, gates in front, and a tile's BN weight
// rows are BN / 2 gates and the BN / 2 ups of the same columns, 32 of each in turn.  A lane then
// holds both projections of an output in tiles 2 j and 2 j + 1 of its sums, and the epilogue stores
// act(gate) * up, and with GATE_ = 2 the two projections too.  4096 x 14336 x 4096 in bf16: silu 757
// us, gelu 775 (1.25 PFLOP/s; the plain product with the same 28672 weight rows 771, as it stores
// twice the outputs); storing the projections too takes 50 us more (235 MB).  1027 x 2560 x 640 in
// fp16: 15.3 us, the plain product 15.2.
template <int TY_, int LAY_, int BM_, int BN_, int WM_, int WN_, int ST_, int KS_ = 1, int GATE_ = 0>
struct Tile {
  static constexpr int TY = TY_, LAY = LAY_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_, KS = KS_, GATE = GATE_;
  static constexpr int OUT_N = GATE ? BN / 2 : BN;  // output columns
  static constexpr bool F8 = TY == T_FP8;
  static constexpr int EB = F8 ? 1 : 2;        // bytes per element
  static constexpr int BK = 128 / EB;          // elements per stage
  static constexpr int WAVES_N = BN / WN, WAVES = BM / WM * WAVES_N, THREADS = 64 * WAVES * KS;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  // 8-bit: the scale dwords of a stage, BM rows', then the weight blocks' (64 per load; the
  // waves past the rows' all bring the latter)
  static constexpr int STAGE = A_BYTES + B_BYTES + (F8 ? 4 * BM + 256 : 0);
  static constexpr int AL = A_BYTES / 1024 / WAVES, BL = B_BYTES / 1024 / WAVES;  // direct loads per wave and stage
  static constexpr int AX = AL + (F8 ? 1 : 0), LOADS = AX + BL;  // with the scales' load
  static constexpr int MT = WM / 32, NT = WN / 32;
  static constexpr int READS = 2 * (MT + NT);                // LDS fragment reads per sub-step
  static constexpr int PRODUCTS = MT * NT * (F8 ? 1 : 2);    // matrix instructions per sub-step
  static constexpr int EPI_ROW = 32 * 2 + 16;                // epilogue staging: 32 rows of 32 16-bit outputs, padded
  static constexpr int RING = ST * STAGE, EPI = KS * RING, GROUPS = EPI + WAVES * 32 * EPI_ROW;
  static constexpr int LDS = GROUPS + WAVES * KS * 768;
  static constexpr bool TA = LAY == L_TN, TB = LAY != L_NT;  // operands stored [contraction, columns]
  static_assert(AL * 1024 * WAVES == A_BYTES && BL * 1024 * WAVES == B_BYTES, "whole loads");
  static_assert(!F8 || WAVES > BM / 64, "waves for the rows' scales and the weights'");
  static_assert(LDS <= 160 * 1024, "LDS of a compute unit");
  static_assert((KS - 1) * 4096 * MT * NT * WAVES <= EPI, "room for the sums");
  static_assert(!GATE || (LAY == L_NT && !F8 && BL * 8 == 32 && NT % 2 == 0), "a wave loads 32 gates or 32 ups");
};

// An operand tile of C rows / columns in LDS.  Row-contiguous operands (TR = 0) lie as rows
// of 128 bytes with the 16-byte chunk c of row r at c ^ (r / 2) % 8: the 16 lanes that a
// 16-byte read serves at a time then touch every bank once.  [contraction, columns] operands
// (TR = 1) lie as rows of 2 C bytes with chunk c of contraction row k at c ^ swz(k): a
// transposing read takes 4 rows x 64 bytes per 32 lanes, which this puts on different banks.
// Direct loads bring 1 KB each, always whole runs of 128 bytes or more: with runs of 64 bytes
// (twice as many requests to L2) the loads alone took 25 % longer.
template <bool TR, int C>
struct Operand {
  static constexpr int PER = TR ? C / 8 : 8;  // 16-byte chunks per LDS row
  static constexpr int ROWS = 64 / PER;       // LDS rows per load
  static_assert(C == 64 || C == 128 || C == 256, "the swizzle below");
  // TR: the 4 rows x 64 bytes of 32 lanes on different banks (rows of 128 bytes: 2 rows cover all)
  static __device__ __forceinline__ int swz(int k) { return C == 64 ? 2 * (k & 2) : 4 * (k & 3); }
  // This lane's place in a load: byte offset of its row, and of its chunk in the row for even
  // loads; the swizzle flips a bit of the latter for odd ones (TR = 1: where a load is 2 rows).
  static __device__ __forceinline__ uint32_t row(int lane, uint32_t ld) { return (uint32_t)(lane / PER) * ld; }
  static __device__ __forceinline__ int chunk(int lane) {
    const int r = lane / PER;
    return 16 * ((lane % PER) ^ (TR ? swz(r) : r >> 1));
  }
  static __device__ __forceinline__ int flip(int q) { return (q & 1) == 0 || (TR && ROWS != 2) ? 0 : TR ? 128 : 64; }
  // LDS offset of this lane's first fragment of the 32-row tiles from r0 (a multiple of 32 x
  // their number); lane half h takes the contraction chunk 4 sub + 2 h + ks of a stage.
  static __device__ __forceinline__ uint32_t frag(int lane, int r0) {
    const int h = lane >> 5, r = lane & 31;
    if (!TR) return (uint32_t)((r0 + r) * 128 + (((2 * h) ^ ((r >> 1) & 7)) << 4));
    // lane j of 16 points at contraction row j / 4, columns 4 (j % 4) .. + 3, and receives
    // column j, the four rows
    const int j = lane & 15, k = 16 * h + (j >> 2), col = r0 + (lane & 16) + 4 * (j & 3);
    return (uint32_t)(k * (2 * C) + (((col >> 3) ^ swz(k)) << 4) + ((col & 7) << 1));
  }
  // Fragment of 16 bytes of tile x from the operand's LDS at offset `at` = frag + its start.
  static __device__ __forceinline__ v4i read(const uint8_t* lds, uint32_t at, int x, int sub, int ks) {
    if (!TR) return *reinterpret_cast<const v4i*>(lds + (at ^ (uint32_t)((4 * sub + ks) << 4)) + x * 4096);
    const uint8_t* p = lds + (at ^ (uint32_t)(x << 6)) + (4 * sub + ks) * 16 * C;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t)p);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t)(p + 4 * 2 * C));
    const int2 a = __builtin_bit_cast(int2, lo), b = __builtin_bit_cast(int2, hi);
    return v4i{a.x, a.y, b.x, b.y};
  }
};

__device__ __forceinline__ int read_word(const uint8_t* lds, uint32_t at) {
  return *reinterpret_cast<const int*>(lds + at);
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

// The gate's activation and its derivative.  silu: g s, s = 1 / (1 + e^-g).  gelu: g P(g), P the
// normal distribution function, P(-z sqrt 2) = e^(-z z) f(z) / 2 with f(z) = e^(z z) erfc(z), z >= 0,
// as t times a polynomial of degree 8 in t = 1 / (1 + z / 2) (fitted to f / t at Chebyshev nodes;
// relative error 5e-7), so P keeps its relative precision for gates far below zero.
enum { ACT_SILU = 0, ACT_GELU = 1 };

__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(x * -1.44269504f); }  // e^-x

__device__ __forceinline__ float2 act_slope(int act, float g) {  // (act(g) / g, act'(g))
  if (act == ACT_SILU) {
    const float s = __builtin_amdgcn_rcpf(1.f + exp_neg(g));
    return make_float2(s, s + g * s * (1.f - s));
  }
  const float w = 0.5f * g * g, e = exp_neg(w);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(g), 0.35355339f, 1.f));
  float f = -0.043854326f;
  f = __builtin_fmaf(f, t, 0.220944047f);
  f = __builtin_fmaf(f, t, -0.377157629f);
  f = __builtin_fmaf(f, t, 0.176279768f);
  f = __builtin_fmaf(f, t, 0.027789898f);
  f = __builtin_fmaf(f, t, 0.185729653f);
  f = __builtin_fmaf(f, t, 0.246055290f);
  f = __builtin_fmaf(f, t, 0.282119066f);
  f = __builtin_fmaf(f, t, 0.282094657f);
  const float q = 0.5f * (f * t) * e, p = g < 0.f ? q : 1.f - q;
  return make_float2(p, __builtin_fmaf(g, 0.39894228f * e, p));
}
__device__ __forceinline__ float act_times(int act, float g, float u) { return g * act_slope(act, g).x * u; }

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
  int cus;                // blocks of the large tiles' launch
  int direct;             // no large tiles: the small ones are counted by themselves
  int rest_least, rest_most;  // small tiles of left-over large ones: their number if this launch is for them
  void* C2;               // gated: both projections, tokens x 2 cols (NULL: not wanted)
  int act;                // gated: ACT_*
};

constexpr int kBig = 256;        // the large tiles: kBig x kBig outputs, one block per compute unit
// Blocks of 256 threads that a grid holds: less than 2^32 work-items.
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;
// A last round of at least this many large tiles (of 256) is not cut up.  (4096 tokens, two
// blocks of small tiles to a compute unit: half a round of large tiles takes 47 us with
// contraction 2048, its small tiles 36; 160 of 256 54 and 56.)
constexpr int kTailShare = 129;
// dW behind whole rounds: its last tiles are the ones of the smallest groups and cost less than a
// round (half a round of 640 tiles, 4 groups: 84 us, cut up 92; a quarter of one is cut up).
constexpr int kTailShareDw = 65;

// Large tiles that a full grid of `cus` blocks takes in whole rounds; the rest is cut into
// small tiles, which fill the chip where a round of few large tiles would leave most
// compute units idle.
__device__ __forceinline__ int whole_rounds(int total, int cus, int share) {
  const int rem = total % cus;
  return rem * 256 >= share * cus ? total : total - rem;
}

// One output tile: its place, and where its operands start.  na, nb: bytes from there to the
// end of the operand's last row (row-contiguous operands); the [contraction, columns] ones
// are bounded by their rows, stage by stage.
struct Work {
  const uint8_t *pa, *pb, *ps;
  int na, nb, ns;
  int stages, kdim;
  Group g;
  int m0, n0;
  bool live;
};

// The stage that is loaded next: ST stages ahead of the one at work, and so at times in the
// next tile.
struct Stream {
  const uint8_t *pa, *pb, *ps;
  int na, nb, ns;
  int k, left;  // stage in the tile; contraction elements from it on
  int xa, xb;   // bytes of a [contraction, columns] row in front of the tile
};

template <class C, int TO>
__global__ void __launch_bounds__(C::THREADS, C::LDS > 80 * 1024 ? C::THREADS / 256 : 2) k_gemm(const GemmArgs p) {
  constexpr int TY = C::TY, LAY = C::LAY, BM = C::BM, BN = C::BN;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = C::KS > 1 ? wave / C::WAVES : 0, wid = wave - kg * C::WAVES;  // its set, and its number there
  const int wm = wid / C::WAVES_N, wn = wid % C::WAVES_N;
  constexpr bool BIG = BM == kBig;
  // ---- the launch's list: large tiles [0, whole), or the small tiles that the others
  // contain, or (direct) all of the small tiles
  const bool cut = !BIG && !p.direct;
  // a unit of the list's order
  const int um = BIG || cut ? kBig : BM, un = BIG || cut ? (C::GATE ? kBig / 2 : kBig) : C::OUT_N;
  const int units_n = (p.cols + un - 1) / un;
  const int units_m = (p.rows + um - 1) / um;  // TN
  Groups gr;
  gr.offsets = p.offsets;
  gr.at = reinterpret_cast<int*>(lds + C::GROUPS + wave * 768);
  gr.E = p.E;
  gr.T = p.T;
  gr.bm = um;
  gr.per_tile = units_n;
  gr.least = p.least;
  gr.most = p.most;
  gr.done = 0;
  const int total = LAY == L_TN ? p.E * units_m * units_n : gr.total();
  // dW: a tile costs its group's rows, so the tiles of the largest groups come first and every
  // other round goes through the blocks backwards, which evens their loads out
  const bool sorted = LAY == L_TN && (BIG || cut) && p.E <= 64;
  if (sorted) gr.sort();
  const int whole = BIG || cut ? whole_rounds(total, p.cus, LAY == L_TN ? kTailShareDw : kTailShare) : 0;
  constexpr int PER_M = kBig / BM, PER = PER_M * (kBig / BN);
  const int rest = total - whole;
  const int list = BIG ? whole : !cut ? total : rest >= p.rest_least && rest <= p.rest_most ? rest * PER : 0;

  const uint32_t lda = (uint32_t)((LAY == L_TN ? p.rows : p.kdim) * C::EB);
  const uint32_t ldb = (uint32_t)((LAY == L_NT ? p.kdim : p.cols) * C::EB);
  const int64_t da = C::TA ? (int64_t)C::BK * lda : 128, db = C::TB ? (int64_t)C::BK * ldb : 128;

  auto locate = [&](int at, Work& w) {
    w.live = at < list;
    w.pa = p.A;
    w.pb = p.B;
    w.ps = p.sa;
    w.na = w.nb = w.ns = w.kdim = 0;
    w.stages = 2;
    w.m0 = w.n0 = 0;
    if (!w.live) return;
    int unit = cut ? whole + at / PER : at;
    const int part = cut ? at % PER : 0;
    int tiles_m;
    if (LAY == L_TN) {
      const int e = unit / (units_m * units_n);
      unit -= e * units_m * units_n;
      if (sorted)
        w.g = Group{__builtin_amdgcn_readfirstlane(gr.at[e]), __builtin_amdgcn_readfirstlane(gr.at[64 + e]),
                    __builtin_amdgcn_readfirstlane(gr.at[128 + e])};
      else
        w.g = group_rows(p.offsets, e, p.T);
      tiles_m = units_m;
    } else {
      w.g = gr.find(unit, unit);
      tiles_m = (w.g.rows + um - 1) / um;
    }
    // patches of 8 row tiles: neighbouring tiles share both operands
    const int patch = unit / (8 * units_n), top = patch * 8;
    const int size = tiles_m - top < 8 ? tiles_m - top : 8;
    const int in = unit - patch * 8 * units_n;
    w.m0 = (top + in % size) * um + part % PER_M * BM;
    w.n0 = in / size * un + part / PER_M * C::OUT_N;
    const int rows = LAY == L_TN ? p.rows : w.g.rows;
    if (w.m0 >= rows || w.n0 >= p.cols) {  // a part of a large tile that hangs over the end
      w.live = false;
      return;
    }
    w.kdim = LAY == L_TN ? w.g.rows : p.kdim;
    const int k = (w.kdim + C::KS * C::BK - 1) / (C::KS * C::BK);
    // a stream that goes on in the next tile is at most one tile ahead; stages past the end
    // read zeros
    w.stages = BIG && k < C::ST ? C::ST : (k < 1 ? 1 : k);
    if (C::TA) {
      w.pa = p.A + (int64_t)w.g.row0 * lda + (int64_t)w.m0 * C::EB;
    } else {
      w.pa = p.A + (int64_t)(w.g.row0 + w.m0) * lda;
      w.na = (rows - w.m0 < BM ? rows - w.m0 : BM) * (int)lda;
    }
    if (LAY == L_NT) {
      w.pb = p.B + ((int64_t)w.g.e * (C::GATE ? 2 : 1) * p.cols + w.n0) * ldb;
      w.nb = (p.cols - w.n0 < C::OUT_N ? p.cols - w.n0 : C::OUT_N) * (int)ldb;
    } else if (LAY == L_NN) {
      w.pb = p.B + (int64_t)w.g.e * p.kdim * ldb + (int64_t)w.n0 * C::EB;
    } else {
      w.pb = p.B + (int64_t)w.g.row0 * ldb + (int64_t)w.n0 * C::EB;
    }
    if (C::F8) {
      if (wid < BM / 64) {
        const int n = rows - w.m0 - 64 * wid;
        w.ps = p.sa + (int64_t)(w.g.row0 + w.m0 + 64 * wid) * p.lds;
        w.ns = n <= 0 ? 0 : (n < 64 ? n : 64) * p.lds;
      } else {
        const int blocks = (p.cols + 127) >> 7, n = blocks - (w.n0 >> 7);
        w.ps = p.sb + ((int64_t)w.g.e * blocks + (w.n0 >> 7)) * p.lds;
        w.ns = (n < (BN + 127) / 128 ? n : (BN + 127) / 128) * p.lds;
      }
    }
  };

  using OA = Operand<C::TA, BM>;
  using OB = Operand<C::TB, BN>;
  // (a wave's loads are consecutive)
  const uint32_t ra = OA::row(lane, lda), rb = OB::row(lane, ldb);
  const int ca = OA::chunk(lane), cb = OB::chunk(lane);
  const uint32_t ring = kg * C::RING;
  const uint32_t fa = ring + OA::frag(lane, wm * C::WM), fb = ring + OB::frag(lane, wn * C::WN) + C::A_BYTES;
  // 8-bit: the first BM / 64 waves bring 64 rows' scale dwords each, the others the weight blocks'
  const uint32_t so = (uint32_t)((wid < BM / 64 ? lane : lane & (BN / 128 > 1 ? 1 : 0)) * p.lds);

  // The stage loads.  Rows past the operand's end and stages past the last read zeros; so do
  // the chunks past a row's end in the last stage, in both operands (what lies there may be a
  // NaN, and 0 x NaN is not 0).  A wave's loads of an operand share one descriptor; the loop
  // is bound by instruction issue, so a load costs one addition besides itself.
  Stream ls;
  rsrc_t dsa, dsb, dss;
  uint32_t va[2], vb[2];  // lane offsets of even and odd loads
  auto begin_tile = [&](const Work& w) {
    // the wave's first row (gated: even waves load gates, odd ones ups)
    const int ga = wid * C::AL * OA::ROWS, gb = C::GATE ? (wid >> 1) * 32 : wid * C::BL * OB::ROWS;
    ls.pa = w.pa + (int64_t)ga * lda + kg * da;
    ls.pb = w.pb + ((int64_t)gb + (C::GATE && (wid & 1) ? p.cols : 0)) * ldb + kg * db;
    ls.ps = w.ps;
    ls.na = w.na - ga * (int)lda - 128 * kg;
    ls.nb = w.nb - gb * (int)ldb - 128 * kg;
    ls.ns = w.ns;
    ls.k = kg;
    ls.left = w.kdim - kg * C::BK;
    ls.xa = w.m0 * C::EB;
    ls.xb = w.n0 * C::EB;
  };
  // Descriptors and lane offsets of the stage, then on to the next one.
  auto begin_stage = [&]() {
    const int rows = ls.left < C::BK ? (ls.left < 0 ? 0 : ls.left) : C::BK;  // contraction rows of the stage
    const int left = ls.left * C::EB;                                        // bytes of a contiguous row
    const int ga = wid * C::AL * OA::ROWS, gb = wid * C::BL * OB::ROWS;
    const int ba = C::TA ? (rows - ga) * (int)lda - ls.xa : ls.na;
    const int bb = C::TB ? (rows - gb) * (int)ldb - ls.xb : ls.nb;
    dsa = make_desc(ls.pa, left > 0 ? ba : 0);
    dsb = make_desc(ls.pb, left > 0 ? bb : 0);
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int xa = ca ^ OA::flip(f), xb = cb ^ OB::flip(f);
      va[f] = C::TA || xa < left ? ra + xa : kOOB;
      vb[f] = C::TB || xb < left ? rb + xb : kOOB;
    }
    if (C::F8) {  // the dword of four 128-blocks that holds this stage's scale
      const int at = (ls.k >> 2) * 4;
      dss = make_desc(ls.ps + at, left > 0 ? ls.ns - at : 0);
    }
    ls.pa += C::KS * da;
    ls.pb += C::KS * db;
    ls.na -= C::KS * 128;
    ls.nb -= C::KS * 128;
    ls.left -= C::KS * C::BK;
    ls.k += C::KS;
  };
  auto issue_b = [&](int q, uint32_t S) {  // load number q of the stage's second operand
    direct_load16(dsb, S + C::A_BYTES + (wid * C::BL + q) * 1024, vb[q & 1] + q * OB::ROWS * ldb);
  };
  auto issue_a = [&](int q, uint32_t S) {  // of the first one; the last is the scales'
    if (q < C::AL)
      direct_load16(dsa, S + (wid * C::AL + q) * 1024, va[q & 1] + q * OA::ROWS * lda);
    else
      direct_load4(dss, S + C::A_BYTES + C::B_BYTES + (wid < BM / 64 ? wid : BM / 64) * 256, so);
  };

  // Fragments of one sub-step in registers.  Two sets alternate: while the matrix cores work
  // on one, the other is read from LDS.
  struct Frag {
    v4i a[C::MT][2], b[C::NT][2];
  };
  struct Scales {
    int x[C::MT], w;
  };
  auto read = [&](int q, uint32_t sa, uint32_t sb, int sub, Frag& f) {  // LDS read number q of a sub-step
    const int x = q >> 1, ks = q & 1;
    if (x < C::NT)
      f.b[x][ks] = OB::read(lds, sb, x, sub, ks);
    else
      f.a[x - C::NT][ks] = OA::read(lds, sa, x - C::NT, sub, ks);
  };
  auto read_scales = [&](int kt, int start, Scales& s) {
    const uint32_t at = ring + start + C::A_BYTES + C::B_BYTES;
    const int sh = 8 * ((C::KS * kt + kg) & 3);
    s.w = (int)((uint32_t)read_word(lds, at + 4 * (BM + (wn * C::WN) / 128)) >> sh);
#pragma unroll
    for (int i = 0; i < C::MT; ++i)
      s.x[i] = (int)((uint32_t)read_word(lds, at + 4 * (wm * C::WM + 32 * i + (lane & 31))) >> sh);
  };
  v16f acc[C::MT][C::NT];
  auto product = [&](int q, const Frag& f, const Scales& s) {  // matrix instruction number q of a sub-step
    const int ks = q / (C::MT * C::NT), i = q % (C::MT * C::NT) / C::NT, j = q % C::NT;
    if (C::F8) {
      const v8i a = __builtin_shufflevector(f.a[i][0], f.a[i][1], 0, 1, 2, 3, 4, 5, 6, 7);
      const v8i b = __builtin_shufflevector(f.b[j][0], f.b[j][1], 0, 1, 2, 3, 4, 5, 6, 7);
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc[i][j], 0, 0, 0, s.w, 0, s.x[i]);
    } else {
      acc[i][j] = mfma16<TY>(f.b[j][ks], f.a[i][ks], acc[i][j]);
    }
  };
  // behind each matrix instruction: LDS reads of sub-step 0; and in each half of sub-step 1 the
  // LDS reads and the direct loads of one operand
  constexpr int PER_P = (C::READS + C::PRODUCTS - 1) / C::PRODUCTS;
  constexpr int HALF = C::PRODUCTS / 2;
  constexpr int RB = (2 * C::NT + HALF - 1) / HALF, RA = (2 * C::MT + HALF - 1) / HALF;
  constexpr int IB = (C::BL + HALF - 1) / HALF, IA = (C::AX + HALF - 1) / HALF;

  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)lds + ring;  // LDS address of the buffers
  const int step = gridDim.x;
  const int slot = xcd_slot(blockIdx.x, step);
  auto tile_of = [&](int round) { return round * step + (sorted && (round & 1) ? step - 1 - slot : slot); };
  int round = 0;
  Work cur, nxt;
  locate(tile_of(0), cur);
  if (BIG ? tile_of(0) >= list : !cur.live) return;  // (small tiles: one per block)
  locate(tile_of(1), nxt);
  begin_tile(cur);
#pragma unroll
  for (int s = 0; s < C::ST; ++s) {
    begin_stage();
#pragma unroll
    for (int q = 0; q < C::BL; ++q) issue_b(q, lds0 + s * C::STAGE);
#pragma unroll
    for (int q = 0; q < C::AX; ++q) issue_a(q, lds0 + s * C::STAGE);
  }
  int ph = 0;  // start of the buffer of the stage at work
  Frag f0, f1;
  Scales sc, sn;
  wait_loads<(C::ST - 1) * C::LOADS>();
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
#pragma unroll
  for (int q = 0; q < C::READS; ++q) read(q, fa, fb, 0, f0);
  if (C::F8) read_scales(0, 0, sc);

  const bool aligned = (int64_t)p.cols * (TO == T_FP32 ? 4 : 2) % 16 == 0;
  constexpr int STORES = C::GATE ? (C::GATE == 2 ? 3 : 1) * C::MT * C::NT : (TO == T_FP32 ? 4 : 2) * C::MT * C::NT;
  int fresh = 0;  // the last tile's STORES stores may be in flight, newer than this tile's first two stages
  // The stages of a block's consecutive tiles are one stream: the first stages of the next
  // tile are loaded during the last ones of this tile, and while its epilogue runs.
  for (;;) {
#pragma unroll
    for (int i = 0; i < C::MT; ++i)
#pragma unroll
      for (int j = 0; j < C::NT; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
#pragma nounroll
    for (int kt = 0; kt < cur.stages; ++kt) {
      const uint32_t S = lds0 + ph;
      const uint32_t sa = fa + ph, sb = fb + ph;
      ph = ph == (C::ST - 1) * C::STAGE ? 0 : ph + C::STAGE;
      const uint32_t na = fa + ph, nb = fb + ph;
      // sub-step 0 from f0; f1 takes sub-step 1
#pragma unroll
      for (int q = 0; q < C::PRODUCTS; ++q) {
        product(q, f0, sc);
#pragma unroll
        for (int r = PER_P * q; r < PER_P * (q + 1) && r < C::READS; ++r) read(r, sa, sb, 1, f1);
        __builtin_amdgcn_sched_barrier(0);
      }
      // Behind this barrier every wave has its fragments of the stage, whose buffer takes stage
      // kt + ST, and the next stage's second operand has landed for all waves; behind the one
      // half a sub-step later the first operand has.  So the loads never run dry: half a stage
      // is in flight at either barrier (with one barrier for both operands the loads alone
      // took 1.5 times the matrix cores' time).
      wait_lgkm();
      if (BIG)
        wait_vm_more<C::AX + (C::ST - 2) * C::LOADS, BIG ? STORES : 0>(fresh);
      else
        wait_vm<C::AX + (C::ST - 2) * C::LOADS>();
      __builtin_amdgcn_s_barrier();
      __asm__ volatile("" ::: "memory");
      if (kt + C::ST == cur.stages) begin_tile(nxt);
      begin_stage();
      // sub-step 1 from f1; f0 takes the next stage's sub-step 0
#pragma unroll
      for (int q = 0; q < C::PRODUCTS; ++q) {
        if (q == HALF) {
          if (BIG)
            wait_vm_more<C::BL + (C::ST - 2) * C::LOADS, BIG ? STORES : 0>(fresh);
          else
            wait_vm<C::BL + (C::ST - 2) * C::LOADS>();
          fresh = 0;
          __builtin_amdgcn_s_barrier();
          __asm__ volatile("" ::: "memory");
          if (C::F8) read_scales(kt + 1 < cur.stages ? kt + 1 : 0, ph, sn);
        }
        product(q, f1, sc);
        if (q < HALF) {
#pragma unroll
          for (int r = RB * q; r < RB * (q + 1) && r < 2 * C::NT; ++r) read(r, na, nb, 0, f0);
#pragma unroll
          for (int r = IB * q; r < IB * (q + 1) && r < C::BL; ++r) issue_b(r, S);
        } else {
#pragma unroll
          for (int r = RA * (q - HALF); r < RA * (q - HALF + 1) && r < 2 * C::MT; ++r) read(2 * C::NT + r, na, nb, 0, f0);
#pragma unroll
          for (int r = IA * (q - HALF); r < IA * (q - HALF + 1) && r < C::AX; ++r) issue_a(r, S);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      sc = sn;
    }

    if (C::KS > 1) {  // the other sets' sums go to the first, which adds them in order and stores
      wait_loads<0>();  // (zeros past the last stage still land in the rings)
      __builtin_amdgcn_s_barrier();
      __asm__ volatile("" ::: "memory");
      constexpr int PIECES = 4 * C::MT * C::NT;  // 16 bytes of each lane
      float4* sums = reinterpret_cast<float4*>(lds) + wid * (64 * PIECES) + lane;
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const v16f& t = acc[i / (4 * C::NT)][i / 4 % C::NT];
        const int a = 4 * (i & 3);
        if (kg > 0) sums[((kg - 1) * C::WAVES * PIECES + i) * 64] = make_float4(t[a], t[a + 1], t[a + 2], t[a + 3]);
      }
      wait_lgkm();
      __builtin_amdgcn_s_barrier();
      __asm__ volatile("" ::: "memory");
      if (kg > 0) return;  // (no barrier follows: one tile per block)
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        v16f& t = acc[i / (4 * C::NT)][i / 4 % C::NT];
        const int a = 4 * (i & 3);
#pragma unroll
        for (int g = 0; g < C::KS - 1; ++g) {
          const float4 o = sums[(g * C::WAVES * PIECES + i) * 64];
          t[a] += o.x;
          t[a + 1] += o.y;
          t[a + 2] += o.z;
          t[a + 3] += o.w;
        }
      }
    }

    // ---- epilogue: lane l holds row l % 32 of a tile and columns 8 a + 4 (l / 32) + 0 .. 3 in
    // registers 4 a .. 4 a + 3.  16-bit outputs pass through LDS, one 32 x 32 tile at a time
    // in a part of the wave's own, so that whole 64-byte row pieces are stored.  Rows and
    // columns past the end are stores past the buffer's, so a wave's stores are always STORES
    // in number and the next tile's first stage need not wait for them.
    if (C::GATE) {
      if (cur.live) {
        uint8_t* stg = lds + C::EPI + wid * 32 * C::EPI_ROW;
        int el = lane;  // (as below)
        __asm__ volatile("" : "+v"(el));
        const int fr = el & 31, h = el >> 5;
        const int rows_left = cur.g.rows - cur.m0 - wm * C::WM;
        const int64_t row = (int64_t)cur.g.row0 + cur.m0 + wm * C::WM;
        const int c0 = cur.n0 + wn * (C::WN / 2);
        const int64_t ldo = (int64_t)p.cols * 2;
        const __amdgpu_buffer_rsrc_t rh = make_rsrc(static_cast<uint8_t*>(p.C) + row * ldo + 2 * c0, C::WM * ldo);
        // both projections: rows of 2 cols numbers, from the gate's column c0 on
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(static_cast<uint8_t*>(p.C2) + (row * ldo + c0) * 2, 2 * C::WM * ldo);
        // one 32 x 32 tile v(a, e) of registers 4 a + e, through LDS as below
        auto put = [&](auto v, const __amdgpu_buffer_rsrc_t& r, uint32_t at, int64_t ld, int live, int cols) {
#pragma unroll
          for (int a = 0; a < 4; ++a)
            *reinterpret_cast<uint2*>(stg + fr * C::EPI_ROW + (8 * a + 4 * h) * 2) =
                make_uint2(pack2<TO>(v(4 * a), v(4 * a + 1)), pack2<TO>(v(4 * a + 2), v(4 * a + 3)));
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int y = 16 * q + (el >> 2), c = el & 3;
            const u4i x = *reinterpret_cast<const u4i*>(stg + y * C::EPI_ROW + 16 * c);
            __builtin_amdgcn_raw_buffer_store_b128(
                x, r, y < live && 8 * c < cols ? at + (uint32_t)(y * ld) + 16 * c : kOOB, 0, 0);
          }
          __builtin_amdgcn_wave_barrier();
        };
#pragma unroll
        for (int i = 0; i < C::MT; ++i) {
          const int live = rows_left - 32 * i;
#pragma unroll
          for (int j = 0; j < C::NT / 2; ++j) {
            __builtin_amdgcn_sched_barrier(0);
            const int cols = p.cols - c0 - 32 * j;
            const v16f &g = acc[i][2 * j], &u = acc[i][C::GATE ? 2 * j + 1 : 0];
            if (C::GATE == 2) {
              const uint32_t o = (uint32_t)(32 * i * 2 * ldo) + 64 * j;
              put([&](int x) { return g[x]; }, rs, o, 2 * ldo, live, cols);
              put([&](int x) { return u[x]; }, rs, o + (uint32_t)ldo, 2 * ldo, live, cols);
            }
            put([&](int x) { return act_times(p.act, g[x], u[x]); }, rh, (uint32_t)(32 * i * ldo) + 64 * j, ldo, live,
                cols);
          }
        }
      }
    } else if (cur.live) {
      uint8_t* stg = lds + C::EPI + wid * 32 * C::EPI_ROW;
      // (a copy of the lane number that the compiler does not see through: it would compute the
      // epilogue's addresses before the stage loop, which has no registers for them)
      int el = lane;
      __asm__ volatile("" : "+v"(el));
      const int fr = el & 31, h = el >> 5;
      constexpr int EO = TO == T_FP32 ? 4 : 2;
      const int rows_left = (LAY == L_TN ? p.rows : cur.g.rows) - cur.m0 - wm * C::WM;
      const int64_t out_row = (LAY == L_TN ? (int64_t)cur.g.e * p.rows : (int64_t)cur.g.row0) + cur.m0 + wm * C::WM;
      const int c0 = cur.n0 + wn * C::WN;
      uint8_t* out = static_cast<uint8_t*>(p.C) + (out_row * p.cols + c0) * EO;
      const int64_t ldo = (int64_t)p.cols * EO;
      const __amdgpu_buffer_rsrc_t ro = make_rsrc(out, C::WM * ldo);
#pragma unroll
      for (int i = 0; i < C::MT; ++i) {
        const int live = rows_left - 32 * i;
#pragma unroll
        for (int j = 0; j < C::NT; ++j) {
          __builtin_amdgcn_sched_barrier(0);  // one tile's outputs at a time
          const int cols = p.cols - c0 - 32 * j;
          const uint32_t o = (uint32_t)((32 * i) * ldo) + 32 * j * EO;
          if (TO == T_FP32) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
              const int c = 8 * a + 4 * h;
              const float4 y = make_float4(acc[i][j][4 * a], acc[i][j][4 * a + 1], acc[i][j][4 * a + 2],
                                           acc[i][j][4 * a + 3]);
              // columns are a multiple of 8 here: whole groups of four
              __builtin_amdgcn_raw_buffer_store_b128(
                  __builtin_bit_cast(u4i, y), ro, fr < live && c < cols ? o + (uint32_t)(fr * ldo) + 4 * c : kOOB, 0, 0);
            }
          } else {
#pragma unroll
            for (int a = 0; a < 4; ++a)
              *reinterpret_cast<uint2*>(stg + fr * C::EPI_ROW + (8 * a + 4 * h) * 2) =
                  make_uint2(pack2<TO>(acc[i][j][4 * a], acc[i][j][4 * a + 1]),
                             pack2<TO>(acc[i][j][4 * a + 2], acc[i][j][4 * a + 3]));
            __builtin_amdgcn_wave_barrier();
            if (aligned) {  // columns are a multiple of 8: whole 16-byte pieces
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int r = 16 * q + (el >> 2), c = el & 3;
                const u4i v = *reinterpret_cast<const u4i*>(stg + r * C::EPI_ROW + 16 * c);
                __builtin_amdgcn_raw_buffer_store_b128(
                    v, ro, r < live && 8 * c < cols ? o + (uint32_t)(r * ldo) + 16 * c : kOOB, 0, 0);
              }
            } else {
#pragma unroll 4
              for (int r = h; r < 32; r += 2) {
                const uint16_t v = *reinterpret_cast<const uint16_t*>(stg + r * C::EPI_ROW + 2 * fr);
                if (r < live && fr < cols) reinterpret_cast<uint16_t*>(out + o + r * ldo)[fr] = v;
              }
            }
            __builtin_amdgcn_wave_barrier();
          }
        }
      }
    }
    fresh = (aligned || C::GATE) && cur.live ? 1 : 0;
    ++round;
    if (tile_of(round) >= list) break;
    cur = nxt;
    locate(tile_of(round + 1), nxt);
  }
  wait_loads<0>();  // the stages loaded past the last tile (zeros)
}

template <class C, int TO>
hipError_t launch_gemm(const GemmArgs& a, int64_t blocks, hipStream_t st) {
  static thread_local int ready_dev = -1;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev != ready_dev) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_gemm<C, TO>), hipFuncAttributeMaxDynamicSharedMemorySize,
                            C::LDS);
    if (e != hipSuccess) return e;
    ready_dev = dev;
  }
  k_gemm<C, TO><<<dim3((unsigned)blocks), C::THREADS, C::LDS, st>>>(a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------ few rows
// Groups of few rows are bound by the weights' bytes.  A tile is 16 weight rows against 16 TT
// token rows; `ks` waves share one, taking runs of 256 bytes of the contraction in turn, and
// their sums meet in LDS in a fixed order (ks = 1: every wave has tiles of its own, and no
// barrier).  Each wave keeps a ring of runs of its own in LDS, filled by direct loads of 4 rows
// x 256 bytes.  The grid is persistent and the runs of a wave's consecutive tiles are one
// stream, so the memory is kept busy across a tile's end.  (Fragments loaded straight into
// registers take 16 bytes from each of 16 rows per 16 lanes: 16-token products then streamed
// 3 TB/s.)  Bound by memory: 14336 x 4096 in 8 bits 13.1 us for 1 token (4.5 TB/s), 13.4 for 16,
// 15.2 for 32; eight bf16 experts of 4096 x 2048, 2 tokens each 25.4 us (5.3 TB/s); 4096 x 4096 in
// 8 bits, 1 token 6.3 us, where launch and first loads count.
// Gated (as in Tile): a tile is 16 gates and the 16 ups of the same columns, with four waves a
// block, as their runs are twice as long; 14336 x 4096 in bf16, 1 token 44 us (5.3 TB/s).
template <int TY_, int TT_, bool GATE_ = false>
struct Few {
  static constexpr int TY = TY_, TT = TT_, WT = GATE_ ? 2 : 1;  // weight tiles
  static constexpr bool F8 = TY == T_FP8, GATE = GATE_;
  static constexpr int WAVES = TT == 1 && !GATE ? 8 : 4, RING = 2;  // streams of a block; runs in flight of each
  static constexpr int RUN = 4096 * (WT + TT) + (F8 ? 512 : 0);     // LDS bytes of a run
  static constexpr int LOADS = 4 * (WT + TT) + (F8 ? 2 : 0);        // direct loads of a run
  static constexpr int TURNS = GATE && TT == 2 ? 1 : 2;             // places of a tile's sums (LDS holds one there)
  static constexpr int SUMS = WAVES * RING * RUN, GROUPS = SUMS + TURNS * WAVES * WT * TT * 1024;
  static_assert(!GATE || !F8, "gated products are 16-bit");
  static constexpr int LDS = GROUPS + WAVES * 768;
  static_assert(LDS <= 160 * 1024 && (RING - 1) * LOADS < 64, "LDS and load counter");
};

template <class C>
__global__ void __launch_bounds__(64 * C::WAVES, 2) k_few(const GemmArgs p, int ks) {
  constexpr int TY = C::TY, TT = C::TT, WT = C::WT, WAVES = C::WAVES, RING = C::RING;
  constexpr bool F8 = C::F8;
  constexpr int EB = F8 ? 1 : 2;
  constexpr int TO = TY == T_FP16 ? T_FP16 : T_BF16;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, q = lane >> 4;
  const int ld = p.kdim * EB;
  const int runs = (ld + 255) >> 8;
  const int tiles_n = (p.cols + 15) >> 4;
  const int blocks = (p.cols + 127) >> 7;
  Groups gr;
  gr.offsets = p.offsets;
  gr.at = reinterpret_cast<int*>(lds + C::GROUPS + wid * 768);
  gr.E = p.E;
  gr.T = p.T;
  gr.bm = 16 * TT;
  gr.per_tile = tiles_n;
  gr.least = p.least;
  gr.most = p.most;
  gr.done = 0;
  const int total = gr.total();

  // A tile: 16 weight rows and up to 16 TT token rows of one group
  struct Place {
    const uint8_t *w, *x, *sw, *sx;
    int wrows, xrows, n0;
    int64_t row0;
  };
  auto locate = [&](int at, Place& t) {
    if (at >= total) {  // past the block's last tile: no bytes
      t.w = p.B;
      t.x = p.A;
      t.sw = p.sb;
      t.sx = p.sa;
      t.wrows = t.xrows = t.n0 = 0;
      t.row0 = 0;
      return;
    }
    int unit;
    const Group g = gr.find(at, unit);
    const int part = unit / tiles_n;  // 16 TT rows of the group
    t.n0 = (unit - part * tiles_n) * 16;
    t.row0 = (int64_t)g.row0 + part * 16 * TT;
    t.xrows = g.rows - part * 16 * TT < 16 * TT ? g.rows - part * 16 * TT : 16 * TT;
    t.wrows = p.cols - t.n0 < 16 ? p.cols - t.n0 : 16;
    t.w = p.B + ((int64_t)g.e * WT * p.cols + t.n0) * ld;
    t.x = p.A + t.row0 * ld;
    t.sw = F8 ? p.sb + ((int64_t)g.e * blocks + (t.n0 >> 7)) * p.lds : nullptr;
    t.sx = F8 ? p.sa + t.row0 * p.lds : nullptr;
  };

  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)lds + wid * RING * C::RUN;
  // Load l of an operand: rows 4 l .. 4 l + 3; the 16-byte chunk c of row r lies at c ^ r % 16,
  // so that the 16 rows' chunks of one column are on different banks.
  const int lrow = lane >> 4, lchunk = lane & 15;
  uint32_t off[4];  // rows 4 l + lrow of the weights, and 16 l' more of the tokens
  int chunk[4];
#pragma unroll
  for (int l = 0; l < 4; ++l) {
    chunk[l] = 16 * (lchunk ^ (4 * l + lrow));
    off[l] = (uint32_t)((4 * l + lrow) * ld) + chunk[l];
  }
  // Rows past the operand's end and chunks past a row's end read zeros (a NaN may lie there).
  auto load_run = [&](const Place& t, int run, int place) {
    const uint32_t S = lds0 + place * C::RUN;
    const int k0 = run << 8, left = ld - k0;
    const rsrc_t rw = make_desc(t.w + k0, t.wrows * ld - k0);
    const rsrc_t rx = make_desc(t.x + k0, t.xrows * ld - k0);
    const rsrc_t ru = C::GATE ? make_desc(t.w + (int64_t)p.cols * ld + k0, t.wrows * ld - k0) : rw;
#pragma unroll
    for (int l = 0; l < 4 * (WT + TT); ++l) {
      const uint32_t o = chunk[l & 3] < left ? off[l & 3] : kOOB;
      direct_load16(l < 4 ? rw : l < 4 * WT ? ru : rx, S + 1024 * l, l < 4 * WT + 4 ? o : o + 16 * ld);
    }
    if (F8) {  // the dword of four 128-blocks that holds the run's two scales
      const int at = (run >> 1) * 4;
      direct_load4(make_desc(t.sx + at, t.xrows * p.lds - at), S + 4096 * (WT + TT), (uint32_t)(lane * p.lds));
      direct_load4(make_desc(t.sw + at, t.wrows > 0 ? 4 : 0), S + 4096 * (WT + TT) + 256, 0);
    }
  };

  const int slots = WAVES / ks, slot = wid / ks, kw = wid - slot * ks;  // tiles at a time; this wave's; its share
  const int step = gridDim.x * slots;
  const int first = xcd_slot(blockIdx.x, gridDim.x) * slots;
  if (first >= total) return;
  const int mine = runs > kw ? (runs - kw + ks - 1) / ks : 0;  // runs of a tile that are this wave's
  // The stream of loads is RING runs ahead, and so in one of the next tiles at times.
  Place lp, cur;
  int la = first + slot, lr = 0;  // its tile, and its run among the wave's
  locate(la, lp);
  auto load_next = [&](int place) {
    if (lr == mine) {
      lr = 0;
      la += step;
      locate(la, lp);
    }
    load_run(lp, kw + lr * ks, place);
    ++lr;
  };
  if (mine > 0)
    for (int r = 0; r < RING; ++r) load_next(r);
  int place = 0, parity = 0;
  for (int base = first; base < total; base += step) {
    const int at = base + slot;  // (past the last tile: no bytes, no outputs)
    v4f acc[WT][TT];
#pragma unroll
    for (int t = 0; t < WT * TT; ++t) acc[t / TT][t % TT] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < mine; ++i) {
      const int run = kw + i * ks;
      wait_loads<(RING - 1) * C::LOADS>();  // all but the newer runs have landed
      __asm__ volatile("" ::: "memory");
      const uint8_t* S = lds + (wid * RING + place) * C::RUN;
      v4i w[WT][4], x[TT][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = ((4 * u + q) ^ fr) << 4;
#pragma unroll
        for (int g = 0; g < WT; ++g) w[g][u] = *reinterpret_cast<const v4i*>(S + 4096 * g + fr * 256 + c);
#pragma unroll
        for (int t = 0; t < TT; ++t) x[t][u] = *reinterpret_cast<const v4i*>(S + 4096 * (WT + t) + fr * 256 + c);
      }
      int sw = 0, sx[TT];
      if (F8) {
        const int sh = 16 * (run & 1);
        sw = (int)((uint32_t)read_word(S, 4096 * (WT + TT) + 256) >> sh);
#pragma unroll
        for (int t = 0; t < TT; ++t)
          sx[t] = (int)((uint32_t)read_word(S, 4096 * (WT + TT) + 4 * (16 * t + fr)) >> sh);
      }
      wait_lgkm();  // the run is in registers: its place takes the next one
      load_next(place);
      place = place == RING - 1 ? 0 : place + 1;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int z = 0; z < WT * TT; ++z) {
          const int g = z / TT, t = z % TT;
          if (F8) {
            const v8i a = __builtin_shufflevector(x[t][2 * u], x[t][2 * u + 1], 0, 1, 2, 3, 4, 5, 6, 7);
            const v8i b = __builtin_shufflevector(w[g][2 * u], w[g][2 * u + 1], 0, 1, 2, 3, 4, 5, 6, 7);
            acc[g][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, acc[g][t], 0, 0, 0, sw >> (8 * u), 0,
                                                                         sx[t] >> (8 * u));
          } else {
#pragma unroll
            for (int v = 2 * u; v < 2 * u + 2; ++v) {
              if (TY == T_BF16)
                acc[g][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf8, w[g][v]), __builtin_bit_cast(bf8, x[t][v]), acc[g][t], 0, 0, 0);
              else
                acc[g][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    __builtin_bit_cast(h8, w[g][v]), __builtin_bit_cast(h8, x[t][v]), acc[g][t], 0, 0, 0);
            }
          }
        }
    }
    // lane l of a tile: token l % 16, columns 4 (l / 16) + 0 .. 3
    auto store = [&](int t, v4f s, void* out, int ldo, int c0) {  // columns from c0 on of rows of ldo
      const int row = 16 * t + fr, col = cur.n0 + 4 * q;
      if (row >= cur.xrows) return;
      uint16_t* y = static_cast<uint16_t*>(out) + (cur.row0 + row) * ldo + c0 + col;
      const uint32_t lo = pack2<TO>(s.x, s.y), hi = pack2<TO>(s.z, s.w);
      if ((p.cols & 3) == 0 && col + 4 <= p.cols) {
        *reinterpret_cast<uint2*>(y) = make_uint2(lo, hi);
      } else {
        const uint16_t o[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (col + c < p.cols) y[c] = o[c];
      }
    };
    auto finish = [&](int t, const v4f (&s)[WT]) {
      if (!C::GATE) {
        store(t, s[0], p.C, p.cols, 0);
        return;
      }
      const v4f &g = s[0], &u = s[WT - 1];
      if (p.C2) {
        store(t, g, p.C2, 2 * p.cols, 0);
        store(t, u, p.C2, 2 * p.cols, p.cols);
      }
      store(t, v4f{act_times(p.act, g.x, u.x), act_times(p.act, g.y, u.y), act_times(p.act, g.z, u.z),
                   act_times(p.act, g.w, u.w)},
            p.C, p.cols, 0);
    };
    if (ks == 1) {
      locate(at, cur);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        v4f s[WT];
#pragma unroll
        for (int g = 0; g < WT; ++g) s[g] = acc[g][t];
        finish(t, s);
      }
    } else {
      // the sums of even and odd tiles take turns, so one barrier a tile is enough
      if (C::TURNS == 1) {
        wait_lgkm();
        __builtin_amdgcn_s_barrier();
        __asm__ volatile("" ::: "memory");
      }
      float* part = reinterpret_cast<float*>(lds + C::SUMS) + parity * WAVES * WT * TT * 256;
      parity = C::TURNS - 1 - parity;
#pragma unroll
      for (int z = 0; z < WT * TT; ++z)
        *reinterpret_cast<v4f*>(part + (wid * WT * TT + z) * 256 + 4 * lane) = acc[z / TT][z % TT];
      wait_lgkm();
      __builtin_amdgcn_s_barrier();
      __asm__ volatile("" ::: "memory");
      if (kw < TT) {  // ks >= TT
        locate(at, cur);
        v4f s[WT];
#pragma unroll
        for (int g = 0; g < WT; ++g) {
          s[g] = v4f{0.f, 0.f, 0.f, 0.f};
          for (int v = 0; v < ks; ++v)
            s[g] += *reinterpret_cast<const v4f*>(part + ((slot * ks + v) * WT * TT + g * TT + kw) * 256 + 4 * lane);
        }
        finish(kw, s);
      }
    }
  }
  wait_loads<0>();
}

template <int TY, int TT, bool GATE>
hipError_t launch_few_tt(const GemmArgs& a, hipStream_t st) {
  using C = Few<TY, TT, GATE>;
  static thread_local int ready_dev = -1;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev != ready_dev) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_few<C>), hipFuncAttributeMaxDynamicSharedMemorySize,
                            C::LDS);
    if (e != hipSuccess) return e;
    ready_dev = dev;
  }
  const int64_t groups = a.E < a.T ? a.E : a.T;
  const int64_t tiles = ((int64_t)a.cols + 15) / 16 * ((a.T + 16 * TT - 1) / (16 * TT) + groups - 1);
  // All waves of a block on one tile, but fewer where a wave would have less than two runs of it
  // and there are tiles enough without (64 experts of 2048 x 1024, a row each in 8 bits: 29 us,
  // with all eight waves on a tile 48; 14336 x 1024, 16 rows: 8.6 against 9.5).
  int ks = C::WAVES;
  const int64_t runs = ((int64_t)a.kdim * (TY == T_FP8 ? 1 : 2) + 255) / 256;
  while (ks > 1 && runs < 2 * ks && tiles * ks >= 2 * (int64_t)a.cus * C::WAVES) ks /= 2;
  const int64_t blocks = (tiles * ks + C::WAVES - 1) / C::WAVES;
  k_few<C><<<dim3((unsigned)(blocks < a.cus ? blocks : a.cus)), 64 * C::WAVES, C::LDS, st>>>(a, ks);
  return hipGetLastError();
}

// 16 token rows at a time also where groups average half as many: one of 17 to 32 rows then
// reads its weights twice, the second time from cache (512 rows in 64 groups of 2048 x 1024 in
// bf16: 54 us, 32 at a time 72; 256 rows in 16 groups of 4096 x 2048: 68 and 60).
template <int TY, bool GATE>
hipError_t launch_few(const GemmArgs& a, hipStream_t st) {
  const int64_t groups = a.E < a.T ? a.E : a.T;
  return a.most <= 16 || a.T <= 8 * groups ? launch_few_tt<TY, 1, GATE>(a, st) : launch_few_tt<TY, 2, GATE>(a, st);
}

// Groups of few rows go to the few-row kernel, the others to the tiled one.  Without the
// offsets (device memory) the host knows only T and E, so it launches whichever can have work;
// a group that is not a kernel's has no tiles there.
constexpr int kFew = 16;

int device_cus() {
  static thread_local int known_dev = -1, cus = 0;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  if (dev != known_dev) {
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 1) return 256;
    known_dev = dev;
  }
  return cus;
}

template <int TY, int LAY, int TO, int GATE = 0>
hipError_t run_gemm(GemmArgs a, hipStream_t st) {
  a.least = 1;
  a.most = 0x7FFFFFFF;
  a.cus = device_cus();
  // The most tiles there can be: exact for dW and without offsets, else each group may add
  // one row tile.
  const int64_t groups = a.E < a.T ? a.E : a.T;
  auto tiles = [&](int64_t b) {
    const int64_t bn = GATE ? b / 2 : b, tn = ((int64_t)a.cols + bn - 1) / bn;
    if (LAY == L_TN) return (int64_t)a.E * (((int64_t)a.rows + b - 1) / b) * tn;
    return (((int64_t)a.T + b - 1) / b + groups - 1) * tn;
  };
  if (LAY == L_NT) {
    // Few rows: 16 to a group on average, or 32 in all, or so little work that tiles would
    // leave most compute units idle (4096 x 4096 in 8 bits: 64 rows 10 us against 23, 128 rows
    // 15 against 23; 14336 x 4096, 64 rows: 27 against 25).  With at most 128 rows in all a
    // group of many rows goes there too, 16 rows at a time, which saves the second launch (8 bits,
    // 128 rows in 8 groups of 4096 x 2048: 25 us against 36; all of them in one group of
    // 14336 x 4096: 56 against 37).  With more rows the limit stays at 32 (1024 rows in 64
    // groups of 4096 x 2048: 124 us, with a limit of 64 141).
    const bool little = (a.T + 32 * groups - 1) / (32 * groups) * tiles(128) * 2 <= a.cus;
    if (little || a.T <= kFew * groups || a.T <= 2 * kFew) {
      const int limit = little || a.T <= 8 * kFew ? 8 * kFew : 2 * kFew;
      // (without offsets the one group's rows are known: it is either kernel's alone)
      if (a.offsets != nullptr || a.T <= limit) {
        GemmArgs f = a;
        f.most = a.T < limit ? a.T : limit;
        const hipError_t e = launch_few<TY, (GATE > 0)>(f, st);
        if (e != hipSuccess || a.T <= limit) return e;
        a.least = limit + 1;
      }
    }
  }
  const int64_t units = tiles(kBig);
  // Small tiles.  A block alone on its compute unit waits for each stage's chain of barrier, LDS
  // reads and products, so where there is one block to a unit at most, sets of waves take the
  // stages in turn (1024 x 1024 outputs, contraction 4096: 64 x 64 tiles with 1, 2, 4 sets 29, 20
  // and 19 us in bf16, 19, 13.5 and 12.6 in 8 bits; 2048^3 in 128 x 128 tiles with 1, 2 sets 25.1
  // and 23.4).  Else two blocks per unit with two stages in flight each.  The 64 x 64 tiles as
  // long as all of them are at work at once (8 bits, 512 of them, contraction 4096: 19 us, 128 x
  // 128 22; 768 of them 31 and 23).
  using Small4 = Tile<TY, LAY, 128, 128, 64, 64, 4, 1, GATE>;
  using SmallK = Tile<TY, LAY, 128, 128, 64, 64, 2, 2, GATE>;
  using Small2 = Tile<TY, LAY, 128, 128, 64, 64, 2, 1, GATE>;
  // They alone: where large tiles would not fill a round, or be mostly empty (groups that
  // average less than a large tile's rows).  The large tiles' blocks are persistent, so they also
  // take what would be more small tiles than a grid holds (thousands of groups of 2^19 outputs).
  const int64_t n = tiles(128);
  if (units * 256 < (int64_t)kTailShare * a.cus || (LAY != L_TN && (int64_t)a.T < kBig * groups && n <= kMaxBlocks)) {
    a.direct = 1;
    const int64_t n64 = tiles(64);
    if (n64 <= a.cus) return launch_gemm<Tile<TY, LAY, 64, 64, 32, 64, 2, 4, GATE>, TO>(a, n64, st);
    if (n64 <= 2 * a.cus) return launch_gemm<Tile<TY, LAY, 64, 64, 32, 64, 2, 2, GATE>, TO>(a, n64, st);
    return n <= a.cus ? launch_gemm<SmallK, TO>(a, n, st) : launch_gemm<Small2, TO>(a, n, st);
  }
  const hipError_t e =
      launch_gemm<Tile<TY, LAY, kBig, kBig, 64, 128, 2, 1, GATE>, TO>(a, units < a.cus ? units : a.cus, st);
  if (e != hipSuccess) return e;
  // What is left over, less than whole_rounds' share of one.  Up to a quarter of a round is one small
  // tile per compute unit at most, and all units load at once there: four stages in flight beat
  // two (dX of 8192 x 4096 x 2048 in 8 groups 158 us against 165) and two sets of waves (166
  // against 170).  More is two blocks to a unit (half a round, 4096 tokens, contraction 2048: 95 us
  // against 105 with four stages and so one block).  Where only the device knows how much is left,
  // both are launched and one of them finds no work (4.5 to 4.8 us).
  const bool sure = LAY == L_TN || a.offsets == nullptr;
  const int64_t most = ((int64_t)(LAY == L_TN ? kTailShareDw : kTailShare) * a.cus - 1) / 256;
  const int64_t quarter = a.cus / 4, left = units % a.cus;
  if (sure && left > most) return hipSuccess;
  const int64_t rest = sure ? left : units < most ? units : most;
  if (rest > 0 && (!sure || rest <= quarter)) {
    a.rest_least = 1;
    a.rest_most = (int)quarter;
    const hipError_t e4 = launch_gemm<Small4, TO>(a, 4 * (rest < quarter ? rest : quarter), st);
    if (e4 != hipSuccess) return e4;
  }
  if (rest <= quarter) return hipSuccess;
  a.rest_least = (int)quarter + 1;
  a.rest_most = (int)most;
  return launch_gemm<Small2, TO>(a, 4 * rest, st);
}

}  // namespace

}  // namespace intlora
