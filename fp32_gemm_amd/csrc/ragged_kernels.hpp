// ragged_kernels.hpp -- the matrix product kernel behind gemm_grouped,
// gemm_grouped_wgrad and igemm.
//
// One template covers three forms of one tile product, D = A * B over a
// reduction of `len` steps, for 32-bit and 16-bit floats and 8-bit integers:
//   kFormNT  A rows are tokens, B rows are output columns; both are contiguous
//            along the reduction (Y = X * W^T, W stored N x K).
//   kFormNN  B rows are reduction steps (Y = X * W, W stored K x N).
//   kFormTN  both operands' rows are reduction steps (dW = X^T * dY).
// The rows of the first two forms, and the reduction of the third, are the
// rows offsets[e] .. offsets[e+1] of group e; the offsets stay on the device.
//
// Everything is laid out in bytes, so that the types share one layout: a slice
// of the reduction is 128 (or 64) bytes of every row that is contiguous along
// it (32 floats, 64 halves, 128 integers), and a lane's matrix-core operand is
// 16 of those bytes.
//
// What bounds it: many rows, the matrix cores and the power they draw (bf16
// 8192 x 8192 x 8192 with transposed weights 808 us, 1362 TFLOP/s at about
// 1.5 GHz; int8 442 us, 2490 TOP/s); few rows, reading the weights (32 experts,
// 16 rows, 2048 to 1024: 10.0 us, 5.2 TB/s); small products, a launch and the
// latencies of the offsets, the first slice and the results (4 us).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ragged_order.hpp"

namespace fp32gemm {

enum Elem { kElemF32 = 0, kElemBF16 = 1, kElemF16 = 2, kElemI8 = 3 };
enum Form { kFormNT = 0, kFormNN = 1, kFormTN = 2 };

constexpr int elem_size(int t) { return t == kElemF32 ? 4 : t == kElemI8 ? 1 : 2; }

struct RaggedArgs {
  const char* A;
  const char* B;
  char* C;
  const int* offsets;     // groups + 1 row numbers; null: one group of all rows
  const float* scale_a;   // 8-bit products: a scale per row,
  const float* scale_b;   // a scale per group and column,
  const float* bias;      // and a bias per group and column, or null
  long long lda, ldb;     // bytes
  long long ldc;          // elements
  long long stride_b;     // bytes between the groups of B
  long long stride_c;     // elements between the groups of C (kFormTN)
  int groups, rows;       // rows: of A (and of B in kFormTN)
  int M, N, K;            // kFormTN: M x N outputs a group; else N columns, K steps
  int out;                // Elem of C
  int longest_first;      // kFormTN: take the groups by falling length
  float alpha, beta;
};

// A tile of one workgroup: BM x BN outputs, WAVES_M x WAVES_N waves that share
// each slice, WAVES_K such groups of waves that take every WAVES_K-th slice
// and add up at the end, S slices of SL bytes in the ring, MF x MF matrix-core blocks,
// registers for PER_SIMD waves on a SIMD.
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int WAVES_K_, int S_, int SL_, int MF_, int PER_SIMD_>
struct RaggedTile {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_,
                       WAVES_K = WAVES_K_, S = S_, SL = SL_, MF = MF_, PER_SIMD = PER_SIMD_;
  static constexpr int WAVES = WAVES_M * WAVES_N;          // waves of one slice
  static constexpr int NT = WAVES * WAVES_K * 64;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  static constexpr int FM = WM / MF, FN = WN / MF;         // blocks of a wave
  static constexpr int STAGE = (BM + BN) * SL;             // bytes of a slice
  static constexpr int RING = STAGE * S * WAVES_K;
  static constexpr int SUMS = (WAVES_K - 1) * BM * BN * 4; // partial sums at the end
  static constexpr int OUT = WAVES * MF * (WN + 1) * 4;    // results on their way to memory
  static constexpr int LDS = RING > SUMS + OUT ? RING : SUMS + OUT;
  static_assert(BM * SL % (1024 * WAVES) == 0 && BN * SL % (1024 * WAVES) == 0, "whole load instructions a wave");
  static_assert(WM % MF == 0 && WN % MF == 0 && LDS <= 160 * 1024, "tile");
};

typedef float rf4 __attribute__((ext_vector_type(4)));
typedef float rf16 __attribute__((ext_vector_type(16)));
typedef int ri4 __attribute__((ext_vector_type(4)));
typedef int ri2 __attribute__((ext_vector_type(2)));
typedef unsigned ru4 __attribute__((ext_vector_type(4)));
typedef unsigned ru2 __attribute__((ext_vector_type(2)));
typedef int ri16 __attribute__((ext_vector_type(16)));
typedef short rs4 __attribute__((ext_vector_type(4)));
typedef __bf16 rb8 __attribute__((ext_vector_type(8)));
typedef _Float16 rh8 __attribute__((ext_vector_type(8)));
typedef __bf16 rb4 __attribute__((ext_vector_type(4)));
typedef _Float16 rh4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char* rlds_t;

// Buffer resources are at most this long; a masked element's offset lies past
// the end of every one of them, so it is not fetched and reads as zero.
constexpr int kRaggedMasked = 0x7FFFFF00;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t ragged_rsrc(const char* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), static_cast<short>(0), bytes,
                                           0x00020000);
}

template <int ELEM, int MF> struct RaggedAcc { using type = rf16; };
template <> struct RaggedAcc<kElemI8, 32> { using type = ri16; };
template <> struct RaggedAcc<kElemF32, 16> { using type = rf4; };
template <> struct RaggedAcc<kElemBF16, 16> { using type = rf4; };
template <> struct RaggedAcc<kElemF16, 16> { using type = rf4; };
template <> struct RaggedAcc<kElemI8, 16> { using type = ri4; };

// acc += b * a on one block: 32 bytes of the reduction with 32 x 32 blocks, 64
// with 16 x 16 ones.  B comes first, so that a lane's results are neighbouring
// columns of one row of C and leave in wide stores.  Floats take four
// instructions; step j multiplies element j of every lane's four, the same
// permutation of the reduction in both operands.
template <int ELEM, int MF, class Acc>
__device__ __forceinline__ void ragged_mma(Acc& acc, const ri4& b, const ri4& a) {
  if constexpr (ELEM == kElemI8) {
    if constexpr (MF == 32) acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, acc, 0, 0, 0);
    else acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, acc, 0, 0, 0);
  } else if constexpr (ELEM == kElemBF16) {
    const rb8 x = __builtin_bit_cast(rb8, b), y = __builtin_bit_cast(rb8, a);
    if constexpr (MF == 32) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, acc, 0, 0, 0);
    else acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, acc, 0, 0, 0);
  } else if constexpr (ELEM == kElemF16) {
    const rh8 x = __builtin_bit_cast(rh8, b), y = __builtin_bit_cast(rh8, a);
    if constexpr (MF == 32) acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, y, acc, 0, 0, 0);
    else acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, acc, 0, 0, 0);
  } else {
    const rf4 x = __builtin_bit_cast(rf4, b), y = __builtin_bit_cast(rf4, a);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (MF == 32) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(x[j], y[j], acc, 0, 0, 0);
      else acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[j], y[j], acc, 0, 0, 0);
    }
  }
}

// ---------------------------------------------------------------------------
// Where a slice of one operand lies in LDS.  R: the tile's rows (ALONG: rows
// are contiguous along the reduction) or columns (rows are reduction steps).
//
// The banks are a sweep of 256 bytes, which a cycle of reads covers: sixteen
// lanes of 16 bytes, 32 of 8 or all 64 of 4.
// ALONG: row r is 128 bytes, its 16-byte piece c at place c ^ (r / 2 & 7): the
// lanes of a fragment read take the same piece of consecutive rows, two of
// which share a sweep.
// Otherwise: reduction step k is a row of R elements.  Halves are read through
// the transposing LDS read: sixteen lanes take 4 steps x 32 bytes, two such
// groups a cycle, either 32 bytes (MF 32) or 8 steps (MF 16) apart; the pieces
// of a step move by 64 bytes for each of the 4 steps and by 32 for the 8.
// Floats are read one by one, steps 4 (MF 32) or 4, 8 and 12 (MF 16) at once,
// which move by 128 and 64 bytes.
template <int ELEM, int R, bool ALONG, int SL>
struct RaggedSlice {
  static constexpr int ES = elem_size(ELEM);
  static constexpr int STEPS = SL / ES;                  // reduction steps of a slice
  static constexpr int ROW = ALONG ? SL : R * ES;        // bytes of a row in LDS
  static constexpr int PIECES = ROW / 16;
  static constexpr int ROWS_PER_LOAD = 1024 / ROW;       // a wave's load fills 1 KiB
  static __device__ __forceinline__ int swizzle(int row) {
    if constexpr (ALONG) return SL == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
    else if constexpr (ES == 2 && ROW >= 256) return (row & 3) << 2 | (row & 8) >> 2;
    else if constexpr (ES == 2) return ((row & 2) << 1 | (row & 8) >> 2) & (PIECES - 1);
    else return ((row & 4) << 1 | (row & 8) >> 1) & (PIECES - 1);
  }
  // Row and piece that lane `lane` of load instruction `i` brings.
  static __device__ __forceinline__ int load_row(int i, int lane) {
    return i * ROWS_PER_LOAD + lane / PIECES;
  }
  static __device__ __forceinline__ int load_piece(int i, int lane) {
    return (lane % PIECES) ^ swizzle(load_row(i, lane));
  }
};

// Loads of one operand's slices by one wave, from memory straight to LDS, 16
// bytes a lane.  The pieces may start at any byte; a piece that starts in a
// row's valid part may run past it by up to 15 bytes, which is still inside
// the operand as long as a later row of at least 16 bytes follows.  Where none
// does (the last slice, or rows shorter than 16 bytes), and where the part past
// the end has to read as zero (the end of a reduction), `fetch` and `put` bring
// the valid bytes and nothing else.
template <int ELEM, int R, bool ALONG, int SL, int WAVES>
struct RaggedLoader {
  using L = RaggedSlice<ELEM, R, ALONG, SL>;
  static constexpr int NI = R * SL / 1024 / WAVES;  // load instructions a wave
  const char* base;  // of the next slice
  long long step;    // bytes to the next slice
  int off[NI];       // this lane's bytes past the base, or kRaggedMasked
  int first;         // the wave's first load instruction
  int valid;         // ALONG: the tile's valid rows; else the valid bytes of a step's row
  int ld;

  __device__ __forceinline__ void init(const char* p, long long ld_bytes, long long step_bytes,
                                       int valid_, int wave, int lane) {
    base = p;
    step = step_bytes;
    ld = static_cast<int>(ld_bytes);
    first = wave * NI;
    valid = valid_;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int row = L::load_row(first + j, lane), c = L::load_piece(first + j, lane) * 16;
      off[j] = (ALONG ? row < valid : c < valid) ? row * ld + c : kRaggedMasked;
    }
  }

  // Sends the next slice to `stage` (this operand's part of a ring stage).
  // Past the reduction's end (`more` false) nothing is fetched, but the
  // instructions are issued, so that every slice counts the same.
  __device__ __forceinline__ void send(rlds_t stage, bool more) {
    const auto r = ragged_rsrc(base, more ? kRaggedMasked : 0);
#pragma unroll
    for (int j = 0; j < NI; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          r, (__attribute__((address_space(3))) void*)(stage + (first + j) * 1024), 16, off[j], 0, 0, 0);
    base += step;
  }

  // Fetches the slice at `p`, of which `left` (bytes ALONG, else steps) exist,
  // into registers.  A piece with fewer than 16 valid bytes is loaded from the
  // 16 bytes that end with them, of which some lie among the `ahead` bytes of
  // the row before p, to be shifted down; `narrow` rows have no 16 bytes and
  // are put together byte by byte.  Masked buffer loads, not branches, keep all
  // of them in flight at once.
  struct Held {
    ri4 reg[NI];
    int back[NI];
  };
  __device__ __forceinline__ void fetch(Held& h, const char* p, int ahead, int left, bool narrow,
                                        int lane) const {
    const auto r = ragged_rsrc(p - ahead, kRaggedMasked);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int row = L::load_row(first + j, lane), c = L::load_piece(first + j, lane) * 16;
      const bool ok = ALONG ? row < valid : row < left;
      const int n = ok ? (ALONG ? left : valid) - c : 0;
      if (narrow) {
        const char* q = p + static_cast<long long>(row) * ld + c;
        unsigned __int128 v = 0;
        for (int b = 0; b < 16 && b < n; ++b)
          v |= static_cast<unsigned __int128>(static_cast<unsigned char>(q[b])) << (8 * b);
        h.reg[j] = __builtin_bit_cast(ri4, v);
        h.back[j] = 0;
      } else {
        h.back[j] = n > 0 && n < 16 ? 16 - n : 0;
        h.reg[j] = __builtin_bit_cast(
            ri4, __builtin_amdgcn_raw_buffer_load_b128(
                     r, n > 0 ? row * ld + ahead + c - h.back[j] : kRaggedMasked, 0, 0));
      }
    }
  }
  // Writes the fetched slice to `stage`.
  __device__ __forceinline__ void put(const Held& h, rlds_t stage, int lane) const {
#pragma unroll
    for (int j = 0; j < NI; ++j)
      *(__attribute__((address_space(3))) ri4*)(stage + (first + j) * 1024 + lane * 16) =
          __builtin_bit_cast(ri4, __builtin_bit_cast(unsigned __int128, h.reg[j]) >> (8 * h.back[j]));
  }
};

// The transposing read.  The restricted pointer tells the compiler that the
// loads to LDS in flight do not write what is read here, which the barrier's
// explicit wait sees to; without it every read would wait for all of them
// (grouped product f16 1000 x 1504 x 784 over 8: 24.6 us, with it 16.8).
typedef __attribute__((address_space(3))) rs4* lds_rs4_t;
__device__ __forceinline__ ri2 read_transposed(lds_rs4_t __restrict__ p) {
  return __builtin_bit_cast(ri2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}

// A lane's 16 operand bytes of a block whose first row or column is `at`, for
// step group `ks` of a slice.
template <int ELEM, int R, bool ALONG, int SL, int MF>
__device__ __forceinline__ ri4 ragged_frag(rlds_t stage, int at, int ks, int lane) {
  using L = RaggedSlice<ELEM, R, ALONG, SL>;
  constexpr int GROUPS = 64 / MF;  // 16-byte pieces of the reduction a block takes
  if constexpr (ALONG) {
    const int row = at + lane % MF;
    const int piece = (ks * GROUPS + lane / MF) ^ L::swizzle(lane % MF);
    return *(__attribute__((address_space(3))) ri4*)(stage + row * SL + piece * 16);
  } else if constexpr (L::ES == 2) {
    // Sixteen lanes read 4 steps x 16 columns (lane s: step s / 4, columns
    // 4 * (s % 4) ..) and each receives one column's four steps.
    const int g = lane / 16, s = lane % 16;
    const int col = at + (MF == 32 ? (g & 1) * 16 : 0) + 4 * (s % 4);
    const int k = ks * 8 * GROUPS + 8 * (MF == 32 ? g >> 1 : g) + s / 4;
    const int piece = (col / 8) ^ L::swizzle(k);
    rlds_t p = stage + k * L::ROW + piece * 16 + 8 * (s & 1);
    const ri2 lo = read_transposed((lds_rs4_t)p), hi = read_transposed((lds_rs4_t)(p + 4 * L::ROW));
    return ri4{lo[0], lo[1], hi[0], hi[1]};
  } else {
    ri4 v;
    const int col = at + lane % MF;
    const int k = ks * 4 * GROUPS + 4 * (lane / MF);
    const int piece = (col / 4) ^ L::swizzle(k);
    rlds_t p = stage + k * L::ROW + piece * 16 + 4 * (col & 3);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *(__attribute__((address_space(3))) int*)(p + j * L::ROW);
    return v;
  }
}

// Waits until at most N of the wave's loads are in flight and its LDS accesses
// are done, then meets the other waves (ALONE: each wave reads only what it
// loaded itself).  __syncthreads() would also wait for the N loads.
template <int N, bool ALONE>
__device__ __forceinline__ void ragged_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  if constexpr (!ALONE) __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
template <int ELEM, int FORM, class T>
__global__ __launch_bounds__(T::NT, T::PER_SIMD) void ragged_kernel(const RaggedArgs p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the stub alone and lacks the matrix builtins
  constexpr bool A_ALONG = FORM != kFormTN, B_ALONG = FORM == kFormNT;
  constexpr int ES = elem_size(ELEM), SL = T::SL, STEPS = SL / ES, MF = T::MF, S = T::S;
  constexpr int GROUPS = 64 / MF, KS = SL / 16 / GROUPS;  // step groups of a slice
  using Acc = typename RaggedAcc<ELEM, MF>::type;
  using LoadA = RaggedLoader<ELEM, T::BM, A_ALONG, SL, T::WAVES>;
  using LoadB = RaggedLoader<ELEM, T::BN, B_ALONG, SL, T::WAVES>;
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS];

  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = wave_all % T::WAVES, kgroup = wave_all / T::WAVES;
  const int tiles_n = (p.N + T::BN - 1) / T::BN;

  // The tile: its group, its window of A, B and C, and the reduction's length.
  int group, rows, len;
  long long row_c;
  const char *a, *b;
  int n0, m_bytes = 0;  // the tile's first column of B, and byte of a step's row of A
  const DeviceWave look{lane};
  const Groups groups{p.offsets, p.groups, p.rows};
  if constexpr (FORM == kFormTN) {
    const TileAt at =
        tile_of_group<T::BM>(look, groups, blockIdx.x, (p.M + T::BM - 1) / T::BM, tiles_n, p.longest_first);
    group = at.group;
    if (group < 0) return;
    const RowSpan s = groups.span(group);
    const int m0 = at.row * T::BM;
    m_bytes = m0 * ES;
    n0 = at.n * T::BN;
    rows = min(T::BM, p.M - m0);
    len = s.hi - s.lo;
    a = p.A + s.lo * p.lda + static_cast<long long>(m0) * ES;
    b = p.B + s.lo * p.ldb + static_cast<long long>(n0) * ES;
    row_c = m0;
  } else {
    const TileAt at = tile_of_rows<T::BM>(look, groups, blockIdx.x, tiles_n);
    group = at.group;
    n0 = at.n * T::BN;
    rows = min(T::BM, at.hi - at.row);
    if (group < 0) return;
    len = p.K;
    a = p.A + at.row * p.lda;
    b = p.B + group * p.stride_b + (B_ALONG ? n0 * p.ldb : static_cast<long long>(n0) * ES);
    row_c = at.row;
  }
  const int cols = min(T::BN, p.N - n0);

  // Slice 0 is the one that goes through registers, if there is one: what is
  // left of the reduction after whole slices, or the last whole slice where
  // rows that are steps end inside a piece.  The others follow in order; group
  // g of waves takes slices g, g + WAVES_K, ...
  const bool cross = (!A_ALONG && rows * ES % 16 != 0) || (!B_ALONG && cols * ES % 16 != 0);
  const int over = len % STEPS, head = over ? over : cross && len > 0 ? STEPS : 0;
  const int whole = (len - head) / STEPS, slices = whole + (head > 0);
  const int turns = (slices + T::WAVES_K - 1) / T::WAVES_K;
  const bool narrow_a = A_ALONG ? len * ES < 16 : p.M * ES < 16;
  const bool narrow_b = B_ALONG ? len * ES < 16 : p.N * ES < 16;
  LoadA la;
  LoadB lb;
  const long long sa = A_ALONG ? SL : STEPS * p.lda, sb = B_ALONG ? SL : STEPS * p.ldb;
  const int skip = kgroup - (head > 0);  // whole slices before this group's first (-1: starts at slice 0)
  la.init(a + skip * sa, p.lda, sa * T::WAVES_K, A_ALONG ? rows : rows * ES, wave, lane);
  lb.init(b + skip * sb, p.ldb, sb * T::WAVES_K, B_ALONG ? cols : cols * ES, wave, lane);
  int left_a = whole - skip, left_b = left_a;  // whole slices from the next on (and slice 0, of group 0)
  const rlds_t ring = (rlds_t)lds + kgroup * (T::STAGE * S);

  auto send_a = [&](int stage) {
    la.send(ring + stage * T::STAGE, left_a > 0);
    left_a -= T::WAVES_K;
  };
  auto send_b = [&](int stage) {
    lb.send(ring + stage * T::STAGE + T::BM * SL, left_b > 0);
    left_b -= T::WAVES_K;
  };

  Acc acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int j = 0; j < T::FN; ++j) acc[i][j] = Acc{};

  // The waves of a tile's rows take its blocks of MF rows in turn, so that in a
  // partly filled tile they have the same number of blocks to leave out.
  const int wave_m = wave / T::WAVES_N, bn = (wave % T::WAVES_N) * T::WN;
  constexpr int MSTEP = T::WAVES_M * MF;
  auto block_row = [&](int i) { return i * MSTEP + wave_m * MF; };

  // Scales and biases of 8-bit products are fetched ahead, from clamped places
  // where the tile ends: a lane's four columns, and a row of each block.
  constexpr int PIECES = T::WN / 4;  // of four columns
  const int cn = n0 + bn;            // the wave's first column
  const int c4 = lane % PIECES, n4 = cn + 4 * c4;
  const float* const sb_row = ELEM == kElemI8 ? p.scale_b + static_cast<long long>(group) * p.N : nullptr;
  const float* const bias_row =
      ELEM == kElemI8 && p.bias ? p.bias + static_cast<long long>(group) * p.N : nullptr;
  float sb4[4] = {}, bias4[4] = {}, scale_m[T::FM] = {};
  if constexpr (ELEM == kElemI8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sb4[i] = sb_row[min(n4 + i, p.N - 1)];
    if (bias_row)
#pragma unroll
      for (int i = 0; i < 4; ++i) bias4[i] = bias_row[min(n4 + i, p.N - 1)];
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
      scale_m[i] = p.scale_a[row_c + min(block_row(i) + lane % MF, rows - 1)];
  }

  auto run = [&](auto blocks) {
    constexpr int NF = decltype(blocks)::value;  // row blocks a wave multiplies
    constexpr bool ALONE = T::WAVES == 1;
    constexpr int NIA = LoadA::NI, NIB = LoadB::NI;
    ri4 fa[2][NF], fb[2][T::FN];
    auto read = [&](int half, rlds_t stage, int ks) {
#pragma unroll
      for (int i = 0; i < NF; ++i)
        fa[half][i] = ragged_frag<ELEM, T::BM, A_ALONG, SL, MF>(stage, block_row(i), ks, lane);
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
        fb[half][j] = ragged_frag<ELEM, T::BN, B_ALONG, SL, MF>(stage + T::BM * SL, bn + j * MF, ks, lane);
    };
    // Order within a step group: the next group's reads and the loads go
    // between the matrix instructions.
    auto schedule = [&](auto loads) {
      constexpr int NM = NF * T::FN * (ELEM == kElemF32 ? 4 : 1), NL = decltype(loads)::value;
      constexpr int RA = A_ALONG ? 1 : ES == 2 ? 2 : 4, RB = B_ALONG ? 1 : ES == 2 ? 2 : 4;
      constexpr int ND = NF * RA + T::FN * RB;
      // The loads write LDS, so they stay behind the reads: reads go in the
      // first part of the group, loads in the second.
      constexpr int DPART = NL ? (NM * ND + ND + NL - 1) / (ND + NL) : NM, LPART = NM - DPART;
      constexpr int DEACH = (ND + DPART - 1) / DPART, LEACH = LPART > 0 ? (NL + LPART - 1) / LPART : NL;
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (i * DEACH < ND) __builtin_amdgcn_sched_group_barrier(0x100, DEACH, 0);
        else if (NL > 0) __builtin_amdgcn_sched_group_barrier(0x020, LEACH, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    ragged_barrier<(S - 2) * (NIA + NIB) + NIA, ALONE>();
    read(0, ring, 0);
    int at = 0;
    // Step group ks of the slice in stage `at` is multiplied from one half of
    // the operand registers while the next one is read to the other half.
    auto step_group = [&](auto group) {
      constexpr int ks = decltype(group)::value, half = ks & 1;
      // The stage's last reads are done before the barrier, so behind it the
      // slice S turns on may take its place, and the next slice is there.
      if constexpr (ks == KS - 1) {
        ragged_barrier<(S - 2) * (NIA + NIB), ALONE>();
        __builtin_amdgcn_sched_barrier(0);
        read(0, ring + (at + 1 == S ? 0 : at + 1) * T::STAGE, 0);
        send_a(at);
      } else {
        read(1 - half, ring + at * T::STAGE, ks + 1);
        if constexpr (ks == 0) send_b(at == 0 ? S - 1 : at - 1);
      }
      // Dense bf16 8192 x 8192 x 8192 with transposed weights: 824 us without
      // the priority, 794 with it; with plain weights no better (897, 917).
      if constexpr (FORM == kFormNT) __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j) ragged_mma<ELEM, MF>(acc[i][j], fb[half][j], fa[half][i]);
      if constexpr (FORM == kFormNT) __builtin_amdgcn_s_setprio(0);
      schedule(std::integral_constant<int, (ks == KS - 1 ? NIA : ks == 0 ? NIB : 0)>{});
    };
    for (int t = 0; t < turns; ++t) {
      step_group(std::integral_constant<int, 0>{});
      step_group(std::integral_constant<int, 1>{});
      if constexpr (KS == 4) {
        step_group(std::integral_constant<int, 2>{});
        step_group(std::integral_constant<int, 3>{});
      }
      at = at + 1 == S ? 0 : at + 1;
    }
  };

  // A slice through registers: `left` steps of the reduction from step `done`.
  typename LoadA::Held ha;
  typename LoadB::Held hb;
  auto fetch = [&](int done, int left) {
    if constexpr (A_ALONG) la.fetch(ha, a + done * ES, done * ES, left * ES, narrow_a, lane);
    else la.fetch(ha, a + done * p.lda, m_bytes, left, narrow_a, lane);
    if constexpr (B_ALONG) lb.fetch(hb, b + done * ES, done * ES, left * ES, narrow_b, lane);
    else lb.fetch(hb, b + done * p.ldb, n0 * ES, left, narrow_b, lane);
  };
  auto put = [&] {
    la.put(ha, ring, lane);
    lb.put(hb, ring + T::BM * SL, lane);
  };

  // Rows of fewer than 16 bytes that are reduction steps: every slice goes
  // through registers.
  auto run_narrow = [&] {
    for (int t = 0; t < turns; ++t) {
      const int done = (t * T::WAVES_K + kgroup) * STEPS;
      fetch(done, min(STEPS, len - done));
      put();
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
          const ri4 fa = ragged_frag<ELEM, T::BM, A_ALONG, SL, MF>(ring, block_row(i), ks, lane);
#pragma unroll
          for (int j = 0; j < T::FN; ++j)
            ragged_mma<ELEM, MF>(
                acc[i][j], ragged_frag<ELEM, T::BN, B_ALONG, SL, MF>(ring + T::BM * SL, bn + j * MF, ks, lane), fa);
        }
      __syncthreads();
    }
  };

  if (FORM != kFormNT && ((!A_ALONG && narrow_a) || (!B_ALONG && narrow_b))) {
    if constexpr (FORM != kFormNT) run_narrow();
  } else {
    // The first S slices are sent ahead (the last one's B in the first group).
    const bool headed = head > 0 && kgroup == 0;
    if (headed) {
      fetch(len - head, head);  // first, for its loads to come back first
      la.base += la.step;
      lb.base += lb.step;
      left_a -= T::WAVES_K;
      left_b -= T::WAVES_K;
    } else {
      send_a(0);
      send_b(0);
    }
#pragma unroll
    for (int s = 1; s < S; ++s) {
      send_a(s);
      if (s < S - 1) send_b(s);
    }
    if (headed) put();
    if constexpr (FORM != kFormTN && T::BM == 256) {
      const int used = (rows + 63) / 64;  // quarters of the tile's rows that hold any
      if (used > 3) run(std::integral_constant<int, 4>{});
      else if (used == 3) run(std::integral_constant<int, 3>{});
      else if (used == 2) run(std::integral_constant<int, 2>{});
      else run(std::integral_constant<int, 1>{});
    } else {
      run(std::integral_constant<int, T::FM>{});
    }
  }
  // The slices past the end, which hold nothing, may still be on their way.
  ragged_barrier<0, false>();

  // Wave groups that took other slices hand over their sums, in a fixed order.
  constexpr int REGS = MF * MF / 64;
  if constexpr (T::WAVES_K > 1) {
    using V = decltype(acc[0][0][0] + acc[0][0][0]);
    __attribute__((address_space(3))) V* sums = (__attribute__((address_space(3))) V*)(rlds_t)lds;
    const int slot = wave * 64 + lane;
    constexpr int EACH = T::WAVES * 64;
    if (kgroup > 0) {
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
#pragma unroll
          for (int r = 0; r < REGS; ++r)
            sums[((((kgroup - 1) * T::FM + i) * T::FN + j) * REGS + r) * EACH + slot] = acc[i][j][r];
    }
    __syncthreads();
    if (kgroup > 0) return;
#pragma unroll
    for (int g = 0; g < T::WAVES_K - 1; ++g)
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
#pragma unroll
          for (int r = 0; r < REGS; ++r)
            acc[i][j][r] += sums[(((g * T::FM + i) * T::FN + j) * REGS + r) * EACH + slot];
  }

  // Results go through LDS, a block of rows at a time, so that the stores of a
  // wave cover whole lines: a lane holds four neighbouring columns of one row
  // in each group of four registers, 32 (MF 16: 16) rows a wave.
  const rlds_t ep = (rlds_t)lds + T::SUMS + wave * (MF * T::WN * 4 + MF * 4);
  const rlds_t ep_scale = ep + MF * T::WN * 4;
  typedef __attribute__((address_space(3))) ri4* lds4_t;
  typedef __attribute__((address_space(3))) float* lds1_t;
  const int osz = p.out == kElemF32 ? 4 : 2;
  char* const c_tile = p.C + (FORM == kFormTN ? group * p.stride_c * osz : 0) + row_c * p.ldc * osz;
  // Sums up to 2^31 are exact; the conversion to 32-bit floats rounds those
  // past 2^24 once, to half a unit in the last place.
  auto value = [&](int bits, float s, float sbc, float bias) {
    if constexpr (ELEM == kElemI8) return static_cast<float>(bits) * (s * sbc) + bias;
    else return __builtin_bit_cast(float, bits);
  };
  const bool four = n4 + 4 <= p.N;
  constexpr int EACH = 64 / PIECES, ITER = MF / EACH;  // rows of a store, stores of a block
  const int c_row = static_cast<int>(p.ldc) * osz;
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
    const int m0 = block_row(i);
    if (m0 >= rows) break;
    {
      const int row = lane % MF;
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
#pragma unroll
        for (int r = 0; r < REGS; r += 4) {
          const int piece = (j * MF + (MF == 32 ? 2 * r : 0)) / 4 + lane / MF;
          const decltype(__builtin_shufflevector(acc[i][j], acc[i][j], 0, 1, 2, 3)) v = {
              acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
          *(lds4_t)(ep + row * (T::WN * 4) + ((piece ^ (row & (PIECES - 1))) * 16)) =
              __builtin_bit_cast(ri4, v);
        }
      if constexpr (ELEM == kElemI8)
        if (lane < MF) *(lds1_t)(ep_scale + lane * 4) = scale_m[i];
    }
    __builtin_amdgcn_wave_barrier();
    ri4 w[ITER];
    float s[ITER];
    int off[ITER];  // of the lane's four results past the tile's start, masked where they are not whole
    const int row0 = m0 + lane / PIECES;
    auto take = [&](int it, ri4& v, float& scale) {
      const int row = it * EACH + lane / PIECES;
      v = *(lds4_t)(ep + row * (T::WN * 4) + ((c4 ^ (row & (PIECES - 1))) * 16));
      scale = ELEM == kElemI8 ? *(lds1_t)(ep_scale + row * 4) : 0.0f;
    };
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      take(it, w[it], s[it]);
      off[it] = four && row0 + it * EACH < rows ? (row0 + it * EACH) * c_row + n4 * osz : kRaggedMasked;
    }
    // Whole fours by masked buffer stores, which may start at any element.
    // Without branches, and with the reads of old values apart, no store waits
    // for the one before it (a 256 x 256 tile of floats: 15.5 thousand cycles
    // with branches, 9.4 so).
    auto emit = [&](auto zero) {
      using O = decltype(zero);
      typedef O Quad __attribute__((ext_vector_type(4)));
      const auto to = ragged_rsrc(c_tile, kRaggedMasked);
      auto store = [&](int it, const float (&v)[4]) {
        Quad q;
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = static_cast<O>(v[e]);
        if constexpr (sizeof(O) == 4)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(ru4, q), to, off[it], 0, 0);
        else
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(ru2, q), to, off[it], 0, 0);
      };
      if (ELEM != kElemI8 && p.beta != 0.0f) {
        Quad old[ITER];
#pragma unroll
        for (int it = 0; it < ITER; ++it)
          if constexpr (sizeof(O) == 4)
            old[it] = __builtin_bit_cast(Quad, __builtin_amdgcn_raw_buffer_load_b128(to, off[it], 0, 0));
          else
            old[it] = __builtin_bit_cast(Quad, __builtin_amdgcn_raw_buffer_load_b64(to, off[it], 0, 0));
#pragma unroll
        for (int it = 0; it < ITER; ++it) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = p.alpha * value(w[it][e], s[it], sb4[e], bias4[e]) + p.beta * static_cast<float>(old[it][e]);
          store(it, v);
        }
      } else {
#pragma unroll
        for (int it = 0; it < ITER; ++it) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = value(w[it][e], s[it], sb4[e], bias4[e]);
            if constexpr (ELEM != kElemI8) v[e] *= p.alpha;
          }
          store(it, v);
        }
      }
      // The one to three results in front of C's last column.
      if (!four && n4 < p.N)
        for (int it = 0; it < ITER && row0 + it * EACH < rows; ++it) {
          ri4 v;
          float scale;
          take(it, v, scale);
          O* const d = reinterpret_cast<O*>(c_tile + static_cast<long long>(row0 + it * EACH) * c_row) + n4;
#pragma unroll
          for (int e = 0; e < 3; ++e)
            if (n4 + e < p.N) {
              float x = value(v[e], scale, sb4[e], bias4[e]);
              if constexpr (ELEM != kElemI8) {
                x *= p.alpha;
                if (p.beta != 0.0f) x += p.beta * static_cast<float>(d[e]);
              }
              d[e] = static_cast<O>(x);
            }
        }
    };
    if (p.out == kElemF32) emit(float{});
    else if (p.out == kElemBF16) emit(__bf16{});
    else emit(_Float16{});
    __builtin_amdgcn_wave_barrier();
  }
#endif
}

// Launches return their own error: hipGetLastError() would also give, and
// clear, one that the program left from an earlier call of its own.
template <int ELEM, int FORM, class T>
hipError_t launch_ragged(const RaggedArgs& a, long long grid, hipStream_t stream) {
  RaggedArgs args = a;
  void* values[] = {&args};
  return hipLaunchKernel(reinterpret_cast<const void*>(&ragged_kernel<ELEM, FORM, T>),
                         dim3(static_cast<unsigned>(grid)), dim3(T::NT), values, 0, stream);
}

// The compiled tiles, by the names of RaggedShape.
//   kWide   eight waves and one workgroup a compute unit.  Weights or operands
//           whose rows are steps come in rows 4 KiB and more apart: shorter
//           slices, a deeper ring (bf16 16384 x 2048 x 4096 over 16: 310 us
//           with 2 slices of 128 bytes, 290 with 3 of 64; transposed weights
//           272 and 288).
//   kMid    two workgroups a compute unit.
//   kDeep   kMid with a ring of four for one workgroup a compute unit, where
//           there are not tiles for two (2048 x 2048 x 8192: 70 us and 86).
//   kSmall  three workgroups a compute unit; five, with rings of two, for
//           weight gradients, whose reductions are often short (bf16, 32
//           experts of 16 rows, 1024 x 1024: 35 us and 43 with rings of three;
//           bf16 products 1024 x 1024 x 8192 65 and 38, f32 4097 x 1024 x 2048
//           over 8 experts 187 and 159).
//   kThin, kSlim: few rows, a slice a wave, so that nobody waits for others.
template <int FORM>
using RaggedWide = std::conditional_t<FORM == kFormNT, RaggedTile<256, 256, 2, 4, 1, 2, 128, 32, 2>,
                                      RaggedTile<256, 256, 2, 4, 1, 3, 64, 32, 2>>;
using RaggedMid = RaggedTile<128, 128, 2, 4, 1, 2, 128, 32, 2>;
using RaggedDeep = RaggedTile<128, 128, 2, 4, 1, 4, 128, 32, 2>;
template <int FORM>
using RaggedSmall = std::conditional_t<FORM == kFormTN, RaggedTile<64, 64, 2, 2, 1, 2, 128, 32, 4>,
                                       RaggedTile<64, 64, 2, 2, 1, 3, 128, 32, 3>>;
using RaggedThin = RaggedTile<16, 32, 1, 1, 4, 2, 128, 16, 3>;
using RaggedSlim = RaggedTile<16, 16, 1, 1, 4, 4, 128, 16, 2>;

enum RaggedShape { kWide, kMid, kDeep, kSmall, kThin, kSlim, kShapes };
constexpr int kRaggedRows[kShapes] = {256, 128, 128, 64, RaggedThin::BM, 16};  // of a tile
constexpr int kRaggedCols[kShapes] = {256, 128, 128, 64, RaggedThin::BN, 16};
constexpr int kRaggedThreads[kShapes] = {512, 512, 512, 256, 256, 256};
static_assert(RaggedWide<kFormNT>::NT == 512 && RaggedMid::NT == 512 && RaggedDeep::NT == 512 &&
              RaggedSmall<kFormNT>::NT == 256 && RaggedThin::NT == 256 && RaggedSlim::NT == 256, "threads");

// The shapes that the plan may choose for a type and form, and no others, are
// compiled.  Where rows of W are steps, few columns are short pieces of many
// rows, and a weight gradient has no few rows.  32-bit products wait for the
// matrix cores, not for loads: there kDeep is never the cheaper of the two but
// for weight gradients.
constexpr bool ragged_compiled(int elem, int form, int shape) {
  return shape == kSlim   ? form == kFormNT
         : shape == kThin ? form != kFormTN
         : shape == kDeep ? elem != kElemF32 || form == kFormTN
                          : true;
}

template <int ELEM, int FORM, int SHAPE, class T>
bool launch_if(int shape, const RaggedArgs& a, long long grid, hipStream_t s, hipError_t& err) {
  if constexpr (ragged_compiled(ELEM, FORM, SHAPE)) {
    if (shape != SHAPE) return false;
    err = launch_ragged<ELEM, FORM, T>(a, grid, s);
    return true;
  } else {
    return false;
  }
}

template <int ELEM, int FORM>
hipError_t launch_shape(int shape, const RaggedArgs& a, long long grid, hipStream_t s) {
  hipError_t err = hipErrorInvalidValue;
  launch_if<ELEM, FORM, kWide, RaggedWide<FORM>>(shape, a, grid, s, err) ||
      launch_if<ELEM, FORM, kMid, RaggedMid>(shape, a, grid, s, err) ||
      launch_if<ELEM, FORM, kDeep, RaggedDeep>(shape, a, grid, s, err) ||
      launch_if<ELEM, FORM, kSmall, RaggedSmall<FORM>>(shape, a, grid, s, err) ||
      launch_if<ELEM, FORM, kThin, RaggedThin>(shape, a, grid, s, err) ||
      launch_if<ELEM, FORM, kSlim, RaggedSlim>(shape, a, grid, s, err);
  return err;
}

// Largest 2-byte or smaller element count a tile's rows may be apart: the byte
// offsets of 256 rows fit the 31 bits of a buffer offset.
constexpr long long kRaggedMaxLd = 1LL << 21;

hipError_t ragged_f32(int form, int shape, const RaggedArgs&, long long grid, hipStream_t);
hipError_t ragged_bf16(int form, int shape, const RaggedArgs&, long long grid, hipStream_t);
hipError_t ragged_f16(int form, int shape, const RaggedArgs&, long long grid, hipStream_t);
hipError_t ragged_i8(int form, int shape, const RaggedArgs&, long long grid, hipStream_t);

}  // namespace fp32gemm
