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
// of the reduction is 128 bytes of every row that is contiguous along it (32
// floats, 64 halves, 128 integers), and a lane's matrix-core operand is 16 of
// those bytes.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

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
  int c_vec;              // C's rows allow stores of four elements
  float alpha, beta;
};

// A tile of one workgroup: BM x BN outputs, WAVES_M x WAVES_N waves that share
// each slice, WAVES_K such groups of waves that take every WAVES_K-th slice
// and add up at the end, S slices in the ring, MF x MF matrix-core blocks.
// DIRECT: slices go from memory to LDS without passing registers, which takes
// operands whose rows are whole, aligned 16-byte pieces.
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int WAVES_K_, int S_, int MF_, bool DIRECT_>
struct RaggedTile {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_,
                       WAVES_K = WAVES_K_, S = DIRECT_ ? S_ : 2, MF = MF_;
  static constexpr bool DIRECT = DIRECT_;
  static constexpr int WAVES = WAVES_M * WAVES_N;          // waves of one slice
  static constexpr int NT = WAVES * WAVES_K * 64;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  static constexpr int FM = WM / MF, FN = WN / MF;         // blocks of a wave
  static constexpr int STAGE = (BM + BN) * 128;            // bytes of a slice
  static constexpr int RING = STAGE * S * WAVES_K;
  static constexpr int SUMS = (WAVES_K - 1) * BM * BN * 4; // partial sums at the end
  static constexpr int LDS = RING > SUMS ? RING : SUMS;
  static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "whole load instructions a wave");
  static_assert(WM % MF == 0 && WN % MF == 0 && LDS <= 160 * 1024, "tile");
};

typedef float rf4 __attribute__((ext_vector_type(4)));
typedef float rf16 __attribute__((ext_vector_type(16)));
typedef int ri4 __attribute__((ext_vector_type(4)));
typedef int ri2 __attribute__((ext_vector_type(2)));
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
// ALONG: row r is 128 bytes, its 16-byte piece c at place c ^ (r & 7).  The
// lanes of a fragment read take the same piece of consecutive rows, which the
// exclusive or spreads over all banks.
// Otherwise: reduction step k is a row of R elements.  Halves are read through
// the transposing LDS read: sixteen lanes take 4 steps x 32 bytes, so the
// pieces of step k move by (k & 3) pairs to keep those four rows on different
// banks; floats are read one by one, the two halves of a wave 4 steps apart,
// which moves by 128 bytes.
template <int ELEM, int R, bool ALONG>
struct RaggedSlice {
  static constexpr int ES = elem_size(ELEM);
  static constexpr int STEPS = 128 / ES;                 // reduction steps of a slice
  static constexpr int ROW = ALONG ? 128 : R * ES;       // bytes of a row in LDS
  static constexpr int PIECES = ROW / 16;
  static constexpr int ROWS_PER_LOAD = 1024 / ROW;       // a wave's load fills 1 KiB
  static __device__ __forceinline__ int swizzle(int row) {
    if constexpr (ALONG) return row & 7;
    else if constexpr (ES == 2) return ((row & 3) << 1) & (PIECES - 1);
    else return ((row & 4) << 1) & (PIECES - 1);
  }
  // Row and piece that lane `lane` of load instruction `i` brings.
  static __device__ __forceinline__ int load_row(int i, int lane) {
    return i * ROWS_PER_LOAD + lane / PIECES;
  }
  static __device__ __forceinline__ int load_piece(int i, int lane) {
    return (lane % PIECES) ^ swizzle(load_row(i, lane));
  }
};

// Loads of one operand's slices by one wave.  `rows_` and `cols_bytes` bound
// the operand's window: ALONG, the valid rows of the tile (the reduction's
// length comes with each slice); otherwise the valid bytes of a step's row.
template <int ELEM, int R, bool ALONG, int WAVES, bool DIRECT>
struct RaggedLoader {
  using L = RaggedSlice<ELEM, R, ALONG>;
  static constexpr int NI = R / 8 / WAVES;  // load instructions a wave: R * 128 / 1024 / WAVES
  static constexpr int LIVE = DIRECT ? 1 : NI;
  const char* base;  // of the next slice
  long long step;    // bytes to the next slice
  int off[NI];       // this lane's bytes past the base, or kRaggedMasked
  int first;         // the wave's first load instruction
  int lane_;
  int bound;         // ALONG: bytes from the base to the last valid row's start; else a row's valid bytes
  int ld;
  ri4 reg[LIVE];
  int more[LIVE];

  __device__ __forceinline__ void init(const char* p, long long ld_bytes, long long step_bytes,
                                       int valid, int wave, int lane) {
    base = p;
    step = step_bytes;
    ld = static_cast<int>(ld_bytes);
    first = wave * NI;
    lane_ = lane;
    bound = ALONG ? (valid - 1) * ld : valid;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int row = L::load_row(first + j, lane), c = L::load_piece(first + j, lane) * 16;
      const bool ok = ALONG ? row < valid : c < valid;
      off[j] = ok ? row * ld + c : kRaggedMasked;
    }
  }

  // Masks what lies at or past the reduction's end in this and all later
  // slices; `left` counts bytes (ALONG) or steps.
  __device__ __forceinline__ void cut(int left) {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int at = ALONG ? L::load_piece(first + j, lane_) * 16 : L::load_row(first + j, lane_);
      if (at >= left) off[j] = kRaggedMasked;
    }
  }

  // Sends the next slice to `stage` (this operand's part of a ring stage).
  __device__ __forceinline__ void send(rlds_t stage) {
    const auto r = ragged_rsrc(base, kRaggedMasked);
#pragma unroll
    for (int j = 0; j < NI; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          r, (__attribute__((address_space(3))) void*)(stage + (first + j) * 1024), 16, off[j], 0, 0, 0);
    base += step;
  }

  // Without direct loads: fetch the next slice into registers.  Pieces of rows
  // that start at any byte are covered by whole dwords and shifted into place.
  // The resource ends with the dword that holds the window's last byte, so no
  // load leaves the dwords the operand itself lies in.
  __device__ __forceinline__ void fetch(int left) {
    const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(base) & 3);
    const int end = ALONG ? bound + (left < 128 ? left : 128)
                          : ((left < L::STEPS ? left : L::STEPS) - 1) * ld + bound;
    const auto r = ragged_rsrc(base - skew, left > 0 ? (end + skew + 3) & ~3 : 0);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int at = off[j] + skew;
      reg[j] = __builtin_bit_cast(ri4, __builtin_amdgcn_raw_buffer_load_b128(r, at & ~3, 0, 0));
      if constexpr (L::ES < 4)
        more[j] = __builtin_amdgcn_raw_buffer_load_b32(r, (at & 3) ? (at & ~3) + 16 : kRaggedMasked, 0, 0);
    }
  }

  // Writes the fetched slice to `stage` and moves on.
  __device__ __forceinline__ void put(rlds_t stage, int left) {
    const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(base) & 3);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      ri4 v = reg[j];
      if constexpr (L::ES < 4) {
        const unsigned s = static_cast<unsigned>(off[j] + skew) & 3u;
        v[0] = __builtin_amdgcn_alignbyte(reg[j][1], reg[j][0], s);
        v[1] = __builtin_amdgcn_alignbyte(reg[j][2], reg[j][1], s);
        v[2] = __builtin_amdgcn_alignbyte(reg[j][3], reg[j][2], s);
        v[3] = __builtin_amdgcn_alignbyte(more[j], reg[j][3], s);
      }
      if constexpr (ALONG) {
        // Bytes past the reduction's end belong to the next row.
        if (left < 128) {
          const int valid = left - L::load_piece(first + j, lane_) * 16;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const int b = valid - 4 * d;
            v[d] = b >= 4 ? v[d] : b <= 0 ? 0 : v[d] & ((1 << (8 * b)) - 1);
          }
        }
      }
      *(__attribute__((address_space(3))) ri4*)(stage + (first + j) * 1024 + lane_ * 16) = v;
    }
    base += step;
  }
};

// A lane's 16 operand bytes of block `f` (of the wave's rows or columns that
// start at `at`) for step group `ks` of a slice.
template <int ELEM, int R, bool ALONG, int MF>
__device__ __forceinline__ ri4 ragged_frag(rlds_t stage, int at, int f, int ks, int lane) {
  using L = RaggedSlice<ELEM, R, ALONG>;
  constexpr int GROUPS = 64 / MF;  // 16-byte pieces of the reduction a block takes
  if constexpr (ALONG) {
    const int row = at + f * MF + lane % MF;
    const int piece = (ks * GROUPS + lane / MF) ^ (lane & 7);
    return *(__attribute__((address_space(3))) ri4*)(stage + row * 128 + piece * 16);
  } else if constexpr (L::ES == 2) {
    // Sixteen lanes read 4 steps x 16 columns (lane s: step s / 4, columns
    // 4 * (s % 4) ..) and each receives one column's four steps.
    const int g = lane / 16, s = lane % 16;
    const int col = at + f * MF + (MF == 32 ? (g & 1) * 16 : 0) + 4 * (s % 4);
    const int k = ks * 8 * GROUPS + 8 * (MF == 32 ? g >> 1 : g) + s / 4;
    const int piece = (col / 8) ^ L::swizzle(s / 4);
    rlds_t p = stage + k * L::ROW + piece * 16 + 8 * (s & 1);
    typedef __attribute__((address_space(3))) rs4* tr_t;
    const ri2 lo = __builtin_bit_cast(ri2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_t)p));
    const ri2 hi = __builtin_bit_cast(ri2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_t)(p + 4 * L::ROW)));
    return ri4{lo[0], lo[1], hi[0], hi[1]};
  } else {
    ri4 v;
    const int col = at + f * MF + lane % MF;
    const int k = ks * 4 * GROUPS + 4 * (lane / MF);
    const int piece = (col / 4) ^ L::swizzle(k);
    rlds_t p = stage + k * L::ROW + piece * 16 + 4 * (col & 3);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *(__attribute__((address_space(3))) int*)(p + j * L::ROW);
    return v;
  }
}

// Waits until at most N of the wave's loads are in flight and its LDS reads
// are done, then meets the other waves (ALONE: each wave reads only what it
// loaded itself).  __syncthreads() would also wait for the N loads.
template <int N, bool ALONE>
__device__ __forceinline__ void ragged_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  if constexpr (!ALONE) __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// Rows of group e, whatever the offsets hold: within 0 .. rows, never negative.
struct RowSpan { int lo, hi; };
__device__ __forceinline__ RowSpan group_rows(const RaggedArgs& p, int e) {
  if (p.offsets == nullptr) return {0, p.rows};
  const int lo = min(max(p.offsets[e], 0), p.rows);
  return {lo, min(max(p.offsets[e + 1], lo), p.rows)};
}

__device__ __forceinline__ int wave_sum_below(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Row tiles of all groups, and the group and row tile of tile `t`.
template <int BM>
__device__ __forceinline__ int count_tiles(const RaggedArgs& p, int lane) {
  if (p.offsets == nullptr) return (p.rows + BM - 1) / BM;
  int n = 0;
  for (int e0 = 0; e0 < p.groups; e0 += 64) {
    if (e0 + lane < p.groups) {
      const RowSpan s = group_rows(p, e0 + lane);
      n += (s.hi - s.lo + BM - 1) / BM;
    }
  }
  return __builtin_amdgcn_readlane(wave_sum_below(n, lane), 63);
}

struct TileAt { int group, tile; };
template <int BM>
__device__ __forceinline__ TileAt find_tile(const RaggedArgs& p, int t, int lane) {
  if (p.offsets == nullptr) return {0, t};
  int before = 0;
  for (int e0 = 0; e0 < p.groups; e0 += 64) {
    int n = 0;
    if (e0 + lane < p.groups) {
      const RowSpan s = group_rows(p, e0 + lane);
      n = (s.hi - s.lo + BM - 1) / BM;
    }
    const int upto = before + wave_sum_below(n, lane);
    const unsigned long long hit = __ballot(upto > t);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      return {e0 + l, t - __builtin_amdgcn_readlane(upto - n, l)};
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return {-1, 0};
}

// Consecutive workgroups run on the eight dies in turn, each with its own L2:
// die x takes the x-th run of consecutive tiles.  Returns -1 past the last.
__device__ __forceinline__ int die_order(int w, int tiles) {
  const int x = w & 7, i = w >> 3, q = tiles >> 3, r = tiles & 7;
  return i < q + (x < r) ? x * q + min(x, r) + i : -1;
}

// Within a run, tiles go down kBand row tiles before the next column, so that
// tiles in flight on a die share operand rows and columns in its L2.
constexpr int kBand = 4;
struct TileRow { int m, n; };
__device__ __forceinline__ TileRow band_order(int id, int tm, int tn) {
  const int band = id / (kBand * tn), first = band * kBand, rows = min(kBand, tm - first);
  const int in = id - first * tn;
  return {first + in % rows, in / rows};
}

// ---------------------------------------------------------------------------
// Four neighbouring outputs of row r from column c.
template <int ELEM, class V4>
__device__ __forceinline__ void ragged_store(const RaggedArgs& p, long long row, int group, int c,
                                             const V4& acc, float sa) {
  if (c >= p.N) return;
  float v[4];
  const bool whole = p.c_vec && c + 4 <= p.N;
  if constexpr (ELEM == kElemI8) {
    // Sums up to 2^31 are exact; the conversion to 32-bit floats rounds those
    // past 2^24 once, to half a unit in the last place.
    const float* sb = p.scale_b + static_cast<long long>(group) * p.N + c;
    const float* bias = p.bias ? p.bias + static_cast<long long>(group) * p.N + c : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < p.N) v[i] = static_cast<float>(acc[i]) * (sa * sb[i]) + (bias ? bias[i] : 0.0f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = p.alpha * acc[i];
  }
  const long long at = row * p.ldc + c;
  if (p.out == kElemF32) {
    float* d = reinterpret_cast<float*>(p.C) + at;
    if (whole) {
      if (ELEM != kElemI8 && p.beta != 0.0f) {
        const rf4 o = *reinterpret_cast<const rf4*>(d);
        for (int i = 0; i < 4; ++i) v[i] += p.beta * o[i];
      }
      *reinterpret_cast<rf4*>(d) = rf4{v[0], v[1], v[2], v[3]};
    } else {
      for (int i = 0; i < 4; ++i)
        if (c + i < p.N) d[i] = ELEM != kElemI8 && p.beta != 0.0f ? v[i] + p.beta * d[i] : v[i];
    }
  } else if (p.out == kElemBF16) {
    __bf16* d = reinterpret_cast<__bf16*>(p.C) + at;
    if (whole) {
      if (ELEM != kElemI8 && p.beta != 0.0f) {
        const rb4 o = *reinterpret_cast<const rb4*>(d);
        for (int i = 0; i < 4; ++i) v[i] += p.beta * static_cast<float>(o[i]);
      }
      *reinterpret_cast<rb4*>(d) = rb4{static_cast<__bf16>(v[0]), static_cast<__bf16>(v[1]),
                                       static_cast<__bf16>(v[2]), static_cast<__bf16>(v[3])};
    } else {
      for (int i = 0; i < 4; ++i)
        if (c + i < p.N)
          d[i] = static_cast<__bf16>(ELEM != kElemI8 && p.beta != 0.0f
                                         ? v[i] + p.beta * static_cast<float>(d[i]) : v[i]);
    }
  } else {
    _Float16* d = reinterpret_cast<_Float16*>(p.C) + at;
    if (whole) {
      if (ELEM != kElemI8 && p.beta != 0.0f) {
        const rh4 o = *reinterpret_cast<const rh4*>(d);
        for (int i = 0; i < 4; ++i) v[i] += p.beta * static_cast<float>(o[i]);
      }
      *reinterpret_cast<rh4*>(d) = rh4{static_cast<_Float16>(v[0]), static_cast<_Float16>(v[1]),
                                       static_cast<_Float16>(v[2]), static_cast<_Float16>(v[3])};
    } else {
      for (int i = 0; i < 4; ++i)
        if (c + i < p.N)
          d[i] = static_cast<_Float16>(ELEM != kElemI8 && p.beta != 0.0f
                                           ? v[i] + p.beta * static_cast<float>(d[i]) : v[i]);
    }
  }
}

template <int ELEM, int FORM, class T>
__global__ __launch_bounds__(T::NT, 2) void ragged_kernel(const RaggedArgs p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the stub alone and lacks the matrix builtins
  constexpr bool A_ALONG = FORM != kFormTN, B_ALONG = FORM == kFormNT;
  constexpr int ES = elem_size(ELEM), STEPS = 128 / ES, MF = T::MF;
  using Acc = typename RaggedAcc<ELEM, MF>::type;
  using LoadA = RaggedLoader<ELEM, T::BM, A_ALONG, T::WAVES, T::DIRECT>;
  using LoadB = RaggedLoader<ELEM, T::BN, B_ALONG, T::WAVES, T::DIRECT>;
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS];

  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = wave_all % T::WAVES, kgroup = wave_all / T::WAVES;
  const int tiles_n = (p.N + T::BN - 1) / T::BN;

  // The tile: its group, its window of A, B and C, and the reduction's length.
  int group, m0, rows, len;
  long long row_c;
  const char *a, *b;
  int n0;
  if constexpr (FORM == kFormTN) {
    // Each group's tiles are dealt out over all dies: groups differ in length.
    const int tiles_m = (p.M + T::BM - 1) / T::BM, each = tiles_m * tiles_n, room = (each + 7) & ~7;
    group = blockIdx.x / room;
    const int id = die_order(blockIdx.x % room, each);
    if (id < 0) return;
    const TileRow at = band_order(id, tiles_m, tiles_n);
    const RowSpan s = group_rows(p, group);
    m0 = at.m * T::BM;
    n0 = at.n * T::BN;
    rows = min(T::BM, p.M - m0);
    len = s.hi - s.lo;
    a = p.A + s.lo * p.lda + static_cast<long long>(m0) * ES;
    b = p.B + s.lo * p.ldb + static_cast<long long>(n0) * ES;
    row_c = m0;
  } else {
    const int tiles_m = count_tiles<T::BM>(p, lane);
    const int id = die_order(blockIdx.x, tiles_m * tiles_n);
    if (id < 0) return;
    const TileRow at = band_order(id, tiles_m, tiles_n);
    const TileAt where = find_tile<T::BM>(p, at.m, lane);
    group = where.group;
    if (group < 0) return;
    const RowSpan s = group_rows(p, group);
    m0 = s.lo + where.tile * T::BM;
    n0 = at.n * T::BN;
    rows = min(T::BM, s.hi - m0);
    len = p.K;
    a = p.A + m0 * p.lda;
    b = p.B + group * p.stride_b + (B_ALONG ? n0 * p.ldb : static_cast<long long>(n0) * ES);
    row_c = m0;
  }
  const int cols = min(T::BN, p.N - n0);

  const int slices = (len + STEPS - 1) / STEPS, turns = (slices + T::WAVES_K - 1) / T::WAVES_K;
  LoadA la;
  LoadB lb;
  {
    const long long sa = A_ALONG ? 128 : STEPS * p.lda, sb = B_ALONG ? 128 : STEPS * p.ldb;
    la.init(a + kgroup * sa, p.lda, sa * T::WAVES_K, A_ALONG ? rows : rows * ES, wave, lane);
    lb.init(b + kgroup * sb, p.ldb, sb * T::WAVES_K, B_ALONG ? cols : cols * ES, wave, lane);
  }
  const rlds_t ring = (rlds_t)lds + kgroup * (T::STAGE * T::S);
  int left = len - kgroup * STEPS;  // reduction steps from the next slice to load
  auto cut = [&] {
    if (left < STEPS) {
      la.cut(A_ALONG ? left * ES : left);
      lb.cut(B_ALONG ? left * ES : left);
    }
  };

  Acc acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int j = 0; j < T::FN; ++j) acc[i][j] = Acc{};

  const int am = (wave / T::WAVES_N) * T::WM, bn = (wave % T::WAVES_N) * T::WN;
  auto multiply = [&](rlds_t stage) {
    constexpr int GROUPS = 64 / MF, KS = 8 / GROUPS;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      ri4 fa[T::FM], fb[T::FN];
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
        fa[i] = ragged_frag<ELEM, T::BM, A_ALONG, MF>(stage, am, i, ks, lane);
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
        fb[j] = ragged_frag<ELEM, T::BN, B_ALONG, MF>(stage + T::BM * 128, bn, j, ks, lane);
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j) ragged_mma<ELEM, MF>(acc[i][j], fb[j], fa[i]);
    }
  };

  constexpr bool ALONE = T::WAVES == 1;
  if constexpr (T::DIRECT) {
    constexpr int NI = LoadA::NI + LoadB::NI;
    auto send = [&](int stage) {
      cut();
      la.send(ring + stage * T::STAGE);
      lb.send(ring + stage * T::STAGE + T::BM * 128);
      left -= STEPS * T::WAVES_K;
    };
#pragma unroll
    for (int s = 0; s < T::S - 1; ++s) send(s);
    int at = 0, next = T::S - 1;
    for (int t = 0; t < turns; ++t) {
      ragged_barrier<(T::S - 2) * NI, ALONE>();
      send(next);
      multiply(ring + at * T::STAGE);
      at = at + 1 == T::S ? 0 : at + 1;
      next = next + 1 == T::S ? 0 : next + 1;
    }
    // The slices past the end, all masked, may still be on their way to LDS.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  } else {
    auto fetch = [&] {
      cut();
      la.fetch(A_ALONG ? left * ES : left);
      lb.fetch(B_ALONG ? left * ES : left);
    };
    auto put = [&](int stage) {
      la.put(ring + stage * T::STAGE, A_ALONG ? left * ES : left);
      lb.put(ring + stage * T::STAGE + T::BM * 128, B_ALONG ? left * ES : left);
      left -= STEPS * T::WAVES_K;
    };
    if (turns > 0) {
      fetch();
      put(0);
    }
    for (int t = 0; t < turns; ++t) {
      __syncthreads();
      if (t + 1 < turns) fetch();
      multiply(ring + (t & 1) * T::STAGE);
      if (t + 1 < turns) put((t + 1) & 1);
    }
  }

  // Wave groups that took other slices hand over their sums, in a fixed order.
  constexpr int REGS = MF * MF / 64;
  if constexpr (T::WAVES_K > 1) {
    using S = decltype(acc[0][0][0] + acc[0][0][0]);
    __attribute__((address_space(3))) S* sums = (__attribute__((address_space(3))) S*)(rlds_t)lds;
    const int slot = wave * 64 + lane;
    constexpr int EACH = T::WAVES * 64;
    __syncthreads();
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

  RaggedArgs q = p;
  if constexpr (FORM == kFormTN)
    q.C += group * p.stride_c * (p.out == kElemF32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
    const int m = am + i * MF + lane % MF;
    if (m >= rows) continue;
    const float sa = ELEM == kElemI8 ? p.scale_a[row_c + m] : 0.0f;
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int r = 0; r < REGS; r += 4) {
        const int n = n0 + bn + j * MF + (MF == 32 ? 2 * r : 0) + 4 * (lane / MF);
        const decltype(__builtin_shufflevector(acc[i][j], acc[i][j], 0, 1, 2, 3)) v = {
            acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
        ragged_store<ELEM>(q, row_c + m, group, n, v, sa);
      }
  }
#endif
}

template <int ELEM, int FORM, class T>
hipError_t launch_ragged(const RaggedArgs& a, long long grid, hipStream_t stream) {
  ragged_kernel<ELEM, FORM, T><<<dim3(static_cast<unsigned>(grid)), dim3(T::NT), 0, stream>>>(a);
  return hipGetLastError();
}

// The compiled tiles, widest first.
using RaggedWide = RaggedTile<256, 256, 2, 4, 1, 2, 32, true>;
using RaggedMid = RaggedTile<128, 128, 2, 2, 1, 2, 32, true>;
using RaggedMidAny = RaggedTile<128, 128, 2, 2, 1, 2, 32, false>;
using RaggedThin = RaggedTile<16, 64, 1, 1, 4, 3, 16, true>;
using RaggedThinAny = RaggedTile<16, 64, 1, 1, 4, 2, 16, false>;

enum RaggedShape { kWide, kMid, kThin };

// Largest 2-byte or smaller element count a tile's rows may be apart: the byte
// offsets of 256 rows fit the 31 bits of a buffer offset.
constexpr long long kRaggedMaxLd = 1LL << 21;

hipError_t ragged_f32(int form, int shape, bool direct, const RaggedArgs&, long long grid, hipStream_t);
hipError_t ragged_bf16(int form, int shape, bool direct, const RaggedArgs&, long long grid, hipStream_t);
hipError_t ragged_f16(int form, int shape, bool direct, const RaggedArgs&, long long grid, hipStream_t);
hipError_t ragged_i8(int form, int shape, bool direct, const RaggedArgs&, long long grid, hipStream_t);

}  // namespace fp32gemm
