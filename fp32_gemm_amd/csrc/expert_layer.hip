// expert_layer.hip -- a whole layer of experts for a few tokens, in two kernels.
//
//   h[t, j] = silu(G_e x_t) * (U_e x_t)   (or silu(U_e x_t)),   e = ids[t, j]
//   y[t] = sum_j share[t, j] D_e h[t, j]
//
// What bounds it is reading the chosen experts' weights, once for each 16 of their
// tokens.  Both kernels multiply an expert's rows by the gathered values of up to 16.  There
// is one workgroup a compute unit; each takes an equal run of all the rows that are to
// be multiplied.  Its eight waves divide the reduction, of 32 rows at a time, or, where
// it is short, two or four times as many rows as well; they add up in LDS in a fixed
// order, and load the next rows meanwhile.  A wave reads 16 rows, 64 bytes of each a step, straight to registers in
// the order in which the matrix instruction takes them: a lane's 16 bytes are its
// operand, so that neither LDS nor a barrier stands between memory and the products.
// The tokens' values, the instruction's other operand, stay in registers for all of
// an expert's rows.
//
// Measured, for the layer of 4096 by 2048 with a gate: one token, 2 of 16 experts in
// bf16 28 us (3.6 TB/s over both kernels), 64 tokens, 16 experts in 8 bits 107 us
// (3.6 TB/s), in bf16 165 to 172 us (4.8 TB/s).  The kernels stream 5 TB/s once they are
// under way; what is left is each kernel's start (launch, ids, first loads: 5 us in
// which little arrives) and the last sums (3 us, 6 for 64 tokens).
//
// Between the two, h is held in 32 bits: as a float where the tokens are floats, else as
// a sum of two bf16, to 2^-17 of itself and with the range of a float.  The matrix
// instruction takes such parts as they lie (rounded to the tokens' type instead, h was
// what results were off by, 2.3e-3 for 1.7e-3, and infinite past 65504 in f16; that took
// 1 us less for one token in bf16, 4 for 64 in 8 bits).
//
// The second kernel leaves an expert's products, not yet shared out, for each pair
// of token and choice; the last workgroup to finish a block of columns adds them up
// for every token, in the order of its choices.
#include "expert_layer.hpp"

#include "ragged_kernels.hpp"

namespace fp32gemm {
namespace {

constexpr int kWaves = 8, kThreads = kWaves * 64, kRows = 16;
constexpr int kGroups = 256;  // workgroups: one a compute unit
static_assert(kThreads >= kLayerPairs, "a thread for each pair");

__device__ __forceinline__ int lanes_below(unsigned long long m) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<unsigned>(m >> 32),
                                   __builtin_amdgcn_mbcnt_lo(static_cast<unsigned>(m), 0));
}

// What the ids say: the experts that any token names, in the order of the pairs
// (token, choice) that name them first, and each one's pairs.  A token that names
// an expert more than once counts once; ids out of range name nothing.  An expert
// whose pairs are more than 16 is taken once for each 16, its weights read as often: the
// entries below, none of which is empty.  There are two ways to them.

// Up to 128 pairs that name up to 32 experts: every wave finds them by itself, two
// pairs a lane and a few instructions for each expert.
constexpr int kFewPairs = 128, kFewExperts = 32;
struct FewPairs {
  int id[2];  // of pairs lane and 64 + lane; -1: none, or an earlier choice of the token is the same

  __device__ __forceinline__ void init(const LayerArgs& p, int lane) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = 64 * k + lane;
      const int e = i < p.T * p.top ? p.ids[i] : -1;
      id[k] = e >= 0 && e < p.experts ? e : -1;
    }
    bool again[2] = {};
    for (int d = 1; d < p.top; ++d) {  // the token's other choices; all lanes fetch
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = 64 * k + lane;
        const int before0 = __shfl(id[0], i - d & 63), before1 = __shfl(id[1], i - d & 63);
        again[k] |= d <= i % p.top && (i - d < 64 ? before0 : before1) == id[k];
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) id[k] = again[k] ? -1 : id[k];
  }
  // Calls visit(expert, entries) for one expert after another until it says no.
  template <class F>
  __device__ __forceinline__ void walk(F visit) const {
    unsigned long long left[2] = {__ballot(id[0] >= 0), __ballot(id[1] >= 0)};
    while (left[0] | left[1]) {
      const int e = left[0] ? __builtin_amdgcn_readlane(id[0], __builtin_ctzll(left[0]))
                            : __builtin_amdgcn_readlane(id[1], __builtin_ctzll(left[1]));
      int n = 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const unsigned long long m = __ballot(id[k] == e);
        left[k] &= ~m;
        n += __builtin_popcountll(m);
      }
      if (!visit(e, (n + 15) / 16)) return;
    }
  }
  __device__ __forceinline__ int entries() const {
    int all = 0;
    walk([&](int, int n) {
      all += n;
      return true;
    });
    return all;
  }
  // Entry v: its expert, and which 16 of its pairs.
  __device__ __forceinline__ void entry(int v, int& e, int& set) const {
    walk([&](int expert, int n) {
      e = expert;
      set = v;
      v -= n;
      return v >= 0;
    });
  }
  // The pairs of expert e from the first-th on, in order, at most 16; returns how many.
  __device__ __forceinline__ int list_pairs(int e, int first, short* list, int lane) const {
    int n = -first;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bool mine = id[k] == e;
      const unsigned long long m = __ballot(mine);
      const int at = n + lanes_below(m);
      if (mine && at >= 0 && at < 16) list[at] = static_cast<short>(64 * k + lane);
      n += __builtin_popcountll(m);
    }
    __builtin_amdgcn_wave_barrier();
    return min(max(n, 0), 16);
  }
};

// More: a table in LDS, made by the whole workgroup.
struct Routing {
  int id[kLayerPairs];    // -1: none, or an earlier choice of the token is the same
  int used[kLayerPairs];  // experts
  int upto[kLayerPairs];  // entries of all experts before it, and its own
  int pairs[kLayerExperts];
  int first[kLayerExperts];
  int count[kWaves];

  // Returns how many entries there are.
  __device__ __forceinline__ int init(const LayerArgs& p) {
    const int i = threadIdx.x, all = p.T * p.top, wave = i >> 6;
    int e = -1;
    if (i < all) {
      e = p.ids[i];
      if (e < 0 || e >= p.experts) e = -1;
      id[i] = e;
      if (e >= 0) {
        first[e] = kLayerPairs;
        pairs[e] = 0;
      }
    }
    __syncthreads();
    const int j = i < all ? i % p.top : 0;
    bool again = false;
    for (int k = 1; k <= j; ++k) again |= id[i - k] == e;
    if (again) e = -1;
    if (e >= 0) {  // whatever the order, the least stays and the sum is the same
      atomicMin(&first[e], i);
      atomicAdd(&pairs[e], 1);
    }
    __syncthreads();
    const bool leads = e >= 0 && first[e] == i;
    const unsigned long long m = __ballot(leads);
    if ((i & 63) == 0) count[wave] = __builtin_popcountll(m);
    if (i < all) id[i] = e;
    __syncthreads();
    int before = 0, experts = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      before += w < wave ? count[w] : 0;
      experts += count[w];
    }
    if (leads) used[before + lanes_below(m)] = e;
    __syncthreads();
    const int mine = i < experts ? (pairs[used[i]] + 15) / 16 : 0;
    const int sum = DeviceWave::sum_below(mine);
    if ((i & 63) == 63) count[wave] = sum;
    __syncthreads();
    before = 0;
    int entries = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      before += w < wave ? count[w] : 0;
      entries += count[w];
    }
    if (i < kLayerPairs) upto[i] = before + sum;
    __syncthreads();
    return entries;
  }
  __device__ __forceinline__ void entry(int v, int& e, int& set) const {
    int lo = 0, hi = kLayerPairs - 1;  // the first expert whose entries go past v
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (upto[mid] > v) hi = mid;
      else lo = mid + 1;
    }
    e = used[lo];
    set = v - (lo > 0 ? upto[lo - 1] : 0);
  }
  __device__ __forceinline__ int list_pairs(int e, int from, int all, short* list, int lane) const {
    int n = -from;
    for (int i0 = 0; i0 < all && n < 16; i0 += 64) {
      const bool mine = i0 + lane < all && id[i0 + lane] == e;
      const unsigned long long m = __ballot(mine);
      const int at = n + lanes_below(m);
      if (mine && at >= 0 && at < 16) list[at] = static_cast<short>(i0 + lane);
      n += __builtin_popcountll(m);
    }
    __builtin_amdgcn_wave_barrier();
    return min(max(n, 0), 16);
  }
};

// ---------------------------------------------------------------------------
// Values that are sums of two bf16: eight first parts, then the eight second ones; rows
// are filled up with zeros to a multiple of eight.
constexpr int kElemPair = 6;
// h, of tokens of type XE.
template <int XE>
constexpr int kHidden = XE == kElemF32 ? kElemF32 : kElemPair;

// How weights of format WE and values of type XE are multiplied.
template <int XE, int WE>
struct Format {
  static constexpr bool SAME = XE == WE, BLOCKS = WE == kElemM4;
  static constexpr bool PAIR = XE == kElemPair, HALVES = PAIR && (WE == kElemBF16 || WE == kElemF16);
  static constexpr int XS = PAIR ? 4 : elem_size(XE);
  static constexpr int PER = WE == kElemM4 ? 32 : 16 / elem_size(WE);  // weights of 16 bytes
  static constexpr int STEP = 4 * PER;                                  // of a step
  static constexpr int XV = PER * XS / 16;                              // 16-byte pieces of values for them
  // Narrow weights become bf16, exactly but for 4-bit ones past 2^128; values become a sum
  // of one, two or three bf16, exactly down to 2^-133, the least bf16, and are multiplied
  // one after another.
  static constexpr int PARTS = SAME ? 1 : XE == kElemBF16 ? 1 : XE == kElemF16 || PAIR ? 2 : 3;
  static constexpr int MMAS = SAME ? 1 : PER / 8;
};

__device__ __forceinline__ rb8 weights_of_8_bits(int lo, int hi) {
  // Whole words until here: seen as bytes, they would be taken apart, and waited for,
  // where they are loaded.
  asm("" : "+v"(lo), "+v"(hi));
  rb8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    r[i] = static_cast<__bf16>(static_cast<float>(static_cast<signed char>((i < 4 ? lo : hi) >> (8 * (i & 3)))));
  return r;
}
__device__ __forceinline__ rb8 weights_of_4_bits(unsigned codes, float scale) {
  typedef __bf16 rb2 __attribute__((ext_vector_type(2)));
  const rb2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0),
            b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1),
            c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2),
            d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return rb8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight weights of f16 as a sum of two bf16, neither of them zero unless the weight is, so
// that an infinite value times the weight is infinite.
__device__ __forceinline__ void weights_of_f16(const ri4& w, rb8 (&part)[2]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = static_cast<float>(__builtin_bit_cast(rh8, w)[i]);
    float top = __builtin_bit_cast(float, __builtin_bit_cast(unsigned, v) & 0xFFFF0000u), rest = v - top;
    if (!(__builtin_fabsf(rest) > 0.0f)) top = rest = 0.5f * v;  // eight bits or fewer, or no number
    part[0][i] = __builtin_bit_cast(__bf16, static_cast<unsigned short>(__builtin_bit_cast(unsigned, top) >> 16));
    part[1][i] = __builtin_bit_cast(__bf16, static_cast<unsigned short>(__builtin_bit_cast(unsigned, rest) >> 16));
  }
}

// Eight values as a sum of bf16.
template <int XE, int PARTS>
__device__ __forceinline__ void split_values(const ri4* raw, int m, rb8 (&part)[PARTS]) {
  if constexpr (XE == kElemBF16) {
    part[0] = __builtin_bit_cast(rb8, raw[m]);
  } else if constexpr (XE == kElemPair) {
    part[0] = __builtin_bit_cast(rb8, raw[2 * m]);
    part[1] = __builtin_bit_cast(rb8, raw[2 * m + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v;
      if constexpr (XE == kElemF16) v = static_cast<float>(__builtin_bit_cast(rh8, raw[m])[i]);
      else v = __builtin_bit_cast(rf4, raw[2 * m + i / 4])[i % 4];
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        const float top = __builtin_bit_cast(float, __builtin_bit_cast(unsigned, v) & 0xFFFF0000u);
        part[k][i] = __builtin_bit_cast(__bf16, static_cast<unsigned short>(__builtin_bit_cast(unsigned, v) >> 16));
        v = v == top ? 0.0f : v - top;  // an infinity leaves nothing
      }
    }
  }
}

// Eight narrow weights, the lowest of `bits`, times eight values.
template <int XE, int WE>
__device__ __forceinline__ void layer_mma_8(rf4& acc, int lo, int hi, const ri4* x, int m, float scale) {
  using Fm = Format<XE, WE>;
  rb8 wb, part[Fm::PARTS];
  if constexpr (Fm::BLOCKS) wb = weights_of_4_bits(static_cast<unsigned>(lo), scale);
  else wb = weights_of_8_bits(lo, hi);
  split_values<XE, Fm::PARTS>(x, m, part);
#pragma unroll
  for (int k = 0; k < Fm::PARTS; ++k) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, part[k], acc, 0, 0, 0);
}
// Eight weights of 16 bits times eight sums of two bf16.
template <int WE>
__device__ __forceinline__ void layer_mma_pairs(rf4& acc, const ri4& w, const ri4* x) {
  rb8 wb[2] = {__builtin_bit_cast(rb8, w), {}};
  if constexpr (WE == kElemF16) weights_of_f16(w, wb);
#pragma unroll
  for (int j = 0; j < (WE == kElemF16 ? 2 : 1); ++j)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], __builtin_bit_cast(rb8, x[k]), acc, 0, 0, 0);
}
// One step of one block of rows and one set of tokens.
template <int XE, int WE>
__device__ __forceinline__ void layer_mma(rf4& acc, const ri4& w, const ri4* x, float scale) {
  using Fm = Format<XE, WE>;
  if constexpr (Fm::SAME) {
    ragged_mma<XE, 16>(acc, w, x[0]);
  } else if constexpr (Fm::HALVES) {
    layer_mma_pairs<WE>(acc, w, x);
  } else {
#pragma unroll
    for (int m = 0; m < Fm::MMAS; ++m)
      layer_mma_8<XE, WE>(acc, Fm::BLOCKS ? w[m] : w[2 * m & 3], Fm::BLOCKS ? 0 : w[2 * m + 1 & 3], x, m, scale);
  }
}

// A wave's part of an expert's rows: NB blocks of 16 rows at a time, a turn of U steps
// of them in hand and one or two more on their way.
//   Q > 0   the tokens' values stay in registers for all rows: Q turns of U steps
//           are all that the wave has of the reduction.
//   Q == 0  they are loaded again with each turn.
template <int XE, int WE, int U, int Q, int NB = 2>
struct Rows {
  using Fm = Format<XE, WE>;
  static constexpr bool KEPT = Q > 0;
  static constexpr int XT = KEPT ? Q : 1;
  static constexpr bool AHEAD = KEPT || U * (NB * 4 + Fm::XV * 4) <= (NB == 1 ? 64 : 48);  // as far as registers go
  struct Held {
    ri4 w[U][NB];
    int s[U][NB];  // 4-bit codes: the blocks' scales, as loaded
    ri4 x[KEPT ? 1 : U][Fm::XV];
  };
  const char* rows[NB];    // the expert's first row of each kind of block
  const char* scales[NB];
  const char* values;
  int lane, last, gap;             // the last row of a block's kind; rows from a set of blocks to the next one
  int blocks = 1, block0 = 0;      // sets of the workgroup, and the wave's
  long long ld, scale_ld;          // bytes between rows
  int row_bytes, steps, full;      // of a row; reduction steps; whole steps of 64 bytes
  int first_step, end_step, turns; // the wave's steps, and its turns
  int x_off;                       // the lane's token past `values`, or kRaggedMasked
  ri4 kept[XT][U][Fm::XV];
  bool tail;                       // this wave takes what whole steps leave

  __device__ __forceinline__ int row_of(int block, int b) const {
    return (block * blocks + block0) * gap + (gap == 32 ? 16 * b : 0);
  }
  __device__ __forceinline__ int lane_row(int row) const { return min(lane % 16, max(last - row, 0)); }
  __device__ __forceinline__ int clamped(int row) const { return min(row, last); }

  // The values of `n` tokens come through LDS, a kilobyte of one token's an
  // instruction: loaded as the products take them, each would touch 64 lines.  Piece c
  // of token t lies at place c ^ t of its row, so that the tokens' reads spread over
  // the banks.
  // More than 16 pieces a lane come in two passes.
  static constexpr int PASSES = XT * U * Fm::XV > 16 ? 2 : 1, PASS = XT * U / PASSES;  // steps of one
  static constexpr int KEEP_ROW = PASS * Fm::STEP * Fm::XS;  // bytes of a token
  static_assert(!KEPT || ((KEEP_ROW & (KEEP_ROW - 1)) == 0 && PASS * PASSES == XT * U), "a power of two");
  __device__ __forceinline__ void send_values(rlds_t room, int pass, int n, const short* list, int top,
                                              long long ldx) const {
    constexpr int PIECES = KEEP_ROW / 16, EACH = PIECES < 64 ? 64 / PIECES : 1;  // tokens an instruction
    const auto v = ragged_rsrc(values, kRaggedMasked);
    const int end = end_step * Fm::STEP * Fm::XS, start = (first_step + pass * PASS) * Fm::STEP * Fm::XS;
    for (int t0 = 0; t0 < n; t0 += EACH)
#pragma unroll
      for (int part = 0; part < (PIECES + 63) / 64; ++part) {
        const int t = t0 + (EACH > 1 ? lane / PIECES : 0), place = part * 64 + lane % (EACH > 1 ? PIECES : 64);
        const int at = start + (place ^ (t & (PIECES - 1) & 15)) * 16;
        const int row = list[min(t, 15)] / top * static_cast<int>(ldx);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            v, (__attribute__((address_space(3))) void*)(room + t0 * KEEP_ROW + part * 1024), 16,
            t < n && at < end ? row + at : kRaggedMasked, 0, 0, 0);
      }
  }
  template <int P>
  __device__ __forceinline__ void keep_values(rlds_t room, int n) {
    constexpr int PIECES = KEEP_ROW / 16;
    const int t = lane % 16;
#pragma unroll
    for (int s = 0; s < PASS; ++s)
#pragma unroll
      for (int i = 0; i < Fm::XV; ++i) {
        const int piece = (s * 4 + lane / 16) * Fm::XV + i;
        const ri4 x = *(__attribute__((address_space(3))) ri4*)(room + t * KEEP_ROW +
                                                               (piece ^ (t & (PIECES - 1) & 15)) * 16);
        kept[(P * PASS + s) / U][(P * PASS + s) % U][i] = t < n ? x : ri4{};
      }
  }
  __device__ __forceinline__ void load(Held& h, int block, int turn) const {
    const int step = first_step + turn * U;
    const bool whole = step + U <= end_step;  // else steps past the wave's last read as zeros
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int row = clamped(row_of(block, b)), in = lane_row(row);
      const auto r = ragged_rsrc(rows[b] + row * ld + step * 64, kRaggedMasked);
      const int off = in * static_cast<int>(ld) + lane / 16 * 16;
      if (whole) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          h.w[u][b] = __builtin_bit_cast(ri4, __builtin_amdgcn_raw_buffer_load_b128(r, off, u * 64, 0));
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
          h.w[u][b] = __builtin_bit_cast(
              ri4, __builtin_amdgcn_raw_buffer_load_b128(r, step + u < end_step ? off : kRaggedMasked, u * 64, 0));
      }
      if constexpr (Fm::BLOCKS) {
        // The scales of four steps are 16 bytes of a row (of two, 8), four for each step,
        // and a lane's the one of its 32 codes.
        const auto q = ragged_rsrc(scales[b] + row * scale_ld + step * 4, kRaggedMasked);
        const int at = in * static_cast<int>(scale_ld);
        if (U == 4 && whole) {
          const ri4 w = __builtin_bit_cast(ri4, __builtin_amdgcn_raw_buffer_load_b128(q, at, 0, 0));
#pragma unroll
          for (int u = 0; u < U; ++u) h.s[u][b] = w[u & 3];
        } else if (U == 2 && whole) {
          const ri2 w = __builtin_bit_cast(ri2, __builtin_amdgcn_raw_buffer_load_b64(q, at, 0, 0));
#pragma unroll
          for (int u = 0; u < U; ++u) h.s[u][b] = w[u & 1];
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u)
            h.s[u][b] = static_cast<int>(
                __builtin_amdgcn_raw_buffer_load_b32(q, step + u < end_step ? at : kRaggedMasked, u * 4, 0));
        }
      }
    }
    if constexpr (!KEPT) {
      const auto v = ragged_rsrc(values, kRaggedMasked);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int off = x_off == kRaggedMasked || step + u >= end_step
                            ? kRaggedMasked : x_off + ((step + u) * Fm::STEP + lane / 16 * Fm::PER) * Fm::XS;
#pragma unroll
        for (int i = 0; i < Fm::XV; ++i)
          h.x[u][i] = __builtin_bit_cast(ri4, __builtin_amdgcn_raw_buffer_load_b128(v, off, i * 16, 0));
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // loads go out before anything waits for earlier ones
  }
  __device__ __forceinline__ float scale_of(int word) const {
    return __builtin_bit_cast(float, (word >> (lane / 16 * 8) & 255) << 23);
  }
  __device__ __forceinline__ void multiply(rf4 (&acc)[NB], const Held& h, int turn) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float scale = Fm::BLOCKS ? scale_of(h.s[u][b]) : 0.0f;
        if constexpr (KEPT) layer_mma<XE, WE>(acc[b], h.w[u][b], kept[turn][u], scale);
        else layer_mma<XE, WE>(acc[b], h.w[u][b], h.x[u], scale);
        // Or all weights are widened first, in registers that are not there.
        if constexpr (!Fm::SAME) __builtin_amdgcn_sched_barrier(0);
      }
  }
  // What whole steps of 64 bytes leave of the rows: nothing past them is read, and
  // what is missing counts as zero.  Where weights are not narrow and rows are 16 bytes
  // or more, the 16 bytes that end with them are loaded with the block's first turn and
  // shifted down (values too, but for pairs, whose rows are filled up); else all of it
  // waits for the turns.
  static constexpr bool RESTS = Fm::SAME || Fm::HALVES;
  struct Rest {
    ri4 w[NB], x[Fm::HALVES ? 2 : 1];
  };
  __device__ __forceinline__ bool ahead_of_rest() const { return RESTS && row_bytes >= 16; }
  __device__ __forceinline__ void load_rest(Rest& h, int block) const {
    const int at = full * 64 + lane / 16 * 16, n = row_bytes - at, back = n > 0 && n < 16 ? 16 - n : 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int row = clamped(row_of(block, b));
      h.w[b] = __builtin_bit_cast(
          ri4, __builtin_amdgcn_raw_buffer_load_b128(ragged_rsrc(rows[b] + row * ld, kRaggedMasked),
                                                     n > 0 ? lane_row(row) * static_cast<int>(ld) + at - back : kRaggedMasked, 0, 0));
    }
    const auto v = ragged_rsrc(values, kRaggedMasked);
    const bool some = n > 0 && x_off != kRaggedMasked;
    if constexpr (Fm::HALVES) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        h.x[k] = __builtin_bit_cast(
            ri4, __builtin_amdgcn_raw_buffer_load_b128(v, some ? x_off + 2 * at + 16 * k : kRaggedMasked, 0, 0));
    } else {
      h.x[0] = __builtin_bit_cast(
          ri4, __builtin_amdgcn_raw_buffer_load_b128(v, some ? x_off + at - back : kRaggedMasked, 0, 0));
    }
  }
  __device__ __forceinline__ void multiply_rest(rf4 (&acc)[NB], const Rest& h) const {
    const int n = row_bytes - (full * 64 + lane / 16 * 16), back = n > 0 && n < 16 ? 16 - n : 0;
    auto down = [&](const ri4& v) { return __builtin_bit_cast(ri4, __builtin_bit_cast(unsigned __int128, v) >> (8 * back)); };
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (Fm::HALVES) layer_mma_pairs<WE>(acc[b], down(h.w[b]), h.x);
      else ragged_mma<XE, 16>(acc[b], down(h.w[b]), down(h.x[0]));
    }
  }
  __device__ __forceinline__ void multiply_tail(rf4 (&acc)[NB], int block) const {
    const int at = full * 64 + lane / 16 * 16, n = row_bytes - at;  // valid bytes from here
    ri4 w[NB];
    float scale[NB] = {};
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int row = clamped(row_of(block, b)), in = lane_row(row);
      const auto r = ragged_rsrc(rows[b] + row * ld, kRaggedMasked);
      const int off = in * static_cast<int>(ld) + at;
      if (row_bytes >= 16) {
        const int back = n > 0 && n < 16 ? 16 - n : 0;
        const ri4 raw = __builtin_bit_cast(
            ri4, __builtin_amdgcn_raw_buffer_load_b128(r, n > 0 ? off - back : kRaggedMasked, 0, 0));
        w[b] = __builtin_bit_cast(ri4, __builtin_bit_cast(unsigned __int128, raw) >> (8 * back));
      } else {
        unsigned __int128 bytes = 0;
#pragma unroll 1
        for (int i = 0; i < 16; ++i)
          bytes |= static_cast<unsigned __int128>(
                       __builtin_amdgcn_raw_buffer_load_b8(r, i < n ? off + i : kRaggedMasked, 0, 0) & 255)
                   << (8 * i);
        w[b] = __builtin_bit_cast(ri4, bytes);
      }
      if constexpr (Fm::BLOCKS) {
        const int byte = __builtin_amdgcn_raw_buffer_load_b8(ragged_rsrc(scales[b] + row * scale_ld, kRaggedMasked),
                                                             n > 0 ? in * static_cast<int>(scale_ld) + at / 16 : kRaggedMasked, 0, 0);
        scale[b] = __builtin_bit_cast(float, (byte & 255) << 23);
      }
    }
    const auto v = ragged_rsrc(values, kRaggedMasked);
    const int first = full * Fm::STEP + lane / 16 * Fm::PER;  // the lane's reduction steps
    // A step's products one after another: written out they would take registers
    // that the whole steps need.
    constexpr int PIECES = Fm::SAME ? 1 : 8 * Fm::XS / 16, EACH = 16 / Fm::XS;  // of values, for a product
#pragma unroll 1
    for (int m = 0; m < Fm::MMAS; ++m) {
      ri4 x[PIECES];
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        x[i] = ri4{};
        if constexpr (Fm::PAIR) {  // rows are filled up to whole pieces
          const int step = first + m * 8;
          x[i] = __builtin_bit_cast(
              ri4, __builtin_amdgcn_raw_buffer_load_b128(
                       v, x_off == kRaggedMasked || step >= steps ? kRaggedMasked : x_off + step * Fm::XS + 16 * i, 0, 0));
          continue;
        }
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
          const int step = first + m * 8 + i * EACH + k;
          const int off = x_off == kRaggedMasked || step >= steps ? kRaggedMasked : x_off + step * Fm::XS;
          if constexpr (Fm::XS == 4)
            x[i][k] = static_cast<int>(__builtin_amdgcn_raw_buffer_load_b32(v, off, 0, 0));
          else
            x[i][k / 2] |= static_cast<int>(static_cast<unsigned>(__builtin_amdgcn_raw_buffer_load_b16(v, off, 0, 0) & 0xFFFF)
                                            << (16 * (k & 1)));
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (Fm::SAME) ragged_mma<XE, 16>(acc[b], w[b], x[0]);
        else if constexpr (Fm::HALVES) layer_mma_pairs<WE>(acc[b], w[b], x);
        else layer_mma_8<XE, WE>(acc[b], w[b][0], w[b][1], x, 0, scale[b]);
        w[b] = Fm::BLOCKS ? ri4{w[b][1], w[b][2], w[b][3], 0} : ri4{w[b][2], w[b][3], 0, 0};
      }
    }
  }
  // Begins to load the second turn of blocks lo .. hi - 1 and waits for the values, which
  // were sent before it: loads arrive in their order.
  __device__ __forceinline__ void load_second(Held& b, int lo, int hi) const {
    if (lo + 1 / XT < hi) {
      load(b, lo + 1 / XT, 1 % XT);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(U * NB + (Fm::BLOCKS ? NB : 0)) : "memory");  // or more
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
  }
  // Blocks lo .. hi - 1; calls end(block, acc) for each, by all waves alike.  `a` holds
  // the first turn, and where values are kept `b` the second one.
  template <class F>
  __device__ __forceinline__ void run(int lo, int hi, Held& a, Held& b, F end) {
    rf4 acc[NB] = {};
    Rest rest;
    auto begin = [&](int block) {
      if constexpr (RESTS)
        if (tail && ahead_of_rest()) load_rest(rest, block);
    };
    auto done = [&](int block) {
      if (tail) {
        if constexpr (RESTS) {
          if (ahead_of_rest()) multiply_rest(acc, rest);
          else multiply_tail(acc, block);
        } else {
          multiply_tail(acc, block);
        }
      }
      end(block, acc);
#pragma unroll
      for (int i = 0; i < NB; ++i) acc[i] = rf4{};
    };
    if constexpr (KEPT) {
      // The turns of a block, or of two, are written out, so that each knows its
      // registers.  Two are on their way while one is multiplied or its sums are
      // shared (one: 8 tokens, 2 choices of 32, 4 bits, 4096 by 2048, when it was built:
      // 52 us for 46).
      constexpr int BLOCKS = Q % 2 ? 2 : 1;
      for (int block = lo; block < hi; block += BLOCKS) {
#pragma unroll
        for (int i = 0; i < BLOCKS * Q; ++i) {
          const int now = block + i / Q, next = block + (i + 2) / Q;
          if (now < hi) {
            if (i % Q == 0) begin(now);
            multiply(acc, i % 2 ? b : a, i % Q);
            if (next < hi) load(i % 2 ? b : a, next, (i + 2) % Q);
            if (i % Q == Q - 1) done(now);
          }
        }
      }
    } else {
      for (int block = lo; block < hi; ++block) {
        int turn = 0;
        begin(block);
        if constexpr (AHEAD) {
          if (block > lo) load(a, block, 0);
          for (; turn + 2 < turns; turn += 2) {
            load(b, block, turn + 1);
            multiply(acc, a, turn);
            load(a, block, turn + 2);
            multiply(acc, b, turn + 1);
          }
          if (turn + 1 < turns) {
            load(b, block, turn + 1);
            multiply(acc, a, turn);
            multiply(acc, b, turn + 1);
          } else {
            multiply(acc, a, turn);
          }
        } else {
          for (; turn < turns; ++turn) {
            if (block > lo || turn > 0) load(a, block, turn);
            multiply(acc, a, turn);
          }
        }
        done(block);
      }
    }
  }
};

template <int WE>
__device__ __forceinline__ int bytes_of_row(int steps) {
  return WE == kElemM4 ? (steps + 1) / 2 : steps * elem_size(WE);
}

__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

template <int XE>
__device__ __forceinline__ void put(char* p, long long i, float v) {
  if constexpr (XE == kElemF32) reinterpret_cast<float*>(p)[i] = v;
  else if constexpr (XE == kElemBF16) reinterpret_cast<__bf16*>(p)[i] = static_cast<__bf16>(v);
  else reinterpret_cast<_Float16*>(p)[i] = static_cast<_Float16>(v);
}

// Value i of a row of h.
template <int HE>
__device__ __forceinline__ void put_hidden(char* p, long long i, float v) {
  if constexpr (HE == kElemF32) {
    reinterpret_cast<float*>(p)[i] = v;
  } else {
    // The nearest bf16, or, where that is infinite and v is not, the one below; what is left rounds again.
    float top = static_cast<float>(static_cast<__bf16>(v));
    if (__builtin_fabsf(top) == __builtin_inff())
      top = __builtin_bit_cast(float, __builtin_bit_cast(unsigned, v) & 0xFFFF0000u);
    __bf16* const q = reinterpret_cast<__bf16*>(p) + (i / 8) * 16 + i % 8;
    q[0] = static_cast<__bf16>(top);
    q[8] = static_cast<__bf16>(v == top ? 0.0f : v - top);
  }
}

// Products that another workgroup adds up: stored and loaded past the caches that
// belong to one die (fences in their place write back, or empty, all of an L2: 4 us
// and more).
__device__ __forceinline__ void publish(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ rf4 published(const float* p) {
  typedef float rf2 __attribute__((ext_vector_type(2)));
  const unsigned long long* const q = reinterpret_cast<const unsigned long long*>(p);
  const rf2 a = __builtin_bit_cast(rf2, __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)),
            b = __builtin_bit_cast(rf2, __hip_atomic_load(q + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  return {a[0], a[1], b[0], b[1]};
}

// Meets the other waves once this one's LDS accesses are done; __syncthreads()
// would also wait for the loads that are on their way.
__device__ __forceinline__ void meet_in_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// Values that stay in registers: U steps and at most MOST turns of them for a wave, so
// U MOST XV pieces of 16 bytes of each token's, at most 16, or 8 that take more room once
// they are split.  WIDE: pairs of which 16 are not enough, up to 32.
template <int XE, int WE, bool WIDE = false>
struct Kept {
  static constexpr int XV = Format<XE, WE>::XV;
  static constexpr int PIECES = WIDE ? 32 : Format<XE, WE>::PARTS == 1 || XE == kElemPair ? 16 : 8;
  static constexpr int U = PIECES / XV < 4 ? PIECES / XV : WIDE || PIECES < 16 ? 2 : 4, MOST = PIECES / (U * XV);
  static constexpr int ROOM = 16 * 64 * (PIECES < 16 ? PIECES : 16);  // bytes of a wave's LDS
};

// One of the two products.  TYPE: the tokens'.  WIDE: the second one with up to 32 pieces
// of a token's values in a wave's registers, a kernel of its own, for with those in reach
// the others spill.
template <int TYPE, int WE, bool IN, bool WIDE = false>
__global__ __launch_bounds__(kThreads, 2) void expert_kernel(const LayerArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int XE = IN ? TYPE : kHidden<TYPE>;
  using Fm = Format<XE, WE>;
  using Keep = Kept<XE, WE, WIDE>;
  constexpr int XV = Fm::XV, U = Keep::U, MOST = Keep::MOST;
  // Values that do not: as many steps as registers hold.
  constexpr int STEP_REGS = 8 + 4 * XV, U0 = STEP_REGS <= (Fm::PAIR ? 12 : 16) ? 4 : STEP_REGS <= 32 ? 2 : 1;
  __shared__ union {
    char values[kWaves][Keep::ROOM];
    float sums[2][kWaves][2][16][kRows + 1];
    struct {
      short pair[kLayerPairs];  // of a choice: the pair that holds its products, or -1
      float share[kLayerPairs];
    } choice;
  } lds __attribute__((aligned(1024)));
  __shared__ union {
    Routing routing;
    int done[kThreads];  // blocks
  } table;
  __shared__ short lists[2][16];
  __shared__ int listed[2], last_blocks;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int depth = IN ? p.D : p.F, wide = IN ? p.F : p.D;  // the reduction, and the outputs of a token
  const bool gate = IN && p.gated;
  // Waves that divide the reduction of the same rows, and sets of rows.  A block is all
  // of a workgroup's rows.
  const int sets = IN ? p.sets_in : p.sets_out, sharers = kWaves / sets;
  const int set_of = wave / sharers, sharer = wave - set_of * sharers;
  const int per = (gate ? 16 : 32) * sets, blocks = (wide + per - 1) / per;
  if constexpr (IN) {  // for the second kernel, whatever the last call left
    const int counters = (p.D + 31) / 32;
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < counters; i += gridDim.x * kThreads) p.finished[i] = 0;
    if (blocks == 0) return;
  }

  FewPairs few;
  int entries;
  if (p.few) {
    few.init(p, lane);
    entries = few.entries();
  } else {
    entries = table.routing.init(p);
  }
  entries = __builtin_amdgcn_readfirstlane(entries);
  // This workgroup's units, a block of an entry each; where nothing is used, y alone
  // is left to be written, block by block.  Each entry that a workgroup begins costs
  // it a few microseconds of latency, so the entries get whole workgroups where that
  // leaves few over (32 experts, 16 tokens, 4 choices, 8 bits, 2048 by 1024, when it was
  // built: 54 us, and 63 with units in equal runs whatever the entry).
  const int owners = max(entries, IN ? 0 : 1), group = blockIdx.x;
  const int each = owners > 0 ? kGroups / owners : 0;
  int begin = 0, end = 0;  // fewer than 2^24 in all: 512 entries of 2^15 blocks
  if (each * owners * 8 >= kGroups * 7) {
    const int v = group / each, part = group - v * each;
    if (v < owners) {
      begin = v * blocks + blocks * part / each;
      end = v * blocks + blocks * (part + 1) / each;
    }
  } else {
    const long long all = owners * blocks;
    begin = static_cast<int>(all * group / kGroups);
    end = static_cast<int>(all * (group + 1) / kGroups);
  }
  const int rows_of = gate ? 2 * wide : wide;
  const int scale_blocks = (depth + 31) / 32;
  const void* const scale_all = IN ? p.scale_in : p.scale_out;

  int turn_of_list = 0;
  for (int unit = begin; entries > 0 && unit < end;) {
    const int v = unit / blocks, lo = unit - v * blocks, hi = min(blocks, lo + (end - unit));
    unit += hi - lo;
    int e = 0, set = 0;
    if (p.few) few.entry(v, e, set);
    else table.routing.entry(v, e, set);
    e = __builtin_amdgcn_readfirstlane(e);
    set = __builtin_amdgcn_readfirstlane(set);
    short* const list = lists[turn_of_list];
    auto find = [&] {
      if (wave == 0) {
        const int found = p.few ? few.list_pairs(e, 16 * set, list, lane)
                                : table.routing.list_pairs(e, 16 * set, p.T * p.top, list, lane);
        if (lane == 0) listed[turn_of_list] = found;
      }
      meet_in_lds();
      return __builtin_amdgcn_readfirstlane(listed[turn_of_list]);
    };
    const float* const row_scale = static_cast<const float*>(scale_all) + static_cast<long long>(e) * rows_of;

    auto work = [&](auto us, auto qs) {
      using R = Rows<XE, WE, decltype(us)::value, decltype(qs)::value>;
      R r;
      r.lane = lane;
      r.ld = IN ? p.ldw_in : p.ldw_out;
      r.scale_ld = scale_blocks;
      r.last = wide - 1;
      r.gap = gate ? 16 : 32;
      r.row_bytes = bytes_of_row<WE>(depth);
      r.steps = depth;
      r.full = depth / Fm::STEP;
      // The waves take equal runs of whole steps, and the last one what is left.
      constexpr int UR = decltype(us)::value;
      r.turns = max((r.full + UR * sharers - 1) / (UR * sharers), 1);
      r.first_step = sharer * r.turns * UR;
      r.end_step = min(r.full, r.first_step + r.turns * UR);
      r.tail = r.full * Fm::STEP < depth && sharer == sharers - 1;
      r.blocks = sets;
      r.block0 = set_of;
      r.values = IN ? p.x : p.h;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const long long row = gate ? b * static_cast<long long>(wide) : 0;
        r.rows[b] = (IN ? p.w_in + e * p.stride_in : p.w_out + e * p.stride_out) + row * r.ld;
        r.scales[b] = static_cast<const char*>(scale_all) + (static_cast<long long>(e) * rows_of + row) * scale_blocks;
      }
      typename R::Held held, second;
      if constexpr (R::KEPT) r.load(held, lo, 0);  // weights first, they take longest
      const int n = find();
      const int pair = list[lane % 16 < n ? lane % 16 : 0];
      r.x_off = lane % 16 >= n ? kRaggedMasked
                : IN           ? pair / p.top * static_cast<int>(p.ldx)
                               : pair * static_cast<int>(p.ldh);
      if constexpr (R::KEPT) {
        const rlds_t room = (rlds_t)&lds.values[wave][0];
        const int choices = IN ? p.top : 1;
        const long long ldx = IN ? p.ldx : p.ldh;
        r.send_values(room, 0, n, list, choices, ldx);
        r.load_second(second, lo, hi);
        r.template keep_values<0>(room, n);
        if constexpr (R::PASSES == 2) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the first pass is read
          r.send_values(room, 1, n, list, choices, ldx);
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
          r.template keep_values<1>(room, n);
        }
        meet_in_lds();  // sums may take their place
      } else {
        r.load(held, lo, 0);
      }
      r.run(lo, hi, held, second, [&](int block, rf4 (&acc)[2]) {
        float (&sums)[kWaves][2][16][kRows + 1] = lds.sums[block & 1];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) sums[wave][b][lane % 16][lane / 16 * 4 + i] = acc[b][i];
        meet_in_lds();
        for (int i = threadIdx.x; i < n * kRows * sets; i += kThreads) {
          const int row = i % kRows, c = i / kRows % n, first = i / kRows / n;
          const int to = list[c], base = block * sets + first;
          float v[2] = {};
          for (int w = first * sharers; w < (first + 1) * sharers; ++w)
#pragma unroll
            for (int b = 0; b < 2; ++b) v[b] += sums[w][b][c][row];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int out = gate ? base * 16 + row : base * 32 + b * 16 + row;
            if constexpr (IN && kHidden<TYPE> == kElemPair) {
              if (out >= wide) {
                if (out < (wide + 7) / 8 * 8) put_hidden<kElemPair>(p.h + to * p.ldh, out, 0.0f);
                continue;
              }
            } else {
              if (out >= wide) break;
            }
            if constexpr (WE == kElemI8) v[b] *= row_scale[gate ? b * wide + out : out];
            if constexpr (!IN) publish(p.z + to * p.ldz + out, v[b]);
            else if (!gate) put_hidden<kHidden<TYPE>>(p.h + to * p.ldh, out, silu(v[b]));
            else if (b == 1) put_hidden<kHidden<TYPE>>(p.h + to * p.ldh, out, silu(v[0]) * v[1]);
          }
        }
      });
      meet_in_lds();  // the sums are read: values or other sums may take their place
    };
    using std::integral_constant;
    const int turns = (depth / Fm::STEP + U * sharers - 1) / (U * sharers);
    const integral_constant<int, U> kept_steps;
    auto keep = [&] {
      if (MOST == 1 || turns <= 1) work(kept_steps, integral_constant<int, 1>{});
      else if (MOST == 2 || turns <= 2) work(kept_steps, integral_constant<int, MOST >= 2 ? 2 : 1>{});
      else work(kept_steps, integral_constant<int, MOST >= 4 ? 4 : 1>{});
    };
    if constexpr (WIDE) {
      if (turns > MOST) work(integral_constant<int, U0>{}, integral_constant<int, 0>{});
      else work(kept_steps, integral_constant<int, MOST>{});
    } else if constexpr (XE == kElemPair) {
      keep();  // or it would be WIDE
    } else {
      if (turns > MOST) work(integral_constant<int, U0>{}, integral_constant<int, 0>{});
      else keep();
    }
    turn_of_list ^= 1;
  }

  if constexpr (!IN) {
    // The last workgroup at a block of columns adds up each token's choices.  The
    // products are where every die sees them once the stores are done, which each
    // wave waits for before the barrier.
    const int pairs = p.T * p.top;
    for (int i = threadIdx.x; i < pairs; i += kThreads) {
      const int e = p.ids[i], t = i / p.top;
      int k = i;
      if (e >= 0 && e < p.experts)
        for (k = t * p.top; p.ids[k] != e; ++k) {}
      else
        k = -1;
      lds.choice.pair[i] = static_cast<short>(k);
      lds.choice.share[i] = p.share[i];
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    // As many blocks at a time as `done` holds.
    for (int at0 = begin; at0 < end; at0 += kThreads) {
      if (threadIdx.x == 0) last_blocks = 0;
      __syncthreads();
      if (at0 + static_cast<int>(threadIdx.x) < end) {
        const int block = (at0 + threadIdx.x) % blocks;
        if (entries == 0 || atomicAdd(&p.finished[block], 1) == entries - 1)
          table.done[atomicAdd(&last_blocks, 1)] = block;
      }
      __syncthreads();
      // Four columns a thread and two such at a time (four: up to a microsecond more).
      constexpr int QUADS = 2;
      const int row_quads = per / 4, quads = last_blocks * row_quads * p.T;  // token by token within a block
      for (int i0 = threadIdx.x; i0 < quads; i0 += QUADS * kThreads) {
        const float* from[QUADS];
        int col[QUADS], token[QUADS];
        rf4 y[QUADS] = {};
#pragma unroll
        for (int k = 0; k < QUADS; ++k) {
          const int i = min(i0 + k * kThreads, quads - 1);
          token[k] = i / row_quads % p.T;
          col[k] = table.done[i / (row_quads * p.T)] * per + i % row_quads * 4;
          from[k] = p.z + min(col[k], (wide - 1) / 4 * 4);  // rows of z are whole lines
        }
        for (int j0 = 0; j0 < p.top; j0 += 2) {
          rf4 z[2][QUADS];
          float share[2][QUADS];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < QUADS; ++k) {
              const int c = token[k] * p.top + min(j0 + j, p.top - 1), pair = lds.choice.pair[c];
              const bool there = pair >= 0 && j0 + j < p.top;
              share[j][k] = there ? lds.choice.share[c] : 0.0f;
              z[j][k] = published(from[k] + (there ? pair : 0) * p.ldz);
              if (!there) z[j][k] = rf4{};
            }
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < QUADS; ++k) y[k] += share[j][k] * z[j][k];
        }
#pragma unroll
        for (int k = 0; k < QUADS; ++k) {
          if (i0 + k * kThreads >= quads) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (col[k] + i >= wide) break;
            const long long at = token[k] * p.ldy + col[k] + i;
            if (TYPE == kElemF32 || p.out32) put<kElemF32>(p.y, at, y[k][i]);
            else put<TYPE>(p.y, at, y[k][i]);
          }
        }
      }
      __syncthreads();  // `done` is read
    }
  }
#endif
}

// The second product where few experts are used: a workgroup takes 16 columns of y
// for all tokens, its waves divide the used experts' rows, end to end, and what each
// finds for a token it adds up in LDS.  No workgroup waits for another's products
// (one token, 2 of 16 experts, 4096 by 2048: the layer takes 28 us so in bf16 and 17
// in 4 bits, 31 and 20 with the kernel above); with more experts than waves each wave
// has too many short pieces (8 bits, 2048 by 1024, 16 tokens, 4 choices of 32: 73 us
// and 59).  What a workgroup reads grows with the hidden width, by all tokens' values
// as well, narrow outputs leave units idle, and wide ones are more workgroups than
// units: several tokens come here where T F F <= 6000 D and D <= 4096 (2 of 8 experts,
// 4096 by 2048: 4 tokens in bf16 69 us and 72 above, 16 in 4 bits 45 and 38; 2048 by 4096:
// one token in bf16 36 and 38, two 52 and 49; 2048 by 2048: 4 tokens 50 and 47; 1024 by
// 512: 8 in 4 bits 17 and 20; 8192 by 1024: 8 in bf16 86 and 83).
constexpr int kDirectTokens = 16, kDirectExperts = kWaves;
constexpr double kDirectWidths = 6000;
template <int TYPE, int WE>
__global__ __launch_bounds__(kThreads, 2) void expert_out_kernel(const LayerArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int XE = kHidden<TYPE>;
  using Fm = Format<XE, WE>;
  constexpr int STEP_REGS = 4 + 4 * Fm::XV, U = STEP_REGS <= 8 ? 8 : STEP_REGS <= 16 ? 4 : STEP_REGS <= 24 ? 2 : 1;
  using R = Rows<XE, WE, U, 0, 1>;
  __shared__ float sums[kWaves][kDirectTokens][kRows + 1];
  __shared__ short lists[kWaves][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  FewPairs few;
  few.init(p, lane);
  for (int i = lane; i < kDirectTokens * (kRows + 1); i += 64) (&sums[wave][0][0])[i] = 0.0f;
  short* const list = lists[wave];
  const int entries = __builtin_amdgcn_readfirstlane(few.entries());
  const int block = blockIdx.x, scale_blocks = (p.F + 31) / 32;
  const int full = p.F / Fm::STEP, turns = max((full + U - 1) / U, 1);
  const int lo = turns * entries * wave / kWaves, hi = turns * entries * (wave + 1) / kWaves;
  for (int at = lo; at < hi;) {
    const int v = at / turns, from = at - v * turns, to = min(turns, from + (hi - at));
    at += to - from;
    int e = 0, set = 0;
    few.entry(v, e, set);
    e = __builtin_amdgcn_readfirstlane(e);
    const int n = __builtin_amdgcn_readfirstlane(few.list_pairs(e, 16 * set, list, lane));
    const int pair = list[lane % 16 < n ? lane % 16 : 0], token = pair / p.top;
    R r;
    r.lane = lane;
    r.ld = p.ldw_out;
    r.scale_ld = scale_blocks;
    r.last = p.D - 1;
    r.gap = 16;
    r.row_bytes = bytes_of_row<WE>(p.F);
    r.steps = p.F;
    r.full = full;
    r.turns = to - from;
    r.first_step = from * U;
    r.end_step = min(full, to * U);
    r.tail = to == turns && full * Fm::STEP < p.F;
    r.values = p.h;
    r.rows[0] = p.w_out + e * p.stride_out;
    r.scales[0] = static_cast<const char*>(p.scale_out) + static_cast<long long>(e) * p.D * scale_blocks;
    r.x_off = lane % 16 < n ? pair * static_cast<int>(p.ldh) : kRaggedMasked;
    float scale[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      scale[i] = WE == kElemI8 ? static_cast<const float*>(p.scale_out)[static_cast<long long>(e) * p.D +
                                                                        min(block * 16 + lane / 16 * 4 + i, p.D - 1)]
                               : 1.0f;
    typename R::Held held, second;
    r.load(held, block, 0);
    float share = 0.0f;  // of all the token's choices of e
    for (int j = token * p.top; j < (token + 1) * p.top; ++j) share += p.ids[j] == e ? p.share[j] : 0.0f;
    r.run(block, block + 1, held, second, [&](int, rf4 (&acc)[1]) {
      if (lane % 16 < n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[wave][token][lane / 16 * 4 + i] += acc[0][i] * scale[i] * share;
    });
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * kRows; i += kThreads) {
    const int t = i / kRows, col = block * 16 + i % kRows;
    if (col >= p.D) continue;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) y += sums[w][t][i % kRows];
    if (TYPE == kElemF32 || p.out32) put<kElemF32>(p.y, t * p.ldy + col, y);
    else put<TYPE>(p.y, t * p.ldy + col, y);
  }
#endif
}

template <int XE, int WE>
hipError_t launch_tokens(const LayerArgs& args, hipStream_t s) {
  LayerArgs a = args;
  void* values[] = {&a};
  const int pairs = a.T * a.top, slots = pairs < a.experts ? pairs : a.experts;
  a.few = pairs <= kFewPairs && slots <= kFewExperts;
  // Rows beside each other where few waves hold the reduction's values and there are
  // rows for two blocks a workgroup all the same.
  auto sets = [&](int hold, int depth, int wide, int per) {  // hold: steps that a wave can keep
    const int steps = depth / Format<XE, WE>::STEP;
    int n = 1;
    while (n < 4 && steps * 2 * n <= hold * kWaves &&
           static_cast<long long>(wide) * slots >= 2LL * kGroups * per * 2 * n)
      n *= 2;
    return n;
  };
  using In = Kept<XE, WE>;
  using Out = Kept<kHidden<XE>, WE>;
  constexpr int kInSteps = In::U * In::MOST, kOutSteps = Out::U * Out::MOST;
  a.sets_in = sets(kInSteps, a.D, a.F, a.gated ? 16 : 32);
  a.sets_out = sets(kOutSteps, a.F, a.D, 32);
  // Hidden widths that need more room, or that in 8 bits have more rows beside each other
  // with it (64 tokens, 4096 by 2048: 42.5 us for 45; in 4 bits alike).
  bool wide = false;
  if constexpr (kHidden<XE> == kElemPair) {
    using More = Kept<kHidden<XE>, WE, true>;
    const int more = sets(More::U * More::MOST, a.F, a.D, 32);
    wide = a.F / Format<XE, WE>::STEP > kOutSteps * kWaves || (WE == kElemI8 && more > a.sets_out);
    if (wide) a.sets_out = more;
  }
  const hipError_t err = hipLaunchKernel(reinterpret_cast<const void*>(&expert_kernel<XE, WE, true>), dim3(kGroups),
                                         dim3(kThreads), values, 0, s);
  if (err != hipSuccess) return err;
  const bool narrow = a.D <= kRows * kGroups && static_cast<double>(a.T) * a.F * a.F <= kDirectWidths * a.D;
  if (a.few && slots <= kDirectExperts && (a.T == 1 || (a.T <= kDirectTokens && narrow)))
    return hipLaunchKernel(reinterpret_cast<const void*>(&expert_out_kernel<XE, WE>),
                           dim3((static_cast<unsigned>(a.D) + kRows - 1) / kRows), dim3(kThreads), values, 0, s);
  const void* out = reinterpret_cast<const void*>(&expert_kernel<XE, WE, false>);
  if constexpr (kHidden<XE> == kElemPair)
    if (wide) out = reinterpret_cast<const void*>(&expert_kernel<XE, WE, false, true>);
  return hipLaunchKernel(out, dim3(kGroups), dim3(kThreads), values, 0, s);
}

template <int XE>
hipError_t launch_type(int weights, const LayerArgs& a, hipStream_t s) {
  if (weights == kElemI8) return launch_tokens<XE, kElemI8>(a, s);
  if (weights == kElemM4) return launch_tokens<XE, kElemM4>(a, s);
  return launch_tokens<XE, XE>(a, s);
}

}  // namespace

hipError_t expert_layer_launch(int type, int weights, const LayerArgs& a, hipStream_t s) {
  return type == kElemF32    ? launch_type<kElemF32>(weights, a, s)
         : type == kElemBF16 ? launch_type<kElemBF16>(weights, a, s)
                             : launch_type<kElemF16>(weights, a, s);
}

}  // namespace fp32gemm
