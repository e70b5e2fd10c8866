// expert_layer.hip -- a whole layer of experts for a few tokens, in two kernels.
//
//   h[t, j] = silu(G_e x_t) * (U_e x_t)   (or silu(U_e x_t)),   e = ids[t, j]
//   y[t] = sum_j share[t, j] D_e h[t, j]
//
// What bounds it is reading the chosen experts' weights, once each.  A wave
// reads 16 rows of weights, 64 bytes of each a step, straight to registers in the
// order in which the matrix instruction takes them: a lane's 16 bytes are its
// operand, so that neither LDS nor a barrier stands between memory and the
// products.  The expert's tokens, gathered, are the instruction's other operand,
// up to 16 of them at once; they come out of the L2.  The eight waves of a
// workgroup divide the reduction and add up in a fixed order.
#include "expert_layer.hpp"

#include "ragged_kernels.hpp"

namespace fp32gemm {
namespace {

constexpr int kWaves = 8, kThreads = kWaves * 64, kRows = 16;
static_assert(kThreads >= kLayerPairs, "a thread for each pair");

// What the ids say, in LDS.  A token that chose an expert more than once counts
// once, with the sum of its shares; ids out of range choose nothing.
struct Routing {
  int id[kLayerPairs];  // -1: none
  float share[kLayerPairs];
  int used[kLayerPairs];  // experts in the order in which the pairs name them
  int first[kLayerExperts];
  int count[kWaves];
};

__device__ __forceinline__ int lanes_below(unsigned long long m) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<unsigned>(m >> 32),
                                   __builtin_amdgcn_mbcnt_lo(static_cast<unsigned>(m), 0));
}

// Returns how many experts are used.  Every thread of the workgroup takes part.
__device__ __forceinline__ int find_routing(Routing& r, const LayerArgs& p) {
  const int i = threadIdx.x, pairs = p.T * p.top, wave = i >> 6;
  int e = -1;
  if (i < pairs) {
    e = p.ids[i];
    if (e < 0 || e >= p.experts) e = -1;
    r.id[i] = e;
    r.share[i] = p.share[i];
    if (e >= 0) r.first[e] = kLayerPairs;
  }
  __syncthreads();
  const int j = i < pairs ? i % p.top : 0;
  bool again = false;
  for (int k = 1; k <= j; ++k) again |= r.id[i - k] == e;
  if (again) e = -1;
  float share = 0.0f;
  if (e >= 0) {
    atomicMin(&r.first[e], i);  // whatever the order, the least stays
    for (int k = 0; j + k < p.top; ++k) share += r.id[i + k] == e ? r.share[i + k] : 0.0f;
  }
  __syncthreads();
  const bool leads = e >= 0 && r.first[e] == i;
  const unsigned long long m = __ballot(leads);
  if ((i & 63) == 0) r.count[wave] = __builtin_popcountll(m);
  if (i < pairs) {
    r.id[i] = e;
    r.share[i] = share;
  }
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += w < wave ? r.count[w] : 0;
    all += r.count[w];
  }
  if (leads) r.used[before + lanes_below(m)] = e;
  __syncthreads();
  return all;
}

// The pairs of expert e, in order, by one wave; returns how many.
__device__ __forceinline__ int list_pairs(const Routing& r, int e, int pairs, short* list, int lane) {
  int n = 0;
  for (int i0 = 0; i0 < pairs; i0 += 64) {
    const bool mine = i0 + lane < pairs && r.id[i0 + lane] == e;
    const unsigned long long m = __ballot(mine);
    if (mine) list[n + lanes_below(m)] = static_cast<short>(i0 + lane);
    n += __builtin_popcountll(m);
  }
  __builtin_amdgcn_wave_barrier();
  return n;
}

// ---------------------------------------------------------------------------
// How weights of format WE and values of type XE are multiplied.
template <int XE, int WE>
struct Format {
  static constexpr bool SAME = XE == WE, BLOCKS = WE == kElemM4;
  static constexpr int XS = elem_size(XE);
  static constexpr int PER = WE == kElemM4 ? 32 : 16 / elem_size(WE);  // weights of 16 bytes
  static constexpr int STEP = 4 * PER;                                  // of a step
  static constexpr int XV = PER * XS / 16;                              // 16-byte pieces of values for them
  // Narrow weights become bf16, exactly; values become a sum of one, two or
  // three bf16, exactly too, and are multiplied one after another.
  static constexpr int PARTS = SAME ? 1 : XE == kElemBF16 ? 1 : XE == kElemF16 ? 2 : 3;
  static constexpr int MMAS = SAME ? 1 : PER / 8;
};

__device__ __forceinline__ rb8 weights_of_8_bits(int lo, int hi) {
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

// Eight values as a sum of bf16.
template <int XE, int PARTS>
__device__ __forceinline__ void split_values(const ri4* raw, int m, rb8 (&part)[PARTS]) {
  if constexpr (XE == kElemBF16) {
    part[0] = __builtin_bit_cast(rb8, raw[m]);
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

// One step of one block of rows and one set of tokens.
template <int XE, int WE>
__device__ __forceinline__ void layer_mma(rf4& acc, const ri4& w, const ri4* x, float scale) {
  using Fm = Format<XE, WE>;
  if constexpr (Fm::SAME) {
    ragged_mma<XE, 16>(acc, w, x[0]);
  } else {
#pragma unroll
    for (int m = 0; m < Fm::MMAS; ++m) {
      rb8 wb, part[Fm::PARTS];
      if constexpr (Fm::BLOCKS) wb = weights_of_4_bits(static_cast<unsigned>(w[m]), scale);
      else wb = weights_of_8_bits(w[2 * m], w[2 * m + 1]);
      split_values<XE, Fm::PARTS>(x, m, part);
#pragma unroll
      for (int k = 0; k < Fm::PARTS; ++k) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, part[k], acc, 0, 0, 0);
    }
  }
}

// The reduction over one expert's rows by one wave: NB blocks of 16 rows, NT
// sets of 16 tokens, U steps on their way at a time and U more in hand.
template <int XE, int WE, int NB, int NT, int U>
struct Stream {
  using Fm = Format<XE, WE>;
  static constexpr int BYTES = 64 * U;  // of a row in a turn
  struct Held {
    ri4 w[U][NB];
    ri4 x[U][NT][Fm::XV];
    int s[U][NB];
  };
  const char* rows[NB];  // the first row of each block
  const char* scales[NB];
  int row_off[NB], scale_off[NB];  // the lane's row past them
  int x_off[NT];                   // the lane's token past `values`, or kRaggedMasked
  const char* values;
  int lane, row_bytes, steps;  // bytes of a row, reduction steps of it

  // A whole turn.
  __device__ __forceinline__ void load(Held& h, int turn) const {
    const int at = turn * BYTES + lane / 16 * 16;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const auto r = ragged_rsrc(rows[b], kRaggedMasked);
#pragma unroll
      for (int u = 0; u < U; ++u)
        h.w[u][b] = __builtin_bit_cast(ri4, __builtin_amdgcn_raw_buffer_load_b128(r, row_off[b] + at, u * 64, 0));
      if constexpr (Fm::BLOCKS) {
        const auto q = ragged_rsrc(scales[b], kRaggedMasked);
#pragma unroll
        for (int u = 0; u < U; ++u)
          h.s[u][b] = __builtin_amdgcn_raw_buffer_load_b8(q, scale_off[b] + turn * (U * 4) + lane / 16, u * 4, 0);
      }
    }
    const auto v = ragged_rsrc(values, kRaggedMasked);
    const int first = (turn * U * Fm::STEP + lane / 16 * Fm::PER) * Fm::XS;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int off = x_off[t] == kRaggedMasked ? kRaggedMasked : x_off[t] + first;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < Fm::XV; ++i)
          h.x[u][t][i] = __builtin_bit_cast(
              ri4, __builtin_amdgcn_raw_buffer_load_b128(v, off, (u * Fm::STEP * Fm::XS) + i * 16, 0));
    }
  }
  __device__ __forceinline__ void multiply(rf4 (&acc)[NB][NT], const Held& h) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float scale = 0.0f;
        if constexpr (Fm::BLOCKS) scale = __builtin_bit_cast(float, (h.s[u][b] & 255) << 23);
#pragma unroll
        for (int t = 0; t < NT; ++t) layer_mma<XE, WE>(acc[b][t], h.w[u][b], h.x[u][t], scale);
      }
  }
  // The last turn, which the rows do not fill: nothing past them is read, and
  // what is missing counts as zero.
  __device__ __forceinline__ void multiply_rest(rf4 (&acc)[NB][NT], int turn) const {
    const auto v = ragged_rsrc(values, kRaggedMasked);
#pragma unroll 1
    for (int u = 0; u < U; ++u) {
      const int at = turn * BYTES + u * 64 + lane / 16 * 16, n = row_bytes - at;  // valid bytes from here
      if (turn * BYTES + u * 64 >= row_bytes) break;
      ri4 w[NB];
      float scale[NB] = {};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const auto r = ragged_rsrc(rows[b], kRaggedMasked);
        if (row_bytes >= 16) {
          const int back = n > 0 && n < 16 ? 16 - n : 0;
          const ri4 raw = __builtin_bit_cast(ri4, __builtin_amdgcn_raw_buffer_load_b128(
                                                     r, n > 0 ? row_off[b] + at - back : kRaggedMasked, 0, 0));
          w[b] = __builtin_bit_cast(ri4, __builtin_bit_cast(unsigned __int128, raw) >> (8 * back));
        } else {
          unsigned __int128 bytes = 0;
#pragma unroll 1
          for (int i = 0; i < 16; ++i)
            bytes |= static_cast<unsigned __int128>(
                         __builtin_amdgcn_raw_buffer_load_b8(r, i < n ? row_off[b] + at + i : kRaggedMasked, 0, 0) & 255)
                     << (8 * i);
          w[b] = __builtin_bit_cast(ri4, bytes);
        }
        if constexpr (Fm::BLOCKS) {
          const int byte = __builtin_amdgcn_raw_buffer_load_b8(ragged_rsrc(scales[b], kRaggedMasked),
                                                               n > 0 ? scale_off[b] + at / 16 : kRaggedMasked, 0, 0);
          scale[b] = __builtin_bit_cast(float, (byte & 255) << 23);
        }
      }
      const int first = (turn * U + u) * Fm::STEP + lane / 16 * Fm::PER;  // the lane's reduction steps
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        ri4 x[Fm::XV];
#pragma unroll
        for (int i = 0; i < Fm::XV; ++i) {
          constexpr int EACH = 16 / Fm::XS;
          x[i] = ri4{};
#pragma unroll
          for (int k = 0; k < EACH; ++k) {
            const int step = first + i * EACH + k;
            const int off = x_off[t] == kRaggedMasked || step >= steps ? kRaggedMasked : x_off[t] + step * Fm::XS;
            if constexpr (Fm::XS == 4)
              x[i][k] = static_cast<int>(__builtin_amdgcn_raw_buffer_load_b32(v, off, 0, 0));
            else
              x[i][k / 2] |= static_cast<int>(static_cast<unsigned>(__builtin_amdgcn_raw_buffer_load_b16(v, off, 0, 0) & 0xFFFF)
                                              << (16 * (k & 1)));
          }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) layer_mma<XE, WE>(acc[b][t], w[b], x, scale[b]);
      }
    }
  }
  // Turns lo .. hi - 1.
  __device__ __forceinline__ void run(rf4 (&acc)[NB][NT], int lo, int hi) const {
    const int whole = min(hi, steps / (Fm::STEP * U));  // by the steps: an odd one is half a byte
    if (lo < whole) {
      Held a, b;
      load(a, lo);
      int t = lo;
      for (; t + 2 < whole; t += 2) {
        load(b, t + 1);
        multiply(acc, a);
        load(a, t + 2);
        multiply(acc, b);
      }
      if (t + 1 < whole) {
        load(b, t + 1);
        multiply(acc, a);
        multiply(acc, b);
      } else {
        multiply(acc, a);
      }
    }
    if (max(lo, whole) < hi) multiply_rest(acc, hi - 1);
  }
  static __device__ __forceinline__ int turns(int row_bytes) { return (row_bytes + BYTES - 1) / BYTES; }
};

template <int WE>
__device__ __forceinline__ int bytes_of_row(int steps) {
  return WE == kElemM4 ? (steps + 1) / 2 : steps * elem_size(WE);
}
// Sets of 16 tokens that share a reading of the weights: four, which is all of
// them, but one where splitting values takes the registers.
template <int XE, int WE>
constexpr int sets_at_once() {
  return Format<XE, WE>::PARTS == 1 ? 4 : 1;
}
// Calls work(sets, first token) for n gathered tokens.
template <int XE, int WE, class F>
__device__ __forceinline__ void for_tokens(int n, F work) {
  if constexpr (sets_at_once<XE, WE>() == 1) {
    for (int c = 0; c < n; c += 16) work(std::integral_constant<int, 1>{}, c);
  } else {
    if (n <= 16) work(std::integral_constant<int, 1>{}, 0);
    else if (n <= 32) work(std::integral_constant<int, 2>{}, 0);
    else work(std::integral_constant<int, 4>{}, 0);
  }
}
// Steps on their way at a time: four of 64 bytes, fewer where the values of many
// tokens, or their parts, fill the registers.
template <int XE, int WE, int NT>
constexpr int steps_at_once() {
  constexpr int values = Format<XE, WE>::XV * NT;
  return Format<XE, WE>::PARTS > 1 && values >= 4 ? 1 : values <= 4 ? 4 : values <= 8 ? 2 : 1;
}

__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

template <int XE>
__device__ __forceinline__ void put(char* p, long long i, float v) {
  if constexpr (XE == kElemF32) reinterpret_cast<float*>(p)[i] = v;
  else if constexpr (XE == kElemBF16) reinterpret_cast<__bf16*>(p)[i] = static_cast<__bf16>(v);
  else reinterpret_cast<_Float16*>(p)[i] = static_cast<_Float16>(v);
}

// ---------------------------------------------------------------------------
// h for one used expert (blockIdx.y) and one block of 16 rows of it, gate and up
// (without a gate: 32 rows).
template <int XE, int WE>
__global__ __launch_bounds__(kThreads, 2) void expert_in_kernel(const LayerArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ union {
    Routing routing;
    float sums[kWaves][2][kLayerTokens][kRows + 1];
  } lds;
  __shared__ short list[kLayerTokens];
  __shared__ int listed;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int used = find_routing(lds.routing, p);
  if (static_cast<int>(blockIdx.y) >= used) return;
  const int e = __builtin_amdgcn_readfirstlane(lds.routing.used[blockIdx.y]);
  const int pairs = p.T * p.top;
  if (wave == 0) {
    const int found = list_pairs(lds.routing, e, pairs, list, lane);
    if (lane == 0) listed = found;
  }
  __syncthreads();
  const int n = __builtin_amdgcn_readfirstlane(listed);

  const int first = blockIdx.x * (p.gated ? kRows : 2 * kRows);
  const int row_bytes = bytes_of_row<WE>(p.D);
  const long long blocks = (p.D + 31) / 32;  // scales of a row of 4-bit weights
  const int rows_of = p.gated ? 2 * p.F : p.F;
  auto work = [&](auto sets, int c0) {
    constexpr int NT = decltype(sets)::value, U = steps_at_once<XE, WE, NT>();
    using S = Stream<XE, WE, 2, NT, U>;
    S s;
    s.lane = lane;
    s.row_bytes = row_bytes;
    s.steps = p.D;
    s.values = p.x;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int f = min(p.gated ? first : first + b * kRows, p.F - 1);
      const int row = p.gated ? b * p.F + f : f;
      const int in = min(lane % 16, p.F - 1 - f);
      s.rows[b] = p.w_in + e * p.stride_in + row * p.ldw_in;
      s.row_off[b] = in * static_cast<int>(p.ldw_in);
      s.scales[b] = static_cast<const char*>(p.scale_in) + (static_cast<long long>(e) * rows_of + row) * blocks;
      s.scale_off[b] = in * static_cast<int>(blocks);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = c0 + t * 16 + lane % 16;
      s.x_off[t] = c < n ? list[min(c, kLayerTokens - 1)] / p.top * static_cast<int>(p.ldx) : kRaggedMasked;
    }
    rf4 acc[2][NT] = {};
    const int turns = S::turns(row_bytes);
    s.run(acc, turns * wave / kWaves, turns * (wave + 1) / kWaves);
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          lds.sums[wave][b][c0 + t * 16 + lane % 16][lane / 16 * 4 + i] = acc[b][t][i];
  };
  for_tokens<XE, WE>(n, work);
  __syncthreads();
  for (int i = threadIdx.x; i < n * kRows; i += kThreads) {
    const int c = i / kRows, row = i % kRows;
    float v[2] = {};
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v[b] += lds.sums[w][b][c][row];
    char* const h = p.h + list[c] * p.ldh;
    const float* const scale = static_cast<const float*>(p.scale_in) + static_cast<long long>(e) * rows_of;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int f = p.gated ? first + row : first + b * kRows + row;
      if (f >= p.F) break;
      if constexpr (WE == kElemI8) v[b] *= scale[p.gated ? b * p.F + f : f];
      if (!p.gated) put<XE>(h, f, silu(v[b]));
      else if (b == 1) put<XE>(h, f, silu(v[0]) * v[1]);
    }
  }
#endif
}

// 16 columns of y for all tokens.  The waves divide the used experts' rows, end
// to end; what each finds for a token it adds up in LDS.
template <int XE, int WE>
__global__ __launch_bounds__(kThreads, 2) void expert_out_kernel(const LayerArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ Routing routing;
  __shared__ float sums[kWaves][kLayerTokens][kRows + 1];
  __shared__ short list[kWaves][kLayerTokens];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int i = threadIdx.x; i < kWaves * kLayerTokens * (kRows + 1); i += kThreads) (&sums[0][0][0])[i] = 0.0f;
  const int used = __builtin_amdgcn_readfirstlane(find_routing(routing, p));  // ends with a barrier
  const int pairs = p.T * p.top;
  const int first = blockIdx.x * kRows, in = min(lane % 16, p.D - 1 - first);
  const int row_bytes = bytes_of_row<WE>(p.F);
  const long long blocks = (p.F + 31) / 32;
  // A turn of the shared division is four steps.
  constexpr int BYTES = 256;
  const int turns = (row_bytes + BYTES - 1) / BYTES;
  const long long all = static_cast<long long>(turns) * used;
  const int lo = static_cast<int>(all * wave / kWaves), hi = static_cast<int>(all * (wave + 1) / kWaves);
  for (int u = lo / max(turns, 1); u * turns < hi; ++u) {
    const int e = __builtin_amdgcn_readfirstlane(routing.used[u]);
    const int from = max(lo - u * turns, 0), to = min(hi - u * turns, turns);
    const int n = __builtin_amdgcn_readfirstlane(list_pairs(routing, e, pairs, list[wave], lane));
    auto work = [&](auto sets, int c0) {
      constexpr int NT = decltype(sets)::value, U = steps_at_once<XE, WE, NT>();
      using S = Stream<XE, WE, 1, NT, U>;
      S s;
      s.lane = lane;
      s.row_bytes = row_bytes;
      s.steps = p.F;
      s.values = p.h;
      s.rows[0] = p.w_out + e * p.stride_out + first * p.ldw_out;
      s.row_off[0] = in * static_cast<int>(p.ldw_out);
      s.scales[0] = static_cast<const char*>(p.scale_out) + (static_cast<long long>(e) * p.D + first) * blocks;
      s.scale_off[0] = in * static_cast<int>(blocks);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int c = c0 + t * 16 + lane % 16;
        s.x_off[t] = c < n ? list[wave][min(c, kLayerTokens - 1)] * static_cast<int>(p.ldh) : kRaggedMasked;
      }
      rf4 acc[1][NT] = {};
      constexpr int PER = BYTES / S::BYTES;
      s.run(acc, from * PER, min(to * PER, S::turns(row_bytes)));
      float scale[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        scale[i] = WE == kElemI8 ? static_cast<const float*>(p.scale_out)[static_cast<long long>(e) * p.D +
                                                                          min(first + lane / 16 * 4 + i, p.D - 1)]
                                 : 1.0f;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int c = c0 + t * 16 + lane % 16;
        if (c < n) {
          const int pair = list[wave][c];
          float* const to_sum = &sums[wave][pair / p.top][lane / 16 * 4];
#pragma unroll
          for (int i = 0; i < 4; ++i) to_sum[i] += acc[0][t][i] * scale[i] * routing.share[pair];
        }
      }
    };
    for_tokens<XE, WE>(n, work);
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * kRows; i += kThreads) {
    const int t = i / kRows, row = i % kRows;
    if (first + row >= p.D) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += sums[w][t][row];
    if (XE == kElemF32 || p.out32) put<kElemF32>(p.y, t * p.ldy + first + row, v);
    else put<XE>(p.y, t * p.ldy + first + row, v);
  }
#endif
}

template <int XE, int WE>
hipError_t launch_layer(const LayerArgs& args, hipStream_t s) {
  LayerArgs a = args;
  void* values[] = {&a};
  const unsigned per = a.gated ? kRows : 2 * kRows;
  const int pairs = a.T * a.top;
  const unsigned slots = static_cast<unsigned>(pairs < a.experts ? pairs : a.experts);
  if (slots > 0 && a.F > 0) {
    const hipError_t err =
        hipLaunchKernel(reinterpret_cast<const void*>(&expert_in_kernel<XE, WE>),
                        dim3((static_cast<unsigned>(a.F) + per - 1) / per, slots), dim3(kThreads), values, 0, s);
    if (err != hipSuccess) return err;
  }
  return hipLaunchKernel(reinterpret_cast<const void*>(&expert_out_kernel<XE, WE>),
                         dim3((static_cast<unsigned>(a.D) + kRows - 1) / kRows), dim3(kThreads), values, 0, s);
}

template <int XE>
hipError_t launch_type(int weights, const LayerArgs& a, hipStream_t s) {
  if (weights == kElemI8) return launch_layer<XE, kElemI8>(a, s);
  if (weights == kElemM4) return launch_layer<XE, kElemM4>(a, s);
  return launch_layer<XE, XE>(a, s);
}

}  // namespace

hipError_t expert_layer_launch(int type, int weights, const LayerArgs& a, hipStream_t s) {
  return type == kElemF32    ? launch_type<kElemF32>(weights, a, s)
         : type == kElemBF16 ? launch_type<kElemBF16>(weights, a, s)
                             : launch_type<kElemF16>(weights, a, s);
}

}  // namespace fp32gemm
