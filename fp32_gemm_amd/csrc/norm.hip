// norm.hip -- the root-mean-square norm of rows, with a residual's addition and
// an 8-bit output, and its gradient.
//
//   h = x + r,  s = (mean h^2 + eps)^(-1/2),  v = h w,  y = s v
//   scale = s max|v| / 127,  code = nearest(127 v / max|v|)
//   dx = s (g - n mean(g n)) + dh,  dw = sum over rows of dy n,  g = dy w, n = h s
//
// Sums of squares, s and the largest |v| are held in 64 bits, so that no row of
// finite numbers overflows and codes are those of the exact quotients.  h is a sum in 32
// bits, and one in 64 in rows where it is infinite in 32.  The largest
// |v| is looked for in 32 bits first; only the 16-byte pieces that may hold it, and
// codes next to a tie, are computed again in 64.
#include "norm.hpp"

#include "ragged_kernels.hpp"

namespace fp32gemm {
namespace {

template <int ELEM>
__device__ __forceinline__ float element(const char* p, long long i) {
  if constexpr (ELEM == kElemF32) return reinterpret_cast<const float*>(p)[i];
  else if constexpr (ELEM == kElemBF16) return static_cast<float>(reinterpret_cast<const __bf16*>(p)[i]);
  else return static_cast<float>(reinterpret_cast<const _Float16*>(p)[i]);
}
template <int ELEM>
__device__ __forceinline__ void set_element(char* p, long long i, float v) {
  if constexpr (ELEM == kElemF32) reinterpret_cast<float*>(p)[i] = v;
  else if constexpr (ELEM == kElemBF16) reinterpret_cast<__bf16*>(p)[i] = static_cast<__bf16>(v);
  else reinterpret_cast<_Float16*>(p)[i] = static_cast<_Float16>(v);
}

// Sixteen bytes of a row: PER elements from any byte on.
template <int ELEM>
struct Piece {
  static constexpr int PER = 16 / elem_size(ELEM);
  ri4 raw;
  __device__ __forceinline__ void load(const char* p, long long piece) { __builtin_memcpy(&raw, p + piece * 16, 16); }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (ELEM == kElemF32) return __builtin_bit_cast(rf4, raw)[i];
    else if constexpr (ELEM == kElemBF16) return static_cast<float>(__builtin_bit_cast(rb8, raw)[i]);
    else return static_cast<float>(__builtin_bit_cast(rh8, raw)[i]);
  }
  static __device__ __forceinline__ void store(char* p, long long piece, const float (&v)[PER]) {
    ri4 w;
    if constexpr (ELEM == kElemF32) {
      w = __builtin_bit_cast(ri4, rf4{v[0], v[1], v[2], v[3]});
    } else if constexpr (ELEM == kElemBF16) {
      rb8 b;
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = static_cast<__bf16>(v[i]);
      w = __builtin_bit_cast(ri4, b);
    } else {
      rh8 b;
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = static_cast<_Float16>(v[i]);
      w = __builtin_bit_cast(ri4, b);
    }
    __builtin_memcpy(p + piece * 16, &w, 16);
  }
};

// PER weights, of the rows' type or (W32) 32-bit floats; ones where there are none.
template <int ELEM, bool W32>
struct Weights {
  static constexpr int PER = Piece<ELEM>::PER, WORDS = W32 ? PER / 4 : 1;
  static constexpr int WELEM = W32 ? kElemF32 : ELEM;
  Piece<WELEM> part[WORDS];
  __device__ __forceinline__ void load(const char* w, long long piece) {
    constexpr int kOne = WELEM == kElemF32 ? 0x3F800000 : WELEM == kElemBF16 ? 0x3F803F80 : 0x3C003C00;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) part[i].raw = ri4{kOne, kOne, kOne, kOne};
    if (w != nullptr)
#pragma unroll
      for (int i = 0; i < WORDS; ++i) part[i].load(w, piece * WORDS + i);
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (W32) return part[i / 4][i % 4];
    else return part[0][i];
  }
  static __device__ __forceinline__ float one(const char* w, long long i) {
    return w == nullptr ? 1.0f : element<WELEM>(w, i);
  }
};

// A value of another lane, by the patterns of a sum over all lanes below.
template <int CTRL, int ROWS>
__device__ __forceinline__ double from_lane(double v, double none) {
  const ru2 w = __builtin_bit_cast(ru2, v), z = __builtin_bit_cast(ru2, none);
  return __builtin_bit_cast(double, ru2{static_cast<unsigned>(__builtin_amdgcn_update_dpp(z[0], w[0], CTRL, ROWS, 0xF, false)),
                                        static_cast<unsigned>(__builtin_amdgcn_update_dpp(z[1], w[1], CTRL, ROWS, 0xF, false))});
}
struct Add {
  static constexpr double kNone = 0.0;
  static __device__ __forceinline__ double of(double a, double b) { return a + b; }
};
struct Larger {
  static constexpr double kNone = 0.0;  // magnitudes
  static __device__ __forceinline__ double of(double a, double b) { return __builtin_fmax(a, b); }
};
// Over the wave, in lane 63.
template <class F>
__device__ __forceinline__ double over_wave(double v) {
  v = F::of(v, from_lane<0x111, 0xF>(v, F::kNone));
  v = F::of(v, from_lane<0x112, 0xF>(v, F::kNone));
  v = F::of(v, from_lane<0x114, 0xF>(v, F::kNone));
  v = F::of(v, from_lane<0x118, 0xF>(v, F::kNone));
  v = F::of(v, from_lane<0x142, 0xA>(v, F::kNone));
  v = F::of(v, from_lane<0x143, 0xC>(v, F::kNone));
  return v;
}
__device__ __forceinline__ double last_lane(double v) {
  const ru2 w = __builtin_bit_cast(ru2, v);
  return __builtin_bit_cast(double, ru2{static_cast<unsigned>(__builtin_amdgcn_readlane(w[0], 63)),
                                        static_cast<unsigned>(__builtin_amdgcn_readlane(w[1], 63))});
}
// Alike in all lanes, so not in the vector registers.
__device__ __forceinline__ double scalar(double v) {
  const ru2 w = __builtin_bit_cast(ru2, v);
  return __builtin_bit_cast(double, ru2{static_cast<unsigned>(__builtin_amdgcn_readfirstlane(w[0])),
                                        static_cast<unsigned>(__builtin_amdgcn_readfirstlane(w[1]))});
}
// Both over the THREADS threads of a row, known to all of them.  `room` holds two
// values a wave; calls that follow one another take rooms in turn.
template <class F, class G, int THREADS>
__device__ __forceinline__ void over_row(double& a, double& b, double (*room)[2]) {
  a = over_wave<F>(a);
  b = over_wave<G>(b);
  if constexpr (THREADS == 64) {
    a = last_lane(a);
    b = last_lane(b);
  } else {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 63) {
      room[wave][0] = a;
      room[wave][1] = b;
    }
    __syncthreads();
    a = room[0][0];
    b = room[0][1];
#pragma unroll
    for (int i = 1; i < THREADS / 64; ++i) {
      a = F::of(a, room[i][0]);
      b = G::of(b, room[i][1]);
    }
  }
}

// 1 / sqrt(m): the instruction's estimate and a step of Newton's method, which
// squares its error; exact limits at 0 and infinity.
__device__ __forceinline__ double inverse_root(double m) {
  const double y = __builtin_amdgcn_rsq(m);
  return m == 0.0 || m == __builtin_inf() ? y : y * __builtin_fma(-0.5 * m * y, y, 1.5);
}

// s in 32 bits, with a power of two of its own where it would leave their range; what
// is multiplied by it is multiplied by `before`, exactly, first.
struct Factor {
  float before, value;
  explicit __device__ __forceinline__ Factor(double s)
      : before(s < 0x1p-100 ? 0x1p-64f : s > 0x1p100 ? 0x1p64f : 1.0f),
        value(static_cast<float>(s < 0x1p-100 ? s * 0x1p64 : s > 0x1p100 ? s * 0x1p-64 : s)) {}
};

// A code decided in 32 bits is off by at most 127 * 5 * 2^-24 < 2^-14 before it is
// rounded (h, v, the largest |v|, its inverse and the product round once each).
// Values that near a tie, and rows whose inverse might leave the range, are multiplied
// in 64 bits, which is off by less than 2^-43, and those that are nearer than kTie
// even then are divided.
constexpr float kNearTie = 0x1p-14f;
constexpr double kTie = 0x1p-40;

constexpr int kNormBlocks = 1 << 23;  // workgroups in x; more rows go on in y
static_assert(256LL * kNormBlocks < 1LL << 32, "threads that HIP takes in a dimension");

// One row by THREADS threads of a workgroup of 256 or as many, KEEP pieces a thread in
// registers as they came; longer rows are read again.  H may be x or r itself: a thread has read
// what it overwrites, and where rows are read twice, H is written the second time.
// Memory-bound without codes: bf16 8192 x 8192 with a residual 102 us, 5.3 TB/s, as a
// copy runs.  With codes as well bound by the two reductions' latencies: 103 us for
// 7 bytes a value, 4.6 TB/s (weights read again for the codes: 114; the largest |v|
// in 64 bits throughout, and a division for every value near a tie: 116).
template <int ELEM, bool W32, int THREADS, int KEEP, bool CODES>
__global__ __launch_bounds__(THREADS < 256 ? 256 : THREADS) void rms_norm_kernel(const NormArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int ROWS = THREADS < 256 ? 256 / THREADS : 1;  // of a workgroup
  using P = Piece<ELEM>;
  using W = Weights<ELEM, W32>;
  constexpr int ES = elem_size(ELEM), PER = P::PER;
  __shared__ double room[3][THREADS / 64][2];
  const int in = threadIdx.x % THREADS;
  const long long block = static_cast<long long>(blockIdx.y) * kNormBlocks + blockIdx.x;
  const long long row = block * ROWS + threadIdx.x / THREADS;
  const bool live = row < p.M;  // uniform in a wave
  const char* const x = p.x + (live ? row : 0) * p.ldx * ES;
  const char* const r = p.r == nullptr ? nullptr : p.r + (live ? row : 0) * p.ldr * ES;
  const int pieces = live ? p.K / PER : 0, rest = live ? p.K % PER : 0;
  const long long last = static_cast<long long>(pieces) * PER + in;
  const bool one = in < rest;

  P kx[KEEP], kr[KEEP];
  W kw[CODES ? KEEP : 1];  // both passes of codes need them
#pragma unroll
  for (int j = 0; j < KEEP; ++j) {
    const int c = in + j * THREADS;
    kx[j].raw = kr[j].raw = ri4{};
    if (c < pieces) {
      kx[j].load(x, c);
      if (r) kr[j].load(r, c);
    }
  }
  if constexpr (CODES)
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if (in + j * THREADS < pieces) kw[j].load(p.w, in + j * THREADS);
  const float x1 = one ? element<ELEM>(x, last) : 0.0f, r1 = one && r ? element<ELEM>(r, last) : 0.0f;
  double sum = 0;
  // In 32 bits: the largest |v| of each piece that is kept, of the others, and NaN
  // once a value is not finite.
  float most[KEEP], most_rest = 0.0f, bad = 0.0f;
  auto take = [&](float a, float b, float w, float& largest) {
    const float h = a + b;
    const double d = h;
    sum = __builtin_fma(d, d, sum);
    if constexpr (CODES) {
      const float v = h * w;
      largest = __builtin_fmaxf(largest, __builtin_fabsf(v));
      bad = __builtin_fmaf(v, 0.0f, bad);
    }
  };
  auto take_piece = [&](const P& a, const P& b, const W& w, float& largest) {
#pragma unroll
    for (int i = 0; i < PER; ++i) take(a[i], b[i], CODES ? w.at(i) : 1.0f, largest);
  };
  // Calls with each piece past the kept ones, which is read again.
  auto others = [&](auto with) {
    for (int c = in + KEEP * THREADS; c < pieces; c += THREADS) {
      P a, b;
      a.load(x, c);
      b.raw = ri4{};
      if (r) b.load(r, c);
      W w;
      w.load(p.w, c);
      with(a, b, w, c);
    }
  };
#pragma unroll
  for (int j = 0; j < KEEP; ++j) {
    most[j] = 0.0f;
    const int c = in + j * THREADS;
    if (c < pieces) take_piece(kx[j], kr[j], kw[CODES ? j : 0], most[j]);
  }
  if (one) take(x1, r1, CODES ? W::one(p.w, last) : 1.0f, most_rest);
  others([&](const P& a, const P& b, const W& w, int) { take_piece(a, b, w, most_rest); });
  double top = 0;
  if constexpr (CODES) {
    float largest = most_rest;
#pragma unroll
    for (int j = 0; j < KEEP; ++j) largest = __builtin_fmaxf(largest, most[j]);
    top = bad == 0.0f ? largest : __builtin_inff();
  }
  over_row<Add, Larger, THREADS>(sum, top, room[0]);
  // Where x + r has passed 32 bits somewhere in the row, or is no number, the thread's
  // values one by one, from memory again: the registers are for the other rows.
  const bool past = __builtin_amdgcn_readfirstlane(r != nullptr && !(sum < __builtin_inf()));
  auto one_by_one = [&](auto with) {
#pragma unroll 1
    for (int c = in; c < pieces; c += THREADS)
#pragma unroll 1
      for (int i = 0; i < PER; ++i) with(static_cast<long long>(c) * PER + i);
    if (one) with(last);
  };
  if (past) {
    sum = 0;
    one_by_one([&](long long i) {
      const double d = static_cast<double>(element<ELEM>(x, i)) + static_cast<double>(element<ELEM>(r, i));
      sum = __builtin_fma(d, d, sum);
    });
    double none = 0;
    over_row<Add, Larger, THREADS>(sum, none, room[1]);
  }
  if constexpr (CODES) {
    // |v| in 32 bits is off by at most 2 * 2^-24 of itself, so the largest lies within
    // 2^-21 of the largest found.  Where that is tiny or no number, all are looked at.
    const double from = top > 0x1p-100 && top < __builtin_inf() ? top * (1.0 - 0x1p-21) : -1.0;
    double exact = 0, wrong = 0;
    auto look = [&](float a, float b, float w) {
      const double v = (static_cast<double>(a) + static_cast<double>(b)) * static_cast<double>(w);
      exact = __builtin_fmax(exact, __builtin_fabs(v));
      wrong = __builtin_fma(v, 0.0, wrong);
    };
    auto look_piece = [&](const P& a, const P& b, const W& w, int) {
#pragma unroll
      for (int i = 0; i < PER; ++i) look(a[i], b[i], w.at(i));
    };
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
      const int c = in + j * THREADS;
      if (c < pieces && most[j] >= from) look_piece(kx[j], kr[j], kw[j], c);
    }
    if (most_rest >= from) {
      if (one) look(x1, r1, W::one(p.w, last));
      others(look_piece);
    }
    if (wrong != 0.0) exact = __builtin_inf();
    double none = 0;
    over_row<Add, Larger, THREADS>(none, exact, room[2]);
    top = exact;
  }
  const double s = inverse_root(__builtin_fma(sum, p.inv_k, static_cast<double>(p.eps)));
  const Factor s32(s);
  const bool usable = top > 0.0 && top < __builtin_inf();
  const bool in_64 = !(top > 0x1p-100 && top < 0x1p100);
  const float inv = in_64 ? 0.0f : 127.0f / static_cast<float>(top);
  if (!live) return;
  if constexpr (CODES)
    if (in == 0) p.scale[row] = top == __builtin_inf() ? __builtin_nanf("") : static_cast<float>(top / 127.0 * s);

  char* const h = p.h ? p.h + row * p.ldh * ES : nullptr;
  char* y = p.y ? p.y + row * p.ldy * (p.out32 ? 4 : ES) : nullptr;
  if (past && y) {  // before H takes the place of x or r
    one_by_one([&](long long i) {
      const double d = static_cast<double>(element<ELEM>(x, i)) + static_cast<double>(element<ELEM>(r, i));
      const float v = static_cast<float>(d * s) * W::one(p.w, i);
      if (ELEM != kElemF32 && p.out32) reinterpret_cast<float*>(y)[i] = v;
      else set_element<ELEM>(y, i, v);
    });
    y = nullptr;
  }
  signed char* const q = CODES ? p.q + row * p.ldq : nullptr;
  // The inverse's estimate, after two steps of Newton's method.
  double inv64 = CODES ? __builtin_amdgcn_rcp(top) : 0.0;
  if constexpr (CODES) {
    inv64 = __builtin_fma(inv64, __builtin_fma(-top, inv64, 1.0), inv64);
    inv64 = __builtin_fma(inv64, __builtin_fma(-top, inv64, 1.0), inv64) * 127.0;
  }
  auto code64 = [&](float a, float b, float w) {
    const double v = (static_cast<double>(a) + static_cast<double>(b)) * static_cast<double>(w);
    double t = v * inv64;
    // (A tiny or huge `top` has no finite estimate: then t is no number near a tie's
    // distance, and is divided.)
    const double off = __builtin_fabs(t - __builtin_rint(t));
    if (!(off < 0.5 - kTie)) t = v * 127.0 / top;
    return usable ? static_cast<int>(__builtin_rint(t)) : 0;
  };
  auto write = [&](const P& a, const P& b, const W& w, int c) {
    float hv[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) hv[i] = a[i] + b[i];
    if (h) P::store(h, c, hv);
    if constexpr (CODES) {
      // t + kSnap is t rounded to an integer, in the low bits of the sum.
      constexpr float kSnap = 1.5f * (1 << 23);
      unsigned code[PER];
      float off = in_64 ? 1.0f : 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float t = hv[i] * w.at(i) * inv, n = t + kSnap;
        off = __builtin_fmaxf(off, __builtin_fabsf(t - (n - kSnap)));
        code[i] = __builtin_bit_cast(unsigned, n);
      }
      if (off > 0.5f - kNearTie)
#pragma unroll
        for (int i = 0; i < PER; ++i) code[i] = static_cast<unsigned>(code64(a[i], b[i], w.at(i)));
      unsigned o[PER / 4];
#pragma unroll
      for (int i = 0; i < PER / 4; ++i)  // the low bytes of four
        o[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(code[4 * i + 3], code[4 * i + 2], 0x0C0C0400u),
                                     __builtin_amdgcn_perm(code[4 * i + 1], code[4 * i], 0x0C0C0400u), 0x05040100u);
      __builtin_memcpy(q + static_cast<long long>(c) * PER, o, PER);
    }
    if (y) {
      float v[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = hv[i] * s32.before * s32.value * w.at(i);
      if (ELEM != kElemF32 && p.out32) __builtin_memcpy(y + static_cast<long long>(c) * PER * 4, v, PER * 4);
      else P::store(y, c, v);
    }
  };
#pragma unroll
  for (int j = 0; j < KEEP; ++j) {
    const int c = in + j * THREADS;
    if (c < pieces) {
      if constexpr (!CODES) kw[0].load(p.w, c);
      write(kx[j], kr[j], kw[CODES ? j : 0], c);
    }
  }
  if (one) {
    const float hv = x1 + r1, w = W::one(p.w, last);
    if (h) set_element<ELEM>(h, last, hv);
    if constexpr (CODES) q[last] = static_cast<signed char>(code64(x1, r1, w));
    if (y) {
      const float v = hv * s32.before * s32.value * w;
      if (ELEM != kElemF32 && p.out32) reinterpret_cast<float*>(y)[last] = v;
      else set_element<ELEM>(y, last, v);
    }
  }
  others(write);
#endif
}

// The gradient: a team of THREADS threads takes every teams-th row, with its sums
// for dw in registers, P pieces a thread (0: any length, the sums in memory), and
// leaves them as a row of `partial`.  Rows with a g past 32 bits, which s may bring back,
// are made in 64 bits, one value after another.  Memory-bound: bf16 16384 x 4096 with dh 114 us,
// 4.7 TB/s, and 5.6 us for the teams' sums.
template <int ELEM, bool W32, int THREADS, int PIECES>
__global__ __launch_bounds__(THREADS < 256 ? 256 : THREADS, PIECES == 4 ? 2 : 4) void rms_norm_grad_kernel(const NormGradArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  using P = Piece<ELEM>;
  using W = Weights<ELEM, W32>;
  constexpr int ES = elem_size(ELEM), PER = P::PER, HELD = PIECES ? PIECES : 1;
  constexpr int TEAMS = THREADS < 256 ? 256 / THREADS : 1;  // of a workgroup
  __shared__ double room[3][THREADS / 64][2];
  const int in = threadIdx.x % THREADS;
  const int team = blockIdx.x * TEAMS + threadIdx.x / THREADS;
  if (team >= p.teams) return;  // uniform in a wave; teams of several waves are whole workgroups
  const int pieces = p.K / PER, rest = p.K % PER;
  const long long last = static_cast<long long>(pieces) * PER + in;
  const bool one = in < rest;
  const float w1 = one ? W::one(p.w, last) : 0.0f;
  float* const part = p.partial ? p.partial + static_cast<long long>(team) * p.K : nullptr;
  float dw[HELD][PER] = {}, dw1 = 0.0f;
  W w[HELD];
  if constexpr (PIECES)
#pragma unroll
    for (int j = 0; j < HELD; ++j)
      if (in + j * THREADS < pieces) w[j].load(p.w, in + j * THREADS);
  int turn = 0;
  for (int row = team; row < p.M; row += p.teams, turn ^= 1) {
    const char* const h = p.h + row * p.ldh * ES;
    const char* const dy = p.dy + row * p.lddy * ES;
    const char* const dh = p.dh ? p.dh + row * p.lddh * ES : nullptr;
    char* const dx = p.dx + row * p.lddx * ES;
    double square = 0, dot = 0;
    float largest = 0.0f;
    auto take = [&](float a, float b, float wv) {
      const double d = a;
      const float g = b * wv;
      square = __builtin_fma(d, d, square);
      dot = __builtin_fma(d, static_cast<double>(g), dot);
      largest = __builtin_fmaxf(largest, __builtin_fabsf(g));
    };
    P kh[HELD], kd[HELD], kr[HELD];
    if constexpr (PIECES) {
#pragma unroll
      for (int j = 0; j < HELD; ++j) {
        const int c = in + j * THREADS;
        kh[j].raw = kd[j].raw = kr[j].raw = ri4{};
        if (c < pieces) {
          kh[j].load(h, c);
          kd[j].load(dy, c);
          if (dh) kr[j].load(dh, c);
        }
      }
#pragma unroll
      for (int j = 0; j < HELD; ++j)
        if (in + j * THREADS < pieces)
#pragma unroll
          for (int i = 0; i < PER; ++i) take(kh[j][i], kd[j][i], w[j].at(i));
    } else {
      for (int c = in; c < pieces; c += THREADS) {
        P a, b;
        a.load(h, c);
        b.load(dy, c);
        w[0].load(p.w, c);
#pragma unroll
        for (int i = 0; i < PER; ++i) take(a[i], b[i], w[0].at(i));
      }
    }
    const float h1 = one ? element<ELEM>(h, last) : 0.0f, d1 = one ? element<ELEM>(dy, last) : 0.0f;
    const float r1 = one && dh ? element<ELEM>(dh, last) : 0.0f;
    if (one) take(h1, d1, w1);
    // |n| is at most 2^15, so where no |g| is larger all that follows stays within 32
    // bits; else the row's sum becomes no number, which its other threads see.
    if (largest > 0x1p100f) dot = __builtin_nan("");
    over_row<Add, Add, THREADS>(square, dot, room[turn]);
    const bool past = __builtin_amdgcn_readfirstlane(!(__builtin_fabs(dot) < __builtin_inf()));
    const double s64 = scalar(inverse_root(__builtin_fma(square, p.inv_k, static_cast<double>(p.eps))));
    const Factor s(s64);
    const float mean = static_cast<float>(dot * p.inv_k * s64);
    auto grad = [&](float a, float b, float r, float wv, float& sums) {
      const float n = a * s.before * s.value;
      sums = __builtin_fmaf(b, n, sums);
      return __builtin_fmaf(__builtin_fmaf(-n, mean, b * wv) * s.before, s.value, r);
    };
    auto piece = [&](const P& a, const P& b, const P& r, const W& wv, int c, float (&sums)[PER]) {
      float v[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = grad(a[i], b[i], r[i], wv.at(i), sums[i]);
      if (!past) P::store(dx, c, v);
    };
    if constexpr (PIECES) {
#pragma unroll
      for (int j = 0; j < HELD; ++j)
        if (in + j * THREADS < pieces) piece(kh[j], kd[j], kr[j], w[j], in + j * THREADS, dw[j]);
    } else {
      for (int c = in; c < pieces; c += THREADS) {
        P a, b, r;
        a.load(h, c);
        b.load(dy, c);
        r.raw = ri4{};
        if (dh) r.load(dh, c);
        w[0].load(p.w, c);
        float sums[PER] = {};
        float* const at = part ? part + static_cast<long long>(c) * PER : nullptr;
        if (at && row != team) __builtin_memcpy(sums, at, PER * 4);
        piece(a, b, r, w[0], c, sums);
        if (at) __builtin_memcpy(at, sums, PER * 4);
      }
    }
    if (one) {
      const float v = grad(h1, d1, r1, w1, dw1);
      if (!past) set_element<ELEM>(dx, last, v);
    }
    if (past) {  // g or what it is made of passes 32 bits, or is no number: in 64, one by one, from memory
      int first = in;
      asm("" : "+v"(first));  // nothing of this is made ready, in registers, for the other rows
      auto one_by_one = [&](auto with) {
#pragma unroll 1
        for (int c = first; c < pieces; c += THREADS)
#pragma unroll 1
          for (int i = 0; i < PER; ++i) with(static_cast<long long>(c) * PER + i);
        if (first < rest) with(static_cast<long long>(pieces) * PER + first);
      };
      auto product = [&](long long i) {
        return static_cast<double>(element<ELEM>(dy, i)) * static_cast<double>(W::one(p.w, i));
      };
      double none = 0;
      dot = 0;
      one_by_one([&](long long i) { dot = __builtin_fma(static_cast<double>(element<ELEM>(h, i)), product(i), dot); });
      over_row<Add, Add, THREADS>(none, dot, room[2]);
      const double middle = dot * p.inv_k * s64;
      one_by_one([&](long long i) {
        const double n = static_cast<double>(element<ELEM>(h, i)) * s64;
        const float v = static_cast<float>(__builtin_fma(-n, middle, product(i)) * s64);
        set_element<ELEM>(dx, i, dh ? v + element<ELEM>(dh, i) : v);
      });
    }
  }
  if (part) {
    if constexpr (PIECES)
#pragma unroll
      for (int j = 0; j < HELD; ++j) {
        const int c = in + j * THREADS;
        if (c < pieces) __builtin_memcpy(part + static_cast<long long>(c) * PER, dw[j], PER * 4);
      }
    if (one) part[last] = dw1;
  }
#endif
}

// dw: the teams' sums, a column by sixteen threads that take every 16th team, in a
// fixed order.
constexpr int kSumColumns = 64, kSumGroups = 16;
constexpr int kSumBlocks = 1 << 21;  // workgroups in x; more columns go on in y
static_assert(1LL * kSumBlocks * kSumColumns * kSumGroups < 1LL << 32, "threads that HIP takes in a dimension");
template <int OUT>
__global__ __launch_bounds__(kSumColumns* kSumGroups) void sum_partial_kernel(const float* partial, int teams, int K,
                                                                             char* dw) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ float sums[kSumGroups][kSumColumns];
  const int c = threadIdx.x % kSumColumns, g = threadIdx.x / kSumColumns;
  const long long col = (static_cast<long long>(blockIdx.y) * kSumBlocks + blockIdx.x) * kSumColumns + c;
  float sum = 0.0f;
  if (col < K)
#pragma unroll 8
    for (int t = g; t < teams; t += kSumGroups) sum += partial[static_cast<long long>(t) * K + col];
  sums[g][c] = sum;
  __syncthreads();
  if (g == 0 && col < K) {
#pragma unroll
    for (int i = 1; i < kSumGroups; ++i) sum += sums[i][c];
    set_element<OUT>(dw, col, sum);
  }
#endif
}

template <int ELEM, bool W32, int THREADS, int KEEP>
const void* norm_kernel(bool codes) {
  return codes ? reinterpret_cast<const void*>(&rms_norm_kernel<ELEM, W32, THREADS, KEEP, true>)
               : reinterpret_cast<const void*>(&rms_norm_kernel<ELEM, W32, THREADS, KEEP, false>);
}

template <int ELEM, bool W32>
hipError_t launch_norm(const NormArgs& args, hipStream_t s) {
  // A wave takes rows of up to two pieces a lane, and where there are rows enough for
  // all waves of up to eight, or four with codes (16384 x 4096, residual and codes:
  // 115 us with eight, 94 by four waves); longer ones go to four waves, or, where
  // few rows leave the card idle and a row's instructions are what takes time, to eight
  // or sixteen (bf16 with a residual, codes: 256 x 8192 7.8 us, and 8.4 by four waves, 256 x
  // 16384 12.6 and 15.8, but 512 x 8192 14.1 and 11.8; Y: 1 x 16384 4.7 and 7.2, 512 x 8192
  // 8.5 and 9.2, but 1024 x 8192 13.3 and 12.9).
  const int pieces = args.K / Piece<ELEM>::PER;
  const bool codes = args.scale != nullptr;
  const bool wave = pieces <= 128 || (pieces <= (codes ? 256 : 512) && args.M >= 4096);
  const bool wide = !wave && args.M <= (codes ? 256 : 512) && pieces > 256 && pieces <= 2048;
  const int threads = wave ? 64 : !wide ? 256 : pieces <= 512 ? 512 : 1024, each = (pieces + threads - 1) / threads;
  const void* const kernel = wave ? (each <= 1   ? norm_kernel<ELEM, W32, 64, 1>(codes)
                                     : each <= 2 ? norm_kernel<ELEM, W32, 64, 2>(codes)
                                     : each <= 4 ? norm_kernel<ELEM, W32, 64, 4>(codes)
                                                 : norm_kernel<ELEM, W32, 64, 8>(codes))
                             : wide ? (pieces <= 512    ? norm_kernel<ELEM, W32, 512, 1>(codes)
                                       : pieces <= 1024 ? norm_kernel<ELEM, W32, 1024, 1>(codes)
                                                        : norm_kernel<ELEM, W32, 1024, 2>(codes))
                                  : (each <= 1   ? norm_kernel<ELEM, W32, 256, 1>(codes)
                                     : each <= 2 ? norm_kernel<ELEM, W32, 256, 2>(codes)
                                     : each <= 4 ? norm_kernel<ELEM, W32, 256, 4>(codes)
                                                 : norm_kernel<ELEM, W32, 256, 8>(codes));
  const unsigned blocks = wave ? (static_cast<unsigned>(args.M) + 3) / 4 : static_cast<unsigned>(args.M);
  const dim3 grid(blocks < kNormBlocks ? blocks : kNormBlocks, (blocks + kNormBlocks - 1) / kNormBlocks);
  NormArgs a = args;
  void* values[] = {&a};
  return hipLaunchKernel(kernel, grid, dim3(wide ? threads : 256), values, 0, s);
}

template <int ELEM, bool W32>
hipError_t launch_grad(const NormGradArgs& args, hipStream_t s) {
  const int pieces = args.K / Piece<ELEM>::PER;
  const void* kernel;
  int threads;
  auto pick = [&](int t, const void* k) {
    threads = t;
    kernel = k;
  };
  if (pieces <= 64) pick(64, reinterpret_cast<const void*>(&rms_norm_grad_kernel<ELEM, W32, 64, 1>));
  else if (pieces <= 128) pick(64, reinterpret_cast<const void*>(&rms_norm_grad_kernel<ELEM, W32, 64, 2>));
  else if (pieces <= 256) pick(256, reinterpret_cast<const void*>(&rms_norm_grad_kernel<ELEM, W32, 256, 1>));
  else if (pieces <= 512) pick(256, reinterpret_cast<const void*>(&rms_norm_grad_kernel<ELEM, W32, 256, 2>));
  else if (pieces <= 1024) pick(256, reinterpret_cast<const void*>(&rms_norm_grad_kernel<ELEM, W32, 256, 4>));
  else if (pieces <= 2048) pick(1024, reinterpret_cast<const void*>(&rms_norm_grad_kernel<ELEM, W32, 1024, 2>));
  else pick(1024, reinterpret_cast<const void*>(&rms_norm_grad_kernel<ELEM, W32, 1024, 0>));
  NormGradArgs a = args;
  void* values[] = {&a};
  const unsigned each = threads < 256 ? 256 / threads : 1;
  return hipLaunchKernel(kernel, dim3((static_cast<unsigned>(args.teams) + each - 1) / each),
                         dim3(threads < 256 ? 256 : threads), values, 0, s);
}

}  // namespace

int norm_teams(long long M) {
  // Every team writes a row of sums: one for at least 16 rows, so that they are
  // few beside the rows, but as many as there are rows until the card is full.
  const long long most = M / 16;
  return static_cast<int>(M <= 512 ? M : most < 512 ? 512 : most < 1024 ? most : 1024);
}

hipError_t rms_norm_launch(int type, bool w32, const NormArgs& a, hipStream_t s) {
  if (type == kElemF32) return launch_norm<kElemF32, false>(a, s);
  if (type == kElemBF16) return w32 ? launch_norm<kElemBF16, true>(a, s) : launch_norm<kElemBF16, false>(a, s);
  return w32 ? launch_norm<kElemF16, true>(a, s) : launch_norm<kElemF16, false>(a, s);
}

hipError_t rms_norm_grad_launch(int type, bool w32, int dw_type, char* dw, const NormGradArgs& a, hipStream_t s) {
  if (a.M > 0) {
    const hipError_t err =
        type == kElemF32    ? launch_grad<kElemF32, false>(a, s)
        : type == kElemBF16 ? (w32 ? launch_grad<kElemBF16, true>(a, s) : launch_grad<kElemBF16, false>(a, s))
                            : (w32 ? launch_grad<kElemF16, true>(a, s) : launch_grad<kElemF16, false>(a, s));
    if (err != hipSuccess) return err;
  }
  if (dw == nullptr) return hipSuccess;
  const float* partial = a.partial;
  int teams = a.M > 0 ? a.teams : 0, K = a.K;
  void* values[] = {&partial, &teams, &K, &dw};
  const void* const kernel = dw_type == kElemF32    ? reinterpret_cast<const void*>(&sum_partial_kernel<kElemF32>)
                             : dw_type == kElemBF16 ? reinterpret_cast<const void*>(&sum_partial_kernel<kElemBF16>)
                                                    : reinterpret_cast<const void*>(&sum_partial_kernel<kElemF16>);
  const unsigned blocks = (static_cast<unsigned>(K) + kSumColumns - 1) / kSumColumns;
  const dim3 grid(blocks < kSumBlocks ? blocks : kSumBlocks, (blocks + kSumBlocks - 1) / kSumBlocks);
  return hipLaunchKernel(kernel, grid, dim3(kSumColumns * kSumGroups), values, 0, s);
}

}  // namespace fp32gemm
