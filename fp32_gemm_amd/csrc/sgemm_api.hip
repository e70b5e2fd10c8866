// sgemm_api.hip -- the C ABI of libfp32_gemm_amd.so: argument validation,
// configuration table, tuned dispatch, introspection, and the host-side
// legality checker and index-map simulator.
//
// The computation is C = alpha*A*B + beta*C on row-major fp32 matrices with
// leading dimensions ("Warp Tiling: A Third Level of Tiling", section "The
// Kernel", epilogue; the launch there puts one workgroup on each output tile).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <vector>

#include "../../include/fp32_gemm.h"
#include "registry.hpp"

#include "instances_index.inc"  // generated by the build: kTables[]

namespace fp32gemm {
hipError_t launch_smem_tiling(const KernelArgs& a, hipStream_t stream);  // ladder.hip

namespace {

struct TunedRule {
  long long M, N, K;  // exact shape this rule was tuned on
  Tile tile;
};

#include "tuned_table.inc"  // kTuned[], kDefaultLarge, kDefaultMedium, kDefaultSmall

constexpr int kMaxRateTiles = 32;
struct RateRow {
  int M, N, K;                       // a measured shape (0, 0, 0: none)
  unsigned char pct[kMaxRateTiles];  // each column tile's rate there, % of the row's best
};

#include "measured_rates.inc"  // kRateTiles[], kScalarRows[], kVectorRows[]
static_assert(sizeof(kRateTiles) / sizeof(kRateTiles[0]) <= kMaxRateTiles, "too many rate columns");

constexpr long long kMaxDim = 1LL << 30;
constexpr long long kMaxLd = kMaxLeadingDim;  // see tile_config.hpp: sized with kMaxTileRows

const std::vector<const ConfigEntry*>& configs() {
  static const std::vector<const ConfigEntry*> list = [] {
    std::vector<const ConfigEntry*> v;
    for (const EntryTable& t : kTables)
      for (int i = 0; i < t.count; ++i)
        if (t.entries[i].launch_vec != nullptr) v.push_back(&t.entries[i]);
    return v;
  }();
  return list;
}

bool same_tile(const Tile& a, const Tile& b) {
  return a.BM == b.BM && a.BN == b.BN && a.BK == b.BK && a.WM == b.WM && a.WN == b.WN &&
         a.WNITER == b.WNITER && a.TM == b.TM && a.TN == b.TN && a.NT == b.NT &&
         a.path == b.path && a.swz == b.swz && a.opt == b.opt;
}

int find_tile(const Tile& t) {
  const auto& c = configs();
  for (size_t i = 0; i < c.size(); ++i)
    if (same_tile(c[i]->tile, t)) return static_cast<int>(i);
  return -1;
}

long long tiles_for(const Tile& t, long long M, long long N) {
  return ((M + t.BM - 1) / t.BM) * ((N + t.BN - 1) / t.BN);
}

// Configuration ids of the tuned rules and of the defaults, resolved once.
struct TunedIds {
  std::vector<int> rule;  // per kTuned entry; -1 if its tuple is not compiled
  int large, medium, small;
};

const TunedIds& tuned_ids() {
  static const TunedIds ids = [] {
    TunedIds t;
    for (const TunedRule& r : kTuned) t.rule.push_back(find_tile(r.tile));
    t.large = find_tile(kDefaultLarge);
    t.medium = find_tile(kDefaultMedium);
    t.small = find_tile(kDefaultSmall);
    return t;
  }();
  return ids;
}

// Which kernel of a configuration a launch runs: the float4 variant's (1) or
// the scalar variant's (0).  Their occupancies can differ, so the split plan
// asks for the right one.
int kernel_variant(bool vec) { return vec ? 1 : 0; }

long long resident_slots(int id, int kv);

// Share of the launched workgroup slots that do work when `tiles` workgroups
// run in waves of `slots` (1 when unknown).
double wave_efficiency(long long tiles, long long slots) {
  if (tiles <= 0 || slots <= 0) return 1.0;
  const long long waves = (tiles + slots - 1) / slots;
  return static_cast<double>(tiles) / static_cast<double>(waves * slots);
}

// Share of the resident workgroup slots that config `id` keeps busy on an
// M x N x K launch, counting the K split of a partly filled last wave that
// its split-K option would make (1 when the slots are unknown).  A launch
// that would split every tile counts as 0: its partial sums all go through
// atomics and a pre-pass, which costs more than the idle slots it fills.
double launch_efficiency(int id, long long M, long long N, long long K, bool vec) {
  const Tile& t = configs()[id]->tile;
  const long long tiles = tiles_for(t, M, N);
  const long long slots = resident_slots(id, kernel_variant(vec));
  if (slots <= 0) return 1.0;
  const long long nk = (std::max(K, 1LL) + t.BK - 1) / t.BK;
  const SplitPlan sp = split_plan(tiles, static_cast<int>(std::min(nk, 0x7FFFFFFFLL)), slots,
                                  (t.opt & kOptSplitK) != 0);
  if (sp.splits > 1 && sp.tiles_full == 0) return 0.0;
  return wave_efficiency(sp.tiles_full + (tiles - sp.tiles_full) * sp.splits, slots);
}

// Shapes without an exact rule, inside the measured-rate table's range,
// choose from that table rather than from the rules: its rows are seeded
// shapes on which every column tile was timed (the scalar variant's rows for
// shapes with N or K not a multiple of 4 or unaligned operands, the float4
// variant's for the rest), so a choice there rests on measurements near the
// shape instead of on the few rules.  The pick is the column with the
// highest weighted sum of log(rate / row's best) over the kRateNeighbours
// rows nearest in (log2 M, log2 N, log2 K), K's difference counting
// kRateKWeight times, each row weighted by exp(-squared distance): the tile
// that loses least near the shape.  A shape the table measured takes that
// row's fastest compiled tile.  A scalar-variant shape reads the float4 rows
// too, among the tiles whose scalar kernel keeps 16-byte loads
// (hybrid_scalar_tile): those kernels run at the float4 kernels' rates but
// for the first K slice, while the table's scalar rows were timed on an
// earlier scalar kernel with 4-byte loads.  Returns -1 if the table names no
// such compiled tile or holds no row to read.
constexpr int kRateNeighbours = 16;
constexpr double kRateKWeight = 0.5;
constexpr long long kRateMinMN = 128, kRateMinK = 32;  // below: the rules decide

struct PreparedRates {
  std::vector<int> col_id;                   // config id per column, -1 if not compiled
  std::vector<bool> col_hybrid;              // the column's tile is hybrid_scalar_tile
  std::vector<double> lm, ln, lk;            // log2 of each row's shape
  std::vector<std::vector<double>> logrel;   // per row, per column: log(pct / 100)
};

template <size_t R>
PreparedRates prepare_rates(const RateRow (&table)[R]) {
  PreparedRates p;
  for (const Tile& t : kRateTiles) {
    p.col_id.push_back(find_tile(t));
    p.col_hybrid.push_back(hybrid_scalar_tile(t));
  }
  for (const RateRow& r : table) {
    if (r.M <= 0 || r.N <= 0 || r.K <= 0) continue;
    p.lm.push_back(std::log2(static_cast<double>(r.M)));
    p.ln.push_back(std::log2(static_cast<double>(r.N)));
    p.lk.push_back(std::log2(static_cast<double>(r.K)));
    std::vector<double> v;
    for (size_t c = 0; c < p.col_id.size(); ++c)
      v.push_back(std::log(std::max<int>(r.pct[c], 1) / 100.0));
    p.logrel.push_back(std::move(v));
  }
  return p;
}

int select_by_rates(long long M, long long N, long long K, bool vec) {
  static const PreparedRates prep = prepare_rates(kVectorRows);
  auto usable = [&](size_t c) { return prep.col_id[c] >= 0 && (vec || prep.col_hybrid[c]); };
  const size_t rows = prep.lm.size(), cols = prep.col_id.size();
  if (rows == 0 || cols == 0) return -1;
  const double xm = std::log2(static_cast<double>(M)), xn = std::log2(static_cast<double>(N));
  const double xk = std::log2(static_cast<double>(std::max(K, 1LL)));
  // The nearest rows, kept sorted by distance (insertion into a short list).
  double near_d[kRateNeighbours];
  size_t near_i[kRateNeighbours];
  int n = 0;
  for (size_t i = 0; i < rows; ++i) {
    const double dm = xm - prep.lm[i], dn = xn - prep.ln[i], dk = xk - prep.lk[i];
    const double d = dm * dm + dn * dn + kRateKWeight * dk * dk;
    if (n == kRateNeighbours && d >= near_d[n - 1]) continue;
    int j = n < kRateNeighbours ? n++ : n - 1;
    for (; j > 0 && near_d[j - 1] > d; --j) {
      near_d[j] = near_d[j - 1];
      near_i[j] = near_i[j - 1];
    }
    near_d[j] = d;
    near_i[j] = i;
  }
  int pick = -1;
  double pick_score = 0.0;
  if (n > 0 && near_d[0] == 0.0) {  // a measured shape: its own fastest tile
    for (size_t c = 0; c < cols; ++c) {
      if (usable(c) && (pick < 0 || prep.logrel[near_i[0]][c] > pick_score)) {
        pick = prep.col_id[c];
        pick_score = prep.logrel[near_i[0]][c];
      }
    }
    if (pick >= 0) return pick;
  }
  double weight[kRateNeighbours];
  for (int j = 0; j < n; ++j) weight[j] = std::exp(-near_d[j]);
  for (size_t c = 0; c < cols; ++c) {
    if (!usable(c)) continue;
    double score = 0.0;
    for (int j = 0; j < n; ++j) score += weight[j] * prep.logrel[near_i[j]][c];
    if (pick < 0 || score > pick_score) {
      pick = prep.col_id[c];
      pick_score = score;
    }
  }
  return pick;
}

// Tuned choice: an exact-shape rule if the tuner recorded one; for a shape
// inside its range, the measured-rate table above.  Otherwise the
// candidates are the rules tuned on shapes that run the same variant
// (float4 or scalar), when there are any: for shapes of at least about a
// GFLOP, among the candidates whose launch keeps at least 85 % of the
// resident slots busy (the split of a partly filled last wave counted), the
// largest block tile wins, then the busier launch, then the nearer rule in
// (log M, log N, log K): a larger tile moves fewer bytes per flop.  Smaller
// shapes, and shapes no candidate fills, take the nearest candidate.  The
// defaults cover an empty table.
int select_config(long long M, long long N, long long K, bool vec) {
  const TunedIds& ids = tuned_ids();
  bool same_variant = false;
  for (size_t i = 0; i < ids.rule.size(); ++i) {
    const TunedRule& r = kTuned[i];
    if (ids.rule[i] >= 0 && r.M > 0 && r.N > 0 && r.K > 0 && ((r.K % 4 == 0 && r.N % 4 == 0) == vec))
      same_variant = true;
  }
  for (size_t i = 0; i < ids.rule.size(); ++i) {
    const TunedRule& r = kTuned[i];
    if (ids.rule[i] >= 0 && r.M == M && r.N == N && r.K == K) return ids.rule[i];
  }
  if (std::min(M, N) >= kRateMinMN && K >= kRateMinK) {
    const int id = select_by_rates(M, N, K, vec);
    if (id >= 0) return id;
  }
  // The fill rule below (largest tile that fills the device) pays where the
  // K loop is long enough for a large tile's operand reuse to matter; with a
  // short K the launch is bound by reading and writing C, and the nearest
  // rule (K weighs as much as M and N) finds the short-K rules instead.
  constexpr double kQuantisationFlop = 1073741824.0;
  constexpr long long kLongK = 256;
  const bool large = 2.0 * static_cast<double>(M) * static_cast<double>(N) * static_cast<double>(K) >=
                     kQuantisationFlop && K >= kLongK;
  int best = -1, best_fit = -1;
  double best_d = 0.0, fit_d = 0.0, fit_eff = 0.0;
  long long fit_area = 0;
  for (size_t i = 0; i < ids.rule.size(); ++i) {
    const TunedRule& r = kTuned[i];
    const int id = ids.rule[i];
    if (r.M <= 0 || r.N <= 0 || r.K <= 0 || id < 0) continue;
    if (r.M == M && r.N == N && r.K == K) return id;
    if (same_variant && ((r.K % 4 == 0 && r.N % 4 == 0) != vec)) continue;
    const double dm = std::log2(static_cast<double>(M) / r.M);
    const double dn = std::log2(static_cast<double>(N) / r.N);
    const double dk = std::log2(static_cast<double>(std::max(K, 1LL)) / r.K);
    const double d = dm * dm + dn * dn + dk * dk;
    if (best < 0 || d < best_d) { best = id; best_d = d; }
    if (!large || resident_slots(id, kernel_variant(vec)) <= 0) continue;  // no device: nearest rule
    const double eff = launch_efficiency(id, M, N, K, vec);
    if (eff < 0.85) continue;
    const long long area = static_cast<long long>(r.tile.BM) * r.tile.BN;
    if (best_fit < 0 || area > fit_area || (area == fit_area && eff > fit_eff) ||
        (area == fit_area && eff == fit_eff && d < fit_d)) {
      best_fit = id;
      fit_area = area;
      fit_eff = eff;
      fit_d = d;
    }
  }
  if (best_fit >= 0) return best_fit;
  if (best >= 0) return best;
  constexpr long long kWorkgroupsWanted = 256;  // one per compute unit
  const Tile* order[] = {&kDefaultLarge, &kDefaultMedium, &kDefaultSmall};
  const int order_ids[] = {ids.large, ids.medium, ids.small};
  for (int i = 0; i < 3; ++i)
    if (order_ids[i] >= 0 && tiles_for(*order[i], M, N) >= kWorkgroupsWanted) return order_ids[i];
  return ids.small >= 0 ? ids.small : 0;
}

int validate(long long M, long long N, long long K, const float* A, long long lda,
             const float* B, long long ldb, const float* C, long long ldc) {
  if (M < 0) return -1;
  if (N < 0) return -2;
  if (K < 0) return -3;
  if (A == nullptr && M > 0 && K > 0) return -5;
  if (lda < std::max(1LL, K)) return -6;
  if (B == nullptr && K > 0 && N > 0) return -7;
  if (ldb < std::max(1LL, N)) return -8;
  if (C == nullptr && M > 0 && N > 0) return -10;
  if (ldc < std::max(1LL, N)) return -11;
  if (M == 0 || N == 0) return SGEMM_OK;
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim || lda > kMaxLd || ldb > kMaxLd || ldc > kMaxLd)
    return SGEMM_ERR_UNSUPPORTED;
  // C's written extent must not meet the extents that are read.
  const uintptr_t c0 = reinterpret_cast<uintptr_t>(C);
  const uintptr_t c1 = c0 + static_cast<uintptr_t>(((M - 1) * ldc + N) * 4);
  if (K > 0) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(A);
    const uintptr_t a1 = a0 + static_cast<uintptr_t>(((M - 1) * lda + K) * 4);
    const uintptr_t b0 = reinterpret_cast<uintptr_t>(B);
    const uintptr_t b1 = b0 + static_cast<uintptr_t>(((K - 1) * ldb + N) * 4);
    if ((c0 < a1 && a0 < c1) || (c0 < b1 && b0 < c1)) return SGEMM_ERR_OVERLAP;
  }
  return SGEMM_OK;
}

bool vector_ok(long long N, long long K, const float* A, long long lda, const float* B,
               long long ldb, const float* C, long long ldc) {
  auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  return K % 4 == 0 && N % 4 == 0 && lda % 4 == 0 && ldb % 4 == 0 && ldc % 4 == 0 &&
         aligned(A) && aligned(B) && aligned(C);
}

thread_local int g_last_hip_error = 0;

constexpr int kMaxDevices = 64;
std::atomic<int> g_device_ok[kMaxDevices];  // 0 unknown, 1 gfx950, 2 not
std::atomic<int> g_device_cus[kMaxDevices];  // compute units, 0 unknown

int device_check() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return SGEMM_ERR_NO_DEVICE;
  if (dev < kMaxDevices) {
    const int known = g_device_ok[dev].load(std::memory_order_relaxed);
    if (known != 0) return known == 1 ? SGEMM_OK : SGEMM_ERR_NO_DEVICE;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return SGEMM_ERR_NO_DEVICE;
  const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < kMaxDevices) {
    g_device_cus[dev].store(prop.multiProcessorCount, std::memory_order_relaxed);
    g_device_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  }
  return ok ? SGEMM_OK : SGEMM_ERR_NO_DEVICE;
}

// Workgroups of config `id` (kernel `kv`, see kernel_variant) that fit on
// the current device at once; 0 if unknown.  Cached per configuration and
// kernel (all devices here are gfx950).
constexpr int kMaxConfigs = 4096;
std::atomic<int> g_blocks_per_cu[kMaxConfigs][2];

long long resident_slots(int id, int kv) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  if (device_check() != SGEMM_OK) return 0;
  const int cus = g_device_cus[dev].load(std::memory_order_relaxed);
  if (id < 0 || id >= kMaxConfigs || cus <= 0) return 0;
  if (kv < 0 || kv > 1) return 0;
  int per_cu = g_blocks_per_cu[id][kv].load(std::memory_order_relaxed);
  if (per_cu == 0) {
    const ConfigEntry* e = configs()[id];
    const void* sym = kv == 1 ? e->sym_vec() : e->sym_scalar();
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, sym, e->tile.NT, 0) != hipSuccess || n <= 0)
      return 0;
    per_cu = n;
    g_blocks_per_cu[id][kv].store(per_cu, std::memory_order_relaxed);
  }
  return static_cast<long long>(cus) * per_cu;
}

void fill_info(int id, const Tile& t, sgemm_config_t* out) {
  out->id = id;
  out->path = t.path;
  out->BM = t.BM; out->BN = t.BN; out->BK = t.BK; out->WM = t.WM; out->WN = t.WN;
  out->WNITER = t.WNITER; out->TM = t.TM; out->TN = t.TN; out->NT = t.NT; out->swz = t.swz;
  out->opt = t.opt;
  out->WMITER = wmiter_of(t, 64);
  out->WSUBM = t.WM / out->WMITER;
  out->WSUBN = t.WN / t.WNITER;
  out->acc_per_lane = acc_per_lane(t, 64);
  out->lds_bytes = lds_bytes(t, kGfx950);
  out->vgpr_estimate = vgpr_estimate(t, 64);
}

Tile tile_from(const int32_t* v) {
  return Tile{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8], v[9], v[10], v[11]};
}

// ---- host simulator --------------------------------------------------------

// Worst bank-conflict degree of one LDS instruction: lanes are served in
// phases of `phase` lanes; within a phase, distinct words that share a bank
// serialise (equal words are broadcast).
struct BankModel {
  int banks;
  int worst = 1;
  void instruction(const std::vector<std::vector<int>>& words_per_lane, int words_per_lane_n) {
    const int phase = std::max(1, banks / words_per_lane_n);
    const int lanes = static_cast<int>(words_per_lane.size());
    for (int p0 = 0; p0 < lanes; p0 += phase) {
      std::vector<std::vector<int>> bank(banks);
      for (int l = p0; l < std::min(lanes, p0 + phase); ++l)
        for (int w : words_per_lane[l]) {
          auto& b = bank[((w % banks) + banks) % banks];
          if (std::find(b.begin(), b.end(), w) == b.end()) b.push_back(w);
        }
      for (auto& b : bank) worst = std::max(worst, static_cast<int>(b.size()));
    }
  }
};

int simulate(const Tile& t, int banks, sgemm_sim_report_t* rep) {
  std::memset(rep, 0, sizeof(*rep));
  const int legal = check_tile(t, kGfx950);
  if (legal != kLegal) { rep->failed_check = legal; return legal; }
  // A k-sliced tuple's two wave groups are copies of one another: each runs
  // the index maps of the half-workgroup tuple, which is what is simulated.
  const Geom g = make_geom(kslices_of(t) > 1 ? half_tile(t) : t);
  const int waves = g.NT / 64;
  auto fail = [&](int n) { rep->failed_check = 100 + n; return 100 + n; };

  // Check 1: each output element of the block tile has exactly one owner.
  std::vector<int> own(g.BM * g.BN, 0);
  for (int w = 0; w < waves; ++w)
    for (int l = 0; l < 64; ++l)
      for (int e = 0; e < g.ACC; ++e) {
        const RC rc = owner(g, w, l, e);
        if (rc.r < 0 || rc.r >= g.BM || rc.c < 0 || rc.c >= g.BN) return fail(1);
        own[rc.r * g.BN + rc.c]++;
      }
  for (int x : own) if (x != 1) return fail(1);

  // LDS contents after one staging round: tag = 1 + element id.
  // A(m,k) -> m*BK + k; B(k,n) -> BM*BK + k*BN + n.
  std::vector<int> lds(g.STAGE, 0);
  auto tagA = [&](int m, int k) { return 1 + m * g.BK + k; };
  auto tagB = [&](int k, int n) { return 1 + g.BM * g.BK + k * g.BN + n; };

  // Checks 2-5 cover the register-staged As[k][m] layout, which direct-LDS
  // MFMA tuples do not use (both of their variants load into As[m][k];
  // checks 6-8).  Direct-LDS VALU tuples keep As[k][m]: check 9 fills the
  // stage from their load maps, and check 4 then reads it as the VALU inner
  // product does.
  BankModel st_a{banks}, st_b{banks}, rd_a{banks}, rd_b{banks};
  const bool staged = (g.opt & kOptDirectLds) == 0;
  const bool valu_direct = !staged && g.path == kPathValu;
  if (valu_direct) {
    for (int fpl : {4, 1}) {
      // Check 9: the A instructions (4 bytes per lane) and B instructions
      // (FPL floats per lane) fill each stage exactly once, lane l of
      // instruction i landing at float i*64 + l (A) or BK*SA + (i*64 + l)*FPL
      // (B), where the layout keeps the element the lane fetches.
      std::vector<int> dl(g.STAGE, 0), hit_a(g.BM * g.BK, 0), hit_b(g.BK * g.BN, 0);
      std::vector<int> cover_a(g.BM * g.BK / 64, 0), cover_b(g.BK * g.BN / (64 * fpl), 0);
      for (int w = 0; w < waves; ++w) {
        for (int j = 0; j < dma_ops_a(g, 1); ++j) {
          const int i = dma_op(g, w, j);
          if (i < 0 || i >= g.BM * g.BK / 64) return fail(9);
          cover_a[i]++;
          for (int l = 0; l < 64; ++l) {
            const MK a = dma_at_src(g, i, l);
            if (a.m < 0 || a.m >= g.BM || a.k < 0 || a.k >= g.BK) return fail(9);
            if (as_index(g, a.k, a.m) != i * 64 + l) return fail(9);
            hit_a[a.m * g.BK + a.k]++;
            dl[i * 64 + l] = tagA(a.m, a.k);
          }
        }
        for (int j = 0; j < dma_ops_b(g, fpl); ++j) {
          const int i = dma_op(g, w, j);
          if (i < 0 || i >= g.BK * g.BN / (64 * fpl)) return fail(9);
          cover_b[i]++;
          for (int l = 0; l < 64; ++l) {
            const KN b = dma_b_src(g, i, l, fpl);
            if (b.k < 0 || b.k >= g.BK || b.n < 0 || b.n % fpl != 0 || b.n + fpl > g.BN) return fail(9);
            const int pos = g.BM * g.BK + (i * 64 + l) * fpl;
            for (int q = 0; q < fpl; ++q) {
              if (dma_bs_index(g, b.k, b.n + q) != pos + q || bs_index(g, b.k, b.n + q) != pos + q)
                return fail(9);
              hit_b[b.k * g.BN + b.n + q]++;
              dl[pos + q] = tagB(b.k, b.n + q);
            }
          }
        }
      }
      for (int x : cover_a) if (x != 1) return fail(9);
      for (int x : cover_b) if (x != 1) return fail(9);
      for (int x : hit_a) if (x != 1) return fail(9);
      for (int x : hit_b) if (x != 1) return fail(9);
      if (fpl == 4) lds = dl;
    }
  }
  // Check 2: A staging covers BM x BK once, into As, without collisions.
  if (staged) {
    std::vector<int> hit(g.BM * g.BK, 0);
    for (int ps = 0; ps < g.PASSES_A; ++ps)
      for (int e = 0; e < 4; ++e) {
        for (int w = 0; w < waves; ++w) {
          std::vector<std::vector<int>> words(64);
          for (int l = 0; l < 64; ++l) {
            const int th = w * 64 + l;
            const int m = stage_a_row(g, th, ps), k = 4 * stage_a_kq(g, th) + e;
            if (m < 0 || m >= g.BM || k < 0 || k >= g.BK) return fail(2);
            hit[m * g.BK + k]++;
            const int idx = as_index(g, k, m);
            if (idx < 0 || idx >= g.BK * g.SA || lds[idx] != 0) return fail(2);
            lds[idx] = tagA(m, k);
            words[l].push_back(idx);
          }
          st_a.instruction(words, 1);
        }
      }
    for (int x : hit) if (x != 1) return fail(2);
  }
  // Check 3: B staging covers BK x BN once; float4 stores aligned and contiguous.
  if (staged) {
    std::vector<int> hit(g.BK * g.BN, 0);
    for (int ps = 0; ps < g.PASSES_B; ++ps)
      for (int w = 0; w < waves; ++w) {
        std::vector<std::vector<int>> words(64);
        for (int l = 0; l < 64; ++l) {
          const int th = w * 64 + l;
          const int k = stage_b_row(g, th, ps), c = 4 * stage_b_nq(g, th);
          if (k < 0 || k >= g.BK || c < 0 || c + 3 >= g.BN) return fail(3);
          const int idx = bs_index(g, k, c);
          if (idx % 4 != 0 || idx < g.BK * g.SA || idx + 3 >= g.STAGE) return fail(3);
          for (int q = 0; q < 4; ++q) {
            if (bs_index(g, k, c + q) != idx + q || lds[idx + q] != 0) return fail(3);
            hit[k * g.BN + c + q]++;
            lds[idx + q] = tagB(k, c + q);
            words[l].push_back(idx + q);
          }
        }
        st_b.instruction(words, 4);
      }
    for (int x : hit) if (x != 1) return fail(3);
  }

  // Check 4: fragment reads return the operands each accumulator needs, and
  // every accumulator sees each k of the slice exactly once.
  for (int w = 0; (staged || valu_direct) && w < waves; ++w) {
    const int wr0 = wave_row0(g, w), wc0 = wave_col0(g, w);
    std::vector<int> kcount(64 * g.ACC * g.BK, 0);
    if (g.path == kPathValu) {
      for (int k = 0; k < g.BK; ++k) {
        // regM / regN as the kernel reads them (128-bit reads).
        std::vector<std::vector<int>> rm(64), rn(64);
        for (int wm = 0; wm < g.WMITER; ++wm)
          for (int i = 0; i < g.TM; i += 4) {
            std::vector<std::vector<int>> words(64);
            for (int l = 0; l < 64; ++l) {
              const int m = wr0 + valu_m(g, l, wm, i);
              const int idx = as_index(g, k, m);
              if (idx % 4 != 0) return fail(4);
              for (int q = 0; q < 4; ++q) {
                if (as_index(g, k, m + q) != idx + q) return fail(4);
                rm[l].push_back(lds[idx + q]);
                words[l].push_back(idx + q);
              }
            }
            rd_a.instruction(words, 4);
          }
        for (int wn = 0; wn < g.WNITER; ++wn)
          for (int j = 0; j < g.TN; j += 4) {
            std::vector<std::vector<int>> words(64);
            for (int l = 0; l < 64; ++l) {
              const int n = wc0 + valu_n(g, l, wn, j);
              const int idx = bs_index(g, k, n);
              if (idx % 4 != 0) return fail(4);
              for (int q = 0; q < 4; ++q) {
                if (bs_index(g, k, n + q) != idx + q) return fail(4);
                rn[l].push_back(lds[idx + q]);
                words[l].push_back(idx + q);
              }
            }
            rd_b.instruction(words, 4);
          }
        for (int l = 0; l < 64; ++l)
          for (int wm = 0; wm < g.WMITER; ++wm)
            for (int i = 0; i < g.TM; ++i)
              for (int wn = 0; wn < g.WNITER; ++wn)
                for (int j = 0; j < g.TN; ++j) {
                  const int e = valu_acc_index(g, wm, i, wn, j);
                  const RC rc = owner(g, w, l, e);
                  if (rm[l][wm * g.TM + i] != tagA(rc.r, k)) return fail(4);
                  if (rn[l][wn * g.TN + j] != tagB(k, rc.c)) return fail(4);
                  kcount[(l * g.ACC + e) * g.BK + k]++;
                }
      }
    } else {
      const int blk = mfma_blk(g), kstep = mfma_kstep(g), regs = mfma_regs(g);
      for (int kk = 0; kk < g.BK; kk += kstep) {
        // Fragment registers as the kernel loads them.
        std::vector<std::vector<int>> fa(64, std::vector<int>(g.WMITER)),
            fb(64, std::vector<int>(g.WNITER));
        for (int wm = 0; wm < g.WMITER; ++wm) {
          std::vector<std::vector<int>> words(64);
          for (int l = 0; l < 64; ++l) {
            const int k = kk + mfma_frag_slot(g, l);
            const int idx = as_index(g, k, wr0 + wm * blk + mfma_frag_row(g, l));
            if (idx < 0 || idx >= g.BK * g.SA) return fail(4);
            fa[l][wm] = lds[idx];
            words[l].push_back(idx);
          }
          rd_a.instruction(words, 1);
        }
        for (int wn = 0; wn < g.WNITER; ++wn) {
          std::vector<std::vector<int>> words(64);
          for (int l = 0; l < 64; ++l) {
            const int k = kk + mfma_frag_slot(g, l);
            const int idx = bs_index(g, k, wc0 + wn * blk + mfma_frag_row(g, l));
            if (idx < g.BK * g.SA || idx >= g.STAGE) return fail(4);
            fb[l][wn] = lds[idx];
            words[l].push_back(idx);
          }
          rd_b.instruction(words, 1);
        }
        // Model of the instruction: D[i][j] += sum_s A[i][s] * B[s][j], where
        // A[i][s] comes from the lane with (frag_row, slot) = (i, s) and
        // B[s][j] from the lane with (frag_row, slot) = (j, s).
        auto lane_of = [&](int row, int s) { return s * blk + row; };
        for (int l = 0; l < 64; ++l)
          for (int wm = 0; wm < g.WMITER; ++wm)
            for (int wn = 0; wn < g.WNITER; ++wn)
              for (int r = 0; r < regs; ++r) {
                const int e = (wm * g.WNITER + wn) * regs + r;
                const RC rc = owner(g, w, l, e);
                const int i = mfma_out_row(g, l, r), j = mfma_out_col(g, l);
                for (int s = 0; s < kstep; ++s) {
                  const int ta = fa[lane_of(i, s)][wm], tb = fb[lane_of(j, s)][wn];
                  // Decode k from the A tag and require the matching B tag.
                  const int ia = ta - 1;
                  const int ma = ia / g.BK, ka = ia % g.BK;
                  if (ta <= 0 || ta > g.BM * g.BK || ma != rc.r) return fail(4);
                  if (tb != tagB(ka, rc.c)) return fail(4);
                  kcount[(l * g.ACC + e) * g.BK + ka]++;
                }
              }
      }
    }
    for (int x : kcount) if (x != 1) return fail(5);
  }

  if ((g.opt & kOptDirectLds) && g.path != kPathValu) {
    // Both variants stage with direct-LDS loads into As[m][k]: 16-byte loads
    // (FPL = 4 floats per lane) in the float4 variant, 4-byte loads (FPL = 1)
    // in the scalar one; the LDS layout and the fragment reads are shared.
    // Because each FPL is checked to land every element at dma_as_index /
    // dma_bs_index, the two may also be mixed, as the scalar variant's
    // hybrid kernels do (A at FPL 1 in slice 0 and 4 after it, B at either).
    BankModel dr_a{banks}, dr_b{banks};
    for (int fpl : {4, 1}) {
      // Check 6: the A instructions fill the A stage exactly once, lane l of
      // instruction i landing at float (i*64 + l)*FPL, which must be where the
      // layout keeps the elements the lane fetches.
      std::vector<int> dl(g.STAGE, 0);
      std::vector<int> cover(g.STAGE / (64 * fpl), 0);
      std::vector<int> hit_a(g.BM * g.BK, 0), hit_b(g.BK * g.BN, 0);
      for (int w = 0; w < waves; ++w) {
        for (int j = 0; j < dma_ops_a(g, fpl); ++j) {
          const int i = dma_op(g, w, j);
          if (i < 0 || i >= g.BM * g.BK / (64 * fpl)) return fail(6);
          cover[i]++;
          for (int l = 0; l < 64; ++l) {
            const MK s = dma_a_src(g, i, l, fpl);
            if (s.m < 0 || s.m >= g.BM || s.k < 0 || s.k % fpl != 0 || s.k + fpl > g.BK) return fail(6);
            for (int q = 0; q < fpl; ++q) {
              hit_a[s.m * g.BK + s.k + q]++;
              if (dma_as_index(g, s.m, s.k + q) != (i * 64 + l) * fpl + q) return fail(6);
              dl[(i * 64 + l) * fpl + q] = tagA(s.m, s.k + q);
            }
          }
        }
        // Check 7: the same for B into Bs[k][n] (after the A stage).
        for (int j = 0; j < dma_ops_b(g, fpl); ++j) {
          const int i = dma_op(g, w, j);
          if (i < 0 || i >= g.BK * g.BN / (64 * fpl)) return fail(7);
          cover[g.BM * g.BK / (64 * fpl) + i]++;
          for (int l = 0; l < 64; ++l) {
            const KN s = dma_b_src(g, i, l, fpl);
            if (s.k < 0 || s.k >= g.BK || s.n < 0 || s.n % fpl != 0 || s.n + fpl > g.BN) return fail(7);
            const int pos = g.BM * g.BK + (i * 64 + l) * fpl;
            for (int q = 0; q < fpl; ++q) {
              hit_b[s.k * g.BN + s.n + q]++;
              if (dma_bs_index(g, s.k, s.n + q) != pos + q) return fail(7);
              dl[pos + q] = tagB(s.k, s.n + q);
            }
          }
        }
      }
      for (int x : cover) if (x != 1) return fail(6);
      for (int x : hit_a) if (x != 1) return fail(6);
      for (int x : hit_b) if (x != 1) return fail(7);

      // Check 8: the k-group fragment reads feed every accumulator each k of
      // the slice exactly once with the matching A and B elements.
      const int blk = mfma_blk(g), slots = dma_slots(g), regs = mfma_regs(g);
      for (int w = 0; w < waves; ++w) {
        const int wr0 = wave_row0(g, w), wc0 = wave_col0(g, w);
        std::vector<int> kcount(64 * g.ACC * g.BK, 0);
        for (int kg = 0; kg < g.BK / dma_kgroup(g); ++kg) {
          std::vector<std::vector<int>> fa(64, std::vector<int>(g.WMITER * 4)),
              fb(64, std::vector<int>(4 * g.WNITER));
          for (int wm = 0; wm < g.WMITER; ++wm) {
            std::vector<std::vector<int>> words(64);
            for (int l = 0; l < 64; ++l) {
              const int m = wr0 + wm * blk + l % blk;
              const int idx = dma_as_index(g, m, dma_k(g, kg, l / blk, 0));
              if (idx < 0 || idx % 4 != 0 || idx + 3 >= g.BM * g.BK) return fail(8);
              for (int q = 0; q < 4; ++q) {
                fa[l][wm * 4 + q] = dl[idx + q];
                words[l].push_back(idx + q);
              }
            }
            if (fpl == 4) dr_a.instruction(words, 4);
          }
          for (int q = 0; q < 4; ++q)
            for (int wn = 0; wn < g.WNITER; ++wn) {
              std::vector<std::vector<int>> words(64);
              for (int l = 0; l < 64; ++l) {
                const int idx = dma_bs_index(g, dma_k(g, kg, l / blk, q), wc0 + wn * blk + l % blk);
                if (idx < g.BM * g.BK || idx >= g.STAGE) return fail(8);
                fb[l][q * g.WNITER + wn] = dl[idx];
                words[l].push_back(idx);
              }
              if (fpl == 4) dr_b.instruction(words, 1);
            }
          for (int l = 0; l < 64; ++l)
            for (int wm = 0; wm < g.WMITER; ++wm)
              for (int wn = 0; wn < g.WNITER; ++wn)
                for (int r = 0; r < regs; ++r) {
                  const int e = (wm * g.WNITER + wn) * regs + r;
                  const RC rc = owner(g, w, l, e);
                  const int i = mfma_out_row(g, l, r), j = mfma_out_col(g, l);
                  for (int q = 0; q < 4; ++q)
                    for (int s2 = 0; s2 < slots; ++s2) {
                      const int ta = fa[s2 * blk + i][wm * 4 + q];
                      const int tb = fb[s2 * blk + j][q * g.WNITER + wn];
                      const int ia = ta - 1;
                      const int ma = ia / g.BK, ka = ia % g.BK;
                      if (ta <= 0 || ta > g.BM * g.BK || ma != rc.r) return fail(8);
                      if (tb != tagB(ka, rc.c)) return fail(8);
                      kcount[(l * g.ACC + e) * g.BK + ka]++;
                    }
                }
        }
        for (int x : kcount) if (x != 1) return fail(8);
      }
    }
    rep->dma_read_a_ways = dr_a.worst;
    rep->dma_read_b_ways = dr_b.worst;
  }
  rep->store_a_ways = st_a.worst;
  rep->store_b_ways = st_b.worst;
  rep->read_a_ways = rd_a.worst;
  rep->read_b_ways = rd_b.worst;
  return 0;
}

}  // namespace

void set_last_hip_error(hipError_t e) { g_last_hip_error = static_cast<int>(e); }  // ragged_api.hip
}  // namespace fp32gemm

using namespace fp32gemm;

extern "C" {

int sgemm_num_configs(void) { return static_cast<int>(configs().size()); }

int sgemm_config_info(int32_t id, sgemm_config_t* out) {
  if (out == nullptr || id < 0 || id >= sgemm_num_configs()) return SGEMM_ERR_BAD_CONFIG;
  fill_info(id, configs()[id]->tile, out);
  return SGEMM_OK;
}

int sgemm_plan(int64_t M, int64_t N, int64_t K, const float* A, int64_t lda, const float* B,
               int64_t ldb, const float* C, int64_t ldc, int32_t cfg_id, sgemm_plan_t* out) {
  const int rc = validate(M, N, K, A, lda, B, ldb, C, ldc);
  if (rc != SGEMM_OK) return rc;
  if (cfg_id >= sgemm_num_configs()) return SGEMM_ERR_BAD_CONFIG;
  const bool vec = vector_ok(N, K, A, lda, B, ldb, C, ldc);
  const int id = cfg_id >= 0 ? cfg_id : select_config(M, N, K, vec);
  if (M > 0 && N > 0 && tiles_for(configs()[id]->tile, M, N) > 0x7FFFFFFFLL)
    return SGEMM_ERR_UNSUPPORTED;
  if (out != nullptr) {
    const Tile& t = configs()[id]->tile;
    out->cfg_id = id;
    out->vector_variant = vec ? 1 : 0;
    const long long tiles = (M == 0 || N == 0) ? 0 : tiles_for(t, M, N);
    const long long slots = resident_slots(id, kernel_variant(vec));
    const SplitPlan sp = split_plan(tiles, static_cast<int>((K + t.BK - 1) / t.BK),
                                    tiles > 0 ? slots : 0, (t.opt & kOptSplitK) != 0);
    out->slots = slots;
    out->grid = sp.tiles_full + (tiles - sp.tiles_full) * sp.splits;
    out->block = t.NT;
    out->tiles_full = sp.tiles_full;
    out->splits = sp.splits;
  }
  return SGEMM_OK;
}

int sgemm_ex(int64_t M, int64_t N, int64_t K, float alpha, const float* A, int64_t lda,
             const float* B, int64_t ldb, float beta, float* C, int64_t ldc, void* stream,
             int32_t cfg_id) {
  int rc = validate(M, N, K, A, lda, B, ldb, C, ldc);
  if (rc != SGEMM_OK) return rc;
  if (M == 0 || N == 0) return SGEMM_OK;
  if (cfg_id >= sgemm_num_configs()) return SGEMM_ERR_BAD_CONFIG;
  rc = device_check();
  if (rc != SGEMM_OK) return rc;
  const bool vec = vector_ok(N, K, A, lda, B, ldb, C, ldc);
  const int id = cfg_id >= 0 ? cfg_id : select_config(M, N, K, vec);
  const ConfigEntry* e = configs()[id];
  if (tiles_for(e->tile, M, N) > 0x7FFFFFFFLL) return SGEMM_ERR_UNSUPPORTED;

  KernelArgs a{};
  a.A = A; a.B = B; a.C = C;
  a.lda = lda; a.ldb = ldb; a.ldc = ldc;
  a.M = static_cast<int>(M); a.N = static_cast<int>(N); a.K = static_cast<int>(K);
  a.alpha = alpha; a.beta = beta;
  const long long slots = (e->tile.opt & kOptSplitK) ? resident_slots(id, kernel_variant(vec)) : 0;
  const hipError_t err =
      (vec ? e->launch_vec : e->launch_scalar)(a, static_cast<hipStream_t>(stream), slots);
  if (err != hipSuccess) {
    g_last_hip_error = static_cast<int>(err);
    return SGEMM_ERR_LAUNCH;
  }
  return SGEMM_OK;
}

int sgemm_ladder(int32_t rung, int64_t M, int64_t N, int64_t K, float alpha, const float* A,
                 int64_t lda, const float* B, int64_t ldb, float beta, float* C, int64_t ldc,
                 void* stream) {
  // Rungs 2 and 3 are VALU tuples: the 128x128x8 tile with 8x8 lane patches
  // and no warp tiling (a wave covers 32 x 128 outputs, the vectorized
  // kernel's thread map), and the warp-tiled 128x64x16 tile with 4x4 patches
  // (the autotuned warp-tiling shape, warp tile widened to 64 x 64 for
  // 64-lane waves); both with the plain, unswizzled LDS layout.
  static constexpr Tile kRung2{128, 128, 8, 32, 128, 1, 8, 8, 256, kPathValu, 0, 0};
  static constexpr Tile kRung3{128, 64, 16, 64, 64, 2, 4, 4, 128, kPathValu, 0, 0};
  if (rung < 1 || rung > 4) return SGEMM_ERR_BAD_CONFIG;
  if (rung == 2 || rung == 3) {
    const int id = find_tile(rung == 2 ? kRung2 : kRung3);
    if (id < 0) return SGEMM_ERR_BAD_CONFIG;
    return sgemm_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream, id);
  }
  if (rung == 4) return sgemm_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream, -1);
  int rc = validate(M, N, K, A, lda, B, ldb, C, ldc);
  if (rc != SGEMM_OK) return rc;
  if (M == 0 || N == 0) return SGEMM_OK;
  rc = device_check();
  if (rc != SGEMM_OK) return rc;
  KernelArgs a{};
  a.A = A; a.B = B; a.C = C;
  a.lda = lda; a.ldb = ldb; a.ldc = ldc;
  a.M = static_cast<int>(M); a.N = static_cast<int>(N); a.K = static_cast<int>(K);
  a.alpha = alpha; a.beta = beta;
  const hipError_t err = launch_smem_tiling(a, static_cast<hipStream_t>(stream));
  if (err != hipSuccess) {
    g_last_hip_error = static_cast<int>(err);
    return SGEMM_ERR_LAUNCH;
  }
  return SGEMM_OK;
}

int sgemm(int64_t M, int64_t N, int64_t K, float alpha, const float* A, int64_t lda,
          const float* B, int64_t ldb, float beta, float* C, int64_t ldc) {
  return sgemm_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, nullptr, -1);
}

const char* sgemm_status_string(int status) {
  switch (status) {
    case SGEMM_OK: return "ok";
    case -1: return "argument 1 (M) is negative";
    case -2: return "argument 2 (N) is negative";
    case -3: return "argument 3 (K) is negative";
    case -5: return "argument 5 (A) is NULL for a non-empty A";
    case -6: return "argument 6 (lda) is smaller than max(1, K)";
    case -7: return "argument 7 (B) is NULL for a non-empty B";
    case -8: return "argument 8 (ldb) is smaller than max(1, N)";
    case -10: return "argument 10 (C) is NULL for a non-empty C";
    case -11: return "argument 11 (ldc) is smaller than max(1, N)";
    case SGEMM_ERR_NO_DEVICE: return "no gfx950 device is current";
    case SGEMM_ERR_BAD_CONFIG: return "unknown configuration id";
    case SGEMM_ERR_OVERLAP: return "C overlaps A or B";
    case SGEMM_ERR_LAUNCH: return "kernel launch failed";
    case SGEMM_ERR_UNSUPPORTED: return "size beyond the supported limits (dims <= 2^30, ld < 2^21)";
    default: return "unknown status";
  }
}

int sgemm_last_hip_error(void) { return g_last_hip_error; }

int sgemm_device_check(void) { return device_check(); }

int sgemm_kernel_attributes(int32_t id, int32_t vector_variant, sgemm_kernel_attr_t* out) {
  if (out == nullptr || id < 0 || id >= sgemm_num_configs()) return SGEMM_ERR_BAD_CONFIG;
  if (vector_variant != 0 && vector_variant != 1) return SGEMM_ERR_BAD_CONFIG;
  const int rc = device_check();
  if (rc != SGEMM_OK) return rc;
  const ConfigEntry* e = configs()[id];
  hipFuncAttributes attr;
  const void* sym = vector_variant ? e->sym_vec() : e->sym_scalar();
  const hipError_t err = hipFuncGetAttributes(&attr, sym);
  if (err != hipSuccess) {
    g_last_hip_error = static_cast<int>(err);
    return SGEMM_ERR_LAUNCH;
  }
  out->num_regs = attr.numRegs;
  out->scratch_bytes = static_cast<int32_t>(attr.localSizeBytes);
  out->lds_bytes = static_cast<int32_t>(attr.sharedSizeBytes);
  out->max_threads = attr.maxThreadsPerBlock;
  return SGEMM_OK;
}

int64_t sgemm_tile_order(int64_t M, int64_t N, int32_t cfg_id, int32_t* rows, int32_t* cols,
                         int64_t capacity) {
  if (M <= 0 || N <= 0 || cfg_id < 0 || cfg_id >= sgemm_num_configs()) return -1;
  const Tile& t = configs()[cfg_id]->tile;
  const long long tm = (M + t.BM - 1) / t.BM, tn = (N + t.BN - 1) / t.BN;
  const long long n = tm * tn;
  if (n > 0x7FFFFFFFLL) return -1;
  const int gm = xcd_group_rows(tm, tn, t.BM, t.BN);
  for (long long id = 0; id < n && id < capacity; ++id) {
    const TileRC rc = tile_of(static_cast<int>(id), static_cast<int>(tm), static_cast<int>(tn), gm,
                              (t.opt & kOptXcdRemap) != 0);
    if (rows) rows[id] = rc.r;
    if (cols) cols[id] = rc.c;
  }
  return n;
}

int sgemm_check_tuple(const int32_t tuple[12], int32_t target) {
  if (tuple == nullptr) return -1;
  if (target == 0) return check_tile(tile_from(tuple), kGfx950);
  if (target == 1) return check_tile(tile_from(tuple), kPageModel);
  return -1;
}

int sgemm_simulate_tuple(const int32_t tuple[12], int32_t banks, sgemm_sim_report_t* out) {
  if (tuple == nullptr || out == nullptr || (banks != 32 && banks != 64)) return -1;
  return simulate(tile_from(tuple), banks, out);
}

}  // extern "C"
