// Decode attention over an 8-bit cache on the 5th-generation tensor cores:
// bf16 queries, head size 128, up to 64 query heads per K/V head.
//
// The cache's e4m3 codes are the A operand of both products (kind::f8f6f4) as
// TMA lands them; no row is converted.  The other operand of such a product is
// e4m3 too, 4 significant bits, so queries and weights enter as two terms:
//   q / w ~ q1 + q2,        q1 = e4m3(q / w),  q2 = e4m3(q / w - q1)
//   P     ~ P1 + P2 / 16,   P1 = e4m3(P),      P2 = e4m3(16 (P - P1))
// With w the power of two that puts a bf16 query's maximum in (224, 448], q1 +
// q2 is exact for elements above 2^-10 of it and off by at most 2^-10 units
// (2^-17 of the maximum) below; both terms' products add up in one
// accumulator.  A weight is off by at most 2^-9 of itself by its terms and 2^-11
// by the fp16 number that they are taken from (a bf16 weight: 2^-8); its terms are
// columns side by side whose results are joined at the end, which gives the second
// term 4 more octaves before it underflows.
//
// With k_t, v_t the codes and a_t, b_t the row scales:
//   S^T[t, i]  = k_t . (q1_i + q2_i)    M = 128 rows, N = heads, K = 2 x 128
//   s_{t,i}    = scale log2(e) w_i a_t S[t, i]
//   p_{t,i}    = 2^(s_{t,i} - m_i),     l_i = sum_t p_{t,i}            (fp32)
//   P_{t,i}    = p_{t,i} b_t 2^(4-E)
//   O^T[c, n] += sum_t v_t[c] P[t, n]   M = 128 columns of V, N = 2 heads, K = 128 rows
//   o_i        = 2^(E-4) (O[c, i] + O[c, i'] / 16) / l_i
// E is the largest value-row exponent seen (of rows that are not all zero; 1, the
// smallest, before any) and m_i is set so that the largest P is 2^4: the e4m3 grid
// (at least 2^-13 in the second term) then lies relative to what a row contributes
// to the output, not to its weight alone, and a heavy row with small values (an
// attention sink) leaves the other rows their precision.  A reference is moved only
// when some P would pass 448.  (Relative errors over 32K rows, queries three times
// as large as normal ones: 0.00159, of which 0.00158 is the output's rounding; with
// 2^2 0.00165, 0 to 1% faster; with 2^6 0.00159, 0.5 to 1.7% slower; a bf16 decode of
// the same values 0.0020.)  Behind a heavy row a long tail's weights can all be below
// that grid: they are dithered before they are rounded, so that their sum stays
// (lowering a reference with a tile's maxima instead cost 24% on 32K-row GQA-8
// caches whose row scales vary: it goes up and down all the time).
//
// Work: two persistent CTAs per SM (a tile's chain of product, softmax and
// product is latency; two chains hide each other's).  CTA c serves K/V head c %
// g over a contiguous run of all sequences' 128-row tiles, balanced in quarter
// tiles with a segment's entry weighed as kSegUnits of them.  The g CTAs of a group
// walk the same rows in step: a cache row's g heads are neighbours in memory,
// 128 bytes each, and reading them together is what DRAM pages want (32 GQA-8
// caches of 8K to 32K rows, 1.44 GB: 287 us head by head, 237 in step).
// Partials of split segments are joined by the merge kernel.  Roles:
//   warp 0, lane 0    K loads;      warp 2, lane 0   V loads (never ahead of K)
//   warp 1, lane 0    S products;   warp 3, lane 0   P.V products
//   warps 4-7, 4-11   query conversion, softmax, epilogue: a thread holds one row
//                     and all heads (up to 32), or half of them
// An ordinary tile has one barrier of the softmax warps, which also tells them
// whether a reference has to move.  Every wait is bounded (one second); on
// expiry the kernel sets MQA_FLAG_PIPE_TIMEOUT, drains its copies and products,
// frees its tensor memory and returns.
//
// Bound: HBM for large caches and groups of up to 16 heads (those 1.44 GB: 223
// us, 6.4 TB/s, where the clocks are good; d + 1 bytes per row instead of 2 d);
// the chain's latency for wider groups (64 MQA caches of 1K to 8K rows with 32
// heads, 80 MB: 33 us, 2.4 TB/s); the fixed costs of a launch for small caches.
#include "q8_tc.cuh"

namespace mqa {
namespace q8 {

namespace {

using namespace sm100;

constexpr int kRows = 128;                      // rows per tile: the products' M
constexpr int kKWarp = 0, kSWarp = 1, kVWarp = 2, kSoftWarp = 4;   // warp 3: P.V products
constexpr int kCtasPerSm = 2;
constexpr uint32_t kTileBytes = kRows * kD;     // 128 rows of codes, 128-byte swizzled
constexpr int kSegUnits = 7;                    // cost of entering a segment, in quarter tiles (measured: 2.7 us, a tile 1.6)
constexpr int kBias = 4;                        // the largest P after a reference is set is 2^kBias
constexpr float kFall = 90.f;                    // octaves that a reference comes down at a time: the sums stay finite
constexpr int kLensCache = 256;
constexpr uint32_t kMaxDynSmem = (233472 - kCtasPerSm * 1024) / kCtasPerSm;

template <int HP>   // heads per segment, padded
struct Cfg {
  // Softmax warps: four, each thread a row and all heads, or eight (half of
  // the heads each) where a row's heads do not fit a thread's registers.
  static constexpr int kSoftWarps = HP <= 32 ? 4 : 8;
  static constexpr int kSoft = 32 * kSoftWarps, kThreads = kSoft + 128;
  static constexpr int CPT = HP / (kSoftWarps / 4);            // heads per thread
  // Registers per thread at launch, and after the roles' warps have given
  // theirs up for the softmax warps: 128 kRegsRoles + kSoft kRegsSoft is what
  // the CTA was launched with.
  static constexpr int kRegs = kSoftWarps == 4 ? 128 : 80;
  static constexpr int kRegsRoles = kSoftWarps == 4 ? 72 : 48, kRegsSoft = kSoftWarps == 4 ? 184 : 96;
  static_assert(128 * kRegsRoles + kSoft * kRegsSoft == kThreads * kRegs && kCtasPerSm * kThreads * kRegs <= 65536, "registers");
  // With few registers per head the logits are taken from tensor memory again
  // instead of being kept.
  static constexpr bool kReload = kSoftWarps == 8;
  static constexpr int SK = 2, SV = HP <= 32 ? 3 : 2;          // ring stages
  static constexpr int kOBufs = HP <= 32 ? 2 : 1;              // O buffers (S has two)
  static constexpr int kN = 2 * HP;                            // columns of P and O: first terms, then second terms
  static constexpr uint32_t kOCol = 2 * HP;                    // tensor memory: S, then O
  static constexpr uint32_t kTmemCols = HP <= 16 ? 128 : 256;  // two CTAs fit the SM's 512
  static_assert(kOCol + kOBufs * kN <= kTmemCols, "tensor memory");
  static_assert(kCtasPerSm * kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory");
  // barriers
  static constexpr int kKFull = 0, kKEmpty = SK, kVFull = 2 * SK, kVEmpty = 2 * SK + SV, kSFull = 2 * SK + 2 * SV,
                       kSEmpty = kSFull + 2, kOFree = kSEmpty + 2, kPFull = kOFree + kOBufs, kOFull = kPFull + 1,
                       kQFull = kOFull + 1, kDone = kQFull + 1, kNumBars = kDone + 1;
  // shared memory
  static constexpr uint32_t kK = 0;
  static constexpr uint32_t kV = kK + SK * kTileBytes;
  static constexpr uint32_t kQ = kV + SV * kTileBytes;
  static constexpr uint32_t kQTerm = HP * kD;                  // Q's two terms, HP rows each
  static constexpr uint32_t kP = kQ + 2 * kQTerm;              // a 128-byte line per row, kN of it used
  static constexpr uint32_t kBar = kP + kRows * 128;
  static constexpr uint32_t kTmemSlot = kBar + kNumBars * 8;
  static constexpr uint32_t kAbort = kTmemSlot + 4;
  static constexpr uint32_t kKIssued = kAbort + 4;
  static constexpr uint32_t kSeg = (kKIssued + 4 + 15) / 16 * 16;  // [2][4] sequence, flags, last unit of a segment
  static constexpr uint32_t kQw = kSeg + 32;                   // [HP] query scales
  static constexpr uint32_t kRed = kQw + HP * 4;               // [4][HP] column maxima per warp
  static constexpr uint32_t kRedL = kRed + 4 * HP * 4;         // [4][HP] column sums per warp
  static constexpr uint32_t kLinv = kRedL + 4 * HP * 4;        // [2][HP]
  static constexpr uint32_t kLse = kLinv + 2 * HP * 4;         // [2][HP]
  static constexpr uint32_t kWarpRefs = kLse + 2 * HP * 4;     // each softmax warp's own: minus the references, how far
                                                               // they move, and the factors of the sums and of O
  static constexpr uint32_t kEred = kWarpRefs + kSoftWarps * 4 * CPT * 4;   // [2][4]
  static constexpr uint32_t kLens = kEred + 32;                // [kLensCache]
  static constexpr uint32_t kSched = (kLens + kLensCache * 4 + 15) / 16 * 16;
  static constexpr uint32_t kAlloc = kSched + 256;
  static_assert(kQ % 1024 == 0 && kP % 1024 == 0, "swizzle atoms need 1024-byte alignment");
  static_assert(kAlloc <= kMaxDynSmem, "shared memory budget");
  static_assert((kThreads / 32 + 6) * 8 <= 256, "schedule scratch");
  static_assert(kThreads >= kLensCache && kRed % 16 == 0 && kQw % 16 == 0 && kWarpRefs % 16 == 0, "tables");
};

template <int N>
__device__ __forceinline__ void soft_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory"); }

// A barrier of the N softmax threads that also reduces a flag, so that every
// thread takes the same branch afterwards.
template <int N>
__device__ __forceinline__ bool soft_barrier_or(bool v) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.or.pred po, 1, %2, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(out) : "r"(uint32_t(v)), "n"(N) : "memory");
  return out != 0;
}

// Reduction over the 32 lanes of W columns (maxima, NaNs passed over, or
// sums); lane l ends with column l % W.  31 shuffles for 32 columns: the warp
// reduction instruction takes one per column and measured three times as long.
template <int W, bool kMax>
__device__ __forceinline__ float transpose_reduce(float (&v)[W], int lane) {
  auto join = [](float x, float y) { return kMax ? fmaxf(x, y) : x + y; };
#pragma unroll
  for (int o = W / 2; o >= 1; o >>= 1) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const float send = upper ? v[k] : v[k + o];
      const float keep = upper ? v[k + o] : v[k];
      v[k] = join(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  float r = v[0];
#pragma unroll
  for (int o = W; o < 32; o <<= 1) r = join(r, __shfl_xor_sync(0xffffffffu, r, o));
  return r;
}

// ------------------------------------------------------------------ work

// This CTA's run of tiles, in the numbering of one head's tiles over all
// sequences (31 bits: the host checks), found as in the bf16 decode: units of
// a quarter tile, kSegUnits more for every sequence.
struct Run {
  int t_begin, t_end;   // tiles
  int seq, base, ubase; // sequence of the first tile, that sequence's first tile and first unit
  int wtotal, active;   // units in all, and groups of CTAs with work
  int pre;              // leading tiles whose loads are already under way
};

// Clamped rows of sequence s.  Where another part joins the partials a
// sequence may have none of its own.
__device__ __forceinline__ int rows_of(const TcArgs& a, int s, bool report) {
  const int n = __ldcg(a.lens + s), c = min(max(n, 0), a.m);
  if (report && (c != n || (n == 0 && !a.partials))) set_flag(a.flags, MQA_FLAG_LEN_CLAMPED);
  return c;
}

__device__ __forceinline__ int units_of(int nb) { return nb > 0 ? kSegUnits + 4 * nb : 0; }

// The thread whose sequences hold the run's first tile calls on_first(seq,
// tile, own, rows) at once, with `own` >= 1 tiles of that sequence belonging to
// the run; it returns how many of them it has begun to load.
template <int kThreads, typename OnFirst>
__device__ Run make_run(const TcArgs& a, int group, bool report, int64_t* scratch, int* lens_tab, OnFirst&& on_first) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.b + kThreads - 1) / kThreads;
  const int s0 = min(a.b, tid * per), s1 = min(a.b, s0 + per);
  const bool tab = a.b <= kLensCache;
  int my_t = 0, my_u = 0;
  for (int s = s0; s < s1; ++s) {
    const int len = rows_of(a, s, report);
    if (tab) lens_tab[s] = len;
    const int nb = tiles_of(span_of(len, a.window), kRows);
    my_t += nb;
    my_u += units_of(nb);
  }
  uint64_t x = (uint64_t(uint32_t(my_t)) << 32) | uint32_t(my_u);   // neither half can carry
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  uint64_t* wsum = reinterpret_cast<uint64_t*>(scratch);
  int* out = reinterpret_cast<int*>(scratch + kThreads / 32);
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  uint64_t tot = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const uint64_t v = wsum[w];
    tot += v;
    if (w < warp) before += v;
  }
  const uint64_t incl = before + x;
  const int T = int(tot >> 32), W = int(uint32_t(tot));
  const int excl_t = int(incl >> 32) - my_t, excl_u = int(uint32_t(incl)) - my_u;
  Run run = {};
  run.wtotal = W;
  // Ranges of four units and more: a range that starts and ends within one
  // sequence then holds a tile's start, so that the parts of a segment lie in
  // consecutive groups; a range may be empty where it covers a segment's entry.
  const int cap = W / 4;
  run.active = cap < a.groups ? cap : a.groups;
  if (group >= run.active) return run;   // uniform across the CTA
  const int q = W / run.active, rm = W - q * run.active;   // group*W/active without a 64-bit division
  const int u0 = group * q + (group * rm) / run.active;
  const int u1 = (group + 1) * q + ((group + 1) * rm) / run.active;
  // Walks this thread's sequences to the one that holds unit u: f(sequence, rows, tiles, tile, its first tile and unit).
  auto locate = [&](int u, auto&& f) {
    if (u < excl_u || u >= excl_u + my_u) return;
    int tb = excl_t, ub = excl_u;
    for (int s = s0; s < s1; ++s) {
      const int len = tab ? lens_tab[s] : rows_of(a, s, false);
      const int nb = tiles_of(span_of(len, a.window), kRows);
      const int su = units_of(nb);
      if (u < ub + su) {
        const int off = u - ub;
        f(s, len, nb, off <= kSegUnits ? 0 : (off - kSegUnits + 3) / 4, tb, ub);
        return;
      }
      tb += nb;
      ub += su;
    }
  };
  if (u1 < W) locate(u1, [&](int, int, int, int k, int tb, int) { out[3] = tb + k; });
  locate(u0, [&](int s, int len, int nb, int k, int tb, int ub) {
    out[0] = tb + k;
    out[1] = s;
    out[2] = tb;
    out[4] = ub;
    int begun = 0;
    if (k < nb) {   // the run's tiles of this sequence: those whose start unit is below u1
      const int lim = u1 - (ub + kSegUnits);
      const int kend = min(nb, lim <= 0 ? 0 : (lim + 3) / 4);
      if (kend > k) begun = on_first(s, k, kend - k, len);
    }
    out[5] = begun;
  });
  __syncthreads();
  run.t_begin = out[0];
  run.seq = out[1];
  run.base = out[2];
  run.t_end = u1 == W ? T : out[3];
  run.ubase = out[4];
  run.pre = out[5];
  return run;
}

struct Roles {
  uint32_t sbase;
  unsigned char* smem;
  uint32_t tmem;
  volatile int* abort;
  int32_t* flags;
  const int* lens_s;   // clamped rows of sequences seq0 .. seq0 + kLensCache - 1
  int seq0;
  int head, group;     // the CTA's K/V head, and its group of CTAs
};

__device__ __forceinline__ int seq_rows(const TcArgs& a, const Roles& r, int s) {
  const int i = s - r.seq0;
  if (i >= 0 && i < kLensCache) return r.lens_s[i];
  return rows_of(a, s, false);
}

__device__ __forceinline__ bool wait_bar(const Roles& r, uint32_t bar, uint32_t parity) {
  if (mbar_wait_asleep(bar, parity, kTimeoutNs)) return true;
  *r.abort = 1;
  set_flag(r.flags, MQA_FLAG_PIPE_TIMEOUT);
  return false;
}

// Walks the CTA's tiles in order, counting (tile, sequence) forward.
struct TileWalk {
  int t, t_end;        // this tile, and the end of the CTA's run
  int k, nb;           // this tile within its sequence, and the sequence's tiles
  int row0, len;       // its first row, and the sequence's rows
  int seq, sidx;       // sequence, and the CTA's count of segments
  int ubase;           // first unit of the sequence
  bool first;          // tile of the segment, within this CTA
  __device__ TileWalk(const TcArgs& a, const Run& run, const Roles& r) : t(run.t_begin - 1), t_end(run.t_end), sidx(-1) {
    int base = run.base;
    ubase = run.ubase;
    set_seq(a, r, run.seq);
    while (run.t_begin >= base + nb) {   // the first tile may lie in a later sequence
      base += nb;
      ubase += units_of(nb);
      set_seq(a, r, seq + 1);
    }
    k = run.t_begin - base - 1;
    row0 += k * kRows;
  }
  __device__ void set_seq(const TcArgs& a, const Roles& r, int s) {
    seq = s;
    len = seq_rows(a, r, s);
    row0 = len - span_of(len, a.window);
    nb = tiles_of(len - row0, kRows);
  }
  __device__ void next(const TcArgs& a, const Roles& r) {
    ++t;
    ++k;
    row0 += kRows;
    first = sidx < 0;
    if (k == nb) {
      first = true;
      ubase += units_of(nb);
      do set_seq(a, r, seq + 1);
      while (nb == 0);
      k = 0;
    }
    if (first) ++sidx;
  }
  __device__ int rows() const { return min(kRows, len - row0); }
  __device__ bool last() const { return k == nb - 1 || t + 1 == t_end; }
  __device__ int seg_t0() const { return t - k; }
  __device__ int seg_last_unit() const { return ubase + kSegUnits + 4 * (nb - 1); }
};

// ------------------------------------------------------------------ loads and products

__device__ __forceinline__ void load_tile(const TcArgs& a, uint32_t dst, const CUtensorMap* map, uint32_t bar, int seq,
                                          int head, int row0, uint64_t pol) {
  mbar_expect_tx(bar, kTileBytes);
  tma_load_3d(dst, map, bar, 0, head, seq * a.m + row0, pol);
}

template <int HP, bool kIsK>
__device__ void producer(const TcArgs& a, const Run& run, const Roles& r, const CUtensorMap* map) {
  using C = Cfg<HP>;
  constexpr int S = kIsK ? C::SK : C::SV;
  constexpr int kFull = kIsK ? C::kKFull : C::kVFull, kEmpty = kIsK ? C::kKEmpty : C::kVEmpty;
  constexpr uint32_t kRing = kIsK ? C::kK : C::kV;
  auto bar = [&](int id) { return r.sbase + C::kBar + 8u * uint32_t(id); };
  const uint64_t pol = l2_evict_first_policy();   // each byte is read once
  volatile int* k_issued = reinterpret_cast<volatile int*>(r.smem + C::kKIssued);
  TileWalk w(a, run, r);
  const int n = run.t_end - run.t_begin;
  int i = 0, st = 0;
  uint32_t ph = 1;   // parity of the stage's previous release
  for (; i < n; ++i) {
    w.next(a, r);
    if (*r.abort) break;
    if (i >= run.pre) {
      if (i >= S && !wait_bar(r, bar(kEmpty + st), ph)) break;
      if (!kIsK) {   // never run ahead of the K producer: the loads go out K(0), V(0), K(1), ...
        uint32_t polls = 0;
        while (*k_issued <= i && !*r.abort && ++polls < (1u << 24)) {}   // cannot stall for good: K gives up on abort
      }
      load_tile(a, r.sbase + kRing + st * kTileBytes, map, bar(kFull + st), w.seq, r.head, w.row0, pol);
    }
    if (kIsK) *k_issued = i + 1;
    if (++st == S) {
      st = 0;
      ph ^= 1u;
    }
  }
  // every copy this thread (or the schedule) issued has landed before the CTA can exit
  for (int j = (i - S > 0 ? i - S : 0); j < i; ++j) mbar_wait_asleep(bar(kFull + j % S), uint32_t(j / S) & 1, kTimeoutNs);
}

// S(i) = K Q^T once K(i), for a segment's first tile its queries, and the S
// buffer are there.
template <int HP>
__device__ void s_issuer(const TcArgs& a, const Run& run, const Roles& r) {
  using C = Cfg<HP>;
  constexpr uint32_t idesc = idesc_code0_f32(kRows, HP, 0, 0);
  const uint64_t kdesc0 = smem_desc_sw128(r.sbase + C::kK, 16, 1024);   // K-major, rows of 128 bytes
  const uint64_t qdesc = smem_desc_sw128(r.sbase + C::kQ, 16, 1024);
  auto bar = [&](int id) { return r.sbase + C::kBar + 8u * uint32_t(id); };
  TileWalk w(a, run, r);
  const int n = run.t_end - run.t_begin;
  int st = 0;
  uint32_t ph = 0;
  for (int i = 0; i < n; ++i) {
    w.next(a, r);
    const int sb = i & 1;
    if (w.first && !wait_bar(r, bar(C::kQFull), uint32_t(w.sidx) & 1)) break;
    if (!wait_bar(r, bar(C::kKFull + st), ph)) break;
    if (i >= 2 && !wait_bar(r, bar(C::kSEmpty + sb), uint32_t((i >> 1) - 1) & 1)) break;
    tc_fence_after();
    const uint64_t ka = kdesc0 + uint64_t((uint32_t(st) * kTileBytes) >> 4);
#pragma unroll
    for (int term = 0; term < 2; ++term)
#pragma unroll
      for (int kk = 0; kk < kD / 32; ++kk)
        mma_e4m3_ss(r.tmem + uint32_t(sb) * HP, ka + ((kk * 32) >> 4), qdesc + ((term * C::kQTerm + kk * 32) >> 4), idesc,
                    term + kk > 0);
    mma_commit(bar(C::kSFull + sb));
    mma_commit(bar(C::kKEmpty + st));
    if (++st == C::SK) {
      st = 0;
      ph ^= 1u;
    }
  }
  // every product issued above has completed before tensor memory is released
  mma_commit(bar(C::kDone));
  mbar_wait_asleep(bar(C::kDone), 0, kTimeoutNs);
}

// O += V^T P(i) once P(i) is written, V(i) has landed and, for a segment's
// first tile, its O buffer has been read by the epilogue of the segment that
// had it before.
template <int HP>
__device__ void pv_issuer(const TcArgs& a, const Run& run, const Roles& r) {
  using C = Cfg<HP>;
  constexpr uint32_t idesc = idesc_code0_f32(kD, C::kN, 1, 1);
  const uint64_t vdesc0 = smem_desc_sw128(r.sbase + C::kV, 16, 1024);   // MN-major: one 128-column atom, 8-row groups
  const uint64_t pdesc = smem_desc_sw128(r.sbase + C::kP, 16, 1024);
  auto bar = [&](int id) { return r.sbase + C::kBar + 8u * uint32_t(id); };
  TileWalk w(a, run, r);
  const int n = run.t_end - run.t_begin;
  int st = 0;
  uint32_t ph = 0;
  for (int i = 0; i < n; ++i) {
    w.next(a, r);
    const int ob = w.sidx % C::kOBufs;
    if (!wait_bar(r, bar(C::kPFull), uint32_t(i & 1))) break;
    if (!wait_bar(r, bar(C::kVFull + st), ph)) break;
    if (w.first && w.sidx >= C::kOBufs && !wait_bar(r, bar(C::kOFree + ob), uint32_t(w.sidx / C::kOBufs - 1) & 1)) break;
    tc_fence_after();
    const uint64_t va = vdesc0 + uint64_t((uint32_t(st) * kTileBytes) >> 4);
    const uint32_t acc0 = w.first ? 0u : 1u;
#pragma unroll
    for (int kk = 0; kk < kRows / 32; ++kk)   // 32 rows: four 8-row groups of 1024 bytes
      mma_e4m3_ss(r.tmem + C::kOCol + uint32_t(ob) * C::kN, va + ((kk * 4096) >> 4), pdesc + ((kk * 4096) >> 4), idesc,
                  kk > 0 ? 1u : acc0);
    mma_commit(bar(C::kOFull));
    mma_commit(bar(C::kVEmpty + st));
    if (++st == C::SV) {
      st = 0;
      ph ^= 1u;
    }
  }
  mma_commit(bar(C::kDone));
  mbar_wait_asleep(bar(C::kDone), 0, kTimeoutNs);
}

// ------------------------------------------------------------------ softmax

// The segment's queries into the Q buffer, eight threads per row.
template <int HP>
__device__ __forceinline__ void convert_queries(const TcArgs& a, const Roles& r, int seq, int tid) {
  using C = Cfg<HP>;
  unsigned char* qs = r.smem + C::kQ;
  float* qw = reinterpret_cast<float*>(r.smem + C::kQw);
  const int part = tid & 7;
  constexpr int kPasses = HP * 8 / C::kSoft;
  QueryPiece q[kPasses];   // all loads first
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    const int n = pass * (C::kSoft / 8) + (tid >> 3);
    q[pass] = load_query(n < a.hq ? a.q + (int64_t(seq) * a.h + int64_t(r.head) * a.hq + n) * kD : nullptr, part);
  }
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    const int n = pass * (C::kSoft / 8) + (tid >> 3);
    uint4 hi, lo;
    const float s = split_query(q[pass], hi, lo);
    unsigned char* at = qs + n * 128 + ((part ^ (n & 7)) << 4);   // HP is a multiple of 8: both terms' rows swizzle alike
    *reinterpret_cast<uint4*>(at) = hi;
    *reinterpret_cast<uint4*>(at + C::kQTerm) = lo;
    if (part == 0) qw[n] = s;
  }
  fence_proxy_async_smem();
  mbar_arrive(r.sbase + C::kBar + 8u * uint32_t(C::kQFull));
}

template <int HP>
__device__ void softmax_epilogue(const TcArgs& a, const Run& run, const Roles& r, int warp, int lane) {
  using C = Cfg<HP>;
  constexpr int CPT = C::CPT, kSoft = C::kSoft;
  constexpr bool kReload = C::kReload;
  constexpr int W = kReload ? 8 : 16;              // columns handled at a time
  auto bar = [&](int id) { return r.sbase + C::kBar + 8u * uint32_t(id); };
  auto wait = [&](int id, uint32_t parity) { return mbar_wait_asleep(bar(id), parity, kTimeoutNs); };
  const int q4 = warp & 3;                         // tensor-memory lane quarter of this warp
  const int grp = (warp - kSoftWarp) >> 2;         // column group: heads [grp*CPT, grp*CPT + CPT)
  const int col0 = grp * CPT;
  const int tid = threadIdx.x - 32 * kSoftWarp;
  const int row = 32 * q4 + lane;                  // row of the tile (S), output column (O)
  const uint32_t t_lane = r.tmem + (uint32_t(32 * q4) << 16);
  float* red = reinterpret_cast<float*>(r.smem + C::kRed);
  float* negm = reinterpret_cast<float*>(r.smem + C::kWarpRefs) + (warp - kSoftWarp) * 4 * CPT;
  float *move = negm + CPT, *alpha_l = negm + 2 * CPT, *alpha_o = negm + 3 * CPT;
  float* redl = reinterpret_cast<float*>(r.smem + C::kRedL);
  float* linv = reinterpret_cast<float*>(r.smem + C::kLinv);
  float* lse2 = reinterpret_cast<float*>(r.smem + C::kLse);
  int* ered = reinterpret_cast<int*>(r.smem + C::kEred);
  int* seg_s = reinterpret_cast<int*>(r.smem + C::kSeg);
  const float* qw = reinterpret_cast<const float*>(r.smem + C::kQw) + col0;
  unsigned char* const line = r.smem + C::kP + row * 128;
  const float c = a.scale * kLog2e;
  uint64_t lsum[CPT / 2];                          // this thread's share of the sums, in pairs
  uint64_t d[(kReload ? W : CPT) / 2];             // s - m, in pairs
  int E = 0;                                       // the value exponent P is relative to
  bool any = false;                                // some value row of the segment so far was not all zeros

  TileWalk w(a, run, r);
  const int n = run.t_end - run.t_begin;
  // This thread's row exponents of the walker's tile; the pointers advance
  // within a segment.
  const uint8_t *ke = nullptr, *ve = nullptr;
  uint32_t nke, nve;
  auto load_exps = [&]() {
    if (w.first) {
      const int64_t at = (int64_t(w.seq) * a.g + r.head) * a.m + w.row0 + row;
      ke = a.ke + at;
      ve = a.ve + at;
    } else {
      ke += kRows;
      ve += kRows;
    }
    const bool in = w.row0 + row < w.len;
    nke = in ? __ldcg(ke) : 0u;
    nve = in ? __ldcg(ve) : 0u;
  };
  w.next(a, r);
  load_exps();
  convert_queries<HP>(a, r, w.seq, tid);
  bool failed = false;
  int pend = -1;       // a finished segment (its count) whose output is still to be written

  // Write segment `sidx`: O^T from tensor memory times 1/l.  Thread `row` holds
  // output column `row` of its heads.
  auto epilogue = [&](int sidx) {
    const int pb = sidx & 1, ob = sidx % C::kOBufs;
    const int seq = seg_s[pb * 4], flags = seg_s[pb * 4 + 1];
    const int64_t seg = int64_t(seq) * a.g + r.head;
    const int64_t slot = tc_slot(r.group, seq, a.g, r.head);
    const bool whole = (flags & 2) && !a.partials;
#pragma unroll
    for (int ch = 0; ch < CPT / W; ++ch) {
      const int cc = col0 + ch * W;
      const uint32_t oc = t_lane + C::kOCol + uint32_t(ob) * C::kN + cc;
      float v[W], v2[W];
      tmem_ld_two<W>(oc, oc + HP, v, v2);
#pragma unroll
      for (int k = 0; k < W; ++k) v[k] = fmaf(v2[k], 0.0625f, v[k]) * linv[pb * HP + cc + k];
      if (whole) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + (int64_t(seq) * a.h + int64_t(r.head) * a.hq + cc) * kD + row;
#pragma unroll
        for (int k = 0; k < W; ++k)
          if (cc + k < a.hq) dst[k * kD] = __float2bfloat16_rn(v[k]);
      } else {
        float* dst = a.ws.part_o + (slot * a.hq + cc) * kD + row;
#pragma unroll
        for (int k = 0; k < W; ++k)
          if (cc + k < a.hq) dst[k * kD] = v[k];
      }
    }
    if (warp == kSoftWarp) {
      if (!whole)
        for (int col = lane; col < a.hq; col += 32) a.ws.part_lse[slot * a.hq + col] = lse2[pb * HP + col];
      if ((flags & 1) && lane == 0)
        a.ws.seg_info[seg] = make_int2(r.group, whole ? -1 : cta_of_unit(seg_s[pb * 4 + 2], run.wtotal, run.active));
    }
    tc_fence_before();
    mbar_arrive(bar(C::kOFree + ob));
  };

  for (int i = 0; i < n; ++i) {
    const float kr = scale_of(nke) * c;
    const int er = int(nve);
    const __half2 dither = row_dither(w.row0 + row);
    const int rows = w.rows(), sidx = w.sidx;
    const bool first = w.first, last = w.last();
    if (last && tid == 0) {   // what the epilogue will need
      const bool owns_first = w.seg_t0() >= run.t_begin, whole = owns_first && w.seg_t0() + w.nb <= run.t_end;
      *reinterpret_cast<int4*>(seg_s + (sidx & 1) * 4) =
          make_int4(w.seq, (owns_first ? 1 : 0) | (whole ? 2 : 0), w.seg_last_unit(), 0);
    }
    if (i + 1 < n) {   // what the next tile needs from memory
      w.next(a, r);
      load_exps();
    }
    const int sb = i & 1;
    const uint64_t kr2 = pack2(kr, kr);
    // W columns' logits minus their references (zero on a segment's first tile)
    auto logits = [&](int ch, uint64_t* x) {
      float s[W];
      tmem_ld<W>(t_lane + uint32_t(sb) * HP + col0 + ch * W, s);
#pragma unroll
      for (int k = 0; k < W; k += 4) {
        uint64_t w0, w1, m0, m1;
        load_pairs(qw + ch * W + k, w0, w1);
        load_pairs(negm + ch * W + k, m0, m1);
        x[k / 2] = fma2(mul2(pack2(s[k], s[k + 1]), w0), kr2, m0);
        x[k / 2 + 1] = fma2(mul2(pack2(s[k + 2], s[k + 3]), w1), kr2, m1);
      }
      if (rows < kRows && row >= rows) {   // past the end: no weight
#pragma unroll
        for (int k = 0; k < W / 2; ++k) x[k] = pack2(-INFINITY, -INFINITY);
      }
    };
    auto release_s = [&]() {   // the buffer may take the next S
      tc_fence_before();
      mbar_arrive(bar(C::kSEmpty + sb));
    };
    const int em4 = __reduce_max_sync(0xffffffffu, er > 1 ? er : 0);   // value exponents, rows of zeros aside
    if (grp == 0 && lane == 0) ered[(i & 1) * 4 + q4] = em4;
    if (first) {
#pragma unroll
      for (int k = 0; k < CPT / 2; ++k) lsum[k] = 0;
      if (lane < CPT) negm[lane] = 0.f;
      __syncwarp();
    }
    if (!wait(C::kSFull + sb, uint32_t(i >> 1) & 1)) failed = true;
    __syncwarp();
    tc_fence_after();
    if (first) soft_barrier<kSoft>();   // the segment's query scales are all written
    // Would some P pass the largest code?
    float top = -INFINITY;
#pragma unroll
    for (int ch = 0; ch < CPT / W; ++ch) {
      uint64_t* x = kReload ? d : d + ch * (W / 2);
      logits(ch, x);
#pragma unroll
      for (int k = 0; k < W / 2; ++k) {
        float x0, x1;
        unpack2(x[k], x0, x1);
        top = fmaxf(top, fmaxf(x0, x1));
      }
    }
    if (!kReload) release_s();
    const bool exceed = !first && top + float(max(er - E, -kSpan) + kBias) > kLogCodeMax;
    // The one barrier of an ordinary tile.  A thread that gave up a wait says so
    // here, a tile late at most, so that all leave together.
    bool full = soft_barrier_or<kSoft>(exceed || failed);
    if (full && soft_barrier_or<kSoft>(failed)) {
      failed = true;
      break;
    }
    full = full || first;
    bool moved[CPT / W];   // chunks with a reference that moves: O and the sums are rescaled there
    if (full) {
      const int* e4 = ered + (i & 1) * 4;
      const int em = max(max(e4[0], e4[1]), max(e4[2], e4[3]));
      const int E_old = E;
      if (first) any = false;
      E = any ? max(E, em) : max(em, 1);   // no value yet: the smallest, so that any value exceeds it
      any = any || em > 0;
      const float off = float(max(er - E, -kSpan));
      float mine = 0.f;      // lane k's: column k's maximum
      if constexpr (kReload) {
#pragma unroll
        for (int ch = 0; ch < CPT / W; ++ch) {
          logits(ch, d);
          float v[W];
#pragma unroll
          for (int k = 0; k < W / 2; ++k) unpack2(d[k], v[2 * k], v[2 * k + 1]);
#pragma unroll
          for (int k = 0; k < W; ++k) v[k] += off;
          const float m = transpose_reduce<W, true>(v, lane);
          mine = lane / W == ch ? m : mine;
        }
      } else {
        float v[CPT];
#pragma unroll
        for (int k = 0; k < CPT / 2; ++k) unpack2(d[k], v[2 * k], v[2 * k + 1]);
#pragma unroll
        for (int k = 0; k < CPT; ++k) v[k] += off;
        mine = transpose_reduce<CPT, true>(v, lane);
      }
      if (lane < CPT) red[q4 * HP + col0 + lane] = mine;
      soft_barrier<kSoft>();
      bool moves = false;
      if (lane < CPT) {   // every warp works out the references of its columns, all to the same result
        const int col = col0 + lane;
        // how far the reference moves, seen from the old one
        float by = fmaxf(fmaxf(red[col], red[HP + col]), fmaxf(red[2 * HP + col], red[3 * HP + col]));
        if (!first) {
          const float shift = float(E_old - E);   // the old reference relative to E
          by = fmaxf(by, fmaxf(shift, -kFall));
          moves = by != shift;
          alpha_l[lane] = ex2_approx(-by);
          alpha_o[lane] = ex2_approx(shift - by);
        }
        negm[lane] -= by;
        move[lane] = -by;
      }
      const uint32_t which = __ballot_sync(0xffffffffu, moves);
      __syncwarp();
#pragma unroll
      for (int ch = 0; ch < CPT / W; ++ch) {
        moved[ch] = ((which >> (ch * W)) & ((1u << W) - 1)) != 0;
        if (first || moved[ch] || E != E_old) {
#pragma unroll
          for (int k = ch * W; k < ch * W + W; k += 4) {
            uint64_t b0, b1;
            if (!kReload) {
              load_pairs(move + k, b0, b1);
              d[k / 2] = add2(d[k / 2], b0);
              d[k / 2 + 1] = add2(d[k / 2 + 1], b1);
            }
            if (!first) {
              load_pairs(alpha_l + k, b0, b1);
              lsum[k / 2] = mul2(lsum[k / 2], b0);
              lsum[k / 2 + 1] = mul2(lsum[k / 2 + 1], b1);
            }
          }
        }
      }
    }
    // P in two terms, into registers before waiting for the previous product
    uint32_t hi[CPT / 4], lo[CPT / 4];
    {
      const int f = er - E + 127 + kBias;   // the factor b_t 2^(kBias - E): a power of two, 0 for a zero scale
      const float ab = er == 0 || f <= 0 ? 0.f : __uint_as_float(uint32_t(min(f, 254)) << 23);
      const uint64_t ab2 = pack2(ab, ab);
#pragma unroll
      for (int ch = 0; ch < CPT / W; ++ch) {
        uint64_t* x = kReload ? d : d + ch * (W / 2);
        if (kReload) logits(ch, x);
#pragma unroll
        for (int k4 = 0; k4 < W / 4; ++k4) {
          uint32_t h[2], l[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x0, x1;
            unpack2(x[2 * k4 + j], x0, x1);
            const uint64_t e = pack2(ex2_approx(x0), ex2_approx(x1));
            uint64_t& ls = lsum[ch * (W / 2) + 2 * k4 + j];
            ls = add2(ls, e);
            float p0, p1;
            unpack2(mul2(e, ab2), p0, p1);
            split2(p0, p1, dither, h[j], l[j]);
          }
          hi[ch * (W / 4) + k4] = h[0] | (h[1] << 16);
          lo[ch * (W / 4) + k4] = l[0] | (l[1] << 16);
        }
      }
      if (kReload) release_s();
    }
    // O(i-1) must be complete before O is rescaled and before P(i) overwrites
    // the P buffer it read; a ragged tile needs its V rows landed before the
    // rows past the end are zeroed.
    if (i > 0 && !wait(C::kOFull, uint32_t(i - 1) & 1)) failed = true;
    if (rows < kRows && !wait(C::kVFull + i % C::SV, uint32_t(i / C::SV) & 1)) failed = true;
    __syncwarp();
    tc_fence_after();
    if (full && !first) {   // rescale what O holds (thread = output column, its heads)
      const uint32_t oc = t_lane + C::kOCol + uint32_t(sidx % C::kOBufs) * C::kN + col0;
#pragma unroll
      for (int ch = 0; ch < CPT / W; ++ch) {
        if (!moved[ch]) continue;
        float v[W], v2[W];
        tmem_ld_two<W>(oc + ch * W, oc + HP + ch * W, v, v2);
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const float al = alpha_o[ch * W + k];
          v[k] *= al;
          v2[k] *= al;
        }
        tmem_st<W>(oc + ch * W, v);
        tmem_st<W>(oc + HP + ch * W, v2);
      }
      tmem_wait_st();
    }
    // P into its lines: byte n of a row's line is column n, 16-byte pieces swizzled
#pragma unroll
    for (int j = 0; j < CPT / 16; ++j) {
      const int p1 = col0 / 16 + j, p2 = (HP + col0) / 16 + j, sw = row & 7;
      *reinterpret_cast<uint4*>(line + ((p1 ^ sw) << 4)) = make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
      *reinterpret_cast<uint4*>(line + ((p2 ^ sw) << 4)) = make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
    }
    if (rows < kRows) {
      // rows past the end were loaded too; zeros in V, so that P = 0 times
      // whatever they hold (NaN codes, say) contributes exactly 0
      unsigned char* vst = r.smem + C::kV + (i % C::SV) * kTileBytes + rows * 128;
      for (int k = tid; k < (kRows - rows) * 8; k += kSoft) *reinterpret_cast<uint4*>(vst + k * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    mbar_arrive(bar(C::kPFull));
    // Off the path to the next product: the previous segment's output (its O is
    // final; with two buffers P.V(i) accumulates into the other one, with one
    // it waits for this), then the next segment's queries (the S products that
    // read the present ones have completed).
    if (pend >= 0) {
      epilogue(pend);
      pend = -1;
    }
    if (last) {
      if (i + 1 < n) {
        if (kReload) soft_barrier<kSoft>();   // the query scales have been read for the last time
        convert_queries<HP>(a, r, w.seq, tid);
      }
#pragma unroll
      for (int ch = 0; ch < CPT / W; ++ch) {
        float v[W];
#pragma unroll
        for (int k = 0; k < W / 2; ++k) unpack2(lsum[ch * (W / 2) + k], v[2 * k], v[2 * k + 1]);
        const float sum = transpose_reduce<W, false>(v, lane);
        if (lane < W) redl[q4 * HP + col0 + ch * W + lane] = sum;
      }
      soft_barrier<kSoft>();
      const int pb = sidx & 1;
      if (q4 == 0 && lane < CPT) {
        const int col = col0 + lane;
        const float l = redl[col] + redl[HP + col] + redl[2 * HP + col] + redl[3 * HP + col];
        linv[pb * HP + col] = scale_of(uint32_t(E)) * (1.f / (1 << kBias)) * rcp_approx(l);
        lse2[pb * HP + col] = lg2_approx(l) - negm[lane];
      }
      pend = sidx;
    }
  }
  if (pend >= 0) {   // the CTA's last segment (all threads come here, or none): wait for its final P.V, then write it
    if (!wait(C::kOFull, uint32_t(n - 1) & 1)) failed = true;
    failed = soft_barrier_or<kSoft>(failed);
    if (!failed) {
      tc_fence_after();
      epilogue(pend);
    }
  }
  if (failed && tid == 0) {
    *r.abort = 1;
    set_flag(r.flags, MQA_FLAG_PIPE_TIMEOUT);
  }
}

template <int HP>
__global__ void __launch_bounds__(Cfg<HP>::kThreads, kCtasPerSm)
    q8_decode_tc_kernel(const TcArgs a, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<HP>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Roles r;
  r.smem = smem_raw;
  r.sbase = smem_u32(smem_raw);
  if (r.sbase & 1023u) {   // the swizzled tiles need a 1024-byte aligned base (uniform across the CTA)
    if (threadIdx.x == 0) set_flag(a.flags, MQA_FLAG_PIPE_TIMEOUT);
    return;
  }
  r.abort = reinterpret_cast<volatile int*>(r.smem + C::kAbort);
  r.flags = a.flags;
  r.group = blockIdx.x / a.g;
  r.head = blockIdx.x - r.group * a.g;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto bar = [&](int id) { return r.sbase + C::kBar + 8u * uint32_t(id); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::SK; ++s) {
      mbar_init(bar(C::kKFull + s), 1);
      mbar_init(bar(C::kKEmpty + s), 1);
    }
    for (int s = 0; s < C::SV; ++s) {
      mbar_init(bar(C::kVFull + s), 1);
      mbar_init(bar(C::kVEmpty + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(C::kSFull + s), 1);
      mbar_init(bar(C::kSEmpty + s), C::kSoft);
    }
    for (int s = 0; s < C::kOBufs; ++s) mbar_init(bar(C::kOFree + s), C::kSoft);
    mbar_init(bar(C::kQFull), C::kSoft);
    mbar_init(bar(C::kPFull), C::kSoft);
    mbar_init(bar(C::kOFull), 1);
    mbar_init(bar(C::kDone), 2);   // one commit from each issuing thread
    *r.abort = 0;
    *reinterpret_cast<int*>(r.smem + C::kKIssued) = 0;
    mbar_fence_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == kSWarp) {
    tmem_alloc(r.sbase + C::kTmemSlot, C::kTmemCols);
    tmem_relinquish();
    tc_fence_before();   // the block barriers of the schedule publish the slot
  }
  // The barriers are initialised before the schedule starts loads on them.
  __syncthreads();
  // Inputs may come from the kernel before this one on the stream (the append).
  // Beside a shared prefix nothing is read that its kernels write, and the first
  // of them has let the others start only after its wait for what came before:
  // that wait stands for this one's, which comes at the end, for the merge.
  // (Inputs are read past the L1, which nothing has cleaned for this grid then.)
  if (!a.partials) asm volatile("griddepcontrol.wait;" ::: "memory");
  int* lens_tab = reinterpret_cast<int*>(r.smem + C::kLens);
  r.lens_s = lens_tab;
  r.seq0 = 0;
  const Run run = make_run<C::kThreads>(
      a, r.group, blockIdx.x == 0, reinterpret_cast<int64_t*>(r.smem + C::kSched), lens_tab,
      [&](int seq, int k0, int own, int len) {
        const uint64_t pol = l2_evict_first_policy();
        const int npre = own < 2 ? own : 2, row0 = len - span_of(len, a.window) + k0 * kRows;
        for (int i = 0; i < npre; ++i) {
          load_tile(a, r.sbase + C::kK + i * kTileBytes, &tm_k, bar(C::kKFull + i), seq, r.head, row0 + i * kRows, pol);
          load_tile(a, r.sbase + C::kV + i * kTileBytes, &tm_v, bar(C::kVFull + i), seq, r.head, row0 + i * kRows, pol);
        }
        return npre;
      });
  if (a.b > kLensCache) {   // the table holds the run's first sequences
    r.seq0 = run.seq;
    if (threadIdx.x < kLensCache && run.seq + int(threadIdx.x) < a.b)
      lens_tab[threadIdx.x] = rows_of(a, run.seq + threadIdx.x, false);
  }
  __syncthreads();
  tc_fence_after();
  r.tmem = *reinterpret_cast<volatile uint32_t*>(r.smem + C::kTmemSlot);
  if (a.no_merge && warp >= kSoftWarp) {   // no merge follows: empty sequences' zero rows
    for (int s = blockIdx.x; s < a.b; s += gridDim.x) {
      if (rows_of(a, s, false) == 0) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + int64_t(s) * a.h * kD);
        for (int k = int(threadIdx.x) - 32 * kSoftWarp; k < a.h * kD / 8; k += C::kSoft) o[k] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  const bool work = run.t_begin < run.t_end;
  if (warp >= kSoftWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoft));
    if (work) softmax_epilogue<HP>(a, run, r, warp, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRoles));
    if (work && lane == 0) {
      if (warp == kKWarp) producer<HP, true>(a, run, r, &tm_k);
      else if (warp == kSWarp) s_issuer<HP>(a, run, r);
      else if (warp == kVWarp) producer<HP, false>(a, run, r, &tm_v);
      else pv_issuer<HP>(a, run, r);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kSWarp) tmem_dealloc(r.tmem, C::kTmemCols);
  if (a.partials) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
}

// ------------------------------------------------------------------ host

template <int HP>
cudaError_t launch(const TcArgs& a, const uint8_t* k, const uint8_t* v, cudaStream_t stream) {
  using C = Cfg<HP>;
  static std::atomic<bool> attr_set[64];   // per device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(q8_decode_tc_kernel<HP>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kAlloc));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true, std::memory_order_relaxed);
  }
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  CUtensorMap tk, tv;
  if (!encode_codes(&tk, k, int64_t(a.b) * a.m, a.g, kRows) || !encode_codes(&tv, v, int64_t(a.b) * a.m, a.g, kRows))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.groups * a.g));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q8_decode_tc_kernel<HP>, a, tk, tv);
}

}  // namespace

bool q8_tc_supported(int d_k, int d_v, int hq, int g) {
  return d_k == kD && d_v == kD && hq >= 1 && hq <= 64 && g <= kMaxCtas;
}

int q8_tc_tile_rows() { return kRows; }

int q8_tc_ctas_per_sm() { return kCtasPerSm; }

// Numbers the kernel keeps in 31 bits: rows (a tile reaches 128 past its
// first), and partition units.
bool q8_tc_fits(int b, int m) {
  return int64_t(b) * m < (int64_t(1) << 31) - 512 &&
         int64_t(b) * (kSegUnits + 4 * ((int64_t(m) + kRows - 1) / kRows)) < (int64_t(1) << 31);
}

cudaError_t launch_q8_decode_tc(const TcArgs& a, const uint8_t* k, const uint8_t* v, cudaStream_t stream) {
  if (!q8_tc_fits(a.b, a.m)) return cudaErrorInvalidValue;
  if (a.hq <= 16) return launch<16>(a, k, v, stream);
  if (a.hq <= 32) return launch<32>(a, k, v, stream);
  return launch<64>(a, k, v, stream);
}

}  // namespace q8
}  // namespace mqa
