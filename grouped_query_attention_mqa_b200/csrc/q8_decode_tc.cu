// Decode attention over an 8-bit cache on the 5th-generation tensor cores, and
// the same for a batch behind one shared prefix: bf16 queries, head size 128,
// up to 64 query heads per K/V head.
//
// The cache's e4m3 codes are the A operand of both products (kind::f8f6f4) as
// TMA lands them; no row is converted.  The other operand of such a product is
// e4m3 too, 4 significant bits, so queries and weights enter as two terms
//   x ~ x1 + x2 / 16,   x1 = e4m3(x),  x2 = e4m3(16 (x - x1)),
// side by side as columns of one product, whose two results are added in fp32.
// A bf16 query scaled by a power of two to a maximum in (224, 448] is
// represented exactly down to 2^-13 of the scaled unit; a weight to 2^-9 of
// itself at worst (a bf16 weight: 2^-8).
//
// With k_t, v_t the codes, a_t, b_t the row scales and w_i the query's scale:
//   S^T[t, n]  = k_t . x_n            M = 128 rows, N = 2 heads' columns, K = 128
//   s_{t,i}    = scale log2(e) w_i a_t (S[t, i] + S[t, i'] / 16)
//   p_{t,i}    = 2^(s_{t,i} - m_i),   l_i = sum_t p_{t,i}            (fp32)
//   P_{t,i}    = p_{t,i} b_t 2^(6-E)  in two terms
//   O^T[c, n] += sum_t v_t[c] P[t, n] M = 128 columns of V, N, K = 128 rows
//   o_i        = 2^(E-6) (O[c, i] + O[c, i'] / 16) / l_i
// E is the largest value-row exponent seen (of rows that are not all zero) and
// m_i is set so that the largest P is 2^6: the e4m3 grid (spacing 2^-9 below
// 2^-6, 2^-13 in the second term) then lies relative to what a row contributes
// to the output, not to its weight alone, and a heavy row with small values (an
// attention sink) leaves the other rows their precision.  A reference is moved
// only when some P would pass 448.
//
// Structure, as in the bf16 decode: one persistent CTA per SM, a contiguous run
// of all segments' tiles each (balanced in quarter tiles, entering a segment
// weighed as a whole tile), partials of split segments joined by a merge
// kernel.  A tile is 256 rows (two 128-row products side by side; 64 KB of K
// and V, which is what one pass through the product-softmax-product chain can
// hide) for up to 32 heads, 128 rows above.  Roles:
//   warp 0, lane 0    K loads;   warp 10, lane 0   V loads (never ahead of K)
//   warp 1, lane 0    S products;   warp 11, lane 0   P.V products
//   warps 2-9         query conversion, softmax, epilogue: two column groups of
//                     four warps, a thread holding one row of each 128-row half
//                     and half of the heads
// Every wait is bounded (one second); on expiry the kernel sets
// MQA_FLAG_PIPE_TIMEOUT, drains its copies and products, frees its tensor
// memory and returns.
//
// Bound: HBM for large caches (d + 1 bytes per row instead of 2 d); the fixed
// costs of a launch for small ones; for a shared prefix, read once per block of
// sequences from L2, the softmax warps.
#include <atomic>
#include <cuda.h>

#include "q8.cuh"
#include "sm100.cuh"

namespace mqa {
namespace q8 {

namespace {

using namespace sm100;

constexpr int kD = 128;
constexpr int kHalfRows = 128;                  // the products' M
constexpr int kThreads = 384;
constexpr int kVWarp = 10, kPvWarp = 11;
constexpr int kSoft = 256;                      // softmax threads (warps 2-9)
constexpr uint32_t kHalfBytes = kHalfRows * kD; // 128 rows of codes, 128-byte swizzled
constexpr uint64_t kTimeoutNs = 1000000000ull;
constexpr int kSegUnits = 4;                    // cost of entering a segment, in quarter tiles
constexpr int kBias = 6;                        // the largest P after a reference is set is 2^kBias
constexpr float kLogCodeMax = 8.807354922f;     // log2(448)
constexpr int kSpan = 60;                       // exponents below E - kSpan count as E - kSpan in the references
constexpr int kLensCache = kThreads;
constexpr uint32_t kMaxDynSmem = 232448;

template <int HP>   // heads per segment, padded
struct Cfg {
  static constexpr int kRH = HP <= 32 ? 2 : 1;                 // 128-row halves per tile
  static constexpr int kRows = kRH * kHalfRows;
  static constexpr int SK = HP <= 32 ? 2 : 4, SV = HP <= 32 ? 3 : 6;
  static constexpr int kN = 2 * HP;                            // columns: first terms, then second terms
  static constexpr uint32_t kTileBytes = kRH * kHalfBytes;
  static constexpr uint32_t kOCol = 2 * kRH * kN;              // tensor memory: S double buffer, then O double buffer
  static constexpr uint32_t kTmemCols = kOCol + 2 * kN <= 256 ? 256 : 512;
  static_assert(kOCol + 2 * kN <= kTmemCols, "tensor memory");
  // barriers
  static constexpr int kKFull = 0, kKEmpty = SK, kVFull = 2 * SK, kVEmpty = 2 * SK + SV, kSFull = 2 * SK + 2 * SV,
                       kSEmpty = kSFull + 2, kPFull = kSEmpty + 2, kOFull = kPFull + 1, kQFull = kOFull + 1,
                       kOFree = kQFull + 2, kDone = kOFree + 2, kNumBars = kDone + 1;
  // shared memory
  static constexpr uint32_t kK = 0;
  static constexpr uint32_t kV = kK + SK * kTileBytes;
  static constexpr uint32_t kQBytes = kN * kD;
  static constexpr uint32_t kQ = kV + SV * kTileBytes;
  static constexpr uint32_t kP = kQ + 2 * kQBytes;             // a 128-byte line per row, kN of it used
  static constexpr uint32_t kBar = kP + kRH * kHalfRows * 128;
  static constexpr uint32_t kTmemSlot = kBar + kNumBars * 8;
  static constexpr uint32_t kAbort = kTmemSlot + 4;
  static constexpr uint32_t kKIssued = kAbort + 4;
  static constexpr uint32_t kQw = (kKIssued + 4 + 15) / 16 * 16;   // [2][HP] query scales
  static constexpr uint32_t kRed = kQw + 2 * HP * 4;           // [4][HP]
  static constexpr uint32_t kMref = kRed + 4 * HP * 4;
  static constexpr uint32_t kAlphaL = kMref + HP * 4;
  static constexpr uint32_t kAlphaO = kAlphaL + HP * 4;
  static constexpr uint32_t kRedL = kAlphaO + HP * 4;          // [4][HP]
  static constexpr uint32_t kLinv = kRedL + 4 * HP * 4;        // [2][HP]
  static constexpr uint32_t kLse = kLinv + 2 * HP * 4;         // [2][HP]
  static constexpr uint32_t kEred = kLse + 2 * HP * 4;         // [4]
  static constexpr uint32_t kLens = kEred + 16;                // [kLensCache]
  static constexpr uint32_t kSched = (kLens + kLensCache * 4 + 15) / 16 * 16;
  static constexpr uint32_t kEnd = kSched + 256;
  static constexpr uint32_t kAlloc = kEnd + 1024;              // room to align the base
  static_assert(kQ % 1024 == 0 && kP % 1024 == 0 && kQBytes % 1024 == 0, "swizzle atoms need 1024-byte alignment");
  static_assert(kAlloc <= kMaxDynSmem, "shared memory budget");
  static_assert((kThreads / 32 + 6) * 8 <= 256, "schedule scratch");
};

__device__ __forceinline__ void soft_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Barriers of the softmax warps that also reduce a flag, so that every thread
// takes the same branch afterwards.
__device__ __forceinline__ bool soft_barrier_and(bool v) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.and.pred po, 1, 256, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(out) : "r"(uint32_t(v)) : "memory");
  return out != 0;
}
__device__ __forceinline__ bool soft_barrier_or(bool v) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.or.pred po, 1, 256, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(out) : "r"(uint32_t(v)) : "memory");
  return out != 0;
}

// Reduction over the 32 lanes of W columns; lane l ends with column l % W.
template <int W, bool kMax>
__device__ __forceinline__ float transpose_reduce(float (&v)[W], int lane) {
#pragma unroll
  for (int o = W / 2; o >= 1; o >>= 1) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const float send = upper ? v[k] : v[k + o];
      const float keep = upper ? v[k + o] : v[k];
      const float recv = __shfl_xor_sync(0xffffffffu, send, o);
      v[k] = kMax ? fmaxf(keep, recv) : keep + recv;
    }
  }
  float r = v[0];
#pragma unroll
  for (int o = W; o < 32; o <<= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, r, o);
    r = kMax ? fmaxf(r, other) : r + other;
  }
  return r;
}

// ------------------------------------------------------------------ work

// Clamped rows of list s.
template <bool kShared>
__device__ __forceinline__ int rows_of(const TcArgs& a, int s, bool report) {
  if constexpr (kShared) {
    const bool pre = s < a.nblk;
    const int m = pre ? a.m_p : a.m;
    const int n = pre ? __ldg(a.plen) : __ldg(a.lens + s - a.nblk);
    const int c = min(max(n, 0), m);
    if (report && c != n) set_flag(a.flags, MQA_FLAG_LEN_CLAMPED);
    return c;
  } else {
    return clamp_len(__ldg(a.lens + s), a.m, a.flags, report);
  }
}

// This CTA's run of tiles (numbers over all segments fit 31 bits: the host
// checks), found as in the bf16 decode: units of a quarter tile, kSegUnits
// more for every segment.
struct Run {
  int t_begin, t_end;   // tiles
  int seq, base, ubase; // list of the first tile, that list's first tile and first unit
  int wtotal, active;
  int pre;              // leading tiles whose loads are already under way
};

__device__ __forceinline__ int units_of(int nb, int g) { return nb > 0 ? g * (kSegUnits + 4 * nb) : 0; }

// The thread whose lists hold the CTA's first tile calls on_first(list, head,
// tile, own, rows, tiles) at once, with `own` >= 1 tiles of that segment
// belonging to the CTA; it returns how many of them it has begun to load.
template <int R, bool kShared, typename OnFirst>
__device__ Run make_run(const TcArgs& a, int cta, int64_t* scratch, int* lens_tab, OnFirst&& on_first) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = a.g;
  const int per = (a.nseq + kThreads - 1) / kThreads;
  const int s0 = min(a.nseq, tid * per), s1 = min(a.nseq, s0 + per);
  int my_t = 0, my_u = 0;
  for (int s = s0; s < s1; ++s) {
    const int len = rows_of<kShared>(a, s, cta == 0);
    if (per == 1) lens_tab[s] = len;
    const int nb = tiles_of(span_of(len, a.window), R);
    my_t += g * nb;
    my_u += units_of(nb, g);
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
  const int cap = W / (kSegUnits + 4);   // every range then holds a tile's start
  run.active = cap < a.grid ? cap : a.grid;
  if (cta >= run.active) return run;     // uniform across the CTA
  const int q = W / run.active, rm = W - q * run.active;   // c*W/A without a 64-bit division
  const int u0 = cta * q + (cta * rm) / run.active;
  const int u1 = (cta + 1) * q + ((cta + 1) * rm) / run.active;
  // Walks this thread's lists to the one that holds unit u: f(list, rows, tiles, first tile, first unit).
  auto locate = [&](int u, auto&& f) {
    if (u < excl_u || u >= excl_u + my_u) return;
    int tb = excl_t, ub = excl_u;
    for (int s = s0; s < s1; ++s) {
      const int len = per == 1 ? lens_tab[s] : rows_of<kShared>(a, s, false);
      const int nb = tiles_of(span_of(len, a.window), R);
      const int su = units_of(nb, g);
      if (u < ub + su) {
        const int seglen = kSegUnits + 4 * nb, rel = u - ub, j = rel / seglen, off = rel - j * seglen;
        f(s, len, nb, j, off <= kSegUnits ? 0 : (off - kSegUnits + 3) / 4, tb, ub);
        return;
      }
      tb += g * nb;
      ub += su;
    }
  };
  if (u1 < W) locate(u1, [&](int, int, int nb, int j, int k, int tb, int) { out[3] = tb + j * nb + k; });
  locate(u0, [&](int s, int len, int nb, int j, int k, int tb, int ub) {
    out[0] = tb + j * nb + k;
    out[1] = s;
    out[2] = tb;
    out[4] = ub;
    int begun = 0;
    if (k < nb) {   // the CTA's tiles of segment j: those whose start unit is below u1
      const int lim = u1 - (ub + j * (kSegUnits + 4 * nb) + kSegUnits);
      const int kend = min(nb, lim <= 0 ? 0 : (lim + 3) / 4);
      if (kend > k) begun = on_first(s, j, k, kend - k, len);
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
  const int* lens_s;   // clamped rows of lists seq0 .. seq0 + kLensCache - 1
  int seq0;
};

template <bool kShared>
__device__ __forceinline__ int list_rows(const TcArgs& a, const Roles& r, int s) {
  const int i = s - r.seq0;
  if (i >= 0 && i < kLensCache) return r.lens_s[i];
  return rows_of<kShared>(a, s, false);
}

__device__ __forceinline__ bool wait_bar(const Roles& r, uint32_t bar, uint32_t parity) {
  if (mbar_wait(bar, parity, kTimeoutNs)) return true;
  *r.abort = 1;
  set_flag(r.flags, MQA_FLAG_PIPE_TIMEOUT);
  return false;
}

// One tile as the roles see it.
struct Tile {
  int seq, head;
  int row0, rows;      // first row of the list's cache, and valid rows
  int sidx;            // the CTA's count of segments
  int seg_t0, nb;      // first tile and tiles of the segment
  bool first, last;    // of the segment, within this CTA
};

// Walks the CTA's tiles in order, counting (tile, head, list) forward.
template <int R, bool kShared>
struct TileWalk {
  int t, base, ubase, seq, head, k, nb, len, lo, sidx;
  __device__ TileWalk(const TcArgs& a, const Run& run, const Roles& r) : t(run.t_begin - 1), sidx(-1) {
    base = run.base;
    ubase = run.ubase;
    set_seq(a, r, run.seq);
    while (run.t_begin >= base + a.g * nb) {   // the first tile may lie in a later list
      base += a.g * nb;
      ubase += units_of(nb, a.g);
      set_seq(a, r, seq + 1);
    }
    const int rel = run.t_begin - base;
    head = rel / nb;
    k = rel - head * nb - 1;
  }
  __device__ void set_seq(const TcArgs& a, const Roles& r, int s) {
    seq = s;
    len = list_rows<kShared>(a, r, s);
    lo = len - span_of(len, a.window);
    nb = tiles_of(len - lo, R);
  }
  __device__ Tile next(const TcArgs& a, const Run& run, const Roles& r) {
    ++t;
    if (++k == nb) {
      k = 0;
      if (++head == a.g) {
        head = 0;
        base += a.g * nb;
        ubase += units_of(nb, a.g);
        do set_seq(a, r, seq + 1);
        while (nb == 0);
      }
    }
    Tile x;
    x.seq = seq;
    x.head = head;
    x.row0 = lo + k * R;
    x.rows = min(R, len - x.row0);
    x.nb = nb;
    x.seg_t0 = base + head * nb;
    x.first = t == run.t_begin || k == 0;
    x.last = k == nb - 1 || t + 1 == run.t_end;
    if (x.first) ++sidx;
    x.sidx = sidx;
    return x;
  }
  __device__ int seg_last_unit() const { return ubase + head * (kSegUnits + 4 * nb) + kSegUnits + 4 * (nb - 1); }
};

// ------------------------------------------------------------------ loads and products

// The maps of one operand: own rows, and the prefix's.
struct Maps {
  const CUtensorMap* own;
  const CUtensorMap* prefix;
};

template <int RH, bool kShared>
__device__ __forceinline__ void load_tile(const TcArgs& a, uint32_t dst, const Maps& maps, uint32_t bar, int seq,
                                          int head, int row0, uint64_t once, uint64_t again) {
  const bool pre = kShared && seq < a.nblk;
  const CUtensorMap* m = pre ? maps.prefix : maps.own;
  const int row = pre ? row0 : (seq - (kShared ? a.nblk : 0)) * a.m + row0;
  mbar_expect_tx(bar, RH * kHalfBytes);
#pragma unroll
  for (int rh = 0; rh < RH; ++rh)
    tma_load_3d(dst + rh * kHalfBytes, m, bar, 0, head, row + rh * kHalfRows, pre ? again : once);
}

// Tiles of the prefix are read again by the other blocks of sequences.
__device__ __forceinline__ uint64_t l2_evict_last_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}

template <int HP, bool kIsK, bool kShared>
__device__ void producer(const TcArgs& a, const Run& run, const Roles& r, const Maps& maps) {
  using C = Cfg<HP>;
  constexpr int S = kIsK ? C::SK : C::SV;
  constexpr int kFull = kIsK ? C::kKFull : C::kVFull, kEmpty = kIsK ? C::kKEmpty : C::kVEmpty;
  constexpr uint32_t kRing = kIsK ? C::kK : C::kV;
  auto bar = [&](int id) { return r.sbase + C::kBar + 8u * uint32_t(id); };
  const uint64_t once = l2_evict_first_policy(), again = kShared ? l2_evict_last_policy() : once;
  volatile int* k_issued = reinterpret_cast<volatile int*>(r.smem + C::kKIssued);
  TileWalk<C::kRows, kShared> w(a, run, r);
  const int n = run.t_end - run.t_begin;
  int i = 0, st = 0;
  uint32_t ph = 1;   // parity of the stage's previous release
  for (; i < n; ++i) {
    const Tile x = w.next(a, run, r);
    if (*r.abort) break;
    if (i >= run.pre) {
      if (i >= S && !wait_bar(r, bar(kEmpty + st), ph)) break;
      if (!kIsK) {   // never run ahead of the K producer: the loads go out K(0), V(0), K(1), ...
        uint32_t polls = 0;
        while (*k_issued <= i && !*r.abort && ++polls < (1u << 24)) {}   // cannot stall for good: K gives up on abort
      }
      load_tile<C::kRH, kShared>(a, r.sbase + kRing + st * C::kTileBytes, maps, bar(kFull + st), x.seq, x.head, x.row0,
                                 once, again);
    }
    if (kIsK) *k_issued = i + 1;
    if (++st == S) {
      st = 0;
      ph ^= 1u;
    }
  }
  // every copy this thread (or the schedule) issued has landed before the CTA can exit
  for (int j = (i - S > 0 ? i - S : 0); j < i; ++j) mbar_wait(bar(kFull + j % S), uint32_t(j / S) & 1, kTimeoutNs);
}

// S(i) = K Q^T once K(i), for a segment's first tile its queries, and S buffer
// i & 1 are there.
template <int HP, bool kShared>
__device__ void s_issuer(const TcArgs& a, const Run& run, const Roles& r) {
  using C = Cfg<HP>;
  constexpr uint32_t idesc = idesc_e4m3_f32(kHalfRows, C::kN, 0, 0);
  const uint64_t kdesc0 = smem_desc_sw128(r.sbase + C::kK, 16, 1024);   // K-major, rows of 128 bytes
  const uint64_t qdesc0 = smem_desc_sw128(r.sbase + C::kQ, 16, 1024);
  auto bar = [&](int id) { return r.sbase + C::kBar + 8u * uint32_t(id); };
  TileWalk<C::kRows, kShared> w(a, run, r);
  const int n = run.t_end - run.t_begin;
  int st = 0;
  uint32_t ph = 0;
  for (int i = 0; i < n; ++i) {
    const Tile x = w.next(a, run, r);
    const int qb = x.sidx & 1;
    if (x.first && !wait_bar(r, bar(C::kQFull + qb), uint32_t(x.sidx >> 1) & 1)) break;
    if (!wait_bar(r, bar(C::kKFull + st), ph)) break;
    if (i >= 2 && !wait_bar(r, bar(C::kSEmpty + (i & 1)), uint32_t((i >> 1) - 1) & 1)) break;
    tc_fence_after();
    const uint64_t ka = kdesc0 + uint64_t((uint32_t(st) * C::kTileBytes) >> 4);
    const uint64_t qa = qdesc0 + uint64_t((uint32_t(qb) * C::kQBytes) >> 4);
    const uint32_t d = r.tmem + uint32_t(i & 1) * (C::kRH * C::kN);
#pragma unroll
    for (int rh = 0; rh < C::kRH; ++rh)
#pragma unroll
      for (int kk = 0; kk < kD / 32; ++kk)
        mma_e4m3_ss(d + rh * C::kN, ka + ((rh * kHalfBytes + kk * 32) >> 4), qa + ((kk * 32) >> 4), idesc, kk > 0);
    mma_commit(bar(C::kSFull + (i & 1)));
    mma_commit(bar(C::kKEmpty + st));
    if (++st == C::SK) {
      st = 0;
      ph ^= 1u;
    }
  }
  // every product issued above has completed before tensor memory is released
  mma_commit(bar(C::kDone));
  mbar_wait(bar(C::kDone), 0, kTimeoutNs);
}

// O += V^T P(i) once P(i) is written, V(i) has landed and, for a segment's
// first tile, its O buffer has been read by the epilogue of the segment two
// back.
template <int HP, bool kShared>
__device__ void pv_issuer(const TcArgs& a, const Run& run, const Roles& r) {
  using C = Cfg<HP>;
  constexpr uint32_t idesc = idesc_e4m3_f32(kD, C::kN, 1, 1);
  const uint64_t vdesc0 = smem_desc_sw128(r.sbase + C::kV, 16, 1024);   // MN-major: one 128-column atom, 8-row groups
  const uint64_t pdesc0 = smem_desc_sw128(r.sbase + C::kP, 16, 1024);
  auto bar = [&](int id) { return r.sbase + C::kBar + 8u * uint32_t(id); };
  TileWalk<C::kRows, kShared> w(a, run, r);
  const int n = run.t_end - run.t_begin;
  int st = 0;
  uint32_t ph = 0;
  for (int i = 0; i < n; ++i) {
    const Tile x = w.next(a, run, r);
    const int ob = x.sidx & 1;
    if (!wait_bar(r, bar(C::kPFull), uint32_t(i & 1))) break;
    if (!wait_bar(r, bar(C::kVFull + st), ph)) break;
    if (x.first && x.sidx >= 2 && !wait_bar(r, bar(C::kOFree + ob), uint32_t((x.sidx >> 1) - 1) & 1)) break;
    tc_fence_after();
    const uint64_t va = vdesc0 + uint64_t((uint32_t(st) * C::kTileBytes) >> 4);
    const uint32_t d = r.tmem + C::kOCol + uint32_t(ob) * C::kN;
    const uint32_t acc0 = x.first ? 0u : 1u;
#pragma unroll
    for (int kk = 0; kk < C::kRows / 32; ++kk)   // 32 rows: four 8-row groups of 1024 bytes
      mma_e4m3_ss(d, va + ((kk * 4096) >> 4), pdesc0 + ((kk * 4096) >> 4), idesc, kk > 0 ? 1u : acc0);
    mma_commit(bar(C::kOFull));
    mma_commit(bar(C::kVEmpty + st));
    if (++st == C::SV) {
      st = 0;
      ph ^= 1u;
    }
  }
  mma_commit(bar(C::kDone));
  mbar_wait(bar(C::kDone), 0, kTimeoutNs);
}

// ------------------------------------------------------------------ softmax

// bf16 query row of column n of a segment, or nullptr.
template <bool kShared>
__device__ __forceinline__ const __nv_bfloat16* query_row(const TcArgs& a, int seq, int head, int n) {
  int s = seq, i = n;
  if constexpr (kShared) {
    if (seq < a.nblk) {
      const int w = n / a.hq;
      i = n - w * a.hq;
      s = w < a.spb ? seq * a.spb + w : a.b;
      if (s >= a.b) return nullptr;
    } else {
      s = seq - a.nblk;
    }
  }
  return i < a.hq ? a.q + (int64_t(s) * a.h + int64_t(head) * a.hq + i) * kD : nullptr;
}

// Columns of a segment that stand for a query.
template <bool kShared>
__device__ __forceinline__ int query_cols(const TcArgs& a, int seq) {
  if constexpr (kShared)
    if (seq < a.nblk) return min(a.spb, a.b - seq * a.spb) * a.hq;
  return a.hq;
}

// The segment's queries, two e4m3 terms each, into Q buffer qb; eight threads
// per row.  A row is scaled by the power of two its largest element asks for.
template <int HP, bool kShared>
__device__ __forceinline__ void convert_queries(const TcArgs& a, const Roles& r, int seq, int head, int qb, int tid) {
  using C = Cfg<HP>;
  unsigned char* qs = r.smem + C::kQ + qb * C::kQBytes;
  float* qw = reinterpret_cast<float*>(r.smem + C::kQw) + qb * HP;
  const int part = tid & 7;
#pragma unroll
  for (int pass = 0; pass < (HP + 31) / 32; ++pass) {
    const int n = pass * 32 + (tid >> 3);
    if (n < HP) {   // whole warps: HP is a multiple of 16, a warp holds four rows
      const __nv_bfloat16* row = query_row<kShared>(a, seq, head, n);
      uint4 w[2] = {};
      if (row != nullptr) {
        w[0] = *reinterpret_cast<const uint4*>(row + part * 16);
        w[1] = *reinterpret_cast<const uint4*>(row + part * 16 + 8);
      }
      float x[16];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t u = k < 4 ? (&w[0].x)[k] : (&w[1].x)[k - 4];
        const float2 f = bf16x2_to_f32x2(u);
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) amax = fabsf(x[k]) < INFINITY ? fmaxf(amax, fabsf(x[k])) : amax;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const uint32_t e = exponent_for(amax);
      const float inv = inverse_scale(e);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t h2[2], l2[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float y[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const float v = x[4 * k + 2 * j + z];
            y[z] = fabsf(v) < INFINITY ? v * inv : NAN;   // an infinite query gives NaN logits, not saturated ones
          }
          h2[j] = to_e4m3x2(y[0], y[1]);
          const float2 f = from_e4m3x2(h2[j]);
          l2[j] = to_e4m3x2((y[0] - f.x) * 16.f, (y[1] - f.y) * 16.f);
        }
        hi[k] = h2[0] | (h2[1] << 16);
        lo[k] = l2[0] | (l2[1] << 16);
      }
      const int n2 = HP + n;
      *reinterpret_cast<uint4*>(qs + n * 128 + ((part ^ (n & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(qs + n2 * 128 + ((part ^ (n2 & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      if (part == 0) qw[n] = scale_of(e);
    }
  }
  fence_proxy_async_smem();
  mbar_arrive(r.sbase + C::kBar + 8u * uint32_t(C::kQFull + qb));
}

// Four weights -> their two e4m3 terms, four codes each.
__device__ __forceinline__ void split4(float p0, float p1, float p2, float p3, uint32_t& hi, uint32_t& lo) {
  const uint32_t ha = to_e4m3x2(p0, p1), hb = to_e4m3x2(p2, p3);
  const float2 fa = from_e4m3x2(ha), fb = from_e4m3x2(hb);
  const uint32_t la = to_e4m3x2((p0 - fa.x) * 16.f, (p1 - fa.y) * 16.f);
  const uint32_t lb = to_e4m3x2((p2 - fb.x) * 16.f, (p3 - fb.y) * 16.f);
  hi = ha | (hb << 16);
  lo = la | (lb << 16);
}

// First and second terms of N columns of this thread's lane.
template <int N>
__device__ __forceinline__ void load_terms(uint32_t t1, uint32_t t2, float (&x1)[N], float (&x2)[N]) {
  if constexpr (N <= 16) {
    tmem_ld_two<N>(t1, t2, x1, x2);
  } else {
    tmem_ld<N>(t1, x1);
    tmem_ld<N>(t2, x2);
  }
}

template <int HP, bool kShared>
__device__ void softmax_epilogue(const TcArgs& a, const Run& run, const Roles& r, int warp, int lane) {
  using C = Cfg<HP>;
  constexpr int RH = C::kRH;
  constexpr int CPT = HP / 2;                      // heads per thread
  constexpr int W = CPT < 16 ? CPT : 16;
  auto bar = [&](int id) { return r.sbase + C::kBar + 8u * uint32_t(id); };
  auto wait = [&](int id, uint32_t parity) { return mbar_wait(bar(id), parity, kTimeoutNs); };
  const int q4 = warp & 3;                         // tensor-memory lane quarter of this warp
  const int grp = (warp - 2) >> 2;                 // column group: heads [grp*CPT, grp*CPT + CPT)
  const int gw = (warp - 2) & 3;
  const int col0 = grp * CPT;
  const int tid = threadIdx.x - 64;
  const int row = 32 * q4 + lane;                  // row of a half (S), output column (O)
  const uint32_t t_lane = r.tmem + (uint32_t(32 * q4) << 16);
  float* red = reinterpret_cast<float*>(r.smem + C::kRed);
  float* mref = reinterpret_cast<float*>(r.smem + C::kMref);
  float* alpha_l = reinterpret_cast<float*>(r.smem + C::kAlphaL);
  float* alpha_o = reinterpret_cast<float*>(r.smem + C::kAlphaO);
  float* redl = reinterpret_cast<float*>(r.smem + C::kRedL);
  float* linv = reinterpret_cast<float*>(r.smem + C::kLinv);
  float* lse2 = reinterpret_cast<float*>(r.smem + C::kLse);
  int* ered = reinterpret_cast<int*>(r.smem + C::kEred);
  const float c = a.scale * kLog2e;
  float lpart[CPT];                                // this thread's share of the sums
  float mr[CPT];                                   // references, mirrored from shared memory
  float d[RH][CPT];                                // s - m
  int E = 0;                                       // the value exponent P is relative to

  TileWalk<C::kRows, kShared> w(a, run, r);
  const int n = run.t_end - run.t_begin;
  Tile nx = w.next(a, run, r);
  int nx_unit = w.seg_last_unit();
  uint32_t nke[RH], nve[RH];                       // the next tile's row exponents
  auto load_exps = [&](const Tile& x) {
    const bool pre = kShared && x.seq < a.nblk;
    const int64_t at = pre ? int64_t(x.head) * a.m_p + x.row0
                           : (int64_t(x.seq - (kShared ? a.nblk : 0)) * a.g + x.head) * a.m + x.row0;
    const uint8_t* ke = (pre ? a.pke : a.ke) + at;
    const uint8_t* ve = (pre ? a.pve : a.ve) + at;
#pragma unroll
    for (int rh = 0; rh < RH; ++rh) {
      const int rr = rh * kHalfRows + row;
      nke[rh] = rr < x.rows ? ke[rr] : 0u;
      nve[rh] = rr < x.rows ? ve[rr] : 0u;
    }
  };
  load_exps(nx);
  convert_queries<HP, kShared>(a, r, nx.seq, nx.head, 0, tid);
  int pv_waited = -1;
  bool failed = false;

  // A finished segment whose output is written one tile later, once the P.V
  // product of its last tile is known to have completed.
  struct Pending {
    bool on, whole, owns_first;
    int sidx, seq, head, last_unit;
  } pend;
  pend.on = false;

  auto epilogue = [&](const Pending& e) {
    const int pb = e.sidx & 1;
    const int64_t seg = int64_t(e.seq) * a.g + e.head;
    const int64_t slot = partial_slot(blockIdx.x, seg);
    const int nc = query_cols<kShared>(a, e.seq);
    const uint32_t oc = t_lane + C::kOCol + uint32_t(pb) * C::kN + col0;
    float v[CPT], v2[CPT];
    load_terms<CPT>(oc, oc + HP, v, v2);
#pragma unroll
    for (int k = 0; k < CPT; ++k) v[k] = fmaf(v2[k], 0.0625f, v[k]) * linv[pb * HP + col0 + k];
    if (!kShared && e.whole) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) +
                           (int64_t(e.seq) * a.h + int64_t(e.head) * a.hq + col0) * kD + row;
#pragma unroll
      for (int k = 0; k < CPT; ++k)
        if (col0 + k < nc) dst[k * kD] = __float2bfloat16_rn(v[k]);
    } else {
      float* dst = a.ws.part_o + (slot * a.cols + col0) * kD + row;
#pragma unroll
      for (int k = 0; k < CPT; ++k)
        if (col0 + k < nc) dst[k * kD] = v[k];
    }
    if (warp == 2) {
      if (kShared || !e.whole)
        for (int col = lane; col < nc; col += 32) a.ws.part_lse[slot * a.cols + col] = lse2[pb * HP + col];
      if (e.owns_first && lane == 0)
        a.ws.seg_info[seg] = make_int2(blockIdx.x, cta_of_unit(e.last_unit, run.wtotal, run.active));
    }
    tc_fence_before();
    mbar_arrive(bar(C::kOFree + pb));
  };

  for (int i = 0; i < n; ++i) {
    const Tile x = nx;
    const int x_unit = nx_unit;
    float kr[RH];
    int er[RH];
    bool valid[RH];
#pragma unroll
    for (int rh = 0; rh < RH; ++rh) {
      valid[rh] = rh * kHalfRows + row < x.rows;
      kr[rh] = scale_of(nke[rh]) * c;
      er[rh] = int(nve[rh]);
    }
    if (i + 1 < n) {   // what the next tile needs from memory
      nx = w.next(a, run, r);
      nx_unit = w.seg_last_unit();
      load_exps(nx);
    }
    if (x.first) {
#pragma unroll
      for (int k = 0; k < CPT; ++k) lpart[k] = 0.f;
    }
    const bool ok = wait(C::kSFull + (i & 1), uint32_t(i >> 1) & 1);
    tc_fence_after();
    if (x.first) soft_barrier();   // the query scales of this segment are all written
    {
      const float* qw = reinterpret_cast<const float*>(r.smem + C::kQw) + (x.sidx & 1) * HP + col0;
      const uint32_t sb = t_lane + uint32_t(i & 1) * (RH * C::kN) + col0;
#pragma unroll
      for (int rh = 0; rh < RH; ++rh) {
        float s2[CPT];
        load_terms<CPT>(sb + rh * C::kN, sb + rh * C::kN + HP, d[rh], s2);
        if (rh == RH - 1) {
          tc_fence_before();
          mbar_arrive(bar(C::kSEmpty + (i & 1)));   // S buffer i&1 may take S(i+2)
        }
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
          const float s = fmaf(s2[k], 0.0625f, d[rh][k]) * qw[k];
          const float m = x.first ? 0.f : mr[k];
          d[rh][k] = valid[rh] ? fmaf(s, kr[rh], -m) : -INFINITY;
        }
      }
    }
    // Would some P pass the largest code?
    bool exceed = false;
    if (!x.first) {
#pragma unroll
      for (int rh = 0; rh < RH; ++rh) {
        float t[CPT];
#pragma unroll
        for (int k = 0; k < CPT; ++k) t[k] = d[rh][k];
#pragma unroll
        for (int span = CPT / 2; span >= 1; span >>= 1)
#pragma unroll
          for (int k = 0; k < span; ++k) t[k] = fmaxf(t[k], t[k + span]);
        exceed |= t[0] + float(max(er[rh] - E, -kSpan) + kBias) > kLogCodeMax;
      }
    }
    const bool full = x.first || soft_barrier_or(exceed);
    if (full) {
      int em = 0;   // the largest value exponent of the tile, rows of zeros aside
#pragma unroll
      for (int rh = 0; rh < RH; ++rh) em = max(em, er[rh] > 1 ? er[rh] : 0);
      em = __reduce_max_sync(0xffffffffu, em);
      if (grp == 0 && lane == 0) ered[gw] = em;
      soft_barrier();
      em = max(max(ered[0], ered[1]), max(ered[2], ered[3]));
      const int E_old = E;
      E = x.first ? em : max(E, em);
      if (E == 0) E = 119;   // no value yet: a middling 2^-8
#pragma unroll
      for (int ch = 0; ch < CPT / W; ++ch) {
        float v[W];
#pragma unroll
        for (int k = 0; k < W; ++k) {
          float t = -INFINITY;
#pragma unroll
          for (int rh = 0; rh < RH; ++rh) t = fmaxf(t, d[rh][ch * W + k] + float(max(er[rh] - E, -kSpan)));
          v[k] = x.first ? t : t + mr[ch * W + k];
        }
        const float mx = transpose_reduce<W, true>(v, lane);
        if (lane < W) red[gw * HP + col0 + ch * W + lane] = mx;
      }
      soft_barrier();
      if (gw == 0) {   // one warp per column group decides for its heads
        for (int col = col0 + lane; col < col0 + CPT; col += 32) {
          float mn = fmaxf(fmaxf(red[col], red[HP + col]), fmaxf(red[2 * HP + col], red[3 * HP + col]));
          if (!x.first) {
            const float old = mref[col], now = old + float(E_old - E);   // the old reference relative to E
            mn = fmaxf(mn, now);
            alpha_l[col] = ex2_approx(old - mn);
            alpha_o[col] = ex2_approx(now - mn);
          }
          mref[col] = mn;
        }
      }
      soft_barrier();
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        const float mn = mref[col0 + k], delta = x.first ? -mn : mr[k] - mn;
#pragma unroll
        for (int rh = 0; rh < RH; ++rh) d[rh][k] += delta;
        mr[k] = mn;
        if (!x.first) lpart[k] *= alpha_l[col0 + k];
      }
    }
    // P in two terms, into registers before waiting for the previous product
    uint32_t hi[RH][CPT / 4], lo[RH][CPT / 4];
#pragma unroll
    for (int rh = 0; rh < RH; ++rh) {
      const int f = er[rh] - E + 127 + kBias;   // the factor b_t 2^(kBias - E): a power of two, 0 for a zero scale
      const float ab = er[rh] == 0 || f <= 0 ? 0.f : __uint_as_float(uint32_t(min(f, 254)) << 23);
#pragma unroll
      for (int k4 = 0; k4 < CPT / 4; ++k4) {
        float p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float e = ex2_approx(d[rh][4 * k4 + k]);
          lpart[4 * k4 + k] += e;
          p[k] = e * ab;
        }
        split4(p[0], p[1], p[2], p[3], hi[rh][k4], lo[rh][k4]);
      }
    }
    // O(i-1) must be complete before O is rescaled and before P(i) overwrites
    // the P buffer it read; a ragged tile needs its V rows landed before the
    // rows past the end are zeroed.
    bool ok2 = true;
    if (i > 0 && pv_waited < i - 1) {
      ok2 = wait(C::kOFull, uint32_t(i - 1) & 1);
      pv_waited = i - 1;
    }
    const int st = i % C::SV;
    if (x.rows < C::kRows) ok2 = wait(C::kVFull + st, uint32_t(i / C::SV) & 1) && ok2;
    if (!soft_barrier_and(ok && ok2)) {
      failed = true;
      break;
    }
    tc_fence_after();
    if (full && !x.first) {   // rescale what O holds (thread = output column, its heads)
      const uint32_t oc = t_lane + C::kOCol + uint32_t(x.sidx & 1) * C::kN + col0;
#pragma unroll
      for (int term = 0; term < 2; ++term) {
        float v[CPT];
        tmem_ld<CPT>(oc + term * HP, v);
#pragma unroll
        for (int k = 0; k < CPT; ++k) v[k] *= alpha_o[col0 + k];
        tmem_st<CPT>(oc + term * HP, v);
      }
      tmem_wait_st();
    }
    // P into its lines: byte n of a row's line is column n, 16-byte pieces swizzled
#pragma unroll
    for (int rh = 0; rh < RH; ++rh) {
      unsigned char* line = r.smem + C::kP + (rh * kHalfRows + row) * 128;
      const int sw = row & 7;
#pragma unroll
      for (int term = 0; term < 2; ++term) {
        const uint32_t* src = term ? lo[rh] : hi[rh];
        const int b0 = term * HP + col0;
        if constexpr (CPT >= 16) {
#pragma unroll
          for (int j = 0; j < CPT / 16; ++j)
            *reinterpret_cast<uint4*>(line + (((b0 / 16 + j) ^ sw) << 4)) =
                make_uint4(src[4 * j], src[4 * j + 1], src[4 * j + 2], src[4 * j + 3]);
        } else {
          static_assert(CPT >= 16 || CPT == 8, "8 heads per thread");
          *reinterpret_cast<uint2*>(line + (((b0 / 16) ^ sw) << 4) + (b0 & 15)) = make_uint2(src[0], src[1]);
        }
      }
    }
    if (x.rows < C::kRows) {
      // rows past the end were loaded too; zeros in V, so that P = 0 times
      // whatever they hold (NaN codes, say) contributes exactly 0
      unsigned char* vst = r.smem + C::kV + st * C::kTileBytes + x.rows * 128;
      for (int k = tid; k < (C::kRows - x.rows) * 8; k += kSoft) *reinterpret_cast<uint4*>(vst + k * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    mbar_arrive(bar(C::kPFull));
    // Off the path to the next product: the next segment's queries, then the
    // previous segment's output (its O buffer is final, and P.V(i) accumulates
    // into the other).  The Q buffer written was last read by S products of the
    // segment before this one, which have completed.
    if (i + 1 < n && nx.first) convert_queries<HP, kShared>(a, r, nx.seq, nx.head, nx.sidx & 1, tid);
    if (pend.on) {
      epilogue(pend);
      pend.on = false;
    }

    if (x.last) {
#pragma unroll
      for (int ch = 0; ch < CPT / W; ++ch) {
        float v[W];
#pragma unroll
        for (int k = 0; k < W; ++k) v[k] = lpart[ch * W + k];
        const float sum = transpose_reduce<W, false>(v, lane);
        if (lane < W) redl[gw * HP + col0 + ch * W + lane] = sum;
      }
      soft_barrier();
      const int pb = x.sidx & 1;
      if (gw == 0)
        for (int col = col0 + lane; col < col0 + CPT; col += 32) {
          const float l = redl[col] + redl[HP + col] + redl[2 * HP + col] + redl[3 * HP + col];
          linv[pb * HP + col] = scale_of(uint32_t(E)) * (1.f / (1 << kBias)) * rcp_approx(l);
          lse2[pb * HP + col] = mref[col] + lg2_approx(l);
        }
      pend.on = true;
      pend.sidx = x.sidx;
      pend.seq = x.seq;
      pend.head = x.head;
      pend.owns_first = x.seg_t0 >= run.t_begin;
      pend.whole = pend.owns_first && x.seg_t0 + x.nb <= run.t_end;
      pend.last_unit = x_unit;
    }
  }
  if (!failed && pend.on) {   // the CTA's last segment: wait for its final P.V, then write it
    bool ok = true;
    if (pv_waited < n - 1) ok = wait(C::kOFull, uint32_t(n - 1) & 1);
    if (soft_barrier_and(ok)) {
      tc_fence_after();
      epilogue(pend);
    } else {
      failed = true;
    }
  }
  if (failed && tid == 0) {
    *r.abort = 1;
    set_flag(r.flags, MQA_FLAG_PIPE_TIMEOUT);
  }
}

// One CTA per SM; 12 warps cap a thread at 168 registers.
template <int HP, bool kShared>
__global__ void __launch_bounds__(kThreads, 1)
    q8_decode_tc_kernel(const TcArgs a, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_pk, const __grid_constant__ CUtensorMap tm_pv) {
  using C = Cfg<HP>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), pad = (1024u - (raw & 1023u)) & 1023u;
  Roles r;
  r.smem = smem_raw + pad;
  r.sbase = raw + pad;
  r.abort = reinterpret_cast<volatile int*>(r.smem + C::kAbort);
  r.flags = a.flags;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto bar = [&](int id) { return r.sbase + C::kBar + 8u * uint32_t(id); };
  const Maps mk = {&tm_k, &tm_pk}, mv = {&tm_v, &tm_pv};
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
      mbar_init(bar(C::kSEmpty + s), kSoft);
      mbar_init(bar(C::kQFull + s), kSoft);
      mbar_init(bar(C::kOFree + s), kSoft);
    }
    mbar_init(bar(C::kPFull), kSoft);
    mbar_init(bar(C::kOFull), 1);
    mbar_init(bar(C::kDone), 2);   // one commit from each issuing thread
    *r.abort = 0;
    *reinterpret_cast<int*>(r.smem + C::kKIssued) = 0;
    mbar_fence_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    if (kShared) {
      prefetch_tensormap(&tm_pk);
      prefetch_tensormap(&tm_pv);
    }
  }
  if (warp == 1) {
    tmem_alloc(r.sbase + C::kTmemSlot, C::kTmemCols);
    tmem_relinquish();
    tc_fence_before();   // the block barriers of the schedule publish the slot
  }
  // The barriers are initialised before the schedule starts loads on them.
  __syncthreads();
  // Inputs may come from the kernel before this one on the stream (the append).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int* lens_tab = reinterpret_cast<int*>(r.smem + C::kLens);
  r.lens_s = lens_tab;
  r.seq0 = 0;
  const Run run = make_run<C::kRows, kShared>(
      a, blockIdx.x, reinterpret_cast<int64_t*>(r.smem + C::kSched), lens_tab,
      [&](int seq, int head, int k0, int own, int len) {
        const uint64_t once = l2_evict_first_policy(), again = kShared ? l2_evict_last_policy() : once;
        const int npre = own < 2 ? own : 2, row0 = len - span_of(len, a.window) + k0 * C::kRows;
        for (int i = 0; i < npre; ++i) {
          load_tile<C::kRH, kShared>(a, r.sbase + C::kK + i * C::kTileBytes, mk, bar(C::kKFull + i), seq, head,
                                     row0 + i * C::kRows, once, again);
          load_tile<C::kRH, kShared>(a, r.sbase + C::kV + i * C::kTileBytes, mv, bar(C::kVFull + i), seq, head,
                                     row0 + i * C::kRows, once, again);
        }
        return npre;
      });
  if (a.nseq > kThreads) {   // the table holds the CTA's first lists
    r.seq0 = run.seq;
    if (run.seq + int(threadIdx.x) < a.nseq) lens_tab[threadIdx.x] = rows_of<kShared>(a, run.seq + threadIdx.x, false);
  }
  __syncthreads();
  tc_fence_after();
  r.tmem = *reinterpret_cast<volatile uint32_t*>(r.smem + C::kTmemSlot);
  if (!kShared && a.no_merge && warp >= 2 && warp < kVWarp) {   // no merge follows: empty sequences' zero rows
    for (int s = blockIdx.x; s < a.b; s += gridDim.x) {
      if (clamp_len(__ldg(a.lens + s), a.m, nullptr, false) == 0) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + int64_t(s) * a.h * kD);
        for (int k = int(threadIdx.x) - 64; k < a.h * kD / 8; k += kSoft) o[k] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  if (run.t_begin < run.t_end) {
    if (warp == 0) {
      if (lane == 0) producer<HP, true, kShared>(a, run, r, mk);
    } else if (warp == 1) {
      if (lane == 0) s_issuer<HP, kShared>(a, run, r);
    } else if (warp == kPvWarp) {
      if (lane == 0) pv_issuer<HP, kShared>(a, run, r);
    } else if (warp == kVWarp) {
      if (lane == 0) producer<HP, false, kShared>(a, run, r, mv);
    } else {
      softmax_epilogue<HP, kShared>(a, run, r, warp, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(r.tmem, C::kTmemCols);
  asm volatile("griddepcontrol.launch_dependents;");
}

// ------------------------------------------------------------------ merge of a shared prefix

// One output row of one head: the partials of its prefix segment (one per CTA
// that held part of it) and of its own rows' segment, weighted with their
// log-sum-exps.  Lists without rows left nothing and are skipped.
constexpr int kMergeThreads = 128;

__global__ void __launch_bounds__(kMergeThreads) q8_merge_shared_kernel(const TcArgs a) {
  const int64_t item = int64_t(blockIdx.x) * (kMergeThreads / 32) + threadIdx.x / 32;   // (sequence, head)
  const int c4 = (threadIdx.x % 32) * 4;
  const bool active = item < int64_t(a.b) * a.h;
  const int s = active ? int(item / a.h) : 0, head = active ? int(item - int64_t(s) * a.h) : 0;
  const int j = head / a.hq, i = head - j * a.hq;
  const bool has[2] = {__ldg(a.plen) > 0, __ldg(a.lens + s) > 0};   // inputs: not written by the kernel before
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  if (!active) return;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    if (!has[part]) continue;
    const int list = part == 0 ? s / a.spb : a.nblk + s;
    const int col = part == 0 ? (s - list * a.spb) * a.hq + i : i;
    const int64_t seg = int64_t(list) * a.g + j;
    const int2 info = a.ws.seg_info[seg];
#pragma unroll 4
    for (int cta = info.x; cta <= info.y; ++cta) {
      const int64_t at = partial_slot(cta, seg) * a.cols + col;
      const float lse = __ldcg(a.ws.part_lse + at);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a.ws.part_o + at * kD + c4));
      const float mn = fmaxf(m, lse);
      const float wo = exp2f(m - mn), wn = exp2f(lse - mn);
      acc.x = acc.x * wo + v.x * wn;
      acc.y = acc.y * wo + v.y * wn;
      acc.z = acc.z * wo + v.z * wn;
      acc.w = acc.w * wo + v.w * wn;
      l = l * wo + wn;
      m = mn;
    }
  }
  const float inv = has[0] || has[1] ? 1.f / l : 0.f;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 out;
  out.x = *reinterpret_cast<const uint32_t*>(&lo);
  out.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + item * kD + c4) = out;
}

// ------------------------------------------------------------------ host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::atomic<EncodeTiledFn> cached{nullptr};
  EncodeTiledFn fn = cached.load(std::memory_order_relaxed);
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      cached.store(fn = reinterpret_cast<EncodeTiledFn>(p), std::memory_order_relaxed);
  }
  return fn;
}

// Codes [rows, g, 128] as (128, g, rows); a box is 128 rows of one K/V head.
bool encode_codes(CUtensorMap* m, const void* base, int64_t rows, int g) {
  const cuuint64_t dims[3] = {cuuint64_t(kD), cuuint64_t(g), cuuint64_t(rows)};
  const cuuint64_t strides[2] = {cuuint64_t(kD), cuuint64_t(g) * kD};
  const cuuint32_t box[3] = {kD, 1, kHalfRows};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HP, bool kShared>
cudaError_t launch(const TcArgs& a, const uint8_t* k, const uint8_t* v, const uint8_t* pk, const uint8_t* pv,
                   cudaStream_t stream) {
  using C = Cfg<HP>;
  static std::atomic<bool> attr_set[64];   // per device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(q8_decode_tc_kernel<HP, kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kAlloc));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true, std::memory_order_relaxed);
  }
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  CUtensorMap tk, tv, tpk, tpv;
  if (!encode_codes(&tk, k, int64_t(a.b) * a.m, a.g) || !encode_codes(&tv, v, int64_t(a.b) * a.m, a.g))
    return cudaErrorInvalidValue;
  if (kShared && (!encode_codes(&tpk, pk, a.m_p, a.g) || !encode_codes(&tpv, pv, a.m_p, a.g)))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q8_decode_tc_kernel<HP, kShared>, a, tk, tv, kShared ? tpk : tk, kShared ? tpv : tv);
}

// Numbers the kernel keeps in 31 bits: rows (a tile's second half reaches 256
// past its first), and partition units.
bool fits(const TcArgs& a, int rows) {
  const int64_t longest = a.m > a.m_p ? a.m : a.m_p;
  return int64_t(a.b) * a.m < (int64_t(1) << 31) - 512 && int64_t(a.m_p) < (int64_t(1) << 31) - 512 &&
         int64_t(a.nseq) * a.g * (kSegUnits + 4 * ((longest + rows - 1) / rows)) < (int64_t(1) << 31);
}

}  // namespace

bool q8_tc_supported(int d_k, int d_v, int hq) { return d_k == kD && d_v == kD && hq >= 1 && hq <= 64; }

int q8_tc_tile_rows(int hq) { return hq <= 32 ? Cfg<32>::kRows : Cfg<64>::kRows; }

int q8_shared_block(int hq) { return 64 / hq; }

cudaError_t launch_q8_decode_tc(const DecodeQ8Args& d, cudaStream_t stream) {
  TcArgs a = {};
  a.o = d.o;
  a.q = static_cast<const __nv_bfloat16*>(d.q);
  a.ke = d.ke;
  a.ve = d.ve;
  a.lens = d.lens;
  a.b = a.nseq = d.b;
  a.h = d.h;
  a.g = d.g;
  a.hq = a.cols = d.hq;
  a.m = d.m_max;
  a.window = d.window;
  a.no_merge = d.no_merge;
  a.scale = d.scale;
  a.ws = d.ws;
  a.flags = d.flags;
  a.grid = d.grid;
  if (!fits(a, q8_tc_tile_rows(a.hq))) return cudaErrorInvalidValue;
  if (a.hq <= 16) return launch<16, false>(a, d.k, d.v, nullptr, nullptr, stream);
  if (a.hq <= 32) return launch<32, false>(a, d.k, d.v, nullptr, nullptr, stream);
  return launch<64, false>(a, d.k, d.v, nullptr, nullptr, stream);
}

cudaError_t launch_q8_decode_shared(const TcArgs& a, const uint8_t* pk, const uint8_t* pv, const uint8_t* k,
                                    const uint8_t* v, cudaStream_t stream) {
  if (!fits(a, Cfg<64>::kRows)) return cudaErrorInvalidValue;
  const cudaError_t e = launch<64, true>(a, k, v, pk, pv, stream);
  if (e != cudaSuccess) return e;
  const int64_t items = int64_t(a.b) * a.h, ctas = (items + kMergeThreads / 32 - 1) / (kMergeThreads / 32);
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q8_merge_shared_kernel, a);
}

}  // namespace q8
}  // namespace mqa
