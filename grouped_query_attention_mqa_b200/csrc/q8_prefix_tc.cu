// A prefix shared by a whole batch, in an 8-bit cache, on the tensor cores:
// every query row of the batch against the prefix's keys and values, computed
// in blocks of 128 rows, so that a staged tile serves 128 rows and the work is
// that of a matrix product, not of a stream.
//
// The rows of one K/V head j are the pairs (sequence, head of the group), in
// that order; a block takes 128 of them.  With x = q / w in two e4m3 terms, the
// codes k, v and the row scales a, b (see the decode kernel for the terms'
// precision):
//   S[r, t]  = (x1_r + x2_r) . k_t     M = 128 query rows, N = 64 keys, K = 2 x 128
//   s_{r,t}  = scale log2(e) w_r a_t S[r, t],   p = 2^(s - m_r),  l_r = sum_t p
//   P[r, t]  = p b_t 2^(6-E)           in two e4m3 terms P1 + P2, P2 = e4m3(P - P1)
//   O[r, c] += sum_t (P1 + P2)[r, t] v_t[c]      M = 128, N = 128, K = 2 x 64
//   o_r      = 2^(E-6) O[r, :] / l_r
// Here query rows are the products' M, so that a row's softmax is one thread's
// own: no barrier and no reduction across threads, and a reference that has to
// move (some P would pass 448) concerns its warp alone.  Both terms of P go into
// one accumulator; the grid that this leaves the small weights is 2^-9 where
// the largest P is 2^6 or more.
//
// Work: all (head, block) segments have the same number of 64-key tiles; the
// persistent CTAs take equal contiguous runs of them, and every (CTA, segment)
// leaves a normalised partial with its log-sum-exp for the merge.  Two CTAs per
// SM hide each other's chain of product, softmax and product.  Roles: warp 0 K
// loads, warp 1 S products, warp 3 P.V products (one lane each); warp 2 V loads
// (one lane) and, with all lanes, the tile's tables: key scales, value factors
// and exponents, and E, which depend on the cached exponents alone (676 of a
// tile's 3,700 cycles while the softmax warps made them); warps 4-7 queries,
// softmax and output, a row per thread.  P has two buffers, so that P(i) need
// not wait for the product of P(i-1).  Every wait is bounded (one second) and
// reported with MQA_FLAG_PIPE_TIMEOUT.
//
// Bound: the softmax threads' instructions and latency (the products need about
// 400 cycles per tile and SM, the exponentials 512).
#include "q8_tc.cuh"

namespace mqa {
namespace q8 {

namespace {

using namespace sm100;

constexpr int kRows = kPrefixRows, kKeys = kPrefixKeys;
constexpr int kThreads = 256, kSoft = 128, kSoftWarp = 4;
constexpr int kCtasPerSm = 2;
constexpr int kRegsRoles = 72, kRegsSoft = 184;   // of the 128 per thread at launch
constexpr int kBias = 6;                          // the largest P after a reference is set is 2^kBias
constexpr int kSK = 2, kSV = 3;                   // ring stages
constexpr uint32_t kTermBytes = kRows * kD, kTileBytes = kKeys * kD;
constexpr uint32_t kTmemCols = 256, kOCol = 2 * kKeys;   // S double buffer, then O

struct Cfg {
  static constexpr int kKFull = 0, kKEmpty = kSK, kVFull = 2 * kSK, kVEmpty = kVFull + kSV, kSFull = kVEmpty + kSV,
                       kSEmpty = kSFull + 2, kPFull = kSEmpty + 2, kOFull = kPFull + 2, kQFull = kOFull + 2,
                       kTabFull = kQFull + 1, kDone = kTabFull + kSV, kNumBars = kDone + 1;
  static constexpr uint32_t kQ = 0;                                 // two terms
  static constexpr uint32_t kK = kQ + 2 * kTermBytes;
  static constexpr uint32_t kV = kK + kSK * kTileBytes;
  static constexpr uint32_t kP = kV + kSV * kTileBytes;             // a row's line: 64 first terms, 64 second terms
  static constexpr uint32_t kPBytes = kRows * 128;                  // two such buffers
  static constexpr uint32_t kBar = kP + 2 * kPBytes;
  static constexpr uint32_t kTmemSlot = kBar + kNumBars * 8;
  static constexpr uint32_t kAbort = kTmemSlot + 4;
  // per V stage: a tile's key scales, value factors, value exponents less E;
  // then E, and how far it rose with this tile
  static constexpr uint32_t kTab = (kAbort + 4 + 15) / 16 * 16;
  static constexpr uint32_t kTabBytes = 3 * kKeys * 4 + 16;
  static constexpr uint32_t kQw = kTab + kSV * kTabBytes;           // [128] query scales
  static constexpr uint32_t kAlloc = kQw + kRows * 4;
  static_assert(kK % 1024 == 0 && kV % 1024 == 0 && kP % 1024 == 0, "swizzle atoms need 1024-byte alignment");
  static_assert(kAlloc <= (233472 - kCtasPerSm * 1024) / kCtasPerSm, "shared memory budget");
  static_assert(128 * kRegsRoles + kSoft * kRegsSoft == kThreads * 128, "registers");
};

struct Roles {
  uint32_t sbase;
  unsigned char* smem;
  uint32_t tmem;
  volatile int* abort;
  int32_t* flags;
  int nb;                // tiles per segment
  int t0, n;             // the CTA's first tile, and how many it has
  int len;               // prefix rows
};

__device__ __forceinline__ bool wait_bar(const Roles& r, uint32_t bar, uint32_t parity) {
  if (mbar_wait_asleep(bar, parity, kTimeoutNs)) return true;
  *r.abort = 1;
  set_flag(r.flags, MQA_FLAG_PIPE_TIMEOUT);
  return false;
}

// Walks the CTA's tiles: segment and tile within it.
struct Walk {
  int seg, k, nb, piece; // piece: segments met so far, less one
  bool first;
  __device__ Walk(const Roles& r) : nb(r.nb), piece(-1), first(false) {
    seg = r.t0 / nb;
    k = r.t0 - seg * nb - 1;
  }
  __device__ void next() {
    first = piece < 0;
    if (++k == nb) {
      k = 0;
      ++seg;
      first = true;
    }
    if (first) ++piece;
  }
};

__device__ __forceinline__ uint64_t l2_evict_last_policy() {   // the tiles are read again by the other blocks
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

__device__ void k_producer(const PrefixArgs& a, const Roles& r, const CUtensorMap* map) {
  auto bar = [&](int id) { return r.sbase + Cfg::kBar + 8u * uint32_t(id); };
  const uint64_t pol = l2_evict_last_policy();
  Walk w(r);
  int i = 0;
  for (; i < r.n; ++i) {
    w.next();
    if (*r.abort) break;
    const int st = i % kSK;
    if (i >= kSK && !wait_bar(r, bar(Cfg::kKEmpty + st), uint32_t(i / kSK - 1) & 1)) break;
    mbar_expect_tx(bar(Cfg::kKFull + st), kTileBytes);
    tma_load_3d(r.sbase + Cfg::kK + st * kTileBytes, map, bar(Cfg::kKFull + st), 0, w.seg / a.blocks, w.k * kKeys, pol);
  }
  // every copy issued has landed before the CTA can exit
  for (int j = (i - kSK > 0 ? i - kSK : 0); j < i; ++j)
    mbar_wait_asleep(bar(Cfg::kKFull + j % kSK), uint32_t(j / kSK) & 1, kTimeoutNs);
}

// V tiles (lane 0) and the tables beside them.  A stage is free again when the
// P.V product of its tile has completed: every softmax thread has then read the
// stage's table, too.
__device__ void v_producer(const PrefixArgs& a, const Roles& r, const CUtensorMap* map, int lane) {
  auto bar = [&](int id) { return r.sbase + Cfg::kBar + 8u * uint32_t(id); };
  const uint64_t pol = l2_evict_last_policy();
  const float c = a.scale * kLog2e;
  Walk w(r);
  // Exponents of keys 2 lane and 2 lane + 1 of the walker's tile.
  uint32_t ke[2], ve[2];
  int head = 0;
  auto load_exps = [&]() {
    if (w.first) head = w.seg / a.blocks;
    const int k0 = w.k * kKeys + 2 * lane;
    const int64_t at = int64_t(head) * a.m_p + k0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      ke[x] = k0 + x < r.len ? a.ke[at + x] : 0u;
      ve[x] = k0 + x < r.len ? a.ve[at + x] : 0u;
    }
  };
  w.next();
  load_exps();
  int E = 0, i = 0;
  bool any = false;      // some value row of the segment so far was not all zeros
  for (; i < r.n; ++i) {
    const int st = i % kSV, k = w.k, at_head = head;
    const bool first = w.first;
    bool go = *r.abort == 0;
    if (i >= kSV) go = mbar_wait_asleep(bar(Cfg::kVEmpty + st), uint32_t(i / kSV - 1) & 1, kTimeoutNs) && go;
    if (!__all_sync(0xffffffffu, go)) {
      if (lane == 0) {
        *r.abort = 1;
        set_flag(r.flags, MQA_FLAG_PIPE_TIMEOUT);
      }
      break;
    }
    if (lane == 0) {
      mbar_expect_tx(bar(Cfg::kVFull + st), kTileBytes);
      tma_load_3d(r.sbase + Cfg::kV + st * kTileBytes, map, bar(Cfg::kVFull + st), 0, at_head, k * kKeys, pol);
    }
    const uint32_t k0 = ke[0], k1 = ke[1], v0 = ve[0], v1 = ve[1];
    if (i + 1 < r.n) {
      w.next();
      load_exps();
    }
    const int em = __reduce_max_sync(0xffffffffu, int(max(v0 > 1 ? v0 : 0u, v1 > 1 ? v1 : 0u)));
    float rise = 0.f;
    if (first) {
      E = em > 0 ? em : 119;   // no value yet: a middling 2^-8
      any = em > 0;
    } else if (em > E || (em > 0 && !any)) {
      rise = float(em - E);
      E = em;
      any = true;
    }
    float* const tab = reinterpret_cast<float*>(r.smem + Cfg::kTab + st * Cfg::kTabBytes);
    reinterpret_cast<float2*>(tab)[lane] = make_float2(scale_of(k0) * c, scale_of(k1) * c);
    const int f0 = int(v0) - E + 127 + kBias, f1 = int(v1) - E + 127 + kBias;   // b_t 2^(kBias - E)
    reinterpret_cast<float2*>(tab + kKeys)[lane] = make_float2(v0 == 0 || f0 <= 0 ? 0.f : __uint_as_float(uint32_t(f0) << 23),
                                                              v1 == 0 || f1 <= 0 ? 0.f : __uint_as_float(uint32_t(f1) << 23));
    reinterpret_cast<float2*>(tab + 2 * kKeys)[lane] =
        make_float2(float(max(int(v0) - E, -kSpan)), float(max(int(v1) - E, -kSpan)));
    if (lane == 0) reinterpret_cast<float2*>(tab + 3 * kKeys)[0] = make_float2(scale_of(uint32_t(E)), rise);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(Cfg::kTabFull + st));
  }
  // every copy issued has landed before the CTA can exit
  if (lane == 0)
    for (int j = (i - kSV > 0 ? i - kSV : 0); j < i; ++j)
      mbar_wait_asleep(bar(Cfg::kVFull + j % kSV), uint32_t(j / kSV) & 1, kTimeoutNs);
}

__device__ void s_issuer(const Roles& r) {
  constexpr uint32_t idesc = idesc_e4m3_f32(kRows, kKeys, 0, 0);
  const uint64_t qdesc = smem_desc_sw128(r.sbase + Cfg::kQ, 16, 1024), kdesc0 = smem_desc_sw128(r.sbase + Cfg::kK, 16, 1024);
  auto bar = [&](int id) { return r.sbase + Cfg::kBar + 8u * uint32_t(id); };
  Walk w(r);
  for (int i = 0; i < r.n; ++i) {
    w.next();
    const int st = i % kSK, sb = i & 1;
    if (w.first && !wait_bar(r, bar(Cfg::kQFull), uint32_t(w.piece) & 1)) break;
    if (!wait_bar(r, bar(Cfg::kKFull + st), uint32_t(i / kSK) & 1)) break;
    if (i >= 2 && !wait_bar(r, bar(Cfg::kSEmpty + sb), uint32_t((i >> 1) - 1) & 1)) break;
    tc_fence_after();
    const uint64_t ka = kdesc0 + uint64_t((uint32_t(st) * kTileBytes) >> 4);
#pragma unroll
    for (int term = 0; term < 2; ++term)
#pragma unroll
      for (int kk = 0; kk < kD / 32; ++kk)
        mma_e4m3_ss(r.tmem + uint32_t(sb) * kKeys, qdesc + ((term * kTermBytes + kk * 32) >> 4), ka + ((kk * 32) >> 4), idesc,
                    term + kk > 0);
    mma_commit(bar(Cfg::kSFull + sb));
    mma_commit(bar(Cfg::kKEmpty + st));
  }
  mma_commit(bar(Cfg::kDone));
  mbar_wait_asleep(bar(Cfg::kDone), 0, kTimeoutNs);
}

__device__ void pv_issuer(const Roles& r) {
  constexpr uint32_t idesc = idesc_e4m3_f32(kRows, kD, 0, 1);
  const uint64_t pdesc = smem_desc_sw128(r.sbase + Cfg::kP, 16, 1024);    // K-major, both terms in a row's 128 bytes
  const uint64_t vdesc0 = smem_desc_sw128(r.sbase + Cfg::kV, 16, 1024);   // MN-major: keys are K
  auto bar = [&](int id) { return r.sbase + Cfg::kBar + 8u * uint32_t(id); };
  Walk w(r);
  for (int i = 0; i < r.n; ++i) {
    w.next();
    const int st = i % kSV, pb = i & 1;
    if (!wait_bar(r, bar(Cfg::kPFull + pb), uint32_t(i >> 1) & 1)) break;
    if (!wait_bar(r, bar(Cfg::kVFull + st), uint32_t(i / kSV) & 1)) break;
    tc_fence_after();
    const uint64_t va = vdesc0 + uint64_t((uint32_t(st) * kTileBytes) >> 4);
#pragma unroll
    for (int term = 0; term < 2; ++term)
#pragma unroll
      for (int kk = 0; kk < kKeys / 32; ++kk)
        mma_e4m3_ss(r.tmem + kOCol, pdesc + ((pb * Cfg::kPBytes + term * kKeys + kk * 32) >> 4), va + ((kk * 4096) >> 4), idesc,
                    !w.first || term + kk > 0);
    mma_commit(bar(Cfg::kOFull + pb));
    mma_commit(bar(Cfg::kVEmpty + st));
  }
  mma_commit(bar(Cfg::kDone));
  mbar_wait_asleep(bar(Cfg::kDone), 0, kTimeoutNs);
}

__device__ void softmax(const PrefixArgs& a, const Roles& r, int warp, int lane) {
  auto bar = [&](int id) { return r.sbase + Cfg::kBar + 8u * uint32_t(id); };
  auto wait = [&](int id, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_asleep(bar(id), parity, kTimeoutNs)); };
  const int q4 = warp & 3, tid = threadIdx.x - 32 * kSoftWarp, row = 32 * q4 + lane;
  const uint32_t t_lane = r.tmem + (uint32_t(32 * q4) << 16);
  float* const qw = reinterpret_cast<float*>(r.smem + Cfg::kQw);
  unsigned char* const lines = r.smem + Cfg::kP + row * 128;
  const int64_t rows_all = int64_t(a.b) * a.hq;
  Walk w(r);

  // The block's queries, eight threads per row.
  auto convert = [&](int seg) {
    const int head = seg / a.blocks;
    const int64_t r0 = int64_t(seg - head * a.blocks) * kRows;
    const int part = tid & 7;
    QueryPiece q[8];   // all loads first
#pragma unroll
    for (int pass = 0; pass < 8; ++pass) {
      const int64_t at = r0 + pass * 16 + (tid >> 3);
      const int s = int(uint32_t(at) / uint32_t(a.hq));   // rows number less than 2^31
      q[pass] = load_query(
          at < rows_all ? a.q + (int64_t(s) * a.h + int64_t(head) * a.hq + (at - int64_t(s) * a.hq)) * kD : nullptr, part);
    }
#pragma unroll
    for (int pass = 0; pass < 8; ++pass) {
      const int n = pass * 16 + (tid >> 3);
      uint4 hi, lo;
      const float sc = split_query(q[pass], hi, lo);
      unsigned char* dst = r.smem + Cfg::kQ + n * 128 + ((part ^ (n & 7)) << 4);
      *reinterpret_cast<uint4*>(dst) = hi;
      *reinterpret_cast<uint4*>(dst + kTermBytes) = lo;
      if (part == 0) qw[n] = sc;
    }
    fence_proxy_async_smem();
    mbar_arrive(bar(Cfg::kQFull));
  };
  // This row's query scale, once all threads have converted block `piece`.  (The
  // next block's come after this one's products, which wait for every thread.)
  auto query_scale = [&](int piece, float& rw) {
    if (!wait(Cfg::kQFull, uint32_t(piece) & 1)) return false;
    rw = qw[row];
    return true;
  };

  w.next();
  convert(w.seg);
  float negm = 0.f, l = 0.f, rw = 0.f;   // minus the row's reference, its sum, its query scale
  bool failed = !query_scale(0, rw);
  for (int i = 0; i < r.n && !failed; ++i) {
    const bool first = w.first;
    const int seg = w.seg, st = i % kSV, pb = i & 1;
    const int valid = min(kKeys, r.len - w.k * kKeys);
    if (i + 1 < r.n) w.next();
    const bool last = i + 1 == r.n || w.first;
    if (!wait(Cfg::kTabFull + st, uint32_t(i / kSV) & 1) || !wait(Cfg::kSFull + pb, uint32_t(i >> 1) & 1)) {
      failed = true;
      break;
    }
    tc_fence_after();
    const float* const ksc = reinterpret_cast<const float*>(r.smem + Cfg::kTab + st * Cfg::kTabBytes);
    const float *const vfac = ksc + kKeys, *const vexp = vfac + kKeys;
    const float2 tile = reinterpret_cast<const float2*>(vexp + kKeys)[0];   // 2^(E-127), rise of E
    if (first) {
      negm = 0.f;
      l = 0.f;
    } else if (tile.y != 0.f) {   // the weights are now relative to a larger exponent, the references with them
      negm += tile.y;
      l *= ex2_approx(tile.y);
    }
    uint64_t x[kKeys / 2];     // s - m, in pairs
    {
      const uint64_t rw2 = pack2(rw, rw), m2 = pack2(negm, negm);
#pragma unroll
      for (int ch = 0; ch < kKeys / 32; ++ch) {
        float s[32];
        tmem_ld32(t_lane + uint32_t(pb) * kKeys + ch * 32, s);
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          uint64_t k0, k1;
          load_pairs(ksc + ch * 32 + k, k0, k1);
          x[(ch * 32 + k) / 2] = fma2(mul2(pack2(s[k], s[k + 1]), k0), rw2, m2);
          x[(ch * 32 + k) / 2 + 1] = fma2(mul2(pack2(s[k + 2], s[k + 3]), k1), rw2, m2);
        }
      }
      tc_fence_before();
      mbar_arrive(bar(Cfg::kSEmpty + pb));   // the buffer may take S(i+2)
      if (valid < kKeys) {
#pragma unroll
        for (int k = 0; k < kKeys / 2; ++k) {
          float x0, x1;
          unpack2(x[k], x0, x1);
          x[k] = pack2(2 * k < valid ? x0 : -INFINITY, 2 * k + 1 < valid ? x1 : -INFINITY);
        }
      }
    }
    // The largest P (relative to 2^kBias): does the reference have to move?
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kKeys; k += 4) {
      uint64_t e0, e1;
      float y0, y1, y2, y3;
      load_pairs(vexp + k, e0, e1);
      unpack2(add2(x[k / 2], e0), y0, y1);
      unpack2(add2(x[k / 2 + 1], e1), y2, y3);
      top = fmaxf(fmaxf(top, y0), y1);
      top = fmaxf(fmaxf(top, y2), y3);
    }
    float alpha = 1.f;
    bool moved = false;
    if (__any_sync(0xffffffffu, first || top > kLogCodeMax - kBias)) {
      const float by = first ? top : fmaxf(top, 0.f);
      const uint64_t b2 = pack2(-by, -by);
#pragma unroll
      for (int k = 0; k < kKeys / 2; ++k) x[k] = add2(x[k], b2);
      negm -= by;
      if (!first) {
        alpha = ex2_approx(-by);
        l *= alpha;
        moved = true;
      }
    }
    // P in two terms
    uint32_t hi[kKeys / 4], lo[kKeys / 4];
    uint64_t sum2 = 0;
#pragma unroll
    for (int k4 = 0; k4 < kKeys / 4; ++k4) {
      uint64_t f[2];
      load_pairs(vfac + 4 * k4, f[0], f[1]);
      uint32_t h[2], lw[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x0, x1, p0, p1;
        unpack2(x[2 * k4 + j], x0, x1);
        const uint64_t e = pack2(ex2_approx(x0), ex2_approx(x1));
        sum2 = add2(sum2, e);
        unpack2(mul2(e, f[j]), p0, p1);
        split2_plain(p0, p1, h[j], lw[j]);
      }
      hi[k4] = h[0] | (h[1] << 16);
      lo[k4] = lw[0] | (lw[1] << 16);
    }
    {
      float s0, s1;
      unpack2(sum2, s0, s1);
      l += s0 + s1;
    }
    // P.V(i-2) must be complete before its P is overwritten, P.V(i-1) before O
    // is rescaled; a ragged tile needs its V rows landed before those past the
    // end are zeroed.
    bool fine = true;
    if (i > 1) fine = wait(Cfg::kOFull + pb, uint32_t((i >> 1) - 1) & 1);
    if (i > 0 && moved) fine = wait(Cfg::kOFull + (pb ^ 1), uint32_t((i - 1) >> 1) & 1) && fine;
    if (valid < kKeys) fine = wait(Cfg::kVFull + st, uint32_t(i / kSV) & 1) && fine;
    if (!fine) {
      failed = true;
      break;
    }
    tc_fence_after();
    if (moved) {               // collective for the warp; alpha = 1 in rows that keep theirs
#pragma unroll
      for (int ch = 0; ch < kD / 32; ++ch) {
        float v[32];
        tmem_ld32(t_lane + kOCol + ch * 32, v);
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] *= alpha;
        tmem_st<32>(t_lane + kOCol + ch * 32, v);
      }
      tmem_wait_st();
    }
    unsigned char* const line = lines + pb * Cfg::kPBytes;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      *reinterpret_cast<uint4*>(line + ((j ^ (row & 7)) << 4)) = make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
      *reinterpret_cast<uint4*>(line + (((4 + j) ^ (row & 7)) << 4)) =
          make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
    }
    if (valid < kKeys) {
      unsigned char* vst = r.smem + Cfg::kV + st * kTileBytes + valid * 128;
      for (int k = tid; k < (kKeys - valid) * 8; k += kSoft) *reinterpret_cast<uint4*>(vst + k * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    mbar_arrive(bar(Cfg::kPFull + pb));
    if (last) {   // the segment's partial; then the next one's queries (its S products wait for them)
      if (!wait(Cfg::kOFull + pb, uint32_t(i >> 1) & 1)) {
        failed = true;
        break;
      }
      tc_fence_after();
      const int64_t slot = int64_t(blockIdx.x) + seg;
      const float inv = tile.x * (1.f / (1 << kBias)) * rcp_approx(l);
      float* dst = a.part_o + (slot * kRows + row) * kD;
      const bool mine = int64_t(seg % a.blocks) * kRows + row < rows_all;
#pragma unroll
      for (int ch = 0; ch < kD / 32; ++ch) {
        float v[32];
        tmem_ld32(t_lane + kOCol + ch * 32, v);
        if (mine) {
#pragma unroll
          for (int k = 0; k < 32; k += 8)   // 32 bytes per lane: whole sectors
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + ch * 32 + k), "f"(v[k] * inv),
                         "f"(v[k + 1] * inv), "f"(v[k + 2] * inv), "f"(v[k + 3] * inv), "f"(v[k + 4] * inv),
                         "f"(v[k + 5] * inv), "f"(v[k + 6] * inv), "f"(v[k + 7] * inv) : "memory");
        }
      }
      if (mine) a.part_lse[slot * kRows + row] = lg2_approx(l) - negm;
      tc_fence_before();   // O has been read before the next P is announced
      if (i + 1 < r.n) {
        convert(w.seg);
        failed = !query_scale(w.piece, rw);
      }
    }
  }
  if (failed && lane == 0) {
    *r.abort = 1;
    set_flag(r.flags, MQA_FLAG_PIPE_TIMEOUT);
  }
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    q8_prefix_tc_kernel(const PrefixArgs a, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Roles r;
  r.smem = smem_raw;
  r.sbase = smem_u32(smem_raw);
  r.abort = reinterpret_cast<volatile int*>(r.smem + Cfg::kAbort);
  r.flags = a.flags;
  if (r.sbase & 1023u) {   // the swizzled tiles need a 1024-byte aligned base (uniform across the CTA)
    if (threadIdx.x == 0) set_flag(a.flags, MQA_FLAG_PIPE_TIMEOUT);
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto bar = [&](int id) { return r.sbase + Cfg::kBar + 8u * uint32_t(id); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSK; ++s) {
      mbar_init(bar(Cfg::kKFull + s), 1);
      mbar_init(bar(Cfg::kKEmpty + s), 1);
    }
    for (int s = 0; s < kSV; ++s) {
      mbar_init(bar(Cfg::kVFull + s), 1);
      mbar_init(bar(Cfg::kVEmpty + s), 1);
      mbar_init(bar(Cfg::kTabFull + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(Cfg::kSFull + s), 1);
      mbar_init(bar(Cfg::kSEmpty + s), kSoft);
      mbar_init(bar(Cfg::kPFull + s), kSoft);
      mbar_init(bar(Cfg::kOFull + s), 1);
    }
    mbar_init(bar(Cfg::kQFull), kSoft);
    mbar_init(bar(Cfg::kDone), 2);   // one commit from each issuing thread
    *r.abort = 0;
    mbar_fence_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(r.sbase + Cfg::kTmemSlot, kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  r.tmem = *reinterpret_cast<volatile uint32_t*>(r.smem + Cfg::kTmemSlot);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // The own rows' kernel may start as this one's CTAs leave room: it reads
  // nothing of this grid's.
  asm volatile("griddepcontrol.launch_dependents;");
  const int given = __ldg(a.len);
  r.len = min(max(given, 0), a.m_p);
  if (r.len != given && blockIdx.x == 0 && threadIdx.x == 0) set_flag(a.flags, MQA_FLAG_LEN_CLAMPED);
  r.nb = prefix_tiles(r.len);
  r.t0 = 0;
  r.n = 0;
  if (r.nb > 0) {
    const int total = a.g * a.blocks * r.nb;
    if (int(blockIdx.x) < total) {
      const PrefixShare share = prefix_share(a.g * a.blocks, r.nb, a.grid);
      r.t0 = share.start(blockIdx.x);
      r.n = share.start(blockIdx.x + 1) - r.t0;
    }
  }
  if (warp >= kSoftWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    if (r.n > 0) softmax(a, r, warp, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRoles));
    if (r.n > 0) {
      if (warp == 2) {
        v_producer(a, r, &tm_v, lane);
      } else if (lane == 0) {
        if (warp == 0) k_producer(a, r, &tm_k);
        else if (warp == 1) s_issuer(r);
        else pv_issuer(r);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(r.tmem, kTmemCols);
}

}  // namespace

cudaError_t launch_q8_prefix(const PrefixArgs& a, const uint8_t* k, const uint8_t* v, cudaStream_t stream) {
  if (int64_t(a.m_p) >= (int64_t(1) << 31) - 512) return cudaErrorInvalidValue;   // row coordinates of a tile
  static std::atomic<bool> attr_set[64];   // per device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(q8_prefix_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Cfg::kAlloc));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true, std::memory_order_relaxed);
  }
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  CUtensorMap tk, tv;
  if (!encode_codes(&tk, k, a.m_p, a.g, kKeys) || !encode_codes(&tv, v, a.m_p, a.g, kKeys)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q8_prefix_tc_kernel, a, tk, tv);
}

}  // namespace q8
}  // namespace mqa
