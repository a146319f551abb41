// A prefix shared by a whole batch, in an 8-bit cache, on the tensor cores:
// every query row of the batch against the prefix's keys and values, computed
// in blocks of 128 rows, so that a staged tile serves 128 rows and the work is
// that of a matrix product, not of a stream.
//
// Two kernels.  The first unpacks the prefix to fp16, once for the whole batch:
// tile by tile of 64 rows, each tile relative to its largest key and its largest
// value exponent,
//   k'_t = code_t 2^(a_t - A),   v'_t = code_t 2^(b_t - B)
// (a code is a multiple of 2^-9: exact down to 2^-15 of the tile's largest scale;
// rows below that are rounded to steps of 2^-24 of it), zeros past the prefix's
// end.  The second is a product with a running softmax over query blocks: the
// rows of one K/V head are the pairs
// (sequence, head of the group), in that order, and with x_r = q_r / w_r in
// fp16 (maximum in (224, 448], bf16's 8 bits exact to 2^-17 of a unit)
//   S[r, t]  = x_r . k'_t              M = 128 query rows, N = 64 keys, K = 128
//   y_{r,t}  = scale log2(e) w_r 2^A S[r, t] + B - B_0
//   P[r, t]  = 2^(y - M_r)  in fp16    (11 bits: a weight is off by 2^-11 of itself at most)
//   O[r, c] += sum_t P[r, t] v'_t[c]   M = 128, N = 128, K = 64 keys (P in tensor memory, where S was)
//   l_r     += sum_t P[r, t] 2^(B_0 - B)   in fp32, before P is rounded
//   o_r      = 2^B_0 O[r, :] / l_r
// B_0 is the B of the first tile that has values (a tile of zeros has B = B_0 - 60
// instead, whatever B_0 becomes): the value exponent enters with the logit, so that
// a reference M_r is the largest contribution to the output, not the largest weight.  fp16 spans 40 octaves: P starts at 2^2, a reference moves only when
// some P would pass 2^15, and weights round to steps of 2^-24, 2^-26 of the
// reference's: 2^18 rows that all lose half a step lose 2^-9 of it.  (Started at
// 2^4: 195 us instead of 190 for 128 sequences behind a 16K prefix with GQA-8
// and row scales that vary, at 2^8 228: the references moved more often.)  The
// maxima are taken before the exponentials; from the finished P, with a second
// pass where one passes 2^15, that took 179 us instead of 155.
// (The same product on the e4m3 codes as they are, with both operands in two
// e4m3 terms and per-row scale tables: 158 us for that prefix when this took
// 116, with a reference moving every third tile; exponents of single rows
// brought to P where a tile's values are far apart: 10% more for every call; a
// quarter or half of the exponentials as a cubic on the FMA pipe: 4 to 10% more.)
// Here query rows are the products' M, so that a row's softmax is one thread's
// own: no barrier and no reduction across threads.
//
// Work: all (head, block) segments have the same number of tiles; the
// persistent CTAs take equal contiguous runs of them (a segment's beginning
// counted as some tiles more), and every (CTA, segment) leaves a normalised
// partial with its log-sum-exp for the merge.  Two CTAs per
// SM hide each other's chain of product, softmax and product.  S has two buffers;
// S(i+2) follows P.V(i), which reads P(i) from S(i)'s place.  Every barrier that
// a role does not wait for tile by tile has one phase per buffer, so that none
// is two phases ahead of what is waited for.  Roles: warp 0 K
// loads, warp 2 V loads, warp 1 S products, warp 3 P.V products (one lane
// each), warps 4-7 queries, softmax and output, a row per thread.  Every wait is
// bounded (one second) and reported with MQA_FLAG_PIPE_TIMEOUT.
//
// Bound: shared memory (per 64-row tile 64 KB of operands read and 32 KB written,
// about 770 cycles at 128 bytes each, of about 1,050 taken) and the softmax
// threads' latency (that prefix: 67 GFLOP and 131 million exponentials in about
// 80 us, 0.8 PFLOP/s; their floors are 41 and 29 us), and at a CTA's ends the
// queries' conversion and the partial outputs.  With P in shared memory, 32 KB
// more per tile, 150 us instead of 143 for that call if no row scales vary; a
// second P buffer there changed nothing.
#include "q8_tc.cuh"

namespace mqa {
namespace q8 {

namespace {

using namespace sm100;

constexpr int kRows = kPrefixRows, kKeys = kPrefixKeys;
constexpr int kThreads = 256, kSoft = 128, kSoftWarp = 4;
constexpr int kCtasPerSm = 2;
constexpr int kRegsRoles = 72, kRegsSoft = 184;   // of the 128 per thread at launch
constexpr float kTopLog = 15.f;                   // P stays below 2^15: half of fp16's range
constexpr int kBias = 2;                          // the largest P after a reference is set is 2^kBias
constexpr int kSK = 2, kSV = 2;                   // ring stages
constexpr uint32_t kQHalf = kRows * 128, kHalf = kKeys * 128;   // 64 columns: 128-byte swizzled rows
constexpr uint32_t kTileBytes = 2 * kHalf;
constexpr uint32_t kTmemCols = 256, kOCol = 2 * kKeys;   // S double buffer, then O

struct Cfg {
  static constexpr int kKFull = 0, kKEmpty = kSK, kVFull = 2 * kSK, kVEmpty = kVFull + kSV, kSFull = kVEmpty + kSV,
                       kSEmpty = kSFull + 2, kPFull = kSEmpty + 2, kOFull = kPFull + 2, kQFull = kOFull + 2,
                       kDone = kQFull + 1, kNumBars = kDone + 1;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + 2 * kQHalf;
  static constexpr uint32_t kV = kK + kSK * kTileBytes;
  static constexpr uint32_t kBox = kV + kSV * kTileBytes;           // outputs on their way: 32 columns of the rows
  static constexpr uint32_t kBar = kBox + kRows * 128;
  static constexpr uint32_t kTmemSlot = kBar + kNumBars * 8;
  static constexpr uint32_t kAbort = kTmemSlot + 4;
  static constexpr uint32_t kQw = kAbort + 4;                       // [128] query scales
  static constexpr uint32_t kAlloc = kQw + kRows * 4;
  static_assert(kK % 1024 == 0 && kV % 1024 == 0, "swizzle atoms need 1024-byte alignment");
  static_assert(kAlloc <= (233472 - kCtasPerSm * 1024) / kCtasPerSm, "shared memory budget");
  static_assert(128 * kRegsRoles + kSoft * kRegsSoft == kThreads * 128, "registers");
};

// ------------------------------------------------------------------ unpacking

constexpr int kUnpackThreads = 256;

// One tile of 64 rows of one K/V head, keys and values, to fp16; (A, B) of the
// tile beside it.  Bound: HBM (128 + 1 bytes read and 256 written per row).
__global__ void __launch_bounds__(kUnpackThreads) q8_unpack_kernel(const PrefixArgs a) {
  __shared__ int top[2][2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int tile = blockIdx.x, head = blockIdx.y, warp = threadIdx.x / 32;
  const int given = __ldg(a.len), len = min(max(given, 0), a.m_p);
  if (given != len && tile == 0 && head == 0 && threadIdx.x == 0) set_flag(a.flags, MQA_FLAG_LEN_CLAMPED);
  const int row0 = tile * kKeys;
  if (row0 >= len) return;
  // threads 0-63 the keys' exponents, 64-127 the values'
  const int64_t e_at = int64_t(head) * a.m_p + row0;
  if (threadIdx.x < 2 * kKeys) {
    const int t = threadIdx.x % kKeys;
    const uint8_t* const exps = threadIdx.x < kKeys ? a.ke : a.ve;
    const uint32_t e = row0 + t < len ? exps[e_at + t] : 0u;
    const int m = __reduce_max_sync(0xffffffffu, int(e > 1 ? e : 0u));   // rows of zeros aside
    if (threadIdx.x % 32 == 0) top[warp / 2][warp % 2] = m;
  }
  // this thread's pieces: 16 codes each, keys first
  constexpr int kPieces = 2 * kKeys * (kD / 16) / kUnpackThreads;
  uint4 w[kPieces];
  uint32_t e[kPieces];
#pragma unroll
  for (int x = 0; x < kPieces; ++x) {
    const int p = x * kUnpackThreads + threadIdx.x, val = p / (kKeys * (kD / 16));
    const int t = (p / (kD / 16)) % kKeys, c = p % (kD / 16);
    w[x] = make_uint4(0, 0, 0, 0);
    e[x] = 0;
    if (row0 + t < len) {
      w[x] = *reinterpret_cast<const uint4*>((val ? a.v : a.k) + ((int64_t(row0) + t) * a.g + head) * kD + c * 16);
      e[x] = (val ? a.ve : a.ke)[e_at + t];
    }
  }
  __syncthreads();
  const int top_k = max(top[0][0], top[0][1]), top_v = max(top[1][0], top[1][1]);
  const int A = max(top_k, 1), B = max(top_v, 1);
  const int64_t out = (int64_t(head) * a.tiles + tile) * kKeys * kD;
#pragma unroll
  for (int x = 0; x < kPieces; ++x) {
    const int p = x * kUnpackThreads + threadIdx.x, val = p / (kKeys * (kD / 16));
    const int t = (p / (kD / 16)) % kKeys, c = p % (kD / 16);
    const int d = int(e[x]) - (val ? B : A);   // 0 at most
    // rows of the smallest scale count as zeros where a tile's values have no other
    const bool none = e[x] == 0 || (val && top_v == 0);
    // The factor 2^d in two, as fp16 ends at 2^-24: the first product is exact (a
    // code is a multiple of 2^-9), the second rounds once.  From 2^-34 on nothing
    // is left of any code.
    const int d1 = max(d, -14), d2 = max(d - d1, -24);
    const __half2 f1 = __float2half2_rn(none ? 0.f : __uint_as_float(uint32_t(127 + d1) << 23));
    const __half2 f2 = __float2half2_rn(__uint_as_float(uint32_t(127 + d2) << 23));
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t u;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(u) : "h"(uint16_t((&w[x].x)[k / 2] >> (16 * (k & 1)))));
      const __half2 y = __hmul2(__hmul2(*reinterpret_cast<const __half2*>(&u), f1), f2);
      h[k] = *reinterpret_cast<const uint32_t*>(&y);
    }
    __half* const dst = (val ? a.v16 : a.k16) + out + t * kD + c * 16;
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]),
                 "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7]) : "memory");
  }
  // a tile whose values are all zeros has no B: 0 tells so
  if (threadIdx.x == 0) a.tile_exps[head * a.tiles + tile] = make_int2(A, top_v);
}

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

template <bool kIsK>
__device__ void producer(const PrefixArgs& a, const Roles& r, const CUtensorMap* map) {
  constexpr int S = kIsK ? kSK : kSV;
  constexpr int kFull = kIsK ? Cfg::kKFull : Cfg::kVFull, kEmpty = kIsK ? Cfg::kKEmpty : Cfg::kVEmpty;
  constexpr uint32_t kRing = kIsK ? Cfg::kK : Cfg::kV;
  auto bar = [&](int id) { return r.sbase + Cfg::kBar + 8u * uint32_t(id); };
  uint64_t pol;   // the tiles are read again by the other blocks
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the unpacked tiles
  Walk w(r);
  int i = 0, head = 0;
  for (; i < r.n; ++i) {
    w.next();
    if (*r.abort) break;
    const int st = i % S;
    if (i >= S && !wait_bar(r, bar(kEmpty + st), uint32_t(i / S - 1) & 1)) break;
    const uint32_t dst = r.sbase + kRing + st * kTileBytes;
    if (w.first) head = w.seg / a.blocks;
    mbar_expect_tx(bar(kFull + st), kTileBytes);
    tma_load_3d(dst, map, bar(kFull + st), 0, w.k * kKeys, head, pol);
    tma_load_3d(dst + kHalf, map, bar(kFull + st), 64, w.k * kKeys, head, pol);
  }
  // every copy issued has landed before the CTA can exit
  for (int j = (i - S > 0 ? i - S : 0); j < i; ++j) mbar_wait_asleep(bar(kFull + j % S), uint32_t(j / S) & 1, kTimeoutNs);
}

__device__ void s_issuer(const Roles& r) {
  constexpr uint32_t idesc = idesc_code0_f32(kRows, kKeys, 0, 0);
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
    for (int kk = 0; kk < kD / 16; ++kk)
      mma_bf16_ss(r.tmem + uint32_t(sb) * kKeys, qdesc + (((kk >> 2) * kQHalf + (kk & 3) * 32) >> 4),
                  ka + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4), idesc, kk > 0);
    mma_commit(bar(Cfg::kSFull + sb));
    mma_commit(bar(Cfg::kKEmpty + st));
  }
  mma_commit(bar(Cfg::kDone));
  mbar_wait_asleep(bar(Cfg::kDone), 0, kTimeoutNs);
}

__device__ void pv_issuer(const Roles& r) {
  constexpr uint32_t idesc = idesc_code0_f32(kRows, kD, 0, 1);
  const uint64_t vdesc0 = smem_desc_sw128(r.sbase + Cfg::kV, kHalf, 1024);   // MN-major: columns are N
  auto bar = [&](int id) { return r.sbase + Cfg::kBar + 8u * uint32_t(id); };
  Walk w(r);
  for (int i = 0; i < r.n; ++i) {
    w.next();
    const int st = i % kSV;
    if (!wait_bar(r, bar(Cfg::kPFull + (i & 1)), uint32_t(i >> 1) & 1)) break;
    if (!wait_bar(r, bar(Cfg::kVFull + st), uint32_t(i / kSV) & 1)) break;
    tc_fence_after();
    const uint64_t va = vdesc0 + uint64_t((uint32_t(st) * kTileBytes) >> 4);
#pragma unroll
    for (int kk = 0; kk < kKeys / 16; ++kk)
      mma_f16_ts(r.tmem + kOCol, r.tmem + uint32_t(i & 1) * kKeys + kk * 8, va + ((kk * 2048) >> 4), idesc, !w.first || kk > 0);
    mma_commit(bar(Cfg::kOFull + (i & 1)));
    mma_commit(bar(Cfg::kSEmpty + (i & 1)));   // the buffer may take S(i+2)
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
  const float c = a.scale * kLog2e;
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
      uint32_t h[8];
      const float sc = half_query(q[pass], h);
      // columns 16 part .. + 15: two 16-byte pieces of the row's line in their 64-column half
      unsigned char* dst = r.smem + Cfg::kQ + (part >> 2) * kQHalf + n * 128;
      const int p0 = (part & 3) * 2;
      *reinterpret_cast<uint4*>(dst + ((p0 ^ (n & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(dst + (((p0 + 1) ^ (n & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
      if (part == 0) qw[n] = sc;
    }
    fence_proxy_async_smem();
    mbar_arrive(bar(Cfg::kQFull));
  };
  // This row's query scale, once all threads have converted block `piece`.  (The
  // next block's come after this one's products, which wait for every thread.)
  auto query_scale = [&](int piece, float& rw) {
    if (!wait(Cfg::kQFull, uint32_t(piece) & 1)) return false;
    rw = qw[row] * c;
    return true;
  };

  w.next();
  convert(w.seg);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the unpacked tiles, from here on
  const int2* tile_exps = a.tile_exps + w.seg / a.blocks * a.tiles;
  int2 exps = tile_exps[w.k];   // the next tile's A and B
  float negm = 0.f, l = 0.f, rw = 0.f;   // minus the row's reference, its sum, its query scale
  int B0 = 0;                            // 0: no value yet
  bool failed = !query_scale(0, rw);
  for (int i = 0; i < r.n && !failed; ++i) {
    const bool first = w.first;
    const int seg = w.seg;
    const int valid = min(kKeys, r.len - w.k * kKeys);
    const int2 e = exps;
    if (i + 1 < r.n) {
      w.next();
      if (w.first) tile_exps = a.tile_exps + w.seg / a.blocks * a.tiles;
      exps = tile_exps[w.k];
    }
    const bool last = i + 1 == r.n || w.first;
    if (first) {
      negm = 0.f;
      l = 0.f;
    }
    if (first || B0 == 0) B0 = e.y;   // O is 0 so far, and l does not depend on B_0
    // B - B_0; a tile of zeros counts for little in the references, not for nothing
    const int rise = e.y > 0 ? min(max(e.y - B0, -126), 126) : -kSpan;
    const float a_t = rw * scale_of(uint32_t(e.x)), shift = float(rise);
    if (!wait(Cfg::kSFull + (i & 1), uint32_t(i >> 1) & 1)) {
      failed = true;
      break;
    }
    tc_fence_after();
    uint64_t y[kKeys / 2];     // y - M, in pairs
    float top4[4];             // their largest, in four chains
    auto largest = [&](int k) {
      float y0, y1;
      unpack2(y[k], y0, y1);
      top4[k % 4] = fmaxf(fmaxf(top4[k % 4], y0), y1);
    };
    auto none = [&]() {
#pragma unroll
      for (int k = 0; k < 4; ++k) top4[k] = -INFINITY;
    };
    {
      const uint64_t a2 = pack2(a_t, a_t), m2 = pack2(negm + shift, negm + shift);
      none();
#pragma unroll
      for (int ch = 0; ch < kKeys / 32; ++ch) {
        float s[32];
        tmem_ld32(t_lane + uint32_t(i & 1) * kKeys + ch * 32, s);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          y[(ch * 32 + k) / 2] = fma2(pack2(s[k], s[k + 1]), a2, m2);
          largest((ch * 32 + k) / 2);
        }
      }
      if (valid < kKeys) {
        none();
#pragma unroll
        for (int k = 0; k < kKeys / 2; ++k) {
          float y0, y1;
          unpack2(y[k], y0, y1);
          y[k] = pack2(2 * k < valid ? y0 : -INFINITY, 2 * k + 1 < valid ? y1 : -INFINITY);
          largest(k);
        }
      }
    }
    // A reference moves if some P of the warp's rows would pass 2^15.
    float alpha = 1.f;
    const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
    const bool move = first || __any_sync(0xffffffffu, top > kTopLog);
    if (move) {
      const float by = first ? top - float(kBias) : fmaxf(top - float(kBias), 0.f);
      const uint64_t b2 = pack2(-by, -by);
#pragma unroll
      for (int k = 0; k < kKeys / 2; ++k) y[k] = add2(y[k], b2);
      negm -= by;
      if (!first) {
        alpha = ex2_approx(-by);
        l *= alpha;
      }
    }
    // P in fp16
    float p[kKeys / 2];        // two fp16 each
    uint64_t sum2 = 0;
#pragma unroll
    for (int k = 0; k < kKeys / 2; ++k) {
      float y0, y1;
      unpack2(y[k], y0, y1);
      const float e0 = ex2_approx(y0), e1 = ex2_approx(y1);
      sum2 = add2(sum2, pack2(e0, e1));
      const __half2 h = __floats2half2_rn(e0, e1);
      p[k] = *reinterpret_cast<const float*>(&h);
    }
    {
      float s0, s1;
      unpack2(sum2, s0, s1);
      l = fmaf(s0 + s1, __uint_as_float(uint32_t(127 - rise) << 23), l);
    }
    if (move && !first) {      // collective for the warp; alpha = 1 in rows that keep theirs
      if (!wait(Cfg::kOFull + ((i - 1) & 1), uint32_t((i - 1) >> 1) & 1)) {   // O holds P.V(i-1)
        failed = true;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int ch = 0; ch < kD / 32; ++ch) {
        float v[32];
        tmem_ld32(t_lane + kOCol + ch * 32, v);
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] *= alpha;
        tmem_st<32>(t_lane + kOCol + ch * 32, v);
      }
    }
    tmem_st<32>(t_lane + uint32_t(i & 1) * kKeys, p);   // where S(i) was
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(bar(Cfg::kPFull + (i & 1)));
    if (last) {   // the segment's partial; then the next one's queries (its S products wait for them)
      if (!wait(Cfg::kOFull + (i & 1), uint32_t(i >> 1) & 1)) {
        failed = true;
        break;
      }
      tc_fence_after();
      const int64_t slot = int64_t(blockIdx.x) + seg;
      const float inv = scale_of(uint32_t(B0)) * rcp_approx(l);
      // 32 columns at a time through the warp's own part of the box, so that whole
      // 128-byte lines leave the SM (a row per lane, 32 bytes each, took four
      // times the requests: 5.5 us at the end of every CTA).
      const int rows_left = int(min(int64_t(kRows), rows_all - int64_t(seg % a.blocks) * kRows)) - 32 * q4;   // of this warp's 32
      const bool mine = lane < rows_left;
      float4* const box = reinterpret_cast<float4*>(r.smem + Cfg::kBox + q4 * 4096);   // [32 rows][8 pieces], swizzled
      float* const dst = a.part_o + (slot * kRows + 32 * q4) * kD;
#pragma unroll
      for (int ch = 0; ch < kD / 32; ++ch) {
        float v[32];
        tmem_ld32(t_lane + kOCol + ch * 32, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          box[lane * 8 + (k ^ (lane & 7))] = make_float4(v[4 * k] * inv, v[4 * k + 1] * inv, v[4 * k + 2] * inv, v[4 * k + 3] * inv);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int rr = 4 * k + lane / 8, piece = lane % 8;
          if (rr < rows_left) *reinterpret_cast<float4*>(dst + rr * kD + ch * 32 + piece * 4) = box[rr * 8 + (piece ^ (rr & 7))];
        }
        __syncwarp();
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
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(Cfg::kSFull + s), 1);
      mbar_init(bar(Cfg::kSEmpty + s), 1);
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
  // The own rows' kernel may start wherever this one leaves room: it reads
  // nothing of this grid's or of the unpacking's, and what came before them is
  // complete (the unpacking let this grid start after its own wait).
  asm volatile("griddepcontrol.launch_dependents;");
  r.len = min(max(__ldcg(a.len), 0), a.m_p);
  r.nb = prefix_tiles(r.len);
  r.t0 = 0;
  r.n = 0;
  if (r.nb > 0) {
    const PrefixShare share(a.g * a.blocks, r.nb, a.grid);
    if (int(blockIdx.x) < share.ctas) {
      r.t0 = share.tile(share.start(blockIdx.x));
      r.n = share.tile(share.start(blockIdx.x + 1)) - r.t0;
    }
  }
  if (warp >= kSoftWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    if (r.n > 0) softmax(a, r, warp, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRoles));
    if (r.n > 0 && lane == 0) {
      if (warp == 0) producer<true>(a, r, &tm_k);
      else if (warp == 1) s_issuer(r);
      else if (warp == 2) producer<false>(a, r, &tm_v);
      else pv_issuer(r);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(r.tmem, kTmemCols);
  // Without tiles nothing here has waited yet: what follows takes this grid's end
  // for the unpacking's too.
  if (r.n == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Unpacked rows [g, rows, 128] fp16 as (128, rows, g); a box is 64 columns of
// 64 rows.
bool encode_unpacked(CUtensorMap* m, const void* base, int64_t rows, int g) {
  const cuuint64_t dims[3] = {cuuint64_t(kD), cuuint64_t(rows), cuuint64_t(g)};
  const cuuint64_t strides[2] = {cuuint64_t(kD) * 2, cuuint64_t(rows) * kD * 2};
  const cuuint32_t box[3] = {64, kKeys, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_q8_prefix(const PrefixArgs& a, cudaStream_t stream) {
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
  if (!encode_unpacked(&tk, a.k16, int64_t(a.tiles) * kKeys, a.g) || !encode_unpacked(&tv, a.v16, int64_t(a.tiles) * kKeys, a.g))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.tiles), unsigned(a.g));
  cfg.blockDim = dim3(kUnpackThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, q8_unpack_kernel, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(unsigned(a.grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg::kAlloc;
  return cudaLaunchKernelEx(&cfg, q8_prefix_tc_kernel, a, tk, tv);
}

}  // namespace q8
}  // namespace mqa
