// Shared pieces of the 8-bit K/V cache: conversions between fp32 and e4m3,
// row scales, and the arguments of the kernels over such caches.
//
// A cached row of one K/V head is d e4m3 codes and an exponent byte E; its
// values are code * s with s the fp32 number whose exponent field is E and
// whose mantissa is 0 (a power of two; 0 for E = 0).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "mqa_q8.h"

namespace mqa {
namespace q8 {

constexpr float kCodeMax = 448.f;   // largest e4m3 value

__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(e << 23); }

// Exponent byte of a row whose largest finite magnitude is `amax`: the
// smallest s with amax <= 448 s.  448 = 1.75 * 2^8, so with amax = 1.m * 2^k
// s is 2^(k-8), or 2^(k-7) when 1.m > 1.75.  Zero and subnormal maxima clamp
// to the smallest normal s (E = 1).
__device__ __forceinline__ uint32_t exponent_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = int(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return uint32_t(e < 1 ? 1 : e);
}

// 1 / scale_of(E) for E from exponent_for (1..247), exact.
__device__ __forceinline__ float inverse_scale(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// Two fp32 -> two e4m3 codes (x0 in the low byte), nearest even, saturating at
// +-448; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float x0, float x1) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
  return r;
}

// Two e4m3 codes (low 16 bits of w) -> two fp32, exact.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(w)));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Attention over an 8-bit cache.
struct DecodeQ8Args {
  void* o;
  const void* q;
  const uint8_t* k;    // [b, m_max, g, d_k] codes
  const uint8_t* ke;   // [b, g, m_max] exponents
  const uint8_t* v;
  const uint8_t* ve;
  const int32_t* lens;
  int b, h, g, m_max, d_k, d_v, hq;
  int window;          // 0: all rows
  int no_merge;        // no segment spans two tiles: every output row is written by the decode itself
  float scale;
  Workspace ws;
  int32_t* flags;
  int grid;
};

cudaError_t launch_q8_append(uint8_t* k, uint8_t* ke, uint8_t* v, uint8_t* ve, const void* k_new, const void* v_new,
                             const int32_t* pos, const int32_t* cu, int b, int total, int m_max, int g, int d_k,
                             int d_v, mqa_dtype_t dtype, int32_t* flags, cudaStream_t stream);
cudaError_t launch_q8_read(void* k_out, void* v_out, const uint8_t* k, const uint8_t* ke, const uint8_t* v,
                           const uint8_t* ve, const int32_t* start, const int32_t* cu, int b, int total, int m_max,
                           int g, int d_k, int d_v, mqa_dtype_t dtype, int32_t* flags, cudaStream_t stream);

// Attention on the tensor cores (bf16, head size 128).
struct TcArgs {
  void* o;
  const __nv_bfloat16* q;
  const uint8_t* ke;     // exponents [b, g, m]
  const uint8_t* ve;
  const int32_t* lens;   // [b]
  int b, h, g, hq, m;
  int window;            // 0: all rows
  int no_merge;          // no segment spans two tiles: every output row is written by the decode itself
  int partials;          // every segment leaves a partial, whole ones too (another part joins them)
  int groups;            // groups of g CTAs, one per K/V head
  float scale;
  Workspace ws;
  int32_t* flags;
};

// Where group `group` leaves its partial of sequence `seq` and K/V head `head`:
// consecutive sequences' groups meet in one group at most, so group + seq is
// theirs alone.  Fewer than (groups + b) g slots.
__device__ __forceinline__ int64_t tc_slot(int group, int seq, int g, int head) {
  return (int64_t(group) + seq) * g + head;
}

// Groups of CTAs for a wish of `ctas` (at least one group).
inline int tc_groups(int ctas, int g) {
  const int n = ctas / g;
  return n < 1 ? 1 : n;
}

bool q8_tc_supported(int d_k, int d_v, int hq, int g);
bool q8_tc_fits(int b, int m);
int q8_tc_tile_rows();
int q8_tc_ctas_per_sm();
cudaError_t launch_q8_decode_tc(const TcArgs& a, const uint8_t* k, const uint8_t* v, cudaStream_t stream);

// A prefix that all sequences share: every query row against it, in blocks of
// kPrefixRows rows of one K/V head.  Leaves a partial per (CTA, block).
constexpr int kPrefixRows = 128, kPrefixKeys = 64;   // query rows of a block, keys of a tile
constexpr int kPrefixMaxCtas = 512;
__device__ __forceinline__ int prefix_tiles(int len) { return (len + kPrefixKeys - 1) / kPrefixKeys; }
// How CTAs share the segments' tiles (`segs` of `nb` each).  A CTA that goes from
// one segment to the next writes an output, converts queries and fills its
// pipeline again, about kPrefixSeam tiles' time, so where CTAs have several
// tiles a segment begins with as many units that are no tiles; a tile is a unit.
// The first `more` CTAs take `each` + 1 units, the others `each`.  (128 GQA-8
// sequences behind 16K rows, 54 tiles a CTA: 167 us with 0, 159 with 4, 155 with
// 8, 160 with 12; 256 MQA ones behind 8K, 7 tiles: 45.5, 38.7 and 38.3 with 0, 4
// and 8.)
constexpr int kPrefixSeam = 8;
struct PrefixShare {
  int nb, seam, ctas, each, more;
  __device__ __forceinline__ PrefixShare(int segs, int nb_, int grid) : nb(nb_) {
    seam = segs * nb >= 4 * grid ? kPrefixSeam : 0;
    const int total = segs * (nb + seam);   // fewer than 2^31
    ctas = min(total, grid);
    each = total / ctas;
    more = total - each * ctas;
  }
  __device__ __forceinline__ int start(int cta) const { return cta * each + min(cta, more); }   // its first unit
  __device__ __forceinline__ int tile(int unit) const {   // tiles before a unit
    if (seam == 0) return unit;
    const int seg = unit / (nb + seam);
    return seg * nb + max(unit - seg * (nb + seam) - seam, 0);
  }
  __device__ __forceinline__ int owner(int seg, int t) const {   // the CTA of a segment's tile
    const int unit = seg * (nb + seam) + seam + t, split = more * (each + 1);
    return unit < split ? unit / (each + 1) : more + (unit - split) / each;
  }
};
struct PrefixArgs {
  const __nv_bfloat16* q;
  const uint8_t* k;      // codes [m_p, g, d]
  const uint8_t* ke;     // exponents [g, m_p]
  const uint8_t* v;
  const uint8_t* ve;
  const int32_t* len;    // [1]
  int b, h, g, hq, m_p;
  int blocks;            // blocks of query rows per K/V head
  int tiles;             // tiles of m_p rows
  __half* k16;           // unpacked [g, tiles * kPrefixKeys, d]
  __half* v16;
  int2* tile_exps;       // [g, tiles]: what the unpacked keys and values are relative to
  float scale;
  float* part_o;         // [slots][kPrefixRows][d], slot = CTA + head * blocks + block
  float* part_lse;       // [slots][kPrefixRows]
  int32_t* flags;
  int grid;
};
cudaError_t launch_q8_prefix(const PrefixArgs& a, cudaStream_t stream);

// Joins the partials of the own rows (and of a prefix, if given).
cudaError_t launch_q8_merge(const TcArgs& a, const PrefixArgs* prefix, cudaStream_t stream);

cudaError_t launch_q8_decode_simt(const DecodeQ8Args& a, mqa_dtype_t dtype, cudaStream_t stream);
int q8_simt_ctas_per_sm(int d_k, int d_v, int hq);
int q8_simt_tile_rows();

}  // namespace q8
}  // namespace mqa
