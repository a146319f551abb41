// Pieces shared by the tensor-core kernels over 8-bit caches: paired fp32
// arithmetic, the two-term e4m3 split of queries and weights, tensor maps.
#pragma once

#include <atomic>
#include <cuda.h>

#include "q8.cuh"
#include "sm100.cuh"

namespace mqa {
namespace sm100 {

// mbar_wait whose polls may sleep in hardware until the phase completes (up to
// `kHintNs` each) instead of returning at once: several CTAs' waiting warps
// then leave the issue slots to the ones that compute (78 -> 75 us where two
// CTAs per SM take a prefix).
__device__ __forceinline__ bool mbar_wait_asleep(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
  constexpr uint32_t kHintNs = 20000;
  uint64_t t0 = 0;
#pragma unroll 1
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kHintNs)
        : "memory");
    if (ok != 0) return true;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    else if (now - t0 > timeout_ns) return false;
  }
}

// mma_bf16_ss with e4m3 inputs (K = 32 per instruction).
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// mma_bf16_ss with the A operand in tensor memory: row m in lane m, two 16-bit
// elements to a column (K-major), eight columns per instruction.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of tcgen05.mma with fp32 sums and input formats of code
// 0: e4m3 x e4m3 in kind::f8f6f4, fp16 x fp16 in kind::f16 (mma_bf16_ss); dense,
// M x N, majors as in idesc_bf16_f32.
__host__ __device__ constexpr uint32_t idesc_code0_f32(int M, int N, int a_mn_major, int b_mn_major) {
  return (1u << 4)                       // D format: f32
         | (uint32_t(a_mn_major) << 15)  // A major
         | (uint32_t(b_mn_major) << 16)  // B major
         | (uint32_t(N >> 3) << 17)      // N / 8
         | (uint32_t(M >> 4) << 24);     // M / 16
}

}  // namespace sm100

namespace q8 {

constexpr int kD = 128;                          // head size
constexpr uint64_t kTimeoutNs = 1000000000ull;   // of any wait
constexpr float kLogCodeMax = 8.807354922f;      // log2(448)
constexpr int kSpan = 60;                        // value exponents below E - kSpan count as E - kSpan in the references

// Two fp32 at a time.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Four floats of shared memory as two pairs.
__device__ __forceinline__ void load_pairs(const float* p, uint64_t& a, uint64_t& b) {
  const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
  a = v.x;
  b = v.y;
}

// Two weights -> their two e4m3 terms (two codes each).  The difference is
// taken in fp16: its 11 bits hold what the second term's 4 can use.  `dither`,
// within half of e4m3's smallest step (2^-9), is added to the second term, in
// both halves: see row_dither.
__device__ __forceinline__ void split2(float p0, float p1, __half2 dither, uint32_t& hi, uint32_t& lo) {
  const __half2 p = __floats2half2_rn(p0, p1);
  const uint32_t pu = *reinterpret_cast<const uint32_t*>(&p);
  uint16_t h, l;
  uint32_t fu;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(pu));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(fu) : "h"(h));
  const __half2 f = *reinterpret_cast<const __half2*>(&fu);
  const __half2 d = __hfma2(__hsub2(p, f), __float2half2_rn(16.f), dither);
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(*reinterpret_cast<const uint32_t*>(&d)));
  hi = h;
  lo = l;
}

// What cache row t adds to its weights before they are rounded: one of 256
// values evenly spread over a step of e4m3's smallest, neighbouring rows' far
// apart (multiples of the golden ratio).  A weight far below a step then becomes
// a step as often as its size says, so that thousands of rows that are each
// lost in the grid behind one heavy row still add up to what they weigh; a
// weight of 0 stays 0.
__device__ __forceinline__ __half2 row_dither(int t) {
  return __float2half2_rn((float((uint32_t(t) * 2654435769u) >> 24) - 127.5f) * (1.f / 131072));
}

// Sixteen elements of a bf16 query row (zeros when row == nullptr), then as two
// e4m3 terms of x / s, sixteen codes each; eight neighbouring lanes hold a row
// (part = lane % 8) and find its power-of-two scale s, which is returned.  x / s reaches (224, 448]; the second term is the rest itself, so
// both products add up in one accumulator.  A bf16 element of x / s
// is exact from 2^-2 on and off by at most 2^-10 below, 2^-17 of the largest.
struct QueryPiece {
  uint4 w[2];
};
__device__ __forceinline__ QueryPiece load_query(const __nv_bfloat16* row, int part) {
  QueryPiece q = {};
  if (row != nullptr) {
    q.w[0] = __ldcg(reinterpret_cast<const uint4*>(row + part * 16));
    q.w[1] = __ldcg(reinterpret_cast<const uint4*>(row + part * 16 + 8));
  }
  return q;
}
// The piece's values over the row's scale, and the scale; an infinite query
// gives NaN logits, not saturated ones.
__device__ __forceinline__ float scale_query(const QueryPiece& q, float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t u = k < 4 ? (&q.w[0].x)[k] : (&q.w[1].x)[k - 4];
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
#pragma unroll
  for (int k = 0; k < 16; ++k) x[k] = fabsf(x[k]) < INFINITY ? x[k] * inv : NAN;
  return scale_of(e);
}
__device__ __forceinline__ float split_query(const QueryPiece& q, uint4& hi, uint4& lo) {
  float x[16];
  const float s = scale_query(q, x);
  uint32_t h[4], l[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t h2[2], l2[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float y0 = x[4 * k + 2 * j], y1 = x[4 * k + 2 * j + 1];
      h2[j] = to_e4m3x2(y0, y1);
      const float2 f = from_e4m3x2(h2[j]);
      l2[j] = to_e4m3x2(y0 - f.x, y1 - f.y);
    }
    h[k] = h2[0] | (h2[1] << 16);
    l[k] = l2[0] | (l2[1] << 16);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
  return s;
}
// The piece in fp16 over the row's scale, and the scale.
__device__ __forceinline__ float half_query(const QueryPiece& q, uint32_t (&h)[8]) {
  float x[16];
  const float s = scale_query(q, x);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const __half2 t = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
    h[k] = *reinterpret_cast<const uint32_t*>(&t);
  }
  return s;
}

// ------------------------------------------------------------------ host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
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

// Codes [rows, g, 128] as (128, g, rows); a box is `box_rows` rows of one K/V
// head.  L2 promotion of 128 bytes: a row of one head is all that is used, and
// 256 would fetch its neighbour's too.
inline bool encode_codes(CUtensorMap* m, const void* base, int64_t rows, int g, int box_rows) {
  const cuuint64_t dims[3] = {cuuint64_t(kD), cuuint64_t(g), cuuint64_t(rows)};
  const cuuint64_t strides[2] = {cuuint64_t(kD), cuuint64_t(g) * kD};
  const cuuint32_t box[3] = {kD, 1, cuuint32_t(box_rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace q8
}  // namespace mqa
