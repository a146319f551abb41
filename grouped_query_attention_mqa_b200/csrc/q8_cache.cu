// The 8-bit cache's rows: quantised as they are written (mqa_q8_append) and
// read back (mqa_q8_read).
//
// Append, per row of one K/V head (the step's "one write-head", velog paper
// review §3, in 8 bits): amax over the row's finite values, s = the smallest
// power of two with amax <= 448 s, code = e4m3(x / s).  The division is a
// multiplication by an exact power of two, so the only rounding is the one to
// e4m3.  Bound: HBM (2 or 4 bytes read and one written per element; the read
// the other way round); a decode step's few rows are bound by the launch.
//
// Both kernels give every thread 8 elements, so d / 8 neighbouring lanes hold
// a row and find its maximum with shuffles: each byte is read once, in one
// pass.  A block takes `rows` consecutive packed rows of all heads, which are
// contiguous in the packed array; its first threads look the rows' sequences
// up (a binary search in the cumulative counts) once for all heads.
#include "q8.cuh"

namespace mqa {
namespace q8 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 256;   // packed rows per block

// (sequence, cache row) of every packed row of the block, or (-1, 0).
__device__ __forceinline__ void locate_rows(int2* where, int r0, int rows, int total, const int32_t* first,
                                            const int32_t* cu, int b, int m_max, int32_t* flags) {
  for (int i = threadIdx.x; i < rows; i += kThreads) {
    const int r = r0 + i;
    int2 at = make_int2(-1, 0);
    if (r < total) {
      int s = r, off = 0;
      bool mine = true;
      if (cu != nullptr) {
        int lo = 0, hi = b;   // the last s with cu[s] <= r
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(cu + mid) <= r) lo = mid;
          else hi = mid;
        }
        const int c0 = __ldg(cu + lo);
        s = lo;
        off = r - c0;
        mine = c0 <= r && c0 >= 0 && r < __ldg(cu + lo + 1);   // holds whatever the counts are
      }
      if (mine) {
        const int64_t p = int64_t(first != nullptr ? __ldg(first + s) : 0) + off;
        if (p >= 0 && p < m_max) at = make_int2(s, int(p));
        else set_flag(flags, MQA_FLAG_POS_SKIPPED);
      }
    }
    where[i] = at;
  }
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
  const float2 a = bf16x2_to_f32x2(w.x), b = bf16x2_to_f32x2(w.y), c = bf16x2_to_f32x2(w.z), d = bf16x2_to_f32x2(w.w);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = c.x, x[5] = c.y, x[6] = d.x, x[7] = d.y;
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

struct CacheArgs {
  uint8_t* codes[2];        // K, V
  uint8_t* exps[2];
  void* packed[2];          // new rows, or rows read
  const int32_t* first;     // cache row of each sequence's first packed row
  const int32_t* cu;
  int b, total, m_max, g, lanes_log2[2];   // lanes_log2: log2 of d / 8
  int rows;                 // packed rows per block
  int32_t* flags;
};

// blockIdx.y: K or V.  kRead: cache -> packed rows, else packed rows -> cache.
template <typename T, bool kRead>
__global__ void __launch_bounds__(kThreads) q8_cache_kernel(const CacheArgs a) {
  __shared__ int2 where[kMaxRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // What follows on the stream may set up now; it waits for this grid's writes.
  asm volatile("griddepcontrol.launch_dependents;");
  const int r0 = blockIdx.x * a.rows;
  const bool val = blockIdx.y != 0;   // values, else keys
  const int ll = val ? a.lanes_log2[1] : a.lanes_log2[0], g = a.g;
  uint8_t* const codes = val ? a.codes[1] : a.codes[0];
  uint8_t* const exps = val ? a.exps[1] : a.exps[0];
  locate_rows(where, r0, a.rows, a.total, a.first, a.cu, a.b, a.m_max, a.flags);
  __syncthreads();
  const int rows = min(a.rows, a.total - r0);
  const int n = (rows * g) << ll;                          // 8-element pieces of this block
  T* const packed = static_cast<T*>(val ? a.packed[1] : a.packed[0]) + ((int64_t(r0) * g) << (ll + 3));
  const int lane_mask = (1 << ll) - 1;
#pragma unroll 4
  for (int i0 = 0; i0 < n; i0 += kThreads) {               // uniform: the shuffles below are warp-wide
    const int i = i0 + int(threadIdx.x);
    const bool in = i < n;
    const int item = in ? i >> ll : 0, row = item / g, head = item - row * g;
    const int2 at = in ? where[row] : make_int2(-1, 0);
    const int c8 = (i & lane_mask) * 8;
    const int64_t code_at = (((int64_t(at.x) * a.m_max + at.y) * g + head) << (ll + 3)) + c8;
    const int64_t exp_at = (int64_t(at.x) * g + head) * a.m_max + at.y;
    if constexpr (kRead) {
      if (at.x >= 0) {
        const uint2 w = *reinterpret_cast<const uint2*>(codes + code_at);
        const float s = scale_of(exps[exp_at]);
        float x[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = from_e4m3x2((k < 2 ? w.x : w.y) >> (16 * (k & 1)));
          x[2 * k] = v.x * s;
          x[2 * k + 1] = v.y * s;
        }
        store8(packed + int64_t(i) * 8, x);
      }
    } else {
      float x[8] = {};
      if (at.x >= 0) load8(packed + int64_t(i) * 8, x);
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float m = fabsf(x[k]);
        amax = m < INFINITY ? fmaxf(amax, m) : amax;       // finite values only
      }
      for (int o = 1; o <= lane_mask; o <<= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const uint32_t e = exponent_for(amax);
      const float inv = inverse_scale(e);
      if (at.x >= 0) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = to_e4m3x2(x[2 * k] * inv, x[2 * k + 1] * inv);
        *reinterpret_cast<uint2*>(codes + code_at) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        if ((i & lane_mask) == 0) exps[exp_at] = uint8_t(e);
      }
    }
  }
}

int log2_lanes(int d) {
  int l = 0;
  while ((8 << l) < d) ++l;
  return l;
}

template <bool kRead>
cudaError_t launch(CacheArgs& a, int d_k, int d_v, mqa_dtype_t dtype, cudaStream_t stream) {
  a.lanes_log2[0] = log2_lanes(d_k);
  a.lanes_log2[1] = log2_lanes(d_v);
  // Four passes of the block per tile where that leaves every SM several
  // blocks, one otherwise (a decode step: as many blocks as there is work for).
  const int64_t pieces = int64_t(a.g) * ((d_k > d_v ? d_k : d_v) / 8);
  const int64_t per = int64_t(a.total) * pieces >= int64_t(148) * 8 * kThreads * 4 ? 4 * kThreads : kThreads;
  const int64_t rows = per / pieces;
  a.rows = int(rows < 1 ? 1 : (rows > kMaxRows ? kMaxRows : rows));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((a.total + a.rows - 1) / a.rows), 2);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (dtype == MQA_BF16) return cudaLaunchKernelEx(&cfg, q8_cache_kernel<__nv_bfloat16, kRead>, a);
  return cudaLaunchKernelEx(&cfg, q8_cache_kernel<float, kRead>, a);
}

}  // namespace

cudaError_t launch_q8_append(uint8_t* k, uint8_t* ke, uint8_t* v, uint8_t* ve, const void* k_new, const void* v_new,
                             const int32_t* pos, const int32_t* cu, int b, int total, int m_max, int g, int d_k,
                             int d_v, mqa_dtype_t dtype, int32_t* flags, cudaStream_t stream) {
  CacheArgs a = {{k, v}, {ke, ve}, {const_cast<void*>(k_new), const_cast<void*>(v_new)}, pos, cu, b, total, m_max, g,
                 {0, 0}, 0, flags};
  return launch<false>(a, d_k, d_v, dtype, stream);
}

cudaError_t launch_q8_read(void* k_out, void* v_out, const uint8_t* k, const uint8_t* ke, const uint8_t* v,
                           const uint8_t* ve, const int32_t* start, const int32_t* cu, int b, int total, int m_max,
                           int g, int d_k, int d_v, mqa_dtype_t dtype, int32_t* flags, cudaStream_t stream) {
  CacheArgs a = {{const_cast<uint8_t*>(k), const_cast<uint8_t*>(v)}, {const_cast<uint8_t*>(ke), const_cast<uint8_t*>(ve)},
                 {k_out, v_out}, start, cu, b, total, m_max, g, {0, 0}, 0, flags};
  return launch<true>(a, d_k, d_v, dtype, stream);
}

}  // namespace q8
}  // namespace mqa
