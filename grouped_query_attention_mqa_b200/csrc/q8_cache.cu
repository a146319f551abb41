// The 8-bit cache's rows: quantised as they are written (mqa_q8_append) and
// read back (mqa_q8_read).
//
// Append, per row of one K/V head (the step's "one write-head", velog paper
// review §3, in 8 bits): amax over the row's finite values, s = the smallest
// power of two with amax <= 448 s, code = e4m3(x / s).  The division is a
// multiplication by an exact power of two, so the only rounding is the one to
// e4m3.  Bound: HBM (2 or 4 bytes read and one written per element; the read
// the other way round): eight bf16 prompts of up to 4,096 rows with 8 heads of
// 128, 118 MB, are written in 23.3 us, 16 of them, 252 MB, read back in 42.5 us
// (5.1 and 5.9 TB/s; the prompts in 20.3 us where the L2 still holds part of
// them).  A decode step's few rows are bound by the launch: 1.8 us in a replayed
// graph, 4.4 in calls from Python.
//
// Both kernels give every thread 16 elements (32-byte loads and stores of bf16,
// 16-byte ones of codes), so d / 16 neighbouring lanes hold a row and find its
// maximum with shuffles: each byte is read once, in one pass.  A block takes
// `rows` consecutive packed rows of all heads, which are contiguous in the
// packed array, and looks their sequences up once for all heads.
#include "q8.cuh"

namespace mqa {
namespace q8 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 256;   // packed rows per block

// Where a packed row lives in the cache: its row among all (sequence, row)
// pairs, and the place of its first head's exponent; `row` < 0: nowhere.
struct __align__(16) Place {
  int64_t row, exp;
};

// The places of packed rows r0 .. r0 + rows - 1 of the block.  Every thread looks
// at a sequence (one round of independent loads); those with rows in the block
// have them written down by their warp.  Whatever the counts are, only
// rows of the block and of the cache are named.
__device__ __forceinline__ void locate_rows(Place* where, int r0, int rows, const int32_t* first, const int32_t* cu, int b,
                                            int m_max, int g, int32_t* flags) {
  auto place = [&](int s, int64_t p) {
    Place at = {-1, 0};
    if (p >= 0 && p < m_max) at = {int64_t(s) * m_max + p, int64_t(s) * g * m_max + p};
    else set_flag(flags, MQA_FLAG_POS_SKIPPED);
    return at;
  };
  if (cu == nullptr) {   // row r is sequence r's
    for (int i = threadIdx.x; i < rows; i += kThreads)
      where[i] = place(r0 + i, first != nullptr ? __ldg(first + r0 + i) : 0);
    __syncthreads();
    return;
  }
  for (int i = threadIdx.x; i < rows; i += kThreads) where[i] = {-1, 0};
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int s0 = int(threadIdx.x) - lane; s0 < b; s0 += kThreads) {
    const int s = s0 + lane;
    int lo = 0, hi = 0;
    int64_t p = 0;       // cache row of the first of this sequence's rows in the block
    if (s < b) {
      const int c0 = __ldg(cu + s), c1 = __ldg(cu + s + 1);
      const int64_t p0 = first != nullptr ? __ldg(first + s) : 0;
      lo = max(c0, r0);
      hi = c0 < 0 ? lo : min(c1, r0 + rows);
      p = p0 + (int64_t(lo) - c0);
    }
    uint32_t found = __ballot_sync(0xffffffffu, lo < hi);
    while (found != 0) {   // the warp's lanes share each such sequence's rows
      const int x = __ffs(found) - 1;
      found &= found - 1;
      // from the block's first row on: r0 + 31 may be past an int
      const int xlo = __shfl_sync(0xffffffffu, lo, x) - r0, xhi = __shfl_sync(0xffffffffu, hi, x) - r0;
      const int64_t xp = __shfl_sync(0xffffffffu, (long long)p, x);
      for (int r = xlo + lane; r < xhi; r += 32) where[r] = place(s0 + x, xp + (r - xlo));
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}

// Sixteen elements as they lie in memory.
template <typename T>
struct Piece;

template <>
struct Piece<__nv_bfloat16> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { load32(p, w); }
  // Largest magnitude as a pair of bf16 patterns (NaNs are passed over);
  // infinities left out if `finite`.
  __device__ __forceinline__ uint32_t top(bool finite) const {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t u = w[k] & 0x7fff7fffu;
      if (finite) {
        if ((u & 0xffffu) >= 0x7f80u) u &= 0xffff0000u;
        if ((u >> 16) >= 0x7f80u) u &= 0xffffu;
      }
      m = join(m, u);
    }
    return m;
  }
  static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  // The joined maximum's fp32 pattern.
  static __device__ __forceinline__ uint32_t pattern(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
  __device__ __forceinline__ float2 pair(int k) const { return bf16x2_to_f32x2(w[k]); }
  __device__ __forceinline__ void set(int k, float x, float y) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(x, y);
    w[k] = *reinterpret_cast<const uint32_t*>(&t);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { store32(p, w); }
};

template <>
struct Piece<float> {
  uint32_t w[16];
  __device__ __forceinline__ void load(const float* p) {
    load32(p, w);
    load32(p + 8, w + 8);
  }
  __device__ __forceinline__ uint32_t top(bool finite) const {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      uint32_t u = w[k] & 0x7fffffffu;
      if (finite && u >= 0x7f800000u) u = 0;
      m = max(m, u);
    }
    return m;
  }
  static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t pattern(uint32_t m) { return m; }
  __device__ __forceinline__ float2 pair(int k) const { return make_float2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1])); }
  __device__ __forceinline__ void set(int k, float x, float y) {
    w[2 * k] = __float_as_uint(x);
    w[2 * k + 1] = __float_as_uint(y);
  }
  __device__ __forceinline__ void store(float* p) const {
    store32(p, w);
    store32(p + 8, w + 8);
  }
};

struct CacheArgs {
  uint8_t* codes[2];        // K, V
  uint8_t* exps[2];
  void* packed[2];          // new rows, or rows read
  const int32_t* first;     // cache row of each sequence's first packed row
  const int32_t* cu;
  int b, total, m_max, g, lanes_log2[2];   // lanes_log2: log2 of d / 16
  int rows;                 // packed rows per block
  unsigned g_inverse;       // floor(2^32 / g) + 1 (g > 1), or 0 where a block has one row
  int32_t* flags;
};

// blockIdx.y: K or V.  kRead: cache -> packed rows, else packed rows -> cache.
// Bound by instructions as much as by HBM: a thread's elements are kept as
// they lie in memory, maxima are taken on their bit patterns.
template <typename T, bool kRead, int kAtOnce>
__global__ void __launch_bounds__(kThreads) q8_cache_kernel(const CacheArgs a) {
  __shared__ Place where[kMaxRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // What follows on the stream may set up now; it waits for this grid's writes.
  asm volatile("griddepcontrol.launch_dependents;");
  const int r0 = blockIdx.x * a.rows;
  const bool val = blockIdx.y != 0;   // values, else keys
  const int ll = val ? a.lanes_log2[1] : a.lanes_log2[0], g = a.g;
  uint8_t* const codes = val ? a.codes[1] : a.codes[0];
  uint8_t* const exps = val ? a.exps[1] : a.exps[0];
  const int rows = min(a.rows, a.total - r0);
  locate_rows(where, r0, rows, a.first, a.cu, a.b, a.m_max, g, a.flags);
  const int n = (rows * g) << ll;                          // pieces of this block
  T* const packed = static_cast<T*>(val ? a.packed[1] : a.packed[0]) + ((int64_t(r0) * g) << (ll + 4));
  const int lane_mask = (1 << ll) - 1;
  // kAtOnce pieces per thread, their loads all in flight before the first is used
  for (int i0 = threadIdx.x; i0 - int(threadIdx.x) < n; i0 += kAtOnce * kThreads) {   // uniform: shuffles below
    int64_t code_at[kAtOnce], exp_at[kAtOnce];
    Piece<T> x[kAtOnce];
    uint4 w[kAtOnce];
    uint32_t e[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kThreads;
      const int item = i >> ll, row = g == 1 ? item : int(__umulhi(unsigned(item), a.g_inverse)),
                head = item - row * g;
      const Place at = i < n ? where[row] : Place{-1, 0};
      code_at[u] = at.row < 0 ? -1 : ((at.row * g + head) << (ll + 4)) + (i & lane_mask) * 16;
      exp_at[u] = at.exp + int64_t(head) * a.m_max;
      if constexpr (kRead) {
        if (code_at[u] >= 0) {
          w[u] = *reinterpret_cast<const uint4*>(codes + code_at[u]);
          e[u] = exps[exp_at[u]];
        }
      } else {
        if (code_at[u] >= 0) {
          x[u].load(packed + int64_t(i) * 16);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[u].set(k, 0.f, 0.f);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kThreads;
      if constexpr (kRead) {
        if (code_at[u] >= 0) {
          const float s = scale_of(e[u]);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 v = from_e4m3x2((&w[u].x)[k / 2] >> (16 * (k & 1)));
            x[u].set(k, v.x * s, v.y * s);
          }
          x[u].store(packed + int64_t(i) * 16);
        }
      } else {
        auto row_top = [&](bool finite) {
          uint32_t m = x[u].top(finite);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < ll) m = Piece<T>::join(m, __shfl_xor_sync(0xffffffffu, m, 1 << k));
          return Piece<T>::pattern(m);
        };
        uint32_t top = row_top(false);
        if (__any_sync(0xffffffffu, top >= 0x7f800000u)) top = row_top(true);   // finite values only
        const uint32_t ex = exponent_for(__uint_as_float(top));
        const float inv = inverse_scale(ex);
        if (code_at[u] >= 0) {
          uint32_t c[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 v = x[u].pair(k);
            c[k] = to_e4m3x2(v.x * inv, v.y * inv);
          }
          *reinterpret_cast<uint4*>(codes + code_at[u]) = make_uint4(c[0] | (c[1] << 16), c[2] | (c[3] << 16), c[4] | (c[5] << 16),
                                                                    c[6] | (c[7] << 16));
          if ((i & lane_mask) == 0) exps[exp_at[u]] = uint8_t(ex);
        }
      }
    }
  }
}

int log2_lanes(int d) {
  int l = 0;
  while ((16 << l) < d) ++l;
  return l;
}

template <bool kRead>
cudaError_t launch(CacheArgs& a, int d_k, int d_v, mqa_dtype_t dtype, cudaStream_t stream) {
  a.lanes_log2[0] = log2_lanes(d_k);
  a.lanes_log2[1] = log2_lanes(d_v);
  // Two pieces per thread and step, four steps, where that leaves every SM
  // several blocks; one piece otherwise (a decode step: as many blocks as there
  // is work for).
  const int64_t pieces = int64_t(a.g) * ((d_k > d_v ? d_k : d_v) / 16);
  const bool large = int64_t(a.total) * pieces >= int64_t(148) * 4 * kThreads * 8;
  const int64_t rows = (large ? 8 * kThreads : kThreads) / pieces;
  a.rows = int(rows < 1 ? 1 : (rows > kMaxRows ? kMaxRows : rows));
  // exact for the block's rows x heads, at most 8 kThreads pieces when it has several rows
  a.g_inverse = a.rows == 1 ? 0u : unsigned((uint64_t(1) << 32) / unsigned(a.g)) + 1u;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((int64_t(a.total) + a.rows - 1) / a.rows), 2);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (dtype == MQA_BF16)
    return large ? cudaLaunchKernelEx(&cfg, q8_cache_kernel<__nv_bfloat16, kRead, 2>, a)
                 : cudaLaunchKernelEx(&cfg, q8_cache_kernel<__nv_bfloat16, kRead, 1>, a);
  return large ? cudaLaunchKernelEx(&cfg, q8_cache_kernel<float, kRead, 2>, a)
               : cudaLaunchKernelEx(&cfg, q8_cache_kernel<float, kRead, 1>, a);
}

}  // namespace

cudaError_t launch_q8_append(uint8_t* k, uint8_t* ke, uint8_t* v, uint8_t* ve, const void* k_new, const void* v_new,
                             const int32_t* pos, const int32_t* cu, int b, int total, int m_max, int g, int d_k,
                             int d_v, mqa_dtype_t dtype, int32_t* flags, cudaStream_t stream) {
  CacheArgs a = {{k, v}, {ke, ve}, {const_cast<void*>(k_new), const_cast<void*>(v_new)}, pos, cu, b, total, m_max, g,
                 {0, 0}, 0, 0, flags};
  return launch<false>(a, d_k, d_v, dtype, stream);
}

cudaError_t launch_q8_read(void* k_out, void* v_out, const uint8_t* k, const uint8_t* ke, const uint8_t* v,
                           const uint8_t* ve, const int32_t* start, const int32_t* cu, int b, int total, int m_max,
                           int g, int d_k, int d_v, mqa_dtype_t dtype, int32_t* flags, cudaStream_t stream) {
  CacheArgs a = {{const_cast<uint8_t*>(k), const_cast<uint8_t*>(v)}, {const_cast<uint8_t*>(ke), const_cast<uint8_t*>(ve)},
                 {k_out, v_out}, start, cu, b, total, m_max, g, {0, 0}, 0, 0, flags};
  return launch<true>(a, d_k, d_v, dtype, stream);
}

}  // namespace q8
}  // namespace mqa
