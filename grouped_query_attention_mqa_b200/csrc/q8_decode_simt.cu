// Decode attention over an 8-bit cache on CUDA cores: fp32 queries, and head
// sizes other than the tensor-core kernel's, keys and values of different
// widths included.
//
// The computation is that of the bf16/fp32 decode (velog paper review §3; GQA
// blog "第三站: GQA") on rows code * s:
//   s_{i,t} = scale * s_t * (q_i . code_t),  w = softmax_t(s),
//   o_i = sum_t (w_{i,t} s'_t) code'_t.
// The row scales are powers of two, applied to the logit and to the weight, so
// the inner products run on the codes themselves (exact in fp32).
//
// Work is split as in the other decodes: persistent CTAs over contiguous runs
// of 64-row tiles, partials of split segments combined by the merge kernel.
//
// Up to four heads per group and equal widths: q8_decode_rows_kernel.  D / 16
// lanes hold a row, sixteen codes each, straight from global memory (no shared
// memory, no barrier until a segment ends); every such group of lanes keeps a
// softmax of its own over the rows it meets, four rows to a step, and the
// groups' results are joined at the end.  Bound: HBM latency at these sizes.
// 12 sequences, 8 K/V heads of 64, windows of up to 1500 rows, fp32, two heads
// each: 12.9 us (25.5 with the tile kernel; 15.7 with four CTAs per SM, whose
// registers spill).
//
// Otherwise q8_decode_simt_kernel.  Bound: the queries' reads of shared memory
// and instruction issue, far from HBM (32 fp32 GQA-8 caches of 2K to 8K rows: 836
// us, 6 TFLOP/s; bf16 at head size 64, 64 MQA caches of 1K to 8K rows with 32
// heads: 326 us, 12 times the bf16 cache's tensor-core decode).  Per tile, codes
// staged by 16-byte cp.async, double buffered, converted once per four lanes of a
// row and used for all heads of the group:
//   logits   four lanes share a row, each taking every fourth word of codes;
//            a word becomes four floats in registers, multiplied with every
//            head's query (16-byte broadcast reads of shared memory);
//   softmax  one warp per head, running max and sum in fp32;
//   values   a thread owns four columns of up to 16 heads and a share of the
//            rows; the shares are added in a fixed order at the segment's end.
#include <atomic>
#include <type_traits>

#include "q8.cuh"

namespace mqa {
namespace q8 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 64;

__device__ __forceinline__ void cp_async16(void* smem, const void* gmem) {
  const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait1() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

template <int DK, int DV>
struct Layout {
  // +16: the four lanes of eight consecutive rows read 32 different banks
  static constexpr int kPitchK = DK + 16, kPitchV = DV + 16;
  static constexpr int kStage = kTile * (kPitchK + kPitchV);
  static constexpr int kRedBytes = ((kWarps + kThreads + 2) * 8 + 15) / 16 * 16;
  // schedule scratch, q [hq][DK], p [hq][kTile], o [hq][DV], m/l/alpha [hq], row scales [2][2][kTile], two stages
  static __host__ __device__ size_t bytes(int hq) {
    return size_t(kRedBytes) + size_t(hq) * (DK + kTile + DV) * 4 + (size_t(3 * hq) * 4 + 15) / 16 * 16 +
           4 * kTile * 4 + 2 * size_t(kStage);
  }
};

// Codes of the tile's valid rows into a stage, and its row scales.
template <int DK, int DV>
__device__ __forceinline__ void load_tile(const DecodeQ8Args& a, unsigned char* stage, float* scales,
                                          const TileCoord& tc) {
  using L = Layout<DK, DV>;
  const int64_t row0 = (int64_t(tc.seq) * a.m_max + tc.row0) * a.g + tc.head;
  for (int i = threadIdx.x; i < tc.rows * (DK / 16); i += kThreads) {
    const int r = i / (DK / 16), c = i - r * (DK / 16);
    cp_async16(stage + r * L::kPitchK + c * 16, a.k + (row0 + int64_t(r) * a.g) * DK + c * 16);
  }
  unsigned char* vs = stage + kTile * L::kPitchK;
  for (int i = threadIdx.x; i < tc.rows * (DV / 16); i += kThreads) {
    const int r = i / (DV / 16), c = i - r * (DV / 16);
    cp_async16(vs + r * L::kPitchV + c * 16, a.v + (row0 + int64_t(r) * a.g) * DV + c * 16);
  }
  const int64_t e0 = (int64_t(tc.seq) * a.g + tc.head) * a.m_max + tc.row0;
  if (threadIdx.x < 2 * kTile) {
    const int r = threadIdx.x & (kTile - 1);
    const uint8_t* e = threadIdx.x < kTile ? a.ke : a.ve;
    scales[threadIdx.x] = r < tc.rows ? scale_of(e[e0 + r]) : 0.f;
  }
}

__device__ __forceinline__ float4 four_codes(const unsigned char* p) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  const float2 a = from_e4m3x2(w), b = from_e4m3x2(w >> 16);
  return make_float4(a.x, a.y, b.x, b.y);
}

// HT: heads a thread holds at a time.
template <int DK, int DV, int HT>
__global__ void __launch_bounds__(kThreads, HT == 4 ? 3 : 2) q8_decode_simt_kernel(const DecodeQ8Args a, int is_f32) {
  using L = Layout<DK, DV>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int hq = a.hq, g = a.g;
  int64_t* red = reinterpret_cast<int64_t*>(smem);
  float* q_s = reinterpret_cast<float*>(smem + L::kRedBytes);
  float* p_s = q_s + hq * DK;
  float* o_s = p_s + hq * kTile;
  float* m_s = o_s + hq * DV;
  float* l_s = m_s + hq;
  float* al_s = l_s + hq;
  float* sc_s = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(m_s) + (size_t(3 * hq) * 4 + 15) / 16 * 16);
  unsigned char* stage = reinterpret_cast<unsigned char*>(sc_s + 4 * kTile);
  const float qscale = a.scale * kLog2e;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  auto store = [&](int64_t at, float x) {
    if (is_f32) static_cast<float*>(a.o)[at] = x;
    else static_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16_rn(x);
  };

  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Sched sc = make_schedule<kThreads>(a.lens, a.b, g, a.m_max, a.window, kTile, a.grid, blockIdx.x, a.flags, red);
  if (a.no_merge) {
    for (int s = blockIdx.x; s < a.b; s += gridDim.x)
      if (clamp_len(__ldg(a.lens + s), a.m_max, nullptr, false) == 0)
        for (int k = threadIdx.x; k < a.h * DV; k += kThreads) store(int64_t(s) * a.h * DV + k, 0.f);
  }
  if (sc.t_begin >= sc.t_end) {
    asm volatile("griddepcontrol.launch_dependents;");
    return;
  }
  Cursor cur = cursor_at(a.lens, a.m_max, a.window, kTile, sc.seq, sc.seq_base);
  Cursor nxt = cur;
  cursor_seek(cur, a.lens, g, a.m_max, a.window, kTile, sc.t_begin);
  load_tile<DK, DV>(a, stage, sc_s, tile_coord(cur, g, kTile, sc.t_begin));
  cp_async_commit();

  // Values: a warp's lanes cover the columns (and, for narrow rows, kSub row
  // shares); the warps are head groups of HT heads times row shares.
  constexpr int kCols = DV / 4, kSub = 32 / kCols;
  int hgroups = 1;
  while (hgroups * HT < hq) hgroups <<= 1;                 // 1, 2, 4 or 8: hq <= 128 and HT = 16 above 4 heads
  const int shares = kWarps / hgroups;                     // row shares among warps
  const int hg = warp & (hgroups - 1), share = warp / hgroups;
  const int c4 = (lane % kCols) * 4, sub = lane / kCols;
  const int h0 = hg * HT;
  float4 acc[HT];
#pragma unroll
  for (int i = 0; i < HT; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);

  for (int64_t t = sc.t_begin; t < sc.t_end; ++t) {
    const int st = int((t - sc.t_begin) & 1);
    cursor_seek(cur, a.lens, g, a.m_max, a.window, kTile, t);
    const TileCoord tc = tile_coord(cur, g, kTile, t);
    if (t == sc.t_begin || tc.k == 0) {   // a new segment: its queries, fresh state
      const int64_t q0 = (int64_t(tc.seq) * a.h + int64_t(tc.head) * hq) * DK;
      for (int i = threadIdx.x; i < hq * DK; i += kThreads)
        q_s[i] = qscale * (is_f32 ? static_cast<const float*>(a.q)[q0 + i]
                                  : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[q0 + i]));
      for (int i = threadIdx.x; i < hq; i += kThreads) {
        m_s[i] = -INFINITY;
        l_s[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < HT; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (t + 1 < sc.t_end) {
      cursor_seek(nxt, a.lens, g, a.m_max, a.window, kTile, t + 1);
      load_tile<DK, DV>(a, stage + (st ^ 1) * L::kStage, sc_s + (st ^ 1) * 2 * kTile, tile_coord(nxt, g, kTile, t + 1));
    }
    cp_async_commit();
    cp_async_wait1();
    __syncthreads();
    const unsigned char* ks = stage + st * L::kStage;
    const unsigned char* vs = ks + kTile * L::kPitchK;
    const float* k_scale = sc_s + st * 2 * kTile;
    const float* v_scale = k_scale + kTile;

    {   // logits (log2 units); -inf past the valid rows
      const int r = threadIdx.x / 4, part = threadIdx.x % 4;   // 64 rows x 4 lanes
      const bool valid = r < tc.rows;
      const float ksc = k_scale[r];
      for (int i0 = 0; i0 < hq; i0 += HT) {
        float s[HT];
#pragma unroll
        for (int i = 0; i < HT; ++i) s[i] = 0.f;
        if (valid) {
#pragma unroll 2
          for (int w = 0; w < DK / 16; ++w) {
            const int c = (w * 4 + part) * 4;
            const float4 k = four_codes(ks + r * L::kPitchK + c);
#pragma unroll
            for (int i = 0; i < HT; ++i) {
              if (i0 + i < hq) {
                const float4 q = *reinterpret_cast<const float4*>(q_s + (i0 + i) * DK + c);
                s[i] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[i]))));
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < HT; ++i) {
          s[i] += __shfl_xor_sync(0xffffffffu, s[i], 1);
          s[i] += __shfl_xor_sync(0xffffffffu, s[i], 2);
          if ((i & 3) == part && i0 + i < hq) p_s[(i0 + i) * kTile + r] = valid ? s[i] * ksc : -INFINITY;
        }
      }
    }
    __syncthreads();

    // online softmax, one warp per head; the weights leave with the value rows' scales
    for (int i = warp; i < hq; i += kWarps) {
      const float s0 = p_s[i * kTile + lane], s1 = p_s[i * kTile + lane + 32];
      float mx = fmaxf(s0, s1);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_old = m_s[i], m_new = fmaxf(m_old, mx);
      const float p0 = exp2f(s0 - m_new), p1 = exp2f(s1 - m_new);
      // rows past the valid ones have weight 0 and scale 0
      p_s[i * kTile + lane] = p0 * v_scale[lane];
      p_s[i * kTile + lane + 32] = p1 * v_scale[lane + 32];
      float sum = p0 + p1;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) {
        const float alpha = exp2f(m_old - m_new);
        al_s[i] = alpha;
        l_s[i] = l_s[i] * alpha + sum;
        m_s[i] = m_new;
      }
    }
    __syncthreads();

#pragma unroll
    for (int i = 0; i < HT; ++i) {
      if (h0 + i < hq) {
        const float al = al_s[h0 + i];
        acc[i].x *= al, acc[i].y *= al, acc[i].z *= al, acc[i].w *= al;
      }
    }
#pragma unroll 1
    for (int r0 = (share * kSub + sub) * 4; r0 < tc.rows; r0 += shares * kSub * 4) {   // four rows at a time
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = r0 + k < tc.rows ? four_codes(vs + (r0 + k) * L::kPitchV + c4) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < HT; ++i) {
        if (h0 + i < hq) {
          const float4 p = *reinterpret_cast<const float4*>(p_s + (h0 + i) * kTile + r0);
          acc[i].x = fmaf(p.x, v[0].x, fmaf(p.y, v[1].x, fmaf(p.z, v[2].x, fmaf(p.w, v[3].x, acc[i].x))));
          acc[i].y = fmaf(p.x, v[0].y, fmaf(p.y, v[1].y, fmaf(p.z, v[2].y, fmaf(p.w, v[3].y, acc[i].y))));
          acc[i].z = fmaf(p.x, v[0].z, fmaf(p.y, v[1].z, fmaf(p.z, v[2].z, fmaf(p.w, v[3].z, acc[i].z))));
          acc[i].w = fmaf(p.x, v[0].w, fmaf(p.y, v[1].w, fmaf(p.z, v[2].w, fmaf(p.w, v[3].w, acc[i].w))));
        }
      }
    }

    if (tc.k == tc.nb - 1 || t + 1 == sc.t_end) {   // the segment ends here (for this CTA)
      const bool owns_first = tc.seg_t0 >= sc.t_begin;
      const bool whole = owns_first && tc.seg_t0 + tc.nb <= sc.t_end;
      const int64_t slot = partial_slot(blockIdx.x, tc.seg);
#pragma unroll
      for (int i = 0; i < HT; ++i) {   // row shares within the warp
#pragma unroll
        for (int o = kCols; o < 32; o <<= 1) {
          acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, o);
          acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, o);
          acc[i].z += __shfl_xor_sync(0xffffffffu, acc[i].z, o);
          acc[i].w += __shfl_xor_sync(0xffffffffu, acc[i].w, o);
        }
      }
      for (int sh = 0; sh < shares; ++sh) {   // then the warps', in order
        if (share == sh && sub == 0) {
#pragma unroll
          for (int i = 0; i < HT; ++i) {
            if (h0 + i < hq) {
              float4* o = reinterpret_cast<float4*>(o_s + (h0 + i) * DV + c4);
              float4 x = acc[i];
              if (sh > 0) {
                const float4 y = *o;
                x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
              }
              *o = x;
            }
          }
        }
        __syncthreads();
      }
      for (int f = threadIdx.x; f < hq * DV; f += kThreads) {
        const int i = f / DV, c = f - i * DV;
        const float x = o_s[f] / l_s[i];
        if (whole) store((int64_t(tc.seq) * a.h + int64_t(tc.head) * hq + i) * DV + c, x);
        else a.ws.part_o[(slot * hq + i) * DV + c] = x;
      }
      if (!whole)
        for (int i = threadIdx.x; i < hq; i += kThreads) a.ws.part_lse[slot * hq + i] = m_s[i] + log2f(l_s[i]);
      if (owns_first && threadIdx.x == 0)
        a.ws.seg_info[tc.seg] = make_int2(blockIdx.x, cta_of_tile(tc.seg_t0 + tc.nb - 1, sc.total, sc.active));
    }
    __syncthreads();
  }
  asm volatile("griddepcontrol.launch_dependents;");
}

// ------------------------------------------------------------------ groups of few heads

__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// The codes of a word's k-th half as two fp32.
__device__ __forceinline__ uint64_t code_pair(const uint4& w, int k) {
  const float2 f = from_e4m3x2((&w.x)[k / 2] >> (16 * (k & 1)));
  return pack2(f.x, f.y);
}

constexpr int kRowThreads = 128, kRowWarps = kRowThreads / 32;

template <int D, int HT>
__global__ void __launch_bounds__(kRowThreads, HT <= 2 ? 3 : 2) q8_decode_rows_kernel(const DecodeQ8Args a, int is_f32) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;    // lanes per row, rows per warp and load
  constexpr int kAtOnce = HT <= 2 ? 4 : 2;               // rows of a lane group per step
  __shared__ int64_t red[kRowWarps + kRowThreads + 2];
  __shared__ float4 o_s[kRowWarps][HT][D / 4];
  __shared__ float m_s[kRowWarps][HT], l_s[kRowWarps][HT];
  const int hq = a.hq, g = a.g;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, part = lane % kLanes, group = lane / kLanes;
  const float qscale = a.scale * kLog2e;

  auto store = [&](int64_t at, float x) {
    if (is_f32) static_cast<float*>(a.o)[at] = x;
    else static_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16_rn(x);
  };

  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Sched sc = make_schedule<kRowThreads>(a.lens, a.b, g, a.m_max, a.window, kTile, a.grid, blockIdx.x, a.flags, red);
  if (a.no_merge) {
    for (int s = blockIdx.x; s < a.b; s += gridDim.x)
      if (clamp_len(__ldg(a.lens + s), a.m_max, nullptr, false) == 0)
        for (int k = threadIdx.x; k < a.h * D; k += kRowThreads) store(int64_t(s) * a.h * D + k, 0.f);
  }
  if (sc.t_begin >= sc.t_end) {
    asm volatile("griddepcontrol.launch_dependents;");
    return;
  }
  Cursor cur = cursor_at(a.lens, a.m_max, a.window, kTile, sc.seq, sc.seq_base);
  for (int64_t t = sc.t_begin; t < sc.t_end;) {
    cursor_seek(cur, a.lens, g, a.m_max, a.window, kTile, t);
    const TileCoord tc = tile_coord(cur, g, kTile, t);
    // the CTA's tiles of this segment: rows tc.row0 .. row_end - 1
    const int64_t t_next = min(sc.t_end, tc.seg_t0 + tc.nb);
    const int row_end = min(cur.len, tc.row0 + int(t_next - t) * kTile);
    const uint8_t* const k_at = a.k + ((int64_t(tc.seq) * a.m_max) * g + tc.head) * D + part * 16;
    const uint8_t* const v_at = a.v + ((int64_t(tc.seq) * a.m_max) * g + tc.head) * D + part * 16;
    const int64_t e0 = (int64_t(tc.seq) * g + tc.head) * a.m_max;
    uint64_t q[HT][8], o[HT][8];
    float m[HT], l[HT];
#pragma unroll
    for (int i = 0; i < HT; ++i) {
      const int64_t at = (int64_t(tc.seq) * a.h + int64_t(tc.head) * hq + i) * D + part * 16;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float2 f = make_float2(0.f, 0.f);
        if (i < hq)
          f = is_f32 ? static_cast<const float2*>(a.q)[at / 2 + k]
                     : __bfloat1622float2(static_cast<const __nv_bfloat162*>(a.q)[at / 2 + k]);
        q[i][k] = pack2(f.x * qscale, f.y * qscale);
        o[i][k] = 0;
      }
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    for (int r0 = tc.row0 + (warp * kAtOnce) * kRows + group; r0 - group < row_end; r0 += kRowWarps * kAtOnce * kRows) {
      uint4 kc[kAtOnce], vc[kAtOnce];
      uint32_t ke[kAtOnce], ve[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int r = r0 + u * kRows;
        kc[u] = vc[u] = make_uint4(0, 0, 0, 0);
        ke[u] = ve[u] = 0;
        if (r < row_end) {
          kc[u] = *reinterpret_cast<const uint4*>(k_at + int64_t(r) * g * D);
          vc[u] = *reinterpret_cast<const uint4*>(v_at + int64_t(r) * g * D);
          ke[u] = a.ke[e0 + r];
          ve[u] = a.ve[e0 + r];
        }
      }
      float s[HT][kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        uint64_t dot[HT];
#pragma unroll
        for (int i = 0; i < HT; ++i) dot[i] = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t c = code_pair(kc[u], k);
#pragma unroll
          for (int i = 0; i < HT; ++i) dot[i] = fma2(q[i][k], c, dot[i]);
        }
        const float ks = scale_of(ke[u]);
#pragma unroll
        for (int i = 0; i < HT; ++i) {
          const float2 f = unpack2(dot[i]);
          float x = f.x + f.y;
#pragma unroll
          for (int w = 1; w < kLanes; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
          s[i][u] = r0 + u * kRows < row_end ? x * ks : -INFINITY;
        }
      }
#pragma unroll
      for (int i = 0; i < HT; ++i) {
        float mn = m[i];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) mn = fmaxf(mn, s[i][u]);
        const float ref = mn == -INFINITY ? 0.f : mn;   // no row yet
        const float alpha = exp2f(m[i] - ref);
        m[i] = mn;
        l[i] *= alpha;
        const uint64_t alpha2 = pack2(alpha, alpha);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[i][k] = fma2(o[i][k], alpha2, 0);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const float p = exp2f(s[i][u] - ref);
          l[i] += p;
          s[i][u] = p * scale_of(ve[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t c = code_pair(vc[u], k);
#pragma unroll
          for (int i = 0; i < HT; ++i) o[i][k] = fma2(pack2(s[i][u], s[i][u]), c, o[i][k]);
        }
    }
    // Join the lane groups, then the warps, in a fixed order.
#pragma unroll
    for (int i = 0; i < HT; ++i) {
      float mw = m[i];
#pragma unroll
      for (int w = kLanes; w < 32; w <<= 1) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, w));
      const float f = exp2f(m[i] - (mw == -INFINITY ? 0.f : mw));
      float lw = l[i] * f;
#pragma unroll
      for (int w = kLanes; w < 32; w <<= 1) lw += __shfl_xor_sync(0xffffffffu, lw, w);
      float x[16];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 y = unpack2(o[i][k]);
        x[2 * k] = y.x * f;
        x[2 * k + 1] = y.y * f;
      }
#pragma unroll
      for (int k = 0; k < 16; ++k)
#pragma unroll
        for (int w = kLanes; w < 32; w <<= 1) x[k] += __shfl_xor_sync(0xffffffffu, x[k], w);
      if (group == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) o_s[warp][i][part * 4 + k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
      }
      if (lane == 0) {
        m_s[warp][i] = mw;
        l_s[warp][i] = lw;
      }
    }
    __syncthreads();
    const bool owns_first = tc.seg_t0 >= sc.t_begin;
    const bool whole = owns_first && tc.seg_t0 + tc.nb <= sc.t_end;
    const int64_t slot = partial_slot(blockIdx.x, tc.seg);
    for (int f = threadIdx.x; f < hq * D; f += kRowThreads) {
      const int i = f / D, c = f - i * D;
      float mx = m_s[0][i];
#pragma unroll
      for (int w = 1; w < kRowWarps; ++w) mx = fmaxf(mx, m_s[w][i]);
      float sum = 0.f, x = 0.f;   // some row is valid, so mx is finite (or everything is NaN)
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) {
        const float e = exp2f(m_s[w][i] - mx);
        sum += l_s[w][i] * e;
        x += reinterpret_cast<const float*>(o_s[w][i])[c] * e;
      }
      x /= sum;
      if (whole) store((int64_t(tc.seq) * a.h + int64_t(tc.head) * hq + i) * D + c, x);
      else a.ws.part_o[(slot * hq + i) * D + c] = x;
      if (!whole && c == 0) a.ws.part_lse[slot * hq + i] = mx + log2f(sum);
    }
    if (owns_first && threadIdx.x == 0)
      a.ws.seg_info[tc.seg] = make_int2(blockIdx.x, cta_of_tile(tc.seg_t0 + tc.nb - 1, sc.total, sc.active));
    __syncthreads();   // the tables are free for the next segment
    t = t_next;
  }
  asm volatile("griddepcontrol.launch_dependents;");
}

// ------------------------------------------------------------------ host

template <int DK, int DV, int HT>
cudaError_t ensure_smem_attr() {
  static std::atomic<bool> done[64];   // per device; any thread may set it (the call is idempotent)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  int optin = 0;
  e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(q8_decode_simt_kernel<DK, DV, HT>, cudaFuncAttributeMaxDynamicSharedMemorySize, optin);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

template <typename Kernel>
cudaError_t launch(Kernel kernel, int threads, size_t smem, const DecodeQ8Args& a, int is_f32, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, is_f32);
}

// Resident CTAs per SM of the tile kernel, cached per (device, h/g).
template <int DK, int DV, int HT>
int occupancy(int hq) {
  static std::atomic<int> cache[64][129];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  const bool cacheable = dev >= 0 && dev < 64 && hq >= 1 && hq <= 128;
  if (cacheable) {
    const int c = cache[dev][hq].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  if (ensure_smem_attr<DK, DV, HT>() != cudaSuccess) return 1;
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, q8_decode_simt_kernel<DK, DV, HT>, kThreads,
                                                    Layout<DK, DV>::bytes(hq)) != cudaSuccess || n < 1)
    n = 1;
  if (cacheable) cache[dev][hq].store(n, std::memory_order_relaxed);
  return n;
}

// Up to four heads of equal widths take the rows kernel: fn(D, HT).
bool rows_kernel(int d_k, int d_v, int hq) { return d_k == d_v && hq <= 4; }

template <typename F>
auto dispatch_rows(int d, int hq, F&& fn) {
  auto heads = [&](auto w) {
    if (hq == 1) return fn(w, std::integral_constant<int, 1>());
    if (hq == 2) return fn(w, std::integral_constant<int, 2>());
    return fn(w, std::integral_constant<int, 4>());
  };
  if (d == 32) return heads(std::integral_constant<int, 32>());
  if (d == 64) return heads(std::integral_constant<int, 64>());
  return heads(std::integral_constant<int, 128>());
}

// fn(DK, DV, HT) for the built widths; four heads at a time for small groups
// (fewer registers, more CTAs per SM), sixteen otherwise.
template <typename F>
auto dispatch(int d_k, int d_v, int hq, F&& fn) {
  auto heads = [&](auto dk, auto dv) {
    if constexpr (decltype(dk)::value != decltype(dv)::value)   // small groups of equal widths have a kernel of their own
      if (hq <= 4) return fn(dk, dv, std::integral_constant<int, 4>());
    return fn(dk, dv, std::integral_constant<int, 16>());
  };
  auto values = [&](auto dk) {
    if (d_v == 32) return heads(dk, std::integral_constant<int, 32>());
    if (d_v == 64) return heads(dk, std::integral_constant<int, 64>());
    return heads(dk, std::integral_constant<int, 128>());
  };
  if (d_k == 32) return values(std::integral_constant<int, 32>());
  if (d_k == 64) return values(std::integral_constant<int, 64>());
  return values(std::integral_constant<int, 128>());
}

}  // namespace

cudaError_t launch_q8_decode_simt(const DecodeQ8Args& a, mqa_dtype_t dtype, cudaStream_t stream) {
  const int is_f32 = dtype == MQA_F32;
  if (rows_kernel(a.d_k, a.d_v, a.hq))
    return dispatch_rows(a.d_k, a.hq, [&](auto d, auto ht) {
      return launch(q8_decode_rows_kernel<decltype(d)::value, decltype(ht)::value>, kRowThreads, 0, a, is_f32, stream);
    });
  return dispatch(a.d_k, a.d_v, a.hq, [&](auto dk, auto dv, auto ht) {
    constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value, HT = decltype(ht)::value;
    const cudaError_t e = ensure_smem_attr<DK, DV, HT>();
    if (e != cudaSuccess) return e;
    return launch(q8_decode_simt_kernel<DK, DV, HT>, kThreads, Layout<DK, DV>::bytes(a.hq), a, is_f32, stream);
  });
}

int q8_simt_tile_rows() { return kTile; }

int q8_simt_ctas_per_sm(int d_k, int d_v, int hq) {
  if (rows_kernel(d_k, d_v, hq)) return hq <= 2 ? 3 : 2;   // the kernel's launch bounds
  return dispatch(d_k, d_v, hq, [&](auto dk, auto dv, auto ht) {
    return occupancy<decltype(dk)::value, decltype(dv)::value, decltype(ht)::value>(hq);
  });
}

}  // namespace q8
}  // namespace mqa
