// Joins the partial outputs of a decode over an 8-bit cache: those that the
// CTAs left of each sequence's own rows and, with a shared prefix, those of the
// prefix's blocks.  A part k is a normalised output o_k with lse_k = log2 of
// its softmax sum; the whole is
//   o = sum_k 2^(lse_k - m) o_k / sum_k 2^(lse_k - m),   m = max_k lse_k.
// Bound: latency (a chain of a few L2 round trips).  An output row has kWarps
// warps, one for a few parts and four for many.  Each reads all the parts' lse,
// a lane each (32 at a time), and so knows all weights before it reads outputs;
// it then sums its share of the parts, every lane four columns, with the loads
// of eight parts in flight; the warps' sums are added in their order.  (33 parts
// behind a 2,000-row prefix: 15 us with one warp a row, 6 with four; 7 parts of
// 8,192 rows: 8 us with one, 14 with four.)
#include "q8.cuh"

namespace mqa {
namespace q8 {

namespace {

constexpr int kThreads = 128, kCtaWarps = kThreads / 32;
constexpr int kHeadSize = 128;
constexpr int kAtOnce = 8;

// (sequence, head) of a warp: below 2^31, as the rows of q.
template <int kWarps>
__global__ void __launch_bounds__(kThreads) q8_merge_kernel(const TcArgs a, const PrefixArgs p, int prefix) {
  __shared__ float4 sums[kWarps > 1 ? kWarps - 1 : 1][32];
  const int warp = kWarps > 1 ? threadIdx.x / 32 : 0, lane = threadIdx.x % 32, c4 = lane * 4;
  const unsigned items = unsigned(a.b) * unsigned(a.h);
  const unsigned item = kWarps > 1 ? blockIdx.x : blockIdx.x * kCtaWarps + threadIdx.x / 32;
  const bool active = item < items;   // warp-uniform; all of a CTA's when its warps share an item
  const int s = active ? int(item / unsigned(a.h)) : 0, head = active ? int(item - unsigned(s) * a.h) : 0;
  const int j = head / a.hq, i = head - j * a.hq;
  // The lengths are inputs, not written by the kernels this one follows.
  const bool has_own = __ldcg(a.lens + s) > 0;
  int pre_n = 0;                    // parts of the row's prefix segment
  int64_t pre_at = 0;               // the first of them, then one every kPrefixRows
  if (prefix) {
    const int nb = prefix_tiles(min(max(__ldcg(p.len), 0), p.m_p));
    const unsigned row = unsigned(s) * unsigned(a.hq) + unsigned(i);
    const int seg = j * p.blocks + int(row / kPrefixRows);
    if (nb > 0) {
      const PrefixShare share(a.g * p.blocks, nb, p.grid);
      const int first = share.owner(seg, 0);
      pre_n = share.owner(seg, nb - 1) - first + 1;
      pre_at = (int64_t(first) + seg) * kPrefixRows + row % kPrefixRows;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  if (!active) return;
  int own_first = 0, own_n = 0;
  float empty = 0.f;                // what a row without parts holds
  if (has_own) {
    const int2 info = a.ws.seg_info[int64_t(s) * a.g + j];
    if (info.y == -1) return;       // written whole
    if (parts_named(info, a.groups)) {
      own_first = info.x;
      own_n = info.y - info.x + 1;
    } else {                        // the decode gave up, and its flag says so
      pre_n = 0;
      empty = NAN;
    }
  }
  const int n = own_n + pre_n;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < n; k0 += 32) {
    const int k = k0 + lane;
    const float* o = nullptr;       // lane k's part
    float lse = -INFINITY;
    if (k < n) {
      const bool own = k >= pre_n;
      const int64_t at = own ? tc_slot(own_first + (k - pre_n), s, a.g, j) * a.hq + i : pre_at + int64_t(k) * kPrefixRows;
      o = (own ? a.ws.part_o : p.part_o) + at * kHeadSize;
      lse = __ldcg((own ? a.ws.part_lse : p.part_lse) + at);
    }
    float mx = lse;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float mn = fmaxf(m, mx);
    const float keep = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float wgt = k < n ? exp2f(lse - mn) : 0.f;
    float sum = wgt;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * keep + sum;
    acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
    m = mn;
    const int cnt = min(32, n - k0);
    for (int x0 = 0; x0 < cnt; x0 += kWarps * kAtOnce) {   // this warp's parts: warp, warp + kWarps, ...
      float4 v[kAtOnce];
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {
        const int part = x0 + warp + kWarps * x;
        const float* at = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), part));
        v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (part < cnt) v[x] = __ldcg(reinterpret_cast<const float4*>(at + c4));
      }
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {   // absent parts have weight 0
        const float w = __shfl_sync(0xffffffffu, wgt, x0 + warp + kWarps * x);
        acc.x = fmaf(w, v[x].x, acc.x);
        acc.y = fmaf(w, v[x].y, acc.y);
        acc.z = fmaf(w, v[x].z, acc.z);
        acc.w = fmaf(w, v[x].w, acc.w);
      }
    }
  }
  static_assert(32 % (kWarps * kAtOnce) == 0, "whole steps in a round of 32 parts");
  if constexpr (kWarps > 1) {
    if (warp > 0) sums[warp - 1][lane] = acc;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int x = 0; x < kWarps - 1; ++x) {
      const float4 v = sums[x][lane];
      acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
    }
  }
  const float inv = n > 0 ? 1.f / l : empty;   // no rows at all: zeros
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 out;
  out.x = *reinterpret_cast<const uint32_t*>(&lo);
  out.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + int64_t(item) * kHeadSize + c4) = out;
}

}  // namespace

cudaError_t launch_q8_merge(const TcArgs& a, const PrefixArgs* prefix, cudaStream_t stream) {
  // About how many parts a row has: CTAs per segment, and one more at each seam.
  int parts = a.groups / a.b + 2;
  if (prefix != nullptr) parts += prefix->grid / (prefix->blocks * a.g) + 2;
  const bool many = parts > 12;
  const unsigned items = unsigned(a.b) * unsigned(a.h);   // fewer than 2^31
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(many ? items : (items + kCtaWarps - 1) / kCtaWarps);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const PrefixArgs p = prefix != nullptr ? *prefix : PrefixArgs{};
  return many ? cudaLaunchKernelEx(&cfg, q8_merge_kernel<kCtaWarps>, a, p, prefix != nullptr ? 1 : 0)
              : cudaLaunchKernelEx(&cfg, q8_merge_kernel<1>, a, p, prefix != nullptr ? 1 : 0);
}

}  // namespace q8
}  // namespace mqa
