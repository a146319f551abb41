// Joins the partial outputs of a decode over an 8-bit cache: those that the
// CTAs left of each sequence's own rows and, with a shared prefix, those of the
// prefix's blocks.  A part k is a normalised output o_k with lse_k = log2 of
// its softmax sum; the whole is
//   o = sum_k 2^(lse_k - m) o_k / sum_k 2^(lse_k - m),   m = max_k lse_k.
// One warp per (sequence, head): its lanes take the parts' lse side by side
// (32 at a time), so that all weights are known before the outputs are read
// and those loads depend on nothing; then every lane sums four columns, in the
// order of the parts.  Bound: latency, and L2 for many parts.
#include "q8.cuh"

namespace mqa {
namespace q8 {

namespace {

constexpr int kThreads = 128;
constexpr int kHeadSize = 128;

__global__ void __launch_bounds__(kThreads) q8_merge_kernel(const TcArgs a, const PrefixArgs p, int prefix) {
  const int64_t item = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;   // (sequence, head)
  const int lane = threadIdx.x % 32, c4 = lane * 4;
  const bool active = item < int64_t(a.b) * a.h;
  const int s = active ? int(item / a.h) : 0, head = active ? int(item - int64_t(s) * a.h) : 0;
  const int j = head / a.hq, i = head - j * a.hq;
  // The lengths are inputs, not written by the kernels this one follows.
  const bool has_own = active && __ldg(a.lens + s) > 0;
  int pre_first = 0, pre_n = 0;     // CTAs that hold parts of the row's prefix segment
  int64_t pre_seg = 0;
  int pre_row = 0;
  if (prefix && active) {
    const int len = min(max(__ldg(p.len), 0), p.m_p), nb = prefix_tiles(len);
    const int64_t row = int64_t(s) * a.hq + i;
    pre_seg = int64_t(j) * p.blocks + row / kPrefixRows;
    pre_row = int(row % kPrefixRows);
    if (nb > 0) {
      const int64_t total = int64_t(a.g) * p.blocks * nb;
      const int ctas = prefix_ctas(total, p.grid);
      pre_first = cta_of_tile(pre_seg * nb, total, ctas);
      pre_n = cta_of_tile(pre_seg * nb + nb - 1, total, ctas) - pre_first + 1;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  if (!active) return;
  int own_first = 0, own_n = 0;
  if (has_own) {
    const int2 info = a.ws.seg_info[int64_t(s) * a.g + j];
    if (info.y < 0) return;         // written whole
    own_first = info.x;
    own_n = info.y - info.x + 1;
  }
  const int n = own_n + pre_n;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < n; k0 += 32) {
    const int k = k0 + lane;
    const float* o = nullptr;       // lane k's part
    float lse = -INFINITY;
    if (k < own_n) {
      const int64_t at = tc_slot(own_first + k, s, a.g, j) * a.hq + i;
      o = a.ws.part_o + at * kHeadSize;
      lse = __ldcg(a.ws.part_lse + at);
    } else if (k < n) {
      const int64_t at = (int64_t(pre_first) + (k - own_n) + pre_seg) * kPrefixRows + pre_row;
      o = p.part_o + at * kHeadSize;
      lse = __ldcg(p.part_lse + at);
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
#pragma unroll 8
    for (int x = 0; x < cnt; ++x) {
      const float w = __shfl_sync(0xffffffffu, wgt, x);
      const float* at = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), x));
      const float4 v = __ldcg(reinterpret_cast<const float4*>(at + c4));
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
  }
  const float inv = n > 0 ? 1.f / l : 0.f;   // no rows at all: zeros
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 out;
  out.x = *reinterpret_cast<const uint32_t*>(&lo);
  out.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + item * kHeadSize + c4) = out;
}

}  // namespace

cudaError_t launch_q8_merge(const TcArgs& a, const PrefixArgs* prefix, cudaStream_t stream) {
  const int64_t items = int64_t(a.b) * a.h, ctas = (items + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q8_merge_kernel, a, prefix != nullptr ? *prefix : PrefixArgs{}, prefix != nullptr ? 1 : 0);
}

}  // namespace q8
}  // namespace mqa
