// The C ABI over 8-bit caches: argument checks, the choice of kernel path and
// CTA count, and the launches.  No allocation, no synchronisation, no
// exceptions.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "q8.cuh"

namespace {

using namespace mqa;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool valid_dtype(int dt) { return dt == MQA_F32 || dt == MQA_BF16; }
bool all_aligned16(std::initializer_list<const void*> ps) {   // and not NULL
  for (const void* p : ps)
    if (p == nullptr || !aligned16(p)) return false;
  return true;
}

// SM count of the current device, cached per device.
int sm_count() {
  static std::atomic<int> cache[64];   // 0 = not yet known; every thread computes the same value
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Head sizes of the append and the read: a row's 16-element pieces fill 1 to 16
// lanes, a power of two.
bool row_width(int d) { return d == 16 || d == 32 || d == 64 || d == 128 || d == 256; }

// Checks shared by the append and the read; MQA_OK with *done set means there
// is nothing to do.
mqa_status_t check_rows(const void* k, const void* ke, const void* v, const void* ve, const void* kp, const void* vp,
                        int b, int total, int m_max, int g, int d_k, int d_v, mqa_dtype_t dtype, bool* done) {
  *done = false;
  if (b < 0 || total < 0 || m_max < 1 || g < 1 || d_k < 1 || d_v < 1 || !valid_dtype(dtype)) return MQA_ERR_INVALID_ARG;
  if (b == 0 || total == 0) {
    *done = true;
    return MQA_OK;
  }
  if (!all_aligned16({k, v}) || !kp || !vp || !aligned32(kp) || !aligned32(vp) || !ke || !ve) return MQA_ERR_INVALID_ARG;
  if (int64_t(b) * g > (int64_t(1) << 30) || int64_t(b) * m_max * g > (int64_t(1) << 40) || g > (1 << 20))
    return MQA_ERR_INVALID_ARG;
  if (!row_width(d_k) || !row_width(d_v)) return MQA_ERR_UNSUPPORTED;
  return MQA_OK;
}

// What the merge kernel reads of a decode.
DecodeArgs merge_args(const q8::DecodeQ8Args& a) {
  DecodeArgs m = {};
  m.o = a.o;
  m.lens = a.lens;
  m.b = a.b;
  m.h = a.h;
  m.g = a.g;
  m.m_max = a.m_max;
  m.d = a.d_v;
  m.dk = a.d_k;
  m.hq = a.hq;
  m.window = a.window;
  m.q_group_heads = a.hq;
  m.scale = a.scale;
  m.ws = a.ws;
  m.flags = a.flags;
  m.grid = a.grid;
  return m;
}

}  // namespace

extern "C" {

mqa_status_t mqa_q8_append(void* k_codes, uint8_t* k_exps, void* v_codes, uint8_t* v_exps, const void* k_new,
                           const void* v_new, const int32_t* pos, const int32_t* cu_new, int b, int total, int m_max,
                           int g, int d_k, int d_v, mqa_dtype_t dtype, int32_t* status_flags, cudaStream_t stream) {
  bool done;
  const mqa_status_t st = check_rows(k_codes, k_exps, v_codes, v_exps, k_new, v_new, b, total, m_max, g, d_k, d_v, dtype, &done);
  if (st != MQA_OK || done) return st;
  if (!all_aligned16({pos}) || (cu_new && !aligned16(cu_new)) || (!cu_new && total != b)) return MQA_ERR_INVALID_ARG;
  if (q8::launch_q8_append(static_cast<uint8_t*>(k_codes), k_exps, static_cast<uint8_t*>(v_codes), v_exps, k_new, v_new,
                           pos, cu_new, b, total, m_max, g, d_k, d_v, dtype, status_flags, stream) != cudaSuccess)
    return MQA_ERR_CUDA;
  return MQA_OK;
}

mqa_status_t mqa_q8_read(void* k_out, void* v_out, const void* k_codes, const uint8_t* k_exps, const void* v_codes,
                         const uint8_t* v_exps, const int32_t* start, const int32_t* cu_rows, int b, int total,
                         int m_max, int g, int d_k, int d_v, mqa_dtype_t dtype, int32_t* status_flags,
                         cudaStream_t stream) {
  bool done;
  const mqa_status_t st = check_rows(k_codes, k_exps, v_codes, v_exps, k_out, v_out, b, total, m_max, g, d_k, d_v, dtype, &done);
  if (st != MQA_OK || done) return st;
  if (!all_aligned16({cu_rows}) || (start && !aligned16(start))) return MQA_ERR_INVALID_ARG;
  if (q8::launch_q8_read(k_out, v_out, static_cast<const uint8_t*>(k_codes), k_exps,
                         static_cast<const uint8_t*>(v_codes), v_exps, start, cu_rows, b, total, m_max, g, d_k, d_v,
                         dtype, status_flags, stream) != cudaSuccess)
    return MQA_ERR_CUDA;
  return MQA_OK;
}

size_t mqa_q8_decode_workspace_size(int b, int h, int g, int d_v) {
  if (b < 0 || h < 1 || g < 1 || h % g != 0 || d_v < 1) return 0;
  return workspace_bytes(b, g, h / g, d_v);
}

mqa_status_t mqa_q8_decode(void* o, const void* q, const void* k_codes, const uint8_t* k_exps, const void* v_codes,
                           const uint8_t* v_exps, const int32_t* lens, int b, int h, int g, int m_max, int d_k,
                           int d_v, float scale, mqa_dtype_t dtype, void* workspace, size_t workspace_bytes_given,
                           int32_t* status_flags, const mqa_decode_opts_t* opts, cudaStream_t stream) {
  if (b < 0 || h < 1 || g < 1 || h % g != 0 || m_max < 1 || d_k < 1 || d_v < 1 || !valid_dtype(dtype) ||
      !std::isfinite(scale))
    return MQA_ERR_INVALID_ARG;
  const int path = opts ? opts->path : MQA_PATH_AUTO;
  if (path < MQA_PATH_AUTO || path > MQA_PATH_TCGEN05) return MQA_ERR_INVALID_ARG;
  if (opts && (opts->num_ctas < 0 || opts->num_ctas > kMaxCtas || opts->window < 0)) return MQA_ERR_INVALID_ARG;
  if (b == 0) return MQA_OK;
  if (!all_aligned16({o, q, k_codes, v_codes, lens}) || !k_exps || !v_exps || !workspace || !aligned256(workspace))
    return MQA_ERR_INVALID_ARG;
  if (int64_t(b) * g > (int64_t(1) << 30) || int64_t(b) * m_max * g > (int64_t(1) << 40) ||
      int64_t(b) * h >= (int64_t(1) << 31))
    return MQA_ERR_INVALID_ARG;
  const int hq = h / g;
  if (workspace_bytes_given < workspace_bytes(b, g, hq, d_v)) return MQA_ERR_INVALID_ARG;
  if ((d_k != 32 && d_k != 64 && d_k != 128) || (d_v != 32 && d_v != 64 && d_v != 128)) return MQA_ERR_UNSUPPORTED;
  const bool simt_ok = int64_t(hq) * d_k <= 4096 && int64_t(hq) * d_v <= 4096;
  const bool tc_ok = dtype == MQA_BF16 && q8::q8_tc_supported(d_k, d_v, hq, g);
  if (path == MQA_PATH_TCGEN05 ? !tc_ok : path == MQA_PATH_SIMT ? !simt_ok : !tc_ok && !simt_ok)
    return MQA_ERR_UNSUPPORTED;
  const bool use_tc = path == MQA_PATH_TCGEN05 || (path == MQA_PATH_AUTO && tc_ok);

  const int sms = sm_count();
  if (sms <= 0) return MQA_ERR_CUDA;
  const int window = opts ? opts->window : 0;
  const int span_max = window > 0 && window < m_max ? window : m_max;
  const Workspace ws = carve_workspace(workspace, b, g, hq);
  const int wish = opts && opts->num_ctas > 0 ? opts->num_ctas
                                              : sms * (use_tc ? q8::q8_tc_ctas_per_sm() : q8::q8_simt_ctas_per_sm(d_k, d_v, hq));
  const int grid = wish < 1 ? 1 : (wish > kMaxCtas ? kMaxCtas : wish);
  if (use_tc) {
    q8::TcArgs a = {};
    a.o = o;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.ke = k_exps;
    a.ve = v_exps;
    a.lens = lens;
    a.b = b;
    a.h = h;
    a.g = g;
    a.hq = hq;
    a.m = m_max;
    a.window = window;
    a.no_merge = span_max <= q8::q8_tc_tile_rows();   // no segment can be split: every row is final as it is
    a.groups = q8::tc_groups(grid, g);
    a.scale = scale;
    a.ws = ws;
    a.flags = status_flags;
    if (!q8::q8_tc_fits(b, m_max)) return MQA_ERR_INVALID_ARG;   // sizes past the kernel's index range
    if (q8::launch_q8_decode_tc(a, static_cast<const uint8_t*>(k_codes), static_cast<const uint8_t*>(v_codes), stream) !=
            cudaSuccess ||
        (!a.no_merge && q8::launch_q8_merge(a, nullptr, stream) != cudaSuccess)) return MQA_ERR_CUDA;
    return MQA_OK;
  }
  q8::DecodeQ8Args a;
  a.o = o;
  a.q = q;
  a.k = static_cast<const uint8_t*>(k_codes);
  a.ke = k_exps;
  a.v = static_cast<const uint8_t*>(v_codes);
  a.ve = v_exps;
  a.lens = lens;
  a.b = b;
  a.h = h;
  a.g = g;
  a.m_max = m_max;
  a.d_k = d_k;
  a.d_v = d_v;
  a.hq = hq;
  a.window = window;
  a.no_merge = span_max <= q8::q8_simt_tile_rows();
  a.scale = scale;
  a.ws = ws;
  a.flags = status_flags;
  a.grid = grid;
  if (q8::launch_q8_decode_simt(a, dtype, stream) != cudaSuccess) return MQA_ERR_CUDA;
  if (!a.no_merge && launch_merge(merge_args(a), dtype, stream) != cudaSuccess) return MQA_ERR_CUDA;
  return MQA_OK;
}

}  // extern "C"

namespace {

// Workspace of a decode behind a shared prefix: the own rows' partials as for
// a decode, then the prefix's (outputs, log-sum-exps), then the prefix unpacked
// (keys, values, what its tiles are relative to).
struct SharedSizes {
  int64_t blocks, tiles;
  size_t own, lse, o, rows, exps;   // bytes of each part
  SharedSizes(int b, int g, int hq, int m_p, int d) {
    blocks = (int64_t(b) * hq + q8::kPrefixRows - 1) / q8::kPrefixRows;
    tiles = (int64_t(m_p) + q8::kPrefixKeys - 1) / q8::kPrefixKeys;
    const size_t part_rows = size_t(q8::kPrefixMaxCtas + blocks * g) * q8::kPrefixRows;
    own = workspace_bytes(b, g, hq, d);
    lse = align256(sizeof(float) * part_rows);
    o = align256(sizeof(float) * part_rows * size_t(d));
    rows = align256(2 * size_t(g) * size_t(tiles) * q8::kPrefixKeys * size_t(d));
    exps = align256(sizeof(int2) * size_t(g) * size_t(tiles));
  }
  size_t total() const { return own + lse + o + 2 * rows + exps; }
};

}  // namespace

extern "C" {

size_t mqa_q8_decode_shared_workspace_size(int b, int h, int g, int m_p, int d) {
  if (b < 0 || h < 1 || g < 1 || h % g != 0 || m_p < 1 || d < 1 || h / g > 64) return 0;
  return SharedSizes(b, g, h / g, m_p, d).total();
}

mqa_status_t mqa_q8_decode_shared(void* o, const void* q, const void* prefix_k, const uint8_t* prefix_k_exps,
                                  const void* prefix_v, const uint8_t* prefix_v_exps, const int32_t* prefix_len,
                                  const void* k_codes, const uint8_t* k_exps, const void* v_codes,
                                  const uint8_t* v_exps, const int32_t* lens, int b, int h, int g, int m_p, int m_s,
                                  int d, float scale, mqa_dtype_t dtype, void* workspace, size_t workspace_bytes_given,
                                  int32_t* status_flags, cudaStream_t stream) {
  if (b < 0 || h < 1 || g < 1 || h % g != 0 || m_p < 1 || m_s < 1 || d < 1 || !valid_dtype(dtype) ||
      !std::isfinite(scale))
    return MQA_ERR_INVALID_ARG;
  if (b == 0) return MQA_OK;
  if (!all_aligned16({o, q, prefix_k, prefix_v, prefix_len, k_codes, v_codes, lens}) || !prefix_k_exps ||
      !prefix_v_exps || !k_exps || !v_exps || !workspace || !aligned256(workspace))
    return MQA_ERR_INVALID_ARG;
  if (int64_t(b) * g > (int64_t(1) << 29) || int64_t(b) * m_s * g > (int64_t(1) << 40) ||
      int64_t(m_p) * g > (int64_t(1) << 40) || int64_t(b) * h >= (int64_t(1) << 31) || !q8::q8_tc_fits(b, m_s) ||
      !q8::q8_tc_fits(1, m_p) || g > 65535 ||   // a grid dimension
      ((int64_t(b) * (h / g) + q8::kPrefixRows - 1) / q8::kPrefixRows) * g *
              ((int64_t(m_p) + q8::kPrefixKeys - 1) / q8::kPrefixKeys + q8::kPrefixSeam) >=
          (int64_t(1) << 31))
    return MQA_ERR_INVALID_ARG;   // past the kernels' index range
  const int hq = h / g;
  if (dtype != MQA_BF16 || !q8::q8_tc_supported(d, d, hq, g)) return MQA_ERR_UNSUPPORTED;
  if (workspace_bytes_given < mqa_q8_decode_shared_workspace_size(b, h, g, m_p, d)) return MQA_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0) return MQA_ERR_CUDA;
  const SharedSizes size(b, g, hq, m_p, d);
  char* at = static_cast<char*>(workspace) + size.own;
  q8::PrefixArgs p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const uint8_t*>(prefix_k);
  p.ke = prefix_k_exps;
  p.v = static_cast<const uint8_t*>(prefix_v);
  p.ve = prefix_v_exps;
  p.len = prefix_len;
  p.b = b;
  p.h = h;
  p.g = g;
  p.hq = hq;
  p.m_p = m_p;
  p.blocks = int(size.blocks);
  p.tiles = int(size.tiles);
  p.scale = scale;
  p.part_lse = reinterpret_cast<float*>(at);
  p.part_o = reinterpret_cast<float*>(at += size.lse);
  p.k16 = reinterpret_cast<__half*>(at += size.o);
  p.v16 = reinterpret_cast<__half*>(at += size.rows);
  p.tile_exps = reinterpret_cast<int2*>(at += size.rows);
  p.flags = status_flags;
  // Two CTAs per SM for a long run of tiles; one when there are only a few, so
  // that the own rows' CTAs fit beside them and the rows have half the parts
  // (12 sequences behind 2,000 rows: 27.4 -> 24.5 us; 256 behind 8,192: 46 -> 52).
  const bool few = size.blocks * g * size.tiles <= int64_t(4) * sms;
  const int ctas = few ? sms : sms * q8::q8_tc_ctas_per_sm();
  p.grid = ctas < q8::kPrefixMaxCtas ? ctas : q8::kPrefixMaxCtas;
  q8::TcArgs a = {};
  a.o = o;
  a.q = p.q;
  a.ke = k_exps;
  a.ve = v_exps;
  a.lens = lens;
  a.b = b;
  a.h = h;
  a.g = g;
  a.hq = hq;
  a.m = m_s;
  a.partials = 1;
  a.groups = q8::tc_groups(ctas, g);
  a.scale = scale;
  a.ws = carve_workspace(workspace, b, g, hq);
  a.flags = status_flags;
  cudaError_t e = q8::launch_q8_prefix(p, stream);
  if (e == cudaSuccess)
    e = q8::launch_q8_decode_tc(a, static_cast<const uint8_t*>(k_codes), static_cast<const uint8_t*>(v_codes), stream);
  if (e == cudaSuccess) e = q8::launch_q8_merge(a, &p, stream);
  return e == cudaSuccess ? MQA_OK : MQA_ERR_CUDA;
}

}  // extern "C"
