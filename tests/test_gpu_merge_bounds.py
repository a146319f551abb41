"""The merge kernels on workspaces that a decode left unfinished: a segment
whose CTAs are not named within the launch's becomes NaN, and no index leaves the
workspace; the segments beside it are joined as ever.  The kernels are called
through a small library of their own, built here from the repository's sources,
since no public call leaves such a workspace."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from grouped_query_attention_mqa_b200 import build as build_

SOURCE = r"""
#include "merge.cu"
#include "q8_merge.cu"
using namespace mqa;

extern "C" {

__attribute__((visibility("default"))) void sizes(int b, int g, int hq, size_t* out) {
  const Workspace w = carve_workspace(nullptr, b, g, hq);
  out[0] = workspace_bytes(b, g, hq, 128);
  out[1] = reinterpret_cast<size_t>(w.part_lse);
  out[2] = reinterpret_cast<size_t>(w.part_o);
}

__attribute__((visibility("default"))) int named(int x, int y, int ctas) { return parts_named(make_int2(x, y), ctas); }

__attribute__((visibility("default"))) int merge_16(void* o, const int32_t* lens, void* ws, int b, int h, int g, int m,
                                                    int ctas, int f32, cudaStream_t stream) {
  DecodeArgs a = {};
  a.o = o;
  a.lens = lens;
  a.b = b;
  a.h = h;
  a.g = g;
  a.m_max = m;
  a.d = a.dk = 128;
  a.hq = a.q_group_heads = h / g;
  a.ws = carve_workspace(ws, b, g, h / g);
  a.grid = ctas;
  return launch_merge(a, f32 ? MQA_F32 : MQA_BF16, stream);
}

__attribute__((visibility("default"))) int merge_8(void* o, const int32_t* lens, void* ws, int b, int h, int g, int m,
                                                   int ctas, int f32, cudaStream_t stream) {
  q8::TcArgs a = {};
  a.o = o;
  a.lens = lens;
  a.b = b;
  a.h = h;
  a.g = g;
  a.m = m;
  a.hq = h / g;
  a.ws = carve_workspace(ws, b, g, h / g);
  a.groups = ctas;
  return q8::launch_q8_merge(a, nullptr, stream);
}
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    folder = tmp_path_factory.mktemp("merge")
    src, out = folder / "merges.cu", folder / "merges.so"
    src.write_text(SOURCE)
    subprocess.run([build_.nvcc()] + build_.ARCH + build_.FLAGS + ["-shared", str(src), "-o", str(out)], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(os.fspath(out))
    ptr, i = ctypes.c_void_p, ctypes.c_int
    for name in ("merge_16", "merge_8"):
        getattr(lib, name).argtypes = [ptr, ptr, ptr] + [i] * 6 + [ptr]
    lib.sizes.argtypes = [i, i, i, ptr]
    lib.sizes.restype = None
    lib.named.argtypes = [i, i, i]
    return lib


LOW, HIGH = -2 ** 31, 2 ** 31 - 1
BAD = [(LOW, HIGH), (HIGH, LOW), (0, HIGH), (-1, 1), (LOW, 3), (3, 1), (HIGH, 0), (7, 8), (1 << 30, (1 << 30) + 1),
       (-2, -2 ** 30)]


def test_which_parts_are_named(lib):
    for x, y in BAD + [(0, -1), (5, -2), (8, 8)]:
        assert not lib.named(x, y, 8)
    for x, y in [(0, 0), (7, 7), (0, 7), (3, 4)]:
        assert lib.named(x, y, 8)


@pytest.mark.gpu
@pytest.mark.parametrize("ctas", [8, 64])      # one warp a row in the 8-bit merge, and four
@pytest.mark.parametrize("name,dtype", [("merge_16", torch.bfloat16), ("merge_16", torch.float32), ("merge_8", torch.bfloat16)])
def test_unfinished_segments_become_nan(lib, name, dtype, ctas):
    b, h, g, hq = 14, 6, 1, 6
    size = np.zeros(3, np.uint64)
    lib.sizes(b, g, hq, size.ctypes.data)
    total, lse_at, o_at = (int(x) for x in size)
    ws = torch.full((total,), 0xA5, dtype=torch.uint8, device="cuda")
    bad = [(x, y + ctas - 8 if (x, y) == (7, 8) else y) for x, y in BAD]
    info = bad + [(0, 1), (3, 3) if name == "merge_16" else (3, -1), (5, 7), (0, HIGH)]
    ws[:8 * b * g] = torch.tensor(info, dtype=torch.int32).view(torch.uint8).flatten().cuda()
    lse = ws[lse_at:o_at].view(torch.float32)
    o = ws[o_at:].view(torch.float32)
    for s, first, values in ((10, 0, [1.0, 3.0]), (12, 5, [2.0, 4.0, 9.0])):
        for k, x in enumerate(values):   # equal weights; slot: CTA + segment
            lse[(first + k + s) * hq:(first + k + s + 1) * hq] = 7.0
            o[(first + k + s) * hq * 128:(first + k + s + 1) * hq * 128] = x
    lens = torch.tensor([300] * 13 + [0], dtype=torch.int32, device="cuda")
    out = torch.full((b, h, 128), 55.0, dtype=dtype, device="cuda")
    st = getattr(lib, name)(out.data_ptr(), lens.data_ptr(), ws.data_ptr(), b, h, g, 1000, ctas, dtype == torch.float32,
                            torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert torch.isnan(out[:10]).all()
    # joined, written whole by the decode, joined, no rows
    for s, want in ((10, 2.0), (11, 55.0), (12, 5.0), (13, 0.0)):
        assert (out[s] == want).all()
