"""mqa_q8_decode against attention in float64 over the cache's values, with
tolerances derived from the arithmetic (``q8_util``).  Rows that do not count
hold NaN codes and infinite scales."""
import math

import numpy as np
import pytest
import torch

from grouped_query_attention_mqa_b200 import binding, q8
from grouped_query_attention_mqa_b200.build import build

from q8_util import assert_within, attention, cache_parts, dev_cache, host_cache, round_to, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    q8.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(rng, lens, h, g, m_max, d_k, d_v, dtype, path, scale=None, window=0, ctas=0, spread=1.0, q_spread=0.0, arrays=None,
        flag=0):
    b = len(lens)
    scale = 1 / math.sqrt(d_k) if scale is None else scale
    arrays = host_cache(rng, b, m_max, g, d_k, d_v, lens, spread) if arrays is None else arrays
    q, q64 = round_to(rows(rng, (b, h, d_k), q_spread), dtype)
    flags = i32([0])
    o = q8.decode(q.cuda(), dev_cache(arrays), i32(lens), scale, path=path, window=window, num_ctas=ctas, status_flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == flag
    ref, tol = attention(q64, cache_parts(arrays, lens, window), g, scale, dtype, two_terms=path != "simt")
    assert_within(o, ref, tol, f"{path} {dtype} h{h} g{g} d{d_k}/{d_v} ctas{ctas}")


SIMT = [  # lens, h, g, m_max, d_k, d_v
    ([1], 1, 1, 1, 32, 32),
    ([1, 2, 63, 64, 65, 127, 128, 129], 8, 2, 130, 64, 64),
    ([300, 7, 299, 1], 16, 16, 300, 128, 128),
    ([500, 77], 32, 1, 500, 128, 128),
    ([130, 64, 3], 24, 2, 200, 64, 128),
    ([65, 200], 12, 4, 200, 32, 64),
    ([100], 128, 1, 128, 32, 32),
    ([257, 31], 34, 2, 260, 128, 32),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SIMT, ids=lambda c: f"h{c[1]}g{c[2]}d{c[4]}_{c[5]}m{c[3]}")
def test_simt(case, dtype):
    lens, h, g, m_max, d_k, d_v = case
    for ctas in (0, 1, 3):
        run(np.random.default_rng(sum(lens) + ctas), lens, h, g, m_max, d_k, d_v, dtype, "simt", ctas=ctas)


@pytest.mark.parametrize("path,dtype,d", [("simt", "f32", 64), ("simt", "bf16", 32)])
@pytest.mark.parametrize("window", [1, 63, 64, 100, 1000])
def test_window(path, dtype, d, window):
    run(np.random.default_rng(window), [1, 64, 65, 300, 299], 8, 2, 300, d, d, dtype, path, window=window)


@pytest.mark.parametrize("path,dtype", [("simt", "f32"), ("simt", "bf16")])
def test_empty_and_clamped_lengths(path, dtype):
    for m_max in (40, 300):   # without and with a merge
        rng = np.random.default_rng(m_max)
        arrays = host_cache(rng, 4, m_max, 2, 128)
        run(rng, [0, 5, -3, m_max + 9], 8, 2, m_max, 128, 128, dtype, path, arrays=arrays,
            flag=binding.MQA_FLAG_LEN_CLAMPED)


@pytest.mark.parametrize("path,dtype", [("simt", "f32"), ("simt", "bf16")])
def test_sharp_and_flat_softmax(path, dtype):
    """Logits of one row far above the others, and all equal; value rows of
    very different magnitude, and rows of zeros."""
    rng = np.random.default_rng(3)
    run(rng, [300, 17], 8, 1, 300, 128, 128, dtype, path, scale=1.0, q_spread=2.0)
    run(rng, [300, 17], 8, 1, 300, 128, 128, dtype, path, scale=0.0)
    run(rng, [600, 90], 8, 2, 600, 128, 128, dtype, path, spread=6.0)
    arrays = host_cache(rng, 2, 400, 1, 128)
    arrays[2][:, ::3] = 0          # zero value rows, as quantised and as new_cache leaves them
    arrays[3][:, :, ::3] = 1
    arrays[2][0, :256] = 0
    arrays[3][0, :, :256] = 0
    run(rng, [400, 399], 8, 1, 400, 128, 128, dtype, path, arrays=arrays)


def test_nan_inputs_show():
    """A NaN in a valid row reaches the heads that read it and no other."""
    rng = np.random.default_rng(4)
    arrays = host_cache(rng, 2, 100, 2, 128)
    arrays[0][0, 50, 0, 3] = 0x7F
    q, _ = round_to(rng.standard_normal((2, 8, 128)), "bf16")
    for path in ("simt",):
        o = q8.decode(q.cuda(), dev_cache(arrays), i32([100, 100]), 0.1, path=path)
        nan = torch.isnan(o).all(-1).cpu().numpy()
        some = torch.isnan(o).any(-1).cpu().numpy()
        assert nan[0, :4].all() and not some[0, 4:].any() and not some[1].any()


def test_append_then_decode_steps():
    """A cache grown step by step by the quantising append, attended to after
    every step on one stream, and the same steps replayed from a graph."""
    rng = np.random.default_rng(12)
    b, h, g, d, m = 5, 16, 2, 128, 40
    cache = q8.new_cache(b, m, g, d)
    kn = torch.zeros((b, g, d), dtype=torch.bfloat16, device="cuda")
    vn, qd = kn.clone(), torch.zeros((b, h, d), dtype=torch.bfloat16, device="cuda")
    pos, lens = i32([0] * b), i32([1] * b)
    step = (q8.AppendPlan(cache, kn, vn, pos), q8.DecodePlan(qd, cache, lens, 0.09))
    graph = None
    from oracle import q8_oracle
    arrays = [np.zeros((b, m, g, d), np.uint8), np.zeros((b, g, m), np.uint8)]
    arrays = arrays + [x.copy() for x in arrays]
    for t in range(m):
        k, k64 = round_to(rows(rng, (b, g, d)), "bf16")
        v, v64 = round_to(rows(rng, (b, g, d)), "bf16")
        q, q64 = round_to(rng.standard_normal((b, h, d)), "bf16")
        kn.copy_(k), vn.copy_(v), qd.copy_(q), pos.fill_(t), lens.fill_(t + 1)
        if t == 3:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step[0].run(), step[1].run()
        if graph is None:
            step[0].run(), step[1].run()
        else:
            graph.replay()
        for i, x in enumerate((k64, v64)):
            c, e = q8_oracle.quantise(x)
            arrays[2 * i][:, t], arrays[2 * i + 1][:, :, t] = c, e
        ref, tol = attention(q64, cache_parts(arrays, [t + 1] * b), g, 0.09, "bf16", two_terms=True)
        assert_within(step[1].out, ref, tol, f"step {t}")


def test_same_call_twice_is_the_same():
    rng = np.random.default_rng(13)
    arrays = host_cache(rng, 3, 900, 2, 64)
    q, _ = round_to(rng.standard_normal((3, 8, 64)), "f32")
    cache, lens = dev_cache(arrays), i32([900, 1, 511])
    a = q8.decode(q.cuda(), cache, lens, 0.2).clone()
    assert torch.equal(a, q8.decode(q.cuda(), cache, lens, 0.2))
