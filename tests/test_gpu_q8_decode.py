"""mqa_q8_decode against attention in float64 over the cache's values, with
tolerances derived from the arithmetic (``q8_util``).  Rows that do not count
hold NaN codes and infinite scales."""
import math

import numpy as np
import pytest
import torch

from grouped_query_attention_mqa_b200 import binding, q8
from grouped_query_attention_mqa_b200.build import build

from oracle import q8_oracle
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


TC = [  # lens, h, g, m_max: tile edges (128 and 256 rows), all group widths, split and whole segments
    ([1], 1, 1, 1),
    ([1, 127, 128, 129, 255, 256, 257], 8, 1, 260),
    ([700, 511, 512, 513], 32, 1, 700),
    ([300, 1, 256], 48, 3, 300),
    ([640, 129, 1000], 64, 1, 1000),
    ([385, 128, 2], 66, 2, 400),
    ([400, 30], 40, 8, 400),
    ([260, 90, 33], 24, 2, 260),
    ([5] * 200 + [600] + [0] * 7 + [128] * 200, 16, 2, 600),     # more sequences than threads of the schedule
]


@pytest.mark.parametrize("case", TC, ids=lambda c: f"b{len(c[0])}h{c[1]}g{c[2]}m{c[3]}")
def test_tensor_cores(case):
    lens, h, g, m_max = case
    for ctas in (0, 1, 5):
        run(np.random.default_rng(sum(lens) + ctas), lens, h, g, m_max, 128, 128, "bf16", "tcgen05", ctas=ctas,
            flag=binding.MQA_FLAG_LEN_CLAMPED if 0 in lens else 0)


def test_tensor_cores_growing_logits():
    """References that have to move, tile after tile: keys (and values) that
    grow along the sequence."""
    rng = np.random.default_rng(21)
    for h in (16, 32, 64):
        arrays = host_cache(rng, 2, 1500, 1, 128)
        for i in (1, 3):
            arrays[i] = (arrays[i] + (np.arange(1500) // 200)[None, None]).astype(np.uint8)
        run(rng, [1500, 1111], h, 1, 1500, 128, 128, "bf16", "tcgen05", arrays=arrays, scale=0.02)
        arrays[3] = arrays[3][:, :, ::-1].copy()
        run(rng, [1500, 1111], h, 1, 1500, 128, 128, "bf16", "tcgen05", arrays=arrays, scale=0.02, ctas=1)


def test_tensor_cores_attention_sink():
    """A heavy row with small values: the others keep their precision."""
    rng = np.random.default_rng(22)
    arrays = host_cache(rng, 1, 4000, 1, 128, spread=0.2)
    q, q64 = round_to(rng.standard_normal((1, 8, 128)), "bf16")
    from oracle import q8_oracle
    k0 = np.ones(128) * 3
    q64[...] = np.abs(q64)
    q = torch.from_numpy(q64).to(torch.bfloat16)
    arrays[0][0, 0, 0], arrays[1][0, 0, 0] = q8_oracle.quantise(k0)
    arrays[3][0, 0, 0] -= 7
    o = q8.decode(q.cuda(), dev_cache(arrays), i32([4000]), 0.04)
    ref, tol = attention(q64, cache_parts(arrays, [4000]), 1, 0.04, "bf16", two_terms=True)
    assert_within(o, ref, tol, "sink")


def test_queries_of_very_different_size():
    """Each query row has a scale of its own; zeros, tiny and huge rows."""
    rng = np.random.default_rng(23)
    arrays = host_cache(rng, 2, 300, 1, 128)
    size = np.exp2(rng.integers(-60, 3, (2, 16, 1)).astype(float))
    size[0, 0] = 0
    q, q64 = round_to(rng.standard_normal((2, 16, 128)) * size, "bf16")
    o = q8.decode(q.cuda(), dev_cache(arrays), i32([300, 200]), 0.3, path="tcgen05")
    ref, tol = attention(q64, cache_parts(arrays, [300, 200]), 1, 0.3, "bf16", two_terms=True)
    assert_within(o, ref, tol)


@pytest.mark.parametrize("path,dtype,d", [("simt", "f32", 64), ("simt", "bf16", 32), ("tcgen05", "bf16", 128)])
@pytest.mark.parametrize("window", [1, 63, 64, 100, 1000])
def test_window(path, dtype, d, window):
    run(np.random.default_rng(window), [1, 64, 65, 300, 299], 8, 2, 300, d, d, dtype, path, window=window)


@pytest.mark.parametrize("path,dtype", [("simt", "f32"), ("simt", "bf16"), ("tcgen05", "bf16")])
def test_empty_and_clamped_lengths(path, dtype):
    for m_max in (40, 300):   # without and with a merge
        rng = np.random.default_rng(m_max)
        arrays = host_cache(rng, 4, m_max, 2, 128)
        run(rng, [0, 5, -3, m_max + 9], 8, 2, m_max, 128, 128, dtype, path, arrays=arrays,
            flag=binding.MQA_FLAG_LEN_CLAMPED)


@pytest.mark.parametrize("path,dtype", [("simt", "f32"), ("simt", "bf16"), ("tcgen05", "bf16")])
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
    for path in ("simt", "tcgen05"):
        o = q8.decode(q.cuda(), dev_cache(arrays), i32([100, 100]), 0.1, path=path)
        nan = torch.isnan(o).all(-1).cpu().numpy()
        some = torch.isnan(o).any(-1).cpu().numpy()
        assert nan[0, :4].all() and not some[0, 4:].any() and not some[1].any()
        bad = q.clone()
        bad[1, 5, 100], bad[0, 6, 0] = float("inf"), float("nan")
        arrays2 = host_cache(np.random.default_rng(5), 2, 100, 2, 128)
        o = q8.decode(bad.cuda(), dev_cache(arrays2), i32([100, 100]), 0.1, path=path)
        some = torch.isnan(o).any(-1).cpu()
        assert bool(torch.isnan(o[1, 5]).all()) and bool(torch.isnan(o[0, 6]).all()) and int(some.sum()) == 2


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


def test_two_captured_calls_do_not_share_a_workspace():
    """Two plans captured into graphs and replayed in turn on two streams."""
    rng = np.random.default_rng(14)
    plans, want = [], []
    for k in range(2):
        arrays = host_cache(rng, 4, 2000, 2, 128)
        lens = [2000, 1500, 3, 900]
        q, q64 = round_to(rng.standard_normal((4, 32, 128)), "bf16")
        plans.append(q8.DecodePlan(q.cuda(), dev_cache(arrays), i32(lens), 0.1))
        want.append(attention(q64, cache_parts(arrays, lens), 2, 0.1, "bf16", two_terms=True))
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for p in plans:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run()
        graphs.append(g)
    for p in plans:
        p.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for p, (ref, tol) in zip(plans, want):
        assert_within(p.out, ref, tol)


def test_calls_on_a_given_stream():
    """Functions (not plans) on a side stream, back to back, with the caller's
    stream busy allocating: each call's workspace belongs to the side stream."""
    rng = np.random.default_rng(15)
    arrays = host_cache(rng, 2, 1200, 2, 128)
    lens = [1200, 700]
    qs = [round_to(rng.standard_normal((2, 32, 128)), "bf16") for _ in range(4)]
    want = [attention(q64, cache_parts(arrays, lens), 2, 0.1, "bf16", two_terms=True) for _, q64 in qs]
    cache, lens_d, qd = dev_cache(arrays), i32(lens), [q.cuda() for q, _ in qs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for q in qd * 5:
        outs.append(q8.decode(q, cache, lens_d, 0.1, stream=side))
        torch.empty(64 << 20, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for k, o in enumerate(outs):
        assert_within(o, *want[k % 4])


def test_refusals_raise():
    cache = q8.new_cache(2, 8, 1, 128)
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.MqaError, match="UNSUPPORTED"):
        q8.decode(q.float(), cache, i32([1, 1]), 1.0, path="tcgen05")
    with pytest.raises(binding.MqaError, match="INVALID_ARG"):
        q8.decode(q, cache, i32([1, 1]), float("nan"))
    with pytest.raises(ValueError):
        q8.decode(q[:1], cache, i32([1, 1]), 1.0)
    with pytest.raises(TypeError):
        q8.decode(q, (cache.k.view(torch.uint8), *cache[1:]), i32([1, 1]), 1.0)
    with pytest.raises(ValueError):
        q8.decode(q, cache, i32([1, 1]).long(), 1.0)
    with pytest.raises(ValueError):
        q8.append(cache, q[:1, :1], q[:1, :1], i32([0, 0]))
    empty = q8.new_cache(0, 8, 1, 128)
    assert q8.decode(q[:0], empty, i32([]), 1.0).shape == (0, 4, 128)


@pytest.mark.parametrize("where", [0, 700, 19999])
@pytest.mark.parametrize("h", [5, 24, 64])
def test_tensor_cores_long_tail_behind_one_heavy_row(h, where):
    """Row ``where`` outweighs each of 20,000 others by up to 2^17, so that the
    others are below a weight's grid relative to it and yet a seventh of the
    result: their weights' roundings, to steps of 2^-13 where the heavy row's P
    is 2^2, must average out.  Weights of 2^-8 of the heavy one and more: 2^-8
    of each at most.  Smaller ones: a rounding is off by less than a step, 2^-15
    of the heavy weight, with a mean of 0 over the dither's 256 values; over n
    rows 2^-15 n^1/2 / 2 is a standard deviation where all differ (half a step
    each, |v| <= 2.5), and 5 of them are allowed."""
    rng = np.random.default_rng(16)
    n, gap = 20000, 17 * np.log(2)
    K = np.zeros((1, n, 1, 128))
    K[0, where, 0, 0] = 1.0
    V = 1.5 + 0.5 * rng.standard_normal((1, n, 1, 128)).clip(-2, 2)
    arrays = []
    for x in (K, V):
        c, e = q8_oracle.quantise(x)
        arrays += [c, np.ascontiguousarray(np.moveaxis(e, 2, 1))]
    q = np.zeros((1, h, 128))
    q[0, :, 0] = np.linspace(0, 1, h)          # gaps of 0 to 17 octaves
    q, q64 = round_to(q, "bf16")
    o = q8.decode(q.cuda(), dev_cache(arrays), i32([n]), float(gap), num_ctas=1)
    ref, tol = attention(q64, cache_parts(arrays, [n]), 1, gap, "bf16", two_terms=False)
    heavy = np.exp(gap * q64[0, :, 0])
    total = heavy + n - 1
    grid = 5 * 2.0 ** -16 * 2.5 * np.sqrt(n) * heavy / total
    M = q64[0, :, :1] * gap
    tol = tol + np.abs(ref) * (2.0 ** -8 + 2 * 2.0 ** -10 / 224 * M) + grid[:, None]
    assert_within(o, ref, tol)


def test_tensor_cores_references_up_and_down():
    """Heavy rows in some tiles and not in others, differently for each head."""
    rng = np.random.default_rng(17)
    n, h = 6000, 24
    K = 0.02 * rng.standard_normal((1, n, 1, 128))
    K[0, rng.integers(0, n, 40), 0, :] *= 40.0
    arrays = []
    for x in (K, rows(rng, (1, n, 1, 128), 3.0)):
        c, e = q8_oracle.quantise(x)
        arrays += [c, np.ascontiguousarray(np.moveaxis(e, 2, 1))]
    run(rng, [n], h, 1, n, 128, 128, "bf16", "tcgen05", scale=1.0, ctas=1, arrays=arrays, q_spread=1.0)


@pytest.mark.parametrize("h,g", [(200, 200), (700, 700), (303, 101)])
def test_tensor_cores_many_kv_heads(h, g):
    """More K/V heads than a grid has CTAs, or a number that does not divide it."""
    run(np.random.default_rng(18), [150, 1, 0, 129], h, g, 150, 128, 128, "bf16", "tcgen05",
        flag=binding.MQA_FLAG_LEN_CLAMPED)   # a decode reports an empty sequence


@pytest.mark.parametrize("path,dtype", [("tcgen05", torch.bfloat16), ("simt", torch.float32)])
def test_offsets_past_32_bits(path, dtype):
    """The last sequences of a cache of more than 2^32 codes against the same
    sequences alone: the same bits."""
    b, m, g = 65, 16384, 32
    big = q8.new_cache(b, m, g, 128)
    assert big.k.numel() > 2 ** 32
    gen = torch.Generator("cuda").manual_seed(19)
    lens = [0] * (b - 2) + [1500, 16384]
    for t, top in ((big.k, 0x7f), (big.v, 0x7f)):   # no NaN
        t.view(torch.uint8)[b - 2:] = torch.randint(0, top, (2, m, g, 128), generator=gen, device="cuda", dtype=torch.uint8)
    for t in (big.k_exp, big.v_exp):
        t[b - 2:] = torch.randint(115, 120, (2, g, m), generator=gen, device="cuda", dtype=torch.uint8)
    small = q8.Cache(*(t[b - 2:].clone() for t in big))
    q = torch.randn((b, 64, 128), generator=gen, device="cuda").to(dtype)
    flags = i32([0])
    o = q8.decode(q, big, i32(lens), 1e-3, path=path, status_flags=flags)
    want = q8.decode(q[b - 2:].contiguous(), small, i32(lens[-2:]), 1e-3, path=path)
    assert torch.equal(o[b - 2:], want) and not o[:b - 2].any() and want.float().abs().min() > 0
    assert int(flags) == binding.MQA_FLAG_LEN_CLAMPED
