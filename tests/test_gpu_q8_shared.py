"""mqa_q8_decode_shared against attention in float64 over the prefix's rows
followed by each sequence's own, with tolerances derived from the arithmetic
(``q8_util``)."""
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


def parts_of(prefix, p_len, arrays, lens):
    p = cache_parts(prefix, [p_len])[0]
    return [p + own for own in cache_parts(arrays, lens)]


def run(rng, lens, h, g, m_p, p_len, m_s, scale=0.09, prefix=None, arrays=None, flag=0, q_spread=0.0):
    b = len(lens)
    prefix = host_cache(rng, 1, m_p, g, 128, lens=[p_len]) if prefix is None else prefix
    arrays = host_cache(rng, b, m_s, g, 128, lens=lens) if arrays is None else arrays
    q, q64 = round_to(rows(rng, (b, h, 128), q_spread), "bf16")
    flags = i32([0])
    o = q8.decode_shared(q.cuda(), dev_cache(prefix), i32([p_len]), dev_cache(arrays), i32(lens), scale, status_flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == flag
    ref, tol = attention(q64, parts_of(prefix, p_len, arrays, lens), g, scale, "bf16", two_terms=True)
    assert_within(o, ref, tol, f"b{b} h{h} g{g} p{p_len}")


CASES = [  # lens, h, g, m_p, p_len, m_s
    ([1], 1, 1, 1, 1, 1),
    ([3, 0, 1], 8, 1, 200, 130, 5),
    ([5, 128, 129, 0, 1, 77, 300, 2, 9], 16, 2, 513, 512, 300),
    ([10, 20], 64, 1, 300, 257, 20),
    ([7] * 13, 24, 2, 150, 150, 9),                  # 12 heads per group: five sequences per block
    ([1, 2, 3], 34, 1, 129, 128, 4),                 # 34 heads: one sequence per block
    ([40, 130, 260], 12, 12, 400, 399, 260),         # one head per group: 64 sequences per block
    ([4] * 130, 4, 1, 700, 650, 4),
    ([0] * 5, 8, 2, 100, 99, 3),                     # nothing but the prefix
    ([2] * 250 + [30], 8, 1, 128, 100, 30),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"b{len(c[0])}h{c[1]}g{c[2]}p{c[4]}")
def test_shared(case):
    lens, h, g, m_p, p_len, m_s = case
    run(np.random.default_rng(sum(lens) + m_p), lens, h, g, m_p, p_len, m_s)


def test_no_prefix_and_no_rows():
    rng = np.random.default_rng(1)
    run(rng, [5, 0, 130], 8, 2, 64, 0, 130)           # the empty sequence's row is zero
    run(rng, [0, 0], 8, 2, 64, 0, 4)


def test_lengths_outside_the_caches_are_clamped():
    rng = np.random.default_rng(2)
    prefix, arrays = host_cache(rng, 1, 50, 1, 128), host_cache(rng, 3, 6, 1, 128)
    for p_len, lens in ((51, [1, 2, 3]), (-4, [6, 2, 0]), (9, [7, -1, 0])):
        run(rng, lens, 8, 1, 50, p_len, 6, prefix=prefix, arrays=arrays, flag=binding.MQA_FLAG_LEN_CLAMPED)


def test_prefix_or_own_rows_dominate():
    """Logits far apart between the two parts, in either direction, and value
    rows of different size."""
    rng = np.random.default_rng(3)
    for up in (0, 1):
        prefix, arrays = host_cache(rng, 1, 700, 2, 128), host_cache(rng, 6, 200, 2, 128)
        (arrays if up else prefix)[1][...] += 4
        (prefix if up else arrays)[3][...] += 9
        run(rng, [200, 1, 130, 199, 0, 60], 16, 2, 700, 690, 200, prefix=prefix, arrays=arrays, scale=0.2)


def test_matches_decode_over_joined_rows():
    """The same rows as one cache through mqa_q8_decode: both within the sum of
    two tolerances of each other (each is within one of the exact output)."""
    rng = np.random.default_rng(4)
    b, g, h, P, m = 5, 2, 16, 300, 40
    lens = [40, 1, 0, 17, 33]
    prefix, arrays = host_cache(rng, 1, P, g, 128), host_cache(rng, b, m, g, 128)
    joined = [np.concatenate([np.repeat(p, b, 0), a], axis=1 if p.ndim == 4 else 2) for p, a in zip(prefix, arrays)]
    q, q64 = round_to(rng.standard_normal((b, h, 128)), "bf16")
    o1 = q8.decode_shared(q.cuda(), dev_cache(prefix), i32([P]), dev_cache(arrays), i32(lens), 0.1)
    o2 = q8.decode(q.cuda(), dev_cache(joined), i32([P + n for n in lens]), 0.1)
    _, tol = attention(q64, parts_of(prefix, P, arrays, lens), g, 0.1, "bf16", two_terms=True)
    assert (np.abs((o1.double() - o2.double()).cpu().numpy()) <= 2 * tol).all()


def test_steps_behind_a_shared_prompt():
    """A served batch: one prompt quantised once, then steps that append each
    sequence's row and attend, captured and replayed."""
    from oracle import q8_oracle
    rng = np.random.default_rng(5)
    b, h, g, P, m = 6, 16, 2, 333, 12
    prefix, cache = q8.new_cache(1, 400, g, 128), q8.new_cache(b, m, g, 128)
    pk, pk64 = round_to(rows(rng, (P, g, 128)), "bf16")
    pv, pv64 = round_to(rows(rng, (P, g, 128)), "bf16")
    q8.append(prefix, pk.cuda(), pv.cuda(), i32([0]), cu_new=i32([0, P]))
    host_prefix = []
    for x in (pk64, pv64):
        c, e = q8_oracle.quantise(x)
        host_prefix += [c[None], np.ascontiguousarray(e.T)[None]]
    kn, vn = (torch.zeros((b, g, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qd = torch.zeros((b, h, 128), dtype=torch.bfloat16, device="cuda")
    pos, lens, p_len = i32([0] * b), i32([1] * b), i32([P])
    step = (q8.AppendPlan(cache, kn, vn, pos), q8.SharedPlan(qd, prefix, p_len, cache, lens, 0.09))
    arrays = [np.zeros((b, m, g, 128), np.uint8), np.zeros((b, g, m), np.uint8)]
    arrays = arrays + [x.copy() for x in arrays]
    graph = None
    for t in range(m):
        k, k64 = round_to(rows(rng, (b, g, 128)), "bf16")
        v, v64 = round_to(rows(rng, (b, g, 128)), "bf16")
        q, q64 = round_to(rng.standard_normal((b, h, 128)), "bf16")
        kn.copy_(k), vn.copy_(v), qd.copy_(q), pos.fill_(t), lens.fill_(t + 1)
        if t == 2:
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
        ref, tol = attention(q64, parts_of(host_prefix, P, arrays, [t + 1] * b), g, 0.09, "bf16", two_terms=True)
        assert_within(step[1].out, ref, tol, f"step {t}")


@pytest.mark.parametrize("spread", [4, 20])
def test_values_of_very_different_size(spread):
    """Value rows up to 2^spread apart within a tile, some of them zero, each
    query on one row.  The unpacked values are off by at most 2^-25 units of
    which their tile's largest row has scale 1: 2^-25 of the scale s."""
    rng = np.random.default_rng(8)
    n, b, h = 500, 40, 8
    K = np.sign(rng.standard_normal((1, n, 1, 128)))
    V = rng.standard_normal((1, n, 1, 128)) * np.exp2(rng.uniform(-spread / 2, spread / 2, (1, n, 1, 1)))
    V[0, ::7] = 0
    prefix = []
    for x in (K, V):
        c, e = q8_oracle.quantise(x)
        prefix += [c, np.ascontiguousarray(np.moveaxis(e, 2, 1))]
    at = rng.integers(0, n, (b, h))
    q, q64 = round_to(K[0, at, 0], "bf16")
    arrays = host_cache(rng, b, 2, 1, 128, lens=[0] * b)
    o = q8.decode_shared(q.cuda(), dev_cache(prefix), i32([n]), dev_cache(arrays), i32([0] * b), 0.5)
    ref, tol = attention(q64, parts_of(prefix, n, arrays, [0] * b), 1, 0.5, "bf16", two_terms=True)
    # and weights to 2^-27 of the largest, relative to the tile's scale, times codes up to 448
    s = q8_oracle.scale_of(prefix[3].astype(np.int64)).max()
    assert_within(o, ref, tol + s * (2.0 ** -25 + 448 * 2.0 ** -27))


def test_many_blocks_with_long_runs():
    """More segments than CTAs could take one each, several tiles a CTA."""
    run(np.random.default_rng(11), [1, 0, 5] * 22, 64, 2, 2500, 2395, 5)


def test_value_sizes_that_rise_along_the_prefix():
    """Each tile's values 2^9 above the one before, and a run of zero rows first."""
    rng = np.random.default_rng(9)
    n = 640
    V = rng.standard_normal((1, n, 2, 128)) * np.exp2(9.0 * (np.arange(n) // 64 - 5))[None, :, None, None]
    for zeros in (0, 130):
        V[0, :zeros] = 0
        prefix = []
        for x in (rng.standard_normal((1, n, 2, 128)), V):
            c, e = q8_oracle.quantise(x)
            prefix += [c, np.ascontiguousarray(np.moveaxis(e, 2, 1))]
        run(rng, [3] * 9, 8, 2, n, n, 4, prefix=prefix, scale=0.3)
        run(rng, [3] * 9, 8, 2, n, 100 + zeros // 5, 4, prefix=prefix, scale=0.3)


def test_long_tail_behind_one_heavy_row():
    """One prefix row outweighs each of 15,000 others by up to 2^17.  Weights are
    fp16 numbers of which a reference starts at 2^2: half a step is 2^-25 at
    most, 2^-27 of the heavy row's, and 2^-12 of a weight above 2^-14."""
    rng = np.random.default_rng(10)
    n, b, h, gap = 15000, 300, 64, 17 * np.log(2)
    K = np.zeros((1, n, 1, 128))
    K[0, 0, 0, 0] = 1.0
    V = 1.5 + 0.5 * rng.standard_normal((1, n, 1, 128)).clip(-2, 2)
    prefix = []
    for x in (K, V):
        c, e = q8_oracle.quantise(x)
        prefix += [c, np.ascontiguousarray(np.moveaxis(e, 2, 1))]
    q = np.zeros((1, h, 128))
    q[0, :, 0] = np.linspace(0, 1, h)
    q, q64 = round_to(q, "bf16")
    arrays = host_cache(rng, 1, 2, 1, 128, lens=[0])
    ref, tol = attention(q64, parts_of(prefix, n, arrays, [0]), 1, gap, "bf16", two_terms=False)
    own = q8.new_cache(b, 2, 1, 128)
    o = q8.decode_shared(q.cuda().expand(b, h, 128).contiguous(), dev_cache(prefix), i32([n]), own, i32([0] * b), float(gap))
    M = q64[0, :, :1] * gap
    tol = tol + np.abs(ref) * (2.0 ** -11 + 2 * 2.0 ** -10 / 224 * M) + n * 2.0 ** -27 * 2.5
    assert_within(o, np.repeat(ref, b, 0), np.repeat(tol, b, 0))


def test_captured_call_follows_the_lengths():
    """One capture, replayed with other prefix and own lengths and queries in
    the same buffers: from none of either to all."""
    rng = np.random.default_rng(12)
    b, h, g, m_p, m_s = 7, 24, 2, 900, 150
    prefix, arrays = host_cache(rng, 1, m_p, g, 128), host_cache(rng, b, m_s, g, 128)
    qd, p_len, lens_d = torch.zeros((b, h, 128), dtype=torch.bfloat16, device="cuda"), i32([0]), i32([0] * b)
    plan = q8.SharedPlan(qd, dev_cache(prefix), p_len, dev_cache(arrays), lens_d, 0.1)
    plan.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    for P, lens in ((900, [150] * b), (0, [0] * b), (64, [0, 1, 2, 128, 129, 150, 0]), (1, [0] * b), (0, [3] * b), (899, [7] * b)):
        q, q64 = round_to(rng.standard_normal((b, h, 128)), "bf16")
        qd.copy_(q), p_len.fill_(P), lens_d.copy_(i32(lens))
        graph.replay()
        ref, tol = attention(q64, parts_of(prefix, P, arrays, lens), g, 0.1, "bf16", two_terms=True)
        assert_within(plan.out, ref, tol, f"prefix {P}")


def test_two_calls_at_once():
    """Two plans, each with its workspace, on two streams without any order
    between them: the same bits as one after the other."""
    rng = np.random.default_rng(13)
    plans = []
    for h, g, m_p in ((32, 4, 3000), (8, 1, 5000)):
        prefix, arrays = host_cache(rng, 1, m_p, g, 128), host_cache(rng, 20, 300, g, 128)
        q, _ = round_to(rng.standard_normal((20, h, 128)), "bf16")
        plans.append(q8.SharedPlan(q.cuda(), dev_cache(prefix), i32([m_p]), dev_cache(arrays),
                                   i32(rng.integers(0, 301, 20).tolist()), 0.1))
    want = [p.run().clone() for p in plans]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in plans]
    for _ in range(20):
        for p, s in zip(plans, streams):
            with torch.cuda.stream(s):
                p.run()
    torch.cuda.synchronize()
    for p, w in zip(plans, want):
        assert torch.equal(p.out, w)


def test_prefix_past_32_bits():
    """A prefix of more than 2^32 codes whose last rows outweigh the rest, against
    the decode over the same rows."""
    m_p, g = 530_000, 64
    prefix = q8.new_cache(1, m_p, g, 128)
    assert prefix.k.numel() > 2 ** 32
    gen = torch.Generator("cuda").manual_seed(20)
    for t in (prefix.k, prefix.v):
        for r in range(0, m_p, 100_000):
            n = min(100_000, m_p - r)
            t.view(torch.uint8)[0, r:r + n] = torch.randint(0, 0x78, (n, g, 128), generator=gen, device="cuda", dtype=torch.uint8)
    prefix.k_exp.fill_(118), prefix.v_exp.fill_(120)
    q = torch.randn((1, g, 128), generator=gen, device="cuda").bfloat16()
    heavy = (q[0].sign() * 256).to(torch.float8_e4m3fn)               # q . k is 128 mean|q| 256 / 512 and more
    prefix.k[0, m_p - 70:] = heavy
    own = q8.new_cache(1, 1, g, 128)
    o = q8.decode_shared(q, prefix, i32([m_p]), own, i32([0]), 0.5)
    want = q8.decode(q, prefix, i32([m_p]), 0.5)
    V = prefix.v[0, m_p - 70:].float() / 128
    near = V.mean(0)                                                   # the heavy rows weigh the same
    # both: 2^-9 of a weight, 2^-8 of the output; the rest weighs nothing
    tol = 2.0 ** -7 * V.abs().mean(0) + 2.0 ** -7 * near.abs()
    assert ((o[0].float() - near).abs() <= tol).all() and ((want[0].float() - near).abs() <= tol).all()
