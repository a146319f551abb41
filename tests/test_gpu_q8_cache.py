"""mqa_q8_append and mqa_q8_read against the float64 oracle of the format:
codes and exponents have one right answer and must equal it; rows that no call
names stay as they were."""
import numpy as np
import pytest
import torch

from grouped_query_attention_mqa_b200 import binding, q8
from grouped_query_attention_mqa_b200.build import build
from oracle import q8_oracle

from q8_util import dev_cache, host_cache, round_to, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    q8.lib()


def host(cache):
    k, ke, v, ve = (t.view(torch.uint8).cpu().numpy() for t in cache)
    return [k, ke, v, ve]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same_codes(a, b):
    """Equal codes; a NaN may have either sign."""
    nan = (a & 0x7F) == 0x7F
    return np.array_equal(nan, (b & 0x7F) == 0x7F) and np.array_equal(a[~nan], b[~nan])


def expect_append(arrays, new, seqs, at):
    """The host cache after rows new = (k, v) [total, g, d] went to (seqs[i], at[i])."""
    out = [x.copy() for x in arrays]
    for i, x in enumerate(new):
        c, e = q8_oracle.quantise(x)
        for r, (s, p) in enumerate(zip(seqs, at)):
            if p is not None and 0 <= p < arrays[0].shape[1]:
                out[2 * i][s, p] = c[r]
                out[2 * i + 1][s, :, p] = e[r]
    return out


def check(cache, want):
    got = host(cache)
    for i in (0, 2):
        assert same_codes(got[i], want[i])
        assert np.array_equal(got[i + 1], want[i + 1])


CASES = [  # b, m_max, g, d_k, d_v, new rows per sequence (None: one each), dtype
    (1, 1, 1, 16, 16, None, "bf16"),
    (5, 33, 3, 128, 128, None, "f32"),
    (64, 17, 1, 128, 64, None, "bf16"),
    (3, 40, 8, 32, 256, [0, 7, 40], "bf16"),
    (4, 129, 5, 64, 64, [1, 128, 0, 63], "f32"),
    (2, 700, 8, 128, 128, [699, 300], "bf16"),
    (7, 11, 2, 256, 16, [3, 0, 0, 11, 1, 2, 5], "bf16"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(map(str, c[:5])))
def test_append_writes_the_oracles_codes(case):
    b, m_max, g, d_k, d_v, new, dtype = case
    rng = np.random.default_rng(b * m_max + d_k)
    n = [1] * b if new is None else new
    total = sum(n)
    before = host_cache(rng, b, m_max, g, d_k, d_v)
    k, k64 = round_to(rows(rng, (total, g, d_k), 4.0), dtype)
    v, v64 = round_to(rows(rng, (total, g, d_v), 4.0), dtype)
    start = [int(rng.integers(0, m_max - x + 1)) for x in n]
    cu = np.concatenate([[0], np.cumsum(n)])
    cache, flags = dev_cache(before), i32([0])
    got = q8.append(cache, k.cuda(), v.cuda(), i32(start), cu_new=None if new is None else i32(cu), status_flags=flags)
    torch.cuda.synchronize()
    assert got.k.data_ptr() == cache.k.data_ptr() and int(flags) == 0
    seqs = [s for s in range(b) for _ in range(n[s])]
    at = [start[s] + i for s in range(b) for i in range(n[s])]
    check(cache, expect_append(before, (k64, v64), seqs, at))


def test_append_special_values():
    """Zeros, subnormals, halves of a step (ties), the largest numbers,
    infinities and NaN, each in rows of their own and mixed."""
    d = 16
    base = np.zeros((12, d), np.float32)
    base[1] = 2.0 ** -140
    base[2] = np.linspace(-448, 448, d)
    base[3, :8] = [17, 19, 18, 1.0625, 1.1875, 240, 248, 464]      # ties and their neighbours
    base[4] = 3.0e38
    base[5, :3] = [np.inf, -np.inf, 1.0]
    base[6, :3] = [np.nan, -np.nan, -3.0]
    base[7] = np.inf
    base[8] = np.nan
    base[9, :2] = [448, 2.0 ** -9]
    base[10, :2] = [448, 2.0 ** -10]                                  # half of the smallest code
    base[11, :4] = [-0.0, 1e-30, -1e-38, 1e-20]
    for dtype in ("f32", "bf16"):
        x, x64 = round_to(base[:, None], dtype)
        y, y64 = round_to(-base[::-1, None], dtype)
        before = host_cache(np.random.default_rng(0), 1, 12, 1, d)
        cache = dev_cache(before)
        q8.append(cache, x.cuda(), y.cuda(), i32([0]), cu_new=i32([0, 12]))
        torch.cuda.synchronize()
        check(cache, expect_append(before, (x64, y64), [0] * 12, range(12)))


def test_append_skips_and_flags_rows_outside_the_cache():
    rng = np.random.default_rng(5)
    before = host_cache(rng, 4, 10, 2, 32)
    k, k64 = round_to(rows(rng, (4, 2, 32)), "bf16")
    for pos in ([-1, 3, 10, 2 ** 31 - 1], [0, 9, 5, -2 ** 31]):
        cache, flags = dev_cache(before), i32([0])
        q8.append(cache, k.cuda(), k.cuda(), i32(pos), status_flags=flags)
        torch.cuda.synchronize()
        assert int(flags) == binding.MQA_FLAG_POS_SKIPPED
        check(cache, expect_append(before, (k64, k64), range(4), pos))
    # packed rows running past the end of the cache: the first ones are written
    cache, flags = dev_cache(before), i32([0])
    q8.append(cache, k.cuda(), k.cuda(), i32([8, 0, 0, 0]), cu_new=i32([0, 4, 4, 4, 4]), status_flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == binding.MQA_FLAG_POS_SKIPPED
    check(cache, expect_append(before, (k64, k64), [0] * 4, [8, 9, None, None]))


def test_append_ignores_rows_of_no_sequence_and_bad_counts():
    rng = np.random.default_rng(6)
    before = host_cache(rng, 3, 20, 1, 64)
    k, k64 = round_to(rows(rng, (9, 1, 64)), "f32")
    cache = dev_cache(before)
    q8.append(cache, k.cuda(), k.cuda(), i32([0, 5, 10]), cu_new=i32([1, 3, 3, 6]))   # rows 0, 6, 7, 8 belong to none
    torch.cuda.synchronize()
    check(cache, expect_append(before, (k64, k64), [0, 0, 0, 2, 2, 2, 0, 0, 0], [None, 0, 1, 10, 11, 12, None, None, None]))
    for cu in ([0, 50, -3, 9], [9, 6, 3, 0], [-5, -4, -3, -2]):   # decreasing or negative: nothing outside is touched
        cache = dev_cache(before)
        q8.append(cache, k.cuda(), k.cuda(), i32([0, 5, 10]), cu_new=i32(cu))
    torch.cuda.synchronize()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(map(str, c[:5])))
def test_read_returns_the_values(case):
    b, m_max, g, d_k, d_v, n, dtype = case
    rng = np.random.default_rng(b + m_max + d_k)
    n = [1] * b if n is None else n
    arrays = host_cache(rng, b, m_max, g, d_k, d_v, spread=4.0)
    cu = np.concatenate([[0], np.cumsum(n)])
    start = [int(rng.integers(0, m_max - x + 1)) for x in n]
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    total = int(cu[-1]) + 2                                          # two packed rows of no sequence
    out = tuple(torch.full((total, g, d), 7.0, dtype=dt, device="cuda") for d in (d_k, d_v))
    flags = i32([0])
    q8.read(dev_cache(arrays), i32(cu), total, start=i32(start), out=out, status_flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == 0
    for i in (0, 1):
        val = q8_oracle.values(arrays[2 * i], arrays[2 * i + 1])
        want = np.concatenate([val[s, start[s]:start[s] + n[s]] for s in range(b)] + [np.full((2, g, val.shape[3]), 7.0)])
        assert np.array_equal(out[i].double().cpu().numpy(), want)   # exact in both types


def test_read_leaves_rows_outside_the_cache_and_reads_odd_exponents():
    rng = np.random.default_rng(8)
    arrays = host_cache(rng, 2, 6, 1, 32)
    arrays[1][0, 0, :3] = [0, 255, 254]
    out = tuple(torch.full((5, 1, 32), 7.0, device="cuda") for _ in range(2))
    flags = i32([0])
    q8.read(dev_cache(arrays), i32([0, 4, 5]), 5, start=i32([-1, 5]), out=out, status_flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == binding.MQA_FLAG_POS_SKIPPED
    with np.errstate(over="ignore", invalid="ignore"):
        val = (q8_oracle.values(arrays[0], arrays[1])).astype(np.float32)
    got = out[0].cpu().numpy()
    assert np.array_equal(got[0], np.full((1, 32), 7.0, np.float32))
    assert np.array_equal(got[1:4], val[0, :3], equal_nan=True) and np.array_equal(got[4], val[1, 5])


def test_what_was_read_and_appended_again_is_the_same_cache():
    rng = np.random.default_rng(9)
    b, m, g, d = 3, 50, 2, 128
    n = [50, 1, 20]
    k, _ = round_to(rows(rng, (sum(n), g, d)), "bf16")
    cu = i32(np.concatenate([[0], np.cumsum(n)]))
    first = q8.append(q8.new_cache(b, m, g, d), k.cuda(), (-k).cuda(), i32([0, 0, 0]), cu_new=cu)
    kk, vv = q8.read(first, cu, sum(n))
    second = q8.append(q8.new_cache(b, m, g, d), kk, vv, i32([0, 0, 0]), cu_new=cu)
    k2, v2 = q8.read(second, cu, sum(n))
    torch.cuda.synchronize()
    assert torch.equal(kk, k2) and torch.equal(vv, v2)


def test_large_offsets():
    """Cache rows past 2^31 bytes: the last sequence of a 2.2 GB code array."""
    b, m_max, g, d = 17, 1 << 20, 1, 128
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB free")
    cache = q8.new_cache(b, m_max, g, d)
    rng = np.random.default_rng(10)
    k, k64 = round_to(rows(rng, (b, g, d)), "bf16")
    q8.append(cache, k.cuda(), (2 * k).cuda(), i32([m_max - 1] * b))
    out = q8.read(cache, i32([0] * b + [2]), 2, start=i32([m_max - 2] * b))
    torch.cuda.synchronize()
    c, e = q8_oracle.quantise(k64)
    want = q8_oracle.TABLE[c] * q8_oracle.scale_of(e)[..., None]
    assert not out[0][0].any() and np.array_equal(out[0][1].double().cpu().numpy(), want[-1])
    assert np.array_equal(out[1][1].double().cpu().numpy(), 2 * want[-1])


def test_plans_streams_and_graphs():
    """A plan on another stream, and captured into a graph that is replayed
    with new rows in the same buffers."""
    rng = np.random.default_rng(11)
    b, m, g, d = 8, 30, 2, 64
    cache = q8.new_cache(b, m, g, d)
    k, _ = round_to(rows(rng, (b, g, d)), "bf16")
    kn, pos = k.cuda(), i32([0] * b)
    plan = q8.AppendPlan(cache, kn, kn, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    want = host_cache(rng, b, m, g, d)
    want = [np.zeros_like(x) for x in want]
    want = expect_append(want, (k.double().numpy(), k.double().numpy()), range(b), [0] * b)
    for step in range(1, 4):
        x, x64 = round_to(rows(rng, (b, g, d)), "bf16")
        kn.copy_(x)
        pos.fill_(step)
        graph.replay()
        want = expect_append(want, (x64, x64), range(b), [step] * b)
    torch.cuda.synchronize()
    check(cache, want)
