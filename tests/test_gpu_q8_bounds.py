"""The precision that include/mqa_q8.h states for the two tensor-core paths,
with the bounds taken row by row (``q8_util.attention`` allows every row the
largest).

Of an output of sum_t w_t v_t (w_t the softmax weights, s_t the value scale that
the path takes row t at, U = max_t w_t s_t):
 - behind a shared prefix s_t is the largest value scale among row t's 64.  P_t,
   proportional to w_t s_t, is one fp16 number of which the largest is 2^2 or
   more: half a step is 2^-11 of it, or 2^-25 among the subnormal ones, 2^-27 of
   the largest; and a rounding to nearest is never off by more than the number:
       sum_t min(w_t, max(2^-11 w_t, 2^-27 U / s_t)) |v_t|.
   Rows 2^-16 and more below s_t lose what is below 2^-25 of it: keys move the
   logits by |scale| sum_c |q_c| 2^-25 s_t' (s_t' the keys' largest), values the
   output by 2^-25 s_t.  A query's elements are fp16 of which the largest has
   224 units: off by 2^-25 of a unit at most.
 - the decode's s_t is the row's own.  P_t is rounded to fp16, 2^-11 of itself,
   then to two e4m3 terms: the first is off by at most 2^-4 of its power of two,
   the second by half a step of that difference, 2^-5 2^-4 = 2^-9 of that power
   of two at most.  Below the second term's smallest step (2^-9 / 16, the largest
   P being 2^4 or more: 2^-17 of U) it is off by less than a step, whichever way
   the dither says.  Signs of v are independent of all that, so such steps add
   up as independent ones: beyond 6 standard deviations with a probability of
   2 exp(-18) (Hoeffding) each:
       (2^-9 + 2^-11) sum_t w_t |v_t| + 6 sqrt(sum_t (2^-17 U / s_t v_t)^2).
   A query's elements: 2^-10 units of which the largest has at least 224.
 - both: logits, sums and the output's rounding as in ``q8_util``."""
import numpy as np
import pytest
import torch

from grouped_query_attention_mqa_b200 import q8
from grouped_query_attention_mqa_b200.build import build
from oracle import q8_oracle
from q8_util import U32, assert_within, dev_cache, host_cache, round_to, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    q8.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def quantised(*arrays):
    """Host cache parts (codes, exponents, ...) of arrays [1, n, g, d]."""
    out = []
    for x in arrays:
        c, e = q8_oracle.quantise(x)
        out += [c, np.ascontiguousarray(np.moveaxis(e, 2, 1))]
    return out


def tile_largest(s):
    """Each row's largest scale among the 64 rows from a multiple of 64 on."""
    n = len(s)
    s = np.concatenate([s, np.zeros(-n % 64)]).reshape(-1, 64).max(1)
    return np.repeat(s, 64)[:n]


def within(o, q64, arrays, n, g, scale, shared):
    """o [b, h, 128] of queries q64 [b, h, 128] that all attend to rows 0..n-1 of
    the one sequence in ``arrays``."""
    k, ke, v, ve = (x[:, :n] if x.ndim == 4 else x[:, :, :n] for x in arrays)
    K, V = q8_oracle.values(k, ke)[0], q8_oracle.values(v, ve)[0]
    ref, tol = np.zeros(q64.shape), np.zeros(q64.shape)
    hq = q64.shape[1] // g
    for j in range(g):
        sk, sv = q8_oracle.scale_of(ke[0, j]), q8_oracle.scale_of(ve[0, j])
        valued = ve[0, j] > 1
        tk, tv = (tile_largest(sk), tile_largest(sv)) if shared else (sk, sv)
        aV = np.abs(V[:, j])
        for i in range(q64.shape[0]):
            qs = q64[i, j * hq:(j + 1) * hq]
            z = qs @ K[:, j].T * scale
            w = np.exp(z - z.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            r, A = w @ V[:, j], w @ aV
            L = (np.abs(qs) @ np.abs(K[:, j]).T).max() * abs(scale)
            M = np.abs(qs).max(1, keepdims=True) * np.abs(K[:, j]).sum(1).max() * abs(scale)
            t = A * (2 * (128 + 4) * U32 * L + (n + 16) * U32) + np.abs(r) * 2.0 ** -8
            U = (w * tv)[:, valued].max(1, keepdims=True) if valued.any() else 0
            with np.errstate(divide="ignore", invalid="ignore"):
                step = np.where(valued, U / tv, 0)
            if shared:
                t = t + np.minimum(w, np.maximum(2.0 ** -11 * w, 2.0 ** -27 * step)) @ aV
                t = t + A * 2 * 2.0 ** -25 / 224 * M
                far = sk < 2.0 ** -15 * tk
                t = t + A * 2 * abs(scale) * np.abs(qs).sum(1, keepdims=True) * 2.0 ** -25 * (tk * far).max()
                t = t + 2.0 ** -25 * (w @ (tv * (sv < 2.0 ** -15 * tv)))[:, None]
            else:
                t = t + (2.0 ** -9 + 2.0 ** -11) * A + 6 * 2.0 ** -17 * np.sqrt(step ** 2 @ aV ** 2)
                t = t + A * 2 * 2.0 ** -10 / 224 * M
            ref[i, j * hq:(j + 1) * hq], tol[i, j * hq:(j + 1) * hq] = r, t
    assert_within(o, ref, tol, "shared" if shared else "decode")


def behind_prefix(q, arrays, n, g, scale):
    """The rows as a prefix behind which every sequence has no rows of its own: a
    few sequences and, so that a CTA takes many tiles, very many with the same
    queries."""
    q, q64 = round_to(q, "bf16")
    b, h = q.shape[:2]
    prefix = dev_cache(arrays)
    for copies in (1, 1 + (1 << 16) // (b * h)):
        o = q8.decode_shared(q.cuda().repeat(copies, 1, 1), prefix, i32([n]), q8.new_cache(b * copies, 1, g, 128),
                             i32([0] * (b * copies)), scale).view(copies, b, h, 128)
        for c in range(0, copies, 1 + copies // 7):
            within(o[c], q64, arrays, n, g, scale, True)


def over_own_rows(q, arrays, n, g, scale):
    """The rows as a sequence's own cache, its tiles split between CTAs and not."""
    q, q64 = round_to(q, "bf16")
    cache = dev_cache(arrays)
    for ctas in (0, 1):
        for s in range(min(q.shape[0], 2)):
            o = q8.decode(q[s:s + 1].cuda(), cache, i32([n]), scale, path="tcgen05", num_ctas=ctas)
            within(o, q64[s:s + 1], arrays, n, g, scale, False)


# ------------------------------------------------------------------ scales far apart within a tile


def sparse_tiles(rng, n, apart):
    """Rows [1, n, 1, 128] with a scale of 2^-apart, but for one row in 64 of scale 1."""
    x = rng.choice([-1.0, 1.0], (1, n, 1, 128)) * rng.uniform(64, 447, (1, n, 1, 128)) * 2.0 ** -apart
    x[..., 0] = 448 * 2.0 ** -apart     # the row's scale
    x[0, ::64] *= 2.0 ** apart
    return x


@pytest.mark.parametrize("apart", [15, 16, 24, 25, 28, 32, 36])
def test_prefix_values_far_below_their_tiles(apart):
    """Each query attends to one row."""
    rng = np.random.default_rng(apart)
    n, b, h = 150, 20, 8
    K = np.sign(rng.standard_normal((1, n, 1, 128)))
    V = sparse_tiles(rng, n, apart)
    at = rng.integers(0, n, (b, h))
    q, q64 = round_to(K[0, at, 0], "bf16")
    prefix = quantised(K, V)
    o = q8.decode_shared(q.cuda(), dev_cache(prefix), i32([n]), q8.new_cache(b, 1, 1, 128), i32([0] * b), 0.5)
    within(o, q64, prefix, n, 1, 0.5, True)


@pytest.mark.parametrize("apart", [15, 16, 23, 24, 25, 26])
def test_prefix_keys_far_below_their_tiles(apart):
    """The large keys are orthogonal to every query, so that the small ones decide."""
    rng = np.random.default_rng(100 + apart)
    n, b, h = 150, 20, 8
    K = sparse_tiles(rng, n, apart)
    K[0, ::64] = 0
    K[..., 0] = 0
    K[0, ::64, :, 0] = 448.0
    K[..., 1] = 448 * 2.0 ** -apart * (K[..., 0] == 0)
    q = rng.standard_normal((b, h, 128)) * 2.0 ** (apart - 8)
    q[..., 0] = 0
    q, q64 = round_to(q, "bf16")
    prefix = quantised(K, rng.standard_normal((1, n, 1, 128)))
    o = q8.decode_shared(q.cuda(), dev_cache(prefix), i32([n]), q8.new_cache(b, 1, 1, 128), i32([0] * b), 0.2)
    within(o, q64, prefix, n, 1, 0.2, True)


# ------------------------------------------------------------------ rows of zeros first


def values_after_zeros(rng, zeros, e, n, g):
    """A cache of n rows, the first of them without a value, the others of scale 2^(e-127)."""
    arrays = host_cache(rng, 1, n, g, 128, spread=0.3)
    arrays[2] = q8_oracle.quantise(rng.choice([-1.0, 1.0], (1, n, g, 128)) * rng.uniform(8, 15, (1, n, g, 128)))[0]
    if e == 250:
        arrays[2] -= 5 << 3             # codes of 128 to 448, 2^-5 of them: below 2^127
    arrays[2][:, :zeros], arrays[3][...] = 0, e
    arrays[3][:, :, :zeros] = 1         # as the append leaves zeros
    return arrays


def heavy_zeros(rng, gap, n, heavy):
    """A cache of n rows and queries; the first rows have no value and outweigh the others by 2^gap."""
    K = 0.05 * rng.standard_normal((1, n, 1, 128))
    K[0, :heavy, 0, 0] += gap * np.log(2)
    V = rng.standard_normal((1, n, 1, 128))
    V[0, :heavy] = 0
    q = 0.05 * rng.standard_normal((3, 8, 128))
    q[..., 0] = 1
    return quantised(K, V), q


@pytest.mark.parametrize("e", [40, 60, 87, 107, 127, 200, 250])
@pytest.mark.parametrize("zeros", [64, 130])
def test_prefix_values_after_tiles_of_zeros(zeros, e):
    """Whole tiles without a value, then values of one scale, whatever it is."""
    rng = np.random.default_rng(zeros + e)
    arrays = values_after_zeros(rng, zeros, e, 400, 2)
    behind_prefix(rng.standard_normal((5, 16, 128)), arrays, 400, 2, 0.09)


@pytest.mark.parametrize("gap", [20, 40])
def test_prefix_values_behind_heavy_tiles_of_zeros(gap):
    rng = np.random.default_rng(gap)
    arrays, q = heavy_zeros(rng, gap, 300, 128)
    behind_prefix(q, arrays, 300, 1, 1.0)


@pytest.mark.parametrize("e", [5, 20, 40, 60, 87, 127, 200, 250])
@pytest.mark.parametrize("h", [16, 128])       # all heads in a thread, or half of them
@pytest.mark.parametrize("zeros", [128, 260])
def test_own_values_after_tiles_of_zeros(zeros, h, e):
    rng = np.random.default_rng(zeros + e + h)
    arrays = values_after_zeros(rng, zeros, e, 700, 2)
    over_own_rows(rng.standard_normal((2, h, 128)), arrays, 700, 2, 0.09)


@pytest.mark.parametrize("gap", [20, 40, 80])
def test_own_values_behind_heavy_tiles_of_zeros(gap):
    rng = np.random.default_rng(gap)
    arrays, q = heavy_zeros(rng, gap, 600, 256)
    over_own_rows(q, arrays, 600, 1, 1.0)


# ------------------------------------------------------------------ many rows, sharp softmaxes, scales of every size


@pytest.mark.parametrize("n,g,h,scale,spread", [
    (1500, 2, 16, 0.09, 1.0), (1500, 1, 32, 0.09, 4.0), (6000, 1, 24, 0.3, 3.0), (2500, 1, 64, 1.0, 1.0),
    (3000, 2, 8, 0.0, 6.0), (700, 1, 8, 0.2, 0.2)])
def test_random_rows(n, g, h, scale, spread):
    rng = np.random.default_rng(n + h)
    arrays, q = host_cache(rng, 1, n, g, 128, spread=spread), rng.standard_normal((6, h, 128))
    behind_prefix(q, arrays, n, g, scale)
    over_own_rows(q, arrays, n, g, scale)


@pytest.mark.parametrize("gap", [4, 12, 20])
def test_some_rows_dominate(gap):
    """One row in 97 outweighs the others by about 2^gap, its values as large as
    theirs or 2^-7 of them."""
    rng = np.random.default_rng(30 + gap)
    n, h = 3000, 32
    K = 0.3 * rng.standard_normal((1, n, 1, 128))
    K[0, ::97, 0, 0] += gap * np.log(2)
    V = rows(rng, (1, n, 1, 128))
    q = 0.3 * rng.standard_normal((4, h, 128))
    q[..., 0] = 1
    for small in (False, True):
        if small:
            V[0, ::97] *= 2.0 ** -7
        behind_prefix(q, quantised(K, V), n, 1, 1.0)
        over_own_rows(q, quantised(K, V), n, 1, 1.0)


# ------------------------------------------------------------------ the same bits again


@pytest.mark.parametrize("op", ["decode", "shared"])
def test_a_call_repeats_itself(op):
    rng = np.random.default_rng(40)
    n, b, g, h = 2000, 12, 2, 32
    prefix, cache = (dev_cache(host_cache(rng, x, y, g, 128)) for x, y in ((1, 1000), (b, n)))
    lens = i32(rng.integers(1, n + 1, b).tolist())
    q = round_to(rng.standard_normal((b, h, 128)), "bf16")[0].cuda()
    plan = q8.DecodePlan(q, cache, lens, 0.1) if op == "decode" else q8.SharedPlan(q, prefix, i32([999]), cache, lens, 0.1)
    first = plan.run().clone()
    for _ in range(50):
        plan.out.fill_(float("nan"))
        assert torch.equal(plan.run(), first)


def test_the_largest_append():
    """As many packed rows as an int counts, all but one of no sequence."""
    total = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        pytest.skip("needs 70 GB free")
    k = torch.empty((total, 1, 16), dtype=torch.bfloat16, device="cuda")
    k[total - 1] = torch.arange(16, device="cuda") - 7.5
    cache = q8.new_cache(1, 4, 1, 16)
    q8.append(cache, k, k, i32([2]), cu_new=i32([total - 1, total]))
    x, _ = q8.read(cache, i32([0, 4]), 4, dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(x[2, 0].cpu(), torch.arange(16) - 7.5) and not x[[0, 1, 3]].any()
