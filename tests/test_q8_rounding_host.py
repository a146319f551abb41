"""What the 8-bit tensor-core paths keep of a weight and of a query, replayed on
the CPU number by number: the bounds that include/mqa_q8.h states hold, and
nothing smaller does."""
import numpy as np
import torch

from oracle import q8_oracle


def e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).to(x.dtype)


def test_weights_in_one_fp16_number():
    """The prefix's: half a step of 11 bits, 2^-11 of a power of two."""
    p = torch.cat([2.0 ** -14 * (1 + torch.rand(200_000, dtype=torch.float64)) * 2.0 ** torch.randint(0, 28, (200_000,)),
                   torch.tensor([1 + 2.0 ** -11], dtype=torch.float64)])
    off = ((p.half().double() - p).abs() / p).max()
    assert 2.0 ** -12 < off <= 2.0 ** -11


def test_weights_in_two_e4m3_terms():
    """The decode's: rounded to fp16, then two e4m3 terms of which the second is 16
    times as large and dithered by up to 2^-10 (its smallest step is 2^-9)."""
    gen = torch.Generator().manual_seed(1)
    p = 2.0 ** torch.randint(-10, 9, (1_000_000,), generator=gen) * (1 + torch.rand(1_000_000, dtype=torch.float64, generator=gen))
    p = p[p <= 448].float()
    h = p.half()
    first = e4m3(h.float())
    rest = h - first.half()
    assert (rest.double() == h.double() - first.double()).all()    # fp16 holds the difference
    worst = 0
    for dither in (-127.5 / 131072, 0.0, 127.5 / 131072):
        got = first.double() + e4m3((16 * rest.float() + dither).half().float()).double() / 16
        off = (got - p.double()).abs()
        assert (off < (2.0 ** -9 + 2.0 ** -11) * p.double() + 2.0 ** -13).all()
        worst = max(worst, (off / p)[p >= 16].max())
    assert 2.0 ** -9 < worst <= 2.0 ** -9 + 2.0 ** -11 + 2.0 ** -13 / 16


def test_queries_in_two_e4m3_terms():
    """Every bf16 number up to 448, the largest of its row in (224, 448]: off by at
    most 2^-10, exact from 2^-2 on."""
    x = torch.arange(0, 0x43E1, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    assert x.max() == 448
    first = e4m3(x)
    off = (first + e4m3(x - first) - x).abs()
    assert off.max() <= 2.0 ** -10 and off[x >= 0.25].max() == 0


def test_a_row_quantised_again_may_get_other_codes_of_the_same_values():
    """228 is nearest to 224 = 448 / 2: read back, the row fits the next smaller scale."""
    codes, exps = q8_oracle.quantise(np.array([[228.0, 1.0, -3.5, 0.0]]))
    val = q8_oracle.TABLE[codes] * q8_oracle.scale_of(exps)[:, None]
    codes2, exps2 = q8_oracle.quantise(val)
    assert exps2 == exps - 1 and val[0, 0] == 224
    assert np.array_equal(q8_oracle.TABLE[codes2], 2 * q8_oracle.TABLE[codes])
