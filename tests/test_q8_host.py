"""The 8-bit cache without a GPU: its format's oracle against torch's e4m3 and
its own definition, the header's symbols, and the refusals of every entry
point (which all come before a launch)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from grouped_query_attention_mqa_b200 import binding, q8
from grouped_query_attention_mqa_b200.build import build
from oracle import q8_oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, OK = binding.MQA_ERR_INVALID_ARG, binding.MQA_ERR_UNSUPPORTED, binding.MQA_OK


@pytest.fixture(scope="module")
def lib():
    build()
    return q8.lib()


def test_header_symbols_are_exported_and_bound(lib):
    text = open(os.path.join(ROOT, "include", "mqa_q8.h")).read()
    names = set(re.findall(r"MQA_API\s+[\w\s\*]+?\b(mqa_\w+)\s*\(", text))
    assert names == set(q8.SIGNATURES)
    for n in names:
        assert hasattr(lib, n)


# ------------------------------------------------------------------ format


def test_table_is_torchs_e4m3():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(q8_oracle.TABLE, t, equal_nan=True)


def test_quantise_matches_torchs_rounding():
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((500, 64)) * np.exp2(rng.integers(-30, 30, (500, 1)))).bfloat16()
    codes, exps = q8_oracle.quantise(x.double().numpy())
    y = x.double() / torch.from_numpy(q8_oracle.scale_of(exps))[:, None]
    assert np.array_equal(codes, y.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_scale_is_the_smallest_that_holds_the_row():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2000, 16)) * np.exp2(rng.integers(-120, 100, (2000, 1)))
    _, exps = q8_oracle.quantise(x)
    s = q8_oracle.scale_of(exps)
    top = np.abs(x).max(1)
    assert (top <= 448 * s).all() and ((top > 448 * s / 2) | (exps == 1)).all()   # E = 1 is the smallest there is


def test_quantising_what_was_read_back_changes_nothing():
    """448 s' >= max|code s| holds for s' = s, and for s / 2 exactly when the
    row's largest code is at most 224: rounding may have taken it there from
    above 224, never below, and then the codes double exactly; values stay."""
    rng = np.random.default_rng(3)
    codes, exps = q8_oracle.quantise(rng.standard_normal((4000, 32)))
    val = q8_oracle.TABLE[codes] * q8_oracle.scale_of(exps)[:, None]
    codes2, exps2 = q8_oracle.quantise(val)
    assert np.array_equal(q8_oracle.TABLE[codes2] * q8_oracle.scale_of(exps2)[:, None], val)


def test_special_values():
    x = np.array([[0.0, -0.0, 0.0, 0.0], [np.nan, 1.0, -2.0, 0.5], [np.inf, 1.0, -np.inf, 0.25], [np.inf, np.nan, 0, 0],
                  [448.0, 1, 2, 3], [449.0, 1, 2, 3], [2.0 ** -140, 0, 0, 0]])
    codes, exps = q8_oracle.quantise(x)
    assert exps.tolist() == [1, 120, 119, 1, 127, 128, 1]
    val = q8_oracle.TABLE[codes] * q8_oracle.scale_of(exps)[:, None]
    assert np.isnan(val[1, 0]) and val[1, 1] == 1.0
    assert val[2].tolist() == [448 * 2.0 ** -8, 1.0, -448 * 2.0 ** -8, 0.25]
    assert codes[0].tolist() == [0, 0x80, 0, 0]


# ------------------------------------------------------------------ refusals

FAKE = ctypes.c_void_p(0x10000)   # aligned, never dereferenced: every call below fails its checks first
ODD = ctypes.c_void_p(0x10008)


def _append(lib, **kw):
    a = dict(k=FAKE, ke=FAKE, v=FAKE, ve=FAKE, kn=FAKE, vn=FAKE, pos=FAKE, cu=FAKE, b=2, total=5, m_max=16, g=1, d_k=128,
             d_v=128, dtype=binding.MQA_BF16)
    a.update(kw)
    return lib.mqa_q8_append(a["k"], a["ke"], a["v"], a["ve"], a["kn"], a["vn"], a["pos"], a["cu"], a["b"], a["total"],
                             a["m_max"], a["g"], a["d_k"], a["d_v"], a["dtype"], None, None)


def _read(lib, **kw):
    a = dict(k=FAKE, ke=FAKE, v=FAKE, ve=FAKE, ko=FAKE, vo=FAKE, start=None, cu=FAKE, b=2, total=5, m_max=16, g=1, d_k=128,
             d_v=128, dtype=binding.MQA_BF16)
    a.update(kw)
    return lib.mqa_q8_read(a["ko"], a["vo"], a["k"], a["ke"], a["v"], a["ve"], a["start"], a["cu"], a["b"], a["total"],
                           a["m_max"], a["g"], a["d_k"], a["d_v"], a["dtype"], None, None)


@pytest.mark.parametrize("call", [_append, _read])
def test_rows_refusals(lib, call):
    for name in ("k", "v", "cu"):
        assert call(lib, **{name: ODD}) == INV
    for name in ("k", "ke", "v", "ve"):
        assert call(lib, **{name: None}) == INV
    assert call(lib, b=-1) == INV and call(lib, total=-1) == INV and call(lib, m_max=0) == INV and call(lib, g=0) == INV
    assert call(lib, dtype=2) == INV
    assert call(lib, d_k=96) == UNS and call(lib, d_v=8) == UNS and call(lib, d_k=512) == UNS
    assert call(lib, b=0) == OK and call(lib, total=0) == OK


def test_append_and_read_refusals_of_their_own(lib):
    assert _append(lib, cu=None) == INV                   # one row per sequence, yet total != b
    assert _append(lib, pos=None) == INV and _append(lib, kn=ODD) == INV and _append(lib, vn=None) == INV
    assert _read(lib, cu=None) == INV and _read(lib, start=ODD) == INV and _read(lib, ko=None) == INV
    half = ctypes.c_void_p(0x10010)                       # packed rows: 32-byte aligned
    assert _append(lib, kn=half) == INV and _read(lib, vo=half) == INV


def _decode(lib, **kw):
    a = dict(o=FAKE, q=FAKE, k=FAKE, ke=FAKE, v=FAKE, ve=FAKE, lens=FAKE, b=2, h=8, g=1, m_max=16, d_k=128, d_v=128,
             scale=1.0, dtype=binding.MQA_BF16, ws=FAKE, ws_bytes=1 << 40, opts=None)
    a.update(kw)
    return lib.mqa_q8_decode(a["o"], a["q"], a["k"], a["ke"], a["v"], a["ve"], a["lens"], a["b"], a["h"], a["g"],
                             a["m_max"], a["d_k"], a["d_v"], a["scale"], a["dtype"], a["ws"], a["ws_bytes"], None,
                             ctypes.byref(binding.DecodeOptions(*a["opts"])) if a["opts"] else None, None)


def test_decode_refusals(lib):
    for name in ("o", "q", "k", "ke", "v", "ve", "lens", "ws"):
        assert _decode(lib, **{name: None}) == INV
    for name in ("o", "q", "k", "v", "lens", "ws"):
        assert _decode(lib, **{name: ODD}) == INV
    assert _decode(lib, ws=ctypes.c_void_p(0x10010)) == INV           # workspace not 256-aligned
    need = lib.mqa_q8_decode_workspace_size(2, 8, 1, 128)
    assert _decode(lib, ws_bytes=need - 1) == INV
    assert _decode(lib, g=3) == INV and _decode(lib, m_max=0) == INV and _decode(lib, dtype=5) == INV
    assert _decode(lib, scale=float("nan")) == INV and _decode(lib, b=-1) == INV
    assert _decode(lib, opts=(9, 0, 0)) == INV and _decode(lib, opts=(0, -1, 0)) == INV
    assert _decode(lib, opts=(0, binding.MQA_MAX_CTAS + 1, 0)) == INV and _decode(lib, opts=(0, 0, -1)) == INV
    assert _decode(lib, d_k=96) == UNS and _decode(lib, d_v=256) == UNS
    assert _decode(lib, dtype=binding.MQA_F32, opts=(2, 0, 0)) == UNS   # tensor cores: bf16
    assert _decode(lib, h=128, opts=(1, 0, 0)) == UNS                   # CUDA cores: h/g * d <= 4096
    assert _decode(lib, h=64, dtype=binding.MQA_F32) == UNS
    assert _decode(lib, b=0) == OK
    size = lib.mqa_q8_decode_workspace_size
    assert size(2, 8, 3, 128) == 0 and size(-1, 8, 1, 128) == 0 and size(0, 8, 1, 128) > 0


def _shared(lib, **kw):
    a = dict(o=FAKE, q=FAKE, pk=FAKE, pke=FAKE, pv=FAKE, pve=FAKE, pl=FAKE, k=FAKE, ke=FAKE, v=FAKE, ve=FAKE, lens=FAKE,
             b=2, h=8, g=1, m_p=64, m_s=16, d=128, scale=1.0, dtype=binding.MQA_BF16, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return lib.mqa_q8_decode_shared(a["o"], a["q"], a["pk"], a["pke"], a["pv"], a["pve"], a["pl"], a["k"], a["ke"],
                                    a["v"], a["ve"], a["lens"], a["b"], a["h"], a["g"], a["m_p"], a["m_s"], a["d"],
                                    a["scale"], a["dtype"], a["ws"], a["ws_bytes"], None, None)


def test_shared_refusals(lib):
    for name in ("o", "q", "pk", "pke", "pv", "pve", "pl", "k", "ke", "v", "ve", "lens", "ws"):
        assert _shared(lib, **{name: None}) == INV
    for name in ("o", "q", "pk", "pv", "pl", "k", "v", "lens", "ws"):
        assert _shared(lib, **{name: ODD}) == INV
    size = lib.mqa_q8_decode_shared_workspace_size
    assert _shared(lib, ws_bytes=size(2, 8, 1, 64, 128) - 1) == INV
    assert _shared(lib, g=3) == INV and _shared(lib, m_p=0) == INV and _shared(lib, m_s=0) == INV and _shared(lib, b=-1) == INV
    assert _shared(lib, scale=float("inf")) == INV and _shared(lib, dtype=9) == INV
    assert _shared(lib, dtype=binding.MQA_F32) == UNS and _shared(lib, d=64) == UNS and _shared(lib, h=65) == UNS
    assert _shared(lib, b=0) == OK
    assert size(2, 8, 3, 64, 128) == 0 and size(2, 65, 1, 64, 128) == 0 and size(2, 8, 1, 0, 128) == 0
    assert size(0, 8, 1, 64, 128) > 0


def test_binding_refuses_other_layouts():
    with pytest.raises(ValueError, match="contiguous CUDA"):
        q8.AppendPlan(q8.new_cache(1, 4, 1, 16, device="cpu"), None, None, None)
