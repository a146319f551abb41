"""Operators of the 8-bit K/V cache: the quantising append, the read-back, single-token attention over the cache, and
single-token attention of a batch whose sequences share one long prefix.  Each case can be run in two forms: the plain one
(elementary torch operations in 32 bits) and, where ``own`` is true, the library's entry points.

The cache.  A row of one K/V head, x[0..d), is stored as d e4m3 codes and one exponent byte E:
    x[c] ~ code[c] * s,   s = the fp32 number whose exponent field is E and whose mantissa is 0 (2^(E-127), 0 for E = 0).
The append takes the smallest power of two s in [2^-126, 2^127] with max|x| <= 448 s over the row's finite values (E = 1 for
a row of zeros) and rounds x/s to e4m3 (nearest, ties to even; infinities saturate, NaN stays NaN).  Both steps are exact
but for that one rounding, so codes and exponents have one right answer.
    codes [b, m_max, g, d] float8_e4m3fn, exponents [b, g, m_max] uint8
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decode step's new rows of a long-context MQA batch: the smallest call, launch latency
        dict(name="append_step_b64_g1", op="append", b=64, g=1, d=128, m_max=1024, new=1, dtype="bf16"),
        # eight prompts of ragged length written behind what their caches already hold
        dict(name="append_prompts_b8_g8", op="append", b=8, g=8, d=128, m_max=8192, new=4096, dtype="bf16"),
        # one cached sequence handed back in fp32, head size 64
        dict(name="read_one_f32_d64", op="read", b=1, g=4, d=64, m_max=2048, rows=1237, dtype="f32"),
        # sixteen cached sequences unpacked for a batched pass over them
        dict(name="read_b16_g8", op="read", b=16, g=8, d=128, m_max=8192, rows=4096, dtype="bf16"),
        # a single user's chat turn
        dict(name="decode_b1_gqa8_m2k", op="decode", b=1, h=32, g=4, d=128, m_max=2048, lo=1900, hi=2048, window=0, dtype="bf16"),
        # the paper-shaped decoder: 128 sequences of up to 128 rows
        dict(name="decode_mqa_b128_m128", op="decode", b=128, h=8, g=1, d=128, m_max=128, lo=1, hi=128, window=0, dtype="bf16"),
        # long-context MQA serving batch
        dict(name="decode_mqa_b64_m8k", op="decode", b=64, h=32, g=1, d=128, m_max=8192, lo=1024, hi=8192, window=0, dtype="bf16"),
        # long-context GQA-8 serving batch: the largest cache
        dict(name="decode_gqa8_b32_m32k", op="decode", b=32, h=64, g=8, d=128, m_max=32768, lo=8192, hi=32768, window=0, dtype="bf16"),
        # fp32 queries at head size 64 with a local window, ragged lengths
        dict(name="decode_f32_d64_window", op="decode", b=12, h=16, g=8, d=64, m_max=3000, lo=1, hi=3000, window=1500, dtype="f32"),
        # a few requests behind one system prompt
        dict(name="shared_b12_gqa4_p2k", op="shared", b=12, h=32, g=8, d=128, m_p=2048, p_len=1999, m_s=256, lo=0, hi=256, dtype="bf16"),
        # a large MQA batch behind one long prompt, short answers so far
        dict(name="shared_b256_mqa_p8k", op="shared", b=256, h=8, g=1, d=128, m_p=8192, p_len=8192, m_s=128, lo=1, hi=128, dtype="bf16"),
        # a GQA-8 batch behind a long document, longer answers
        dict(name="shared_b128_gqa8_p16k", op="shared", b=128, h=64, g=8, d=128, m_p=16384, p_len=16001, m_s=1024, lo=1, hi=1024, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "decode", "shared", "shared"])
    while True:
        if op in ("append", "read"):
            c = dict(op=op, b=_log(rng, 1, 128), g=_log(rng, 1, 32), d=rng.choice([32, 64, 128, 128]), m_max=_log(rng, 64, 8192),
                     dtype=rng.choice(["bf16", "bf16", "f32"]))
            most = c["m_max"]
            if op == "append":
                c["new"] = 1 if rng.random() < 0.5 else _log(rng, 2, most)
            else:
                c["rows"] = _log(rng, 1, most)
            if c["b"] * c["m_max"] * c["g"] * c["d"] > 8 * 8192 * 8 * 128:
                continue
        elif op == "decode":
            d = rng.choice([32, 64, 128, 128, 128, 128])
            dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
            g, hq = _log(rng, 1, 32), rng.choice([1, 2, 4, 8, 12, 16, 32] + ([64] if dtype == "bf16" and d == 128 else []))
            m_max = _log(rng, 64, 32768)
            hi = rng.randint(max(1, m_max // 2), m_max)
            c = dict(op=op, b=_log(rng, 1, 256), h=g * hq, g=g, d=d, m_max=m_max, lo=rng.randint(0, hi), hi=hi,
                     window=rng.choice([0, 0, 0, _log(rng, 1, m_max)]), dtype=dtype)
            if c["b"] * m_max * g > 16 * 32768 or c["b"] * c["h"] * m_max > 32 * 64 * 16384:
                continue
        else:
            g, hq = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 8, 8, 12, 16, 32])
            m_p, m_s = _log(rng, 128, 16384), _log(rng, 1, 1024)
            c = dict(op=op, b=_log(rng, 2, 256), h=g * hq, g=g, d=128, m_p=m_p, p_len=rng.randint(1, m_p), m_s=m_s, lo=rng.randint(0, m_s), hi=m_s,
                     dtype="bf16")
            if c["b"] * c["h"] * m_p > 128 * 64 * 8192 or c["b"] * m_s * g > 128 * 1024 * 4:
                continue
        return c


def _lengths(case, lo, hi):
    """The case's lengths: part of the case, the same for every seed."""
    r = random.Random("%s %d %d %d" % (case["op"], case["b"], lo, hi))
    n = [r.randint(lo, hi) for _ in range(case["b"])]
    n[r.randrange(len(n))] = hi
    return n


def _new_rows(case):
    """New rows of each sequence (append), or rows read of each (read)."""
    if case["op"] == "append":
        return [1] * case["b"] if case["new"] == 1 else _lengths(case, max(1, case["new"] // 4), case["new"])
    return _lengths(case, max(1, case["rows"] // 4), case["rows"])


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    d, g, b = case["d"], case["g"], case["b"]
    row = d + 1  # a stored row: its codes and its exponent
    if case["op"] in ("append", "read"):
        rows = 2 * sum(_new_rows(case)) * g
        return {"bytes": rows * (d * e + row), "flops": rows * d * 2}
    if case["op"] == "decode":
        w = case["window"] or case["m_max"]
        rows = sum(min(n, w) for n in _lengths(case, case["lo"], case["hi"]))
        return {"bytes": 2 * rows * g * row + 2 * b * case["h"] * d * e, "flops": 4 * rows * case["h"] * d}
    own_rows = sum(_lengths(case, case["lo"], case["hi"]))
    return {"bytes": 2 * (own_rows + case["p_len"]) * g * row + 2 * b * case["h"] * d * e,
            "flops": 4 * (own_rows + b * case["p_len"]) * case["h"] * d}


# ------------------------------------------------------------------ the format, in plain torch


def _scale(exps):
    return (exps.to(torch.int32) << 23).view(torch.float32)


def _quantise(x):
    """(codes, exponents) of rows x[..., d]."""
    x = x.float()
    a = x.abs()
    top = torch.where(torch.isfinite(a), a, torch.zeros_like(a)).amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -126)).clamp(-126, 127)
    back = ((127 - e).int() << 23).view(torch.float32)  # 2^-e, a normal number: e <= 120 for finite rows
    return (x * back[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _values(codes, exps):
    """fp32 rows [b, m, g, d] of codes [b, m, g, d] and exponents [b, g, m]."""
    return codes.float() * _scale(exps).transpose(1, 2)[..., None]


# ------------------------------------------------------------------ inputs


def _rows(shape, gen):
    """Rows as a projection gives them: normal, their magnitude varying from row to row."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return x * torch.exp2(torch.randn(shape[:-1] + (1,), generator=gen, device="cuda"))


def _cache(b, m, g, d, gen):
    k, ke = _quantise(_rows((b, m, g, d), gen))
    v, ve = _quantise(_rows((b, m, g, d), gen))
    return [k, ke.transpose(1, 2).contiguous(), v, ve.transpose(1, 2).contiguous()]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cumulative(n):
    c = [0]
    for x in n:
        c.append(c[-1] + x)
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, op, b, g, d = _DTYPES[case["dtype"]], case["op"], case["b"], case["g"], case["d"]
    st = dict(case=case)
    if op in ("append", "read"):
        st["cache"] = _cache(b, case["m_max"], g, d, gen)
        n = _new_rows(case)
        cu = _cumulative(n)
        r = random.Random("start %d" % case["m_max"])
        start = [r.randint(0, case["m_max"] - x) for x in n]
        st["start"], st["total"] = _i32(start), cu[-1]
        st["cu"] = None if op == "append" and case["new"] == 1 else _i32(cu)
        # where the plain form finds each packed row: its sequence and its cache row
        st["seq"] = torch.tensor([s for s, x in enumerate(n) for _ in range(x)], device="cuda")
        st["row"] = torch.tensor([start[s] + i for s, x in enumerate(n) for i in range(x)], device="cuda")
        if op == "append":
            st["k_new"] = _rows((cu[-1], g, d), gen).to(dt)
            st["v_new"] = _rows((cu[-1], g, d), gen).to(dt)
    else:
        st["q"] = torch.randn((b, case["h"], d), generator=gen, device="cuda").to(dt)
        st["lens"] = _i32(_lengths(case, case["lo"], case["hi"]))
        st["scale"] = 1.0 / math.sqrt(d)
        if op == "decode":
            st["cache"] = _cache(b, case["m_max"], g, d, gen)
        else:
            st["prefix"] = _cache(1, case["m_p"], g, d, gen)
            st["p_len"] = _i32([case["p_len"]])
            st["cache"] = _cache(b, case["m_s"], g, d, gen)
    if own:  # the library's pre-marshalled call, as a serving loop keeps it
        st["plan"] = _plan(st)
    return st


def _plan(st):
    from grouped_query_attention_mqa_b200 import q8

    case = st["case"]
    cache = q8.Cache(*st["cache"])
    if case["op"] == "append":
        return q8.AppendPlan(cache, st["k_new"], st["v_new"], st["start"], cu_new=st["cu"])
    if case["op"] == "read":
        return q8.ReadPlan(cache, st["cu"], st["total"], start=st["start"], dtype=_DTYPES[case["dtype"]])
    if case["op"] == "decode":
        return q8.DecodePlan(st["q"], cache, st["lens"], st["scale"], window=case["window"])
    return q8.SharedPlan(st["q"], q8.Cache(*st["prefix"]), st["p_len"], cache, st["lens"], st["scale"])


# ------------------------------------------------------------------ one pass


def _attend(q, keys, values, valid, scale):
    """o [b, g, n, d] of q [b, g, n, d] over keys and values [b, m, g, d] (or [1, m, g, d]) where valid [b, m]; also the
    row maxima and sums, so that two sets of rows can be joined."""
    s = torch.matmul(q, keys.permute(0, 2, 3, 1)) * scale
    s = torch.where(valid[:, None, None, :], s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    o = torch.matmul(p, values.permute(0, 2, 1, 3))
    return o, top, p.sum(-1, keepdim=True)


def _mask(values, valid):
    """Rows that count for nothing hold zeros, whatever was left in them."""
    return torch.where(valid[:, :, None, None], values, torch.zeros_like(values))


def run(st):
    if own:
        return st["plan"].run()
    case, op = st["case"], st["case"]["op"]
    if op == "append":
        for new, codes, exps in ((st["k_new"], st["cache"][0], st["cache"][1]), (st["v_new"], st["cache"][2], st["cache"][3])):
            c, e = _quantise(new)
            codes.view(torch.uint8)[st["seq"], st["row"]] = c.view(torch.uint8)
            exps.transpose(1, 2)[st["seq"], st["row"]] = e
        return tuple(st["cache"])
    if op == "read":
        k, ke, v, ve = st["cache"]
        dt = _DTYPES[case["dtype"]]
        return tuple((c.view(torch.uint8)[st["seq"], st["row"]].view(torch.float8_e4m3fn).float()
                      * _scale(e.transpose(1, 2)[st["seq"], st["row"]])[..., None]).to(dt) for c, e in ((k, ke), (v, ve)))
    q, b, g, d = st["q"], case["b"], case["g"], case["d"]
    hq = case["h"] // g
    k, ke, v, ve = st["cache"]
    at = torch.arange(k.shape[1], device=q.device)
    lens = st["lens"][:, None]
    valid = at[None] < lens
    if op == "decode" and case["window"]:
        valid = valid & (at[None] >= lens - case["window"])
    qf = q.float().view(b, g, hq, d)
    o, top, total = _attend(qf, _mask(_values(k, ke), valid), _mask(_values(v, ve), valid), valid, st["scale"])
    if op == "shared":
        pk, pke, pv, pve = st["prefix"]
        keep = torch.arange(pk.shape[1], device=q.device)[None] < st["p_len"][:, None]
        # the whole batch's queries against the one prefix
        q1 = qf.permute(1, 0, 2, 3).reshape(1, g, b * hq, d)
        po, ptop, ptotal = _attend(q1, _mask(_values(pk, pke), keep), _mask(_values(pv, pve), keep), keep, st["scale"])
        po, ptop, ptotal = (x.view(g, b, hq, -1).permute(1, 0, 2, 3) for x in (po, ptop, ptotal))
        m = torch.maximum(top, ptop)
        m = torch.where(m > -math.inf, m, torch.zeros_like(m))
        o = o * torch.exp(top - m) + po * torch.exp(ptop - m)
        total = total * torch.exp(top - m) + ptotal * torch.exp(ptop - m)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.reshape(b, case["h"], d).to(q.dtype)


# ------------------------------------------------------------------ 64 bits, from the definition


def _two_to(e):
    """2^e in 64 bits, by its bits (a power function may be an ulp off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def exact(case, seed):
    st = prepare(dict(case), seed)
    op = case["op"]
    if op == "read":
        out = []
        for codes, exps in ((st["cache"][0], st["cache"][1]), (st["cache"][2], st["cache"][3])):
            power = _two_to(exps.long() - 127)  # [b, g, m]
            out.append(torch.stack([codes[s, r].double() * power[s, :, r, None] for s, r in zip(st["seq"].tolist(), st["row"].tolist())])
                       if st["total"] <= 4096 else codes.double()[st["seq"], st["row"]] * power.permute(0, 2, 1)[st["seq"], st["row"]].unsqueeze(-1))
        return tuple(out)
    if op == "append":
        # codes: the nearest of the 256 values of e4m3, found among them; exponents: by trying powers of two
        out = []
        table = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8).view(torch.float8_e4m3fn).double()
        table = table[torch.isfinite(table)].unique()
        for new, codes, exps in ((st["k_new"], st["cache"][0], st["cache"][1]), (st["v_new"], st["cache"][2], st["cache"][3])):
            x = new.double()
            e = torch.full(x.shape[:-1], -126, device="cuda")
            top = x.abs().amax(-1)
            for p in range(-126, 127):
                e += (top > 448.0 * 2.0 ** p).long()
            y = x * _two_to(-e)[..., None]
            hi = torch.searchsorted(table, y.contiguous()).clamp(1, table.numel() - 1)
            lo = hi - 1
            up, down = table[hi] - y, y - table[lo]
            # a tie goes to the value whose last mantissa bit is 0: of two neighbours that is the one that is a multiple of twice their distance
            gap = table[hi] - table[lo]
            even_hi = torch.remainder(table[hi], 2 * gap) == 0
            near = torch.where((up < down) | ((up == down) & even_hi), table[hi], table[lo])
            full = codes.double()
            full[st["seq"], st["row"]] = near
            out += [full, None]
        return tuple(out)
    b, h, g, d, q = case["b"], case["h"], case["g"], case["d"], st["q"].double()
    hq = h // g

    def rows(cache, s, a, n):
        """Keys and values [g, n - a, d] of rows a..n of sequence s."""
        got = []
        for codes, exps in ((cache[0], cache[1]), (cache[2], cache[3])):
            got.append(codes[s, a:n].double().permute(1, 0, 2) * _two_to(exps[s, :, a:n].long() - 127)[..., None])
        return got

    out = torch.zeros((b, h, d), dtype=torch.float64, device="cuda")
    prefix = rows(st["prefix"], 0, 0, case["p_len"]) if op == "shared" else None
    for s, n in enumerate(st["lens"].tolist()):
        a = max(0, n - case["window"]) if op == "decode" and case["window"] else 0
        k, v = rows(st["cache"], s, a, n)
        qs = q[s].view(g, hq, d)
        logits, parts = [qs @ k.transpose(1, 2)], [v]
        if prefix is not None:
            logits, parts = [qs @ prefix[0].transpose(1, 2)] + logits, [prefix[1]] + parts
        z = torch.cat(logits, -1) * st["scale"]
        if z.shape[-1] == 0:
            continue
        w = torch.softmax(z, -1)
        at = 0
        for part in parts:
            out[s] += (w[..., at:at + part.shape[1]] @ part).reshape(h, d)
            at += part.shape[1]
    return out
