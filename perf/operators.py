"""The operators that are measured, as cases: a 4-bit KV cache and attention over a window.

* ``kv_append_q4`` / ``kv_read_q4``: new fp32 K/V rows of a ragged batch are quantised into a cache
  of 4-bit e2m1 codes with one e4m3 scale per 16 dims, and rows of such a cache are read back as
  the values they stand for.
* ``attn_decode_q4``: grouped-query decode attention over that cache, dense or with a sliding
  window and a few first positions (sinks) that stay visible.
* ``attn_decode_f16_window``: the same visibility rule over the f16 cache.

``run`` computes them in plain torch operations, or calls the library where ``own`` is true.
"""

import math
import random

import torch

own = False

HEADS = ((4, 1), (32, 8), (48, 4), (16, 16), (24, 8), (8, 2), (20, 4))


# ------------------------------------------------------------------------------------ cases

def _append(name, n_seq, new_min, new_max, hk, d, cap, k_exp=0, v_exp=0):
    return {"name": name, "op": "append", "n_seq": n_seq, "new_min": new_min, "new_max": new_max,
            "n_kv_heads": hk, "head_dim": d, "cap": cap, "k_exp": k_exp, "v_exp": v_exp}


def _read(name, n_seq, new_min, new_max, hk, d, cap, half):
    return {"name": name, "op": "read", "n_seq": n_seq, "new_min": new_min, "new_max": new_max,
            "n_kv_heads": hk, "head_dim": d, "cap": cap, "k_exp": 0, "v_exp": -2, "half": half}


def _decode(name, op, n_seq, rows, h, hk, d, cap, len_min, len_max, window, n_sink):
    return {"name": name, "op": op, "n_seq": n_seq, "rows": rows, "n_heads": h, "n_kv_heads": hk,
            "head_dim": d, "cap": cap, "len_min": len_min, "len_max": len_max, "window": window,
            "n_sink": n_sink}


def listed():
    return [
        # one user's decode step: the new token's K/V rows go into the cache
        _append("append one token", 1, 1, 1, 8, 128, 4096),
        # a batch's decode step, some sequences idle in it
        _append("append batch step", 64, 0, 1, 8, 128, 1024, k_exp=1, v_exp=-3),
        # prompts of uneven length entering the cache at once
        _append("append prompts", 9, 700, 4100, 8, 128, 4608),
        # a short prefix copied out as the f16 rows that a dense prefill reads
        _read("read prefix f16", 1, 333, 333, 4, 256, 1024, True),
        # whole sequences read back in fp32
        _read("read sequences fp32", 6, 1, 8192, 8, 128, 8192, False),
        # one short row: latency
        _decode("q4 one short row", "q4", 1, 1, 4, 1, 64, 256, 256, 256, 0, 0),
        # one row of a wide head over a long context
        _decode("q4 wide head", "q4", 1, 1, 48, 4, 256, 8192, 8191, 8191, 0, 0),
        # a serving batch of mixed lengths, up to 32768 positions
        _decode("q4 long batch", "q4", 16, 1, 32, 8, 128, 32768, 1024, 32768, 0, 0),
        # rows of one sequence (drafted tokens, a small prefill chunk) through window and sinks
        _decode("q4 window rows", "q4", 2, 16, 32, 8, 64, 8192, 5000, 8100, 2048, 4),
        # one row of a long context, seen through a window
        _decode("f16 window one row", "f16w", 1, 1, 32, 8, 64, 16384, 16001, 16001, 1024, 4),
        # a serving batch of mixed lengths, shorter and longer than the window
        _decode("f16 window batch", "f16w", 64, 1, 32, 8, 128, 8192, 0, 8192, 4096, 4),
        # a chunk of a prompt: causal rows of one sequence
        _decode("f16 window chunk", "f16w", 1, 512, 32, 8, 128, 8192, 6500, 6500, 2048, 16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges: sizes spread over their logarithm, none costlier than the
    largest listed case (cache elements, new rows and score counts are capped by theirs)."""
    op = rng.choice(("append", "read", "q4", "q4", "f16w", "f16w"))
    d = rng.choice((64, 128, 128, 256))
    if op in ("append", "read"):
        hk = rng.choice((1, 2, 4, 8, 16))
        n_seq = _log(rng, 1, 64)
        # at most the listed prompts' 21600 new rows of 8 heads of 128
        top = max(1, min(8192, 21600 * 1024 // (n_seq * hk * d)))
        hi = _log(rng, 1, top)
        lo = rng.randint(0, hi)
        cap = -(-(hi + rng.randint(0, 400)) // 16) * 16
        if op == "append":
            return {k: v for k, v in _append("", n_seq, lo, hi, hk, d, cap, rng.randint(-6, 6),
                                             rng.randint(-6, 6)).items() if k != "name"}
        return {k: v for k, v in _read("", n_seq, lo, hi, hk, d, cap,
                                       rng.random() < 0.5).items() if k != "name"}
    h, hk = rng.choice(HEADS)
    n_seq = _log(rng, 1, 64)
    rows = 1 if rng.random() < 0.6 else _log(rng, 2, 512)
    if rows > 1:
        n_seq = max(1, min(n_seq, 4, 512 // rows))
    # at most 2^28 cache elements a side, and 512 rows x 32 heads x 6500 scores
    top = min(32768, (1 << 28) // (n_seq * hk * d), 512 * 32 * 6500 // (n_seq * rows * h))
    hi = _log(rng, max(rows, 16), max(top, max(rows, 16)))
    lo = rng.randint(0, hi)
    cap = -(-hi // 16) * 16
    window = _log(rng, 1, hi) if op == "f16w" or rng.random() < 0.5 else 0
    n_sink = rng.choice((0, 1, 4, 16, 33)) if window else 0
    return {k: v for k, v in _decode("", op, n_seq, rows, h, hk, d, cap, lo, hi, window,
                                     n_sink).items() if k != "name"}


def _ints(case):
    """The case's lengths: fixed by the case, so that its work is too.  append / read: new rows per
    sequence and the first position; decode: per row, rows of a sequence being consecutive."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] in ("append", "read"):
        n = [rng.randint(case["new_min"], case["new_max"]) for _ in range(case["n_seq"])]
        if not sum(n):
            n[0] = max(1, case["new_max"])
        return n, [rng.randint(0, case["cap"] - x) for x in n]
    last = [rng.randint(case["len_min"], case["len_max"]) for _ in range(case["n_seq"])]
    r = case["rows"]
    return [max(0, x - (r - 1 - i)) for x in last for i in range(r)], None


# ------------------------------------------------------------------------------------ plain form

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x, exp):
    """x [..., D] fp32 -> (codes [..., D] uint8, scales [..., D/16] fp32): y = x / 2^exp; the scale
    of 16 dims is amax|y| / 6 rounded to e4m3, a code the e2m1 value nearest to y / scale, ties to
    the even code in both.  NaN counts as 0."""
    y = torch.where(torch.isnan(x), 0.0, x) * 2.0 ** -exp
    y = y.unflatten(-1, (-1, 16))
    v = y.abs().amax(-1, keepdim=True).double() / 6
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    s = torch.where(torch.isinf(v), 448.0, torch.round(v / step) * step).clamp(max=448.0).float()
    a = y.abs()
    code = ((a > 0.25 * s).to(torch.uint8) + (a >= 0.75 * s) + (a > 1.25 * s) + (a >= 1.75 * s)
            + (a > 2.5 * s) + (a >= 3.5 * s) + (a > 5.0 * s))
    code = torch.where(s > 0, code, 0)
    code = code + 8 * ((y < 0) & (code > 0)).to(torch.uint8)
    return code.flatten(-2), s.squeeze(-1)


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _values(packed, scales, exp, table):
    """Packed codes [..., D/2] and e4m3 scale bytes [..., D/16] -> fp32 [..., D]."""
    code = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float() * 2.0 ** exp
    return (table[code.int()].unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _places(state):
    """(sequence, position) of every row of the ragged batch."""
    r = torch.arange(state["n_rows"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(state["row_off"], r, right=True) - 1
    return seq, (state["t0"][seq] + r - state["row_off"][seq]).long()


def _plain_append(s):
    seq, pos = _places(s)
    at = (seq[:, None], torch.arange(s["kq"].shape[1], device="cuda")[None], pos[:, None])
    out = []
    for x, q, sc, exp in ((s["k_new"], s["kq"], s["ksc"], s["k_exp"]),
                          (s["v_new"], s["vq"], s["vsc"], s["v_exp"])):
        code, scale = _quantise(x, exp)
        q[at] = _pack(code)
        sc[at] = scale.to(torch.float8_e4m3fn).view(torch.uint8)
        out.append(_values(q[at], sc[at], exp, s["table"]))
    return out


def _plain_read(s):
    seq, pos = _places(s)
    at = (seq[:, None], torch.arange(s["kq"].shape[1], device="cuda")[None], pos[:, None])
    return [_values(s["kq"][at], s["ksc"][at], s["k_exp"], s["table"]).to(s["dtype"]),
            _values(s["vq"][at], s["vsc"][at], s["v_exp"], s["table"]).to(s["dtype"])]


def _plain_decode(s, k, v):
    """k, v [n_seq][Hk][n][D] fp32; a row of length L sees positions j < L with j < n_sink or
    j >= L - window (all of them without a window)."""
    q = s["q"]
    t, h, d = q.shape
    n_seq, hk, n = k.shape[:3]
    r, g = t // n_seq, h // hk
    qs = q.view(n_seq, r, hk, g, d).transpose(1, 2).reshape(n_seq, hk, r * g, d)
    x = (qs @ k.transpose(-1, -2) * s["scale"]).view(n_seq, hk, r, g, n)
    j = torch.arange(n, device=q.device)
    length = s["kv_len"].view(n_seq, 1, r, 1, 1)
    see = j < length
    if s["window"]:
        see = see & ((j >= length - s["window"]) | (j < s["n_sink"]))
    x = torch.where(see, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = (p.view(n_seq, hk, r * g, n) @ v).view(n_seq, hk, r, g, d)
    o = torch.where(total > 0, o / total, 0.0)
    return o.transpose(1, 2).reshape(t, h, d)


# ------------------------------------------------------------------------------------ state

def _rows(gen, *shape):
    """K or V rows as a model makes them: normal values, a few channels several times larger."""
    x = torch.randn(shape, generator=gen, device="cuda")
    big = torch.rand(shape[-1], generator=gen, device="cuda") < 0.03
    return x * torch.where(big, 6.0, 1.0)


def _cache(gen, n_seq, hk, cap, d, exp):
    code, scale = _quantise(_rows(gen, n_seq, hk, cap, d), exp)
    return _pack(code), scale.to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n_seq, hk, d, cap = (case[x] for x in ("n_seq", "n_kv_heads", "head_dim", "cap"))
    first, t0 = _ints(case)
    s = dict(op=case["op"], table=torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda"))
    if case["op"] in ("append", "read"):
        s["k_exp"], s["v_exp"] = case["k_exp"], case["v_exp"]
        off = [sum(first[:i]) for i in range(n_seq + 1)]
        s["row_off"] = torch.tensor(off, dtype=torch.int32, device="cuda")
        s["t0"] = torch.tensor(t0, dtype=torch.int32, device="cuda")
        s["n_rows"] = off[-1]
        s["dtype"] = torch.float16 if case.get("half") else torch.float32
        s["kq"], s["ksc"] = _cache(gen, n_seq, hk, cap, d, s["k_exp"])
        s["vq"], s["vsc"] = _cache(gen, n_seq, hk, cap, d, s["v_exp"])
        if case["op"] == "append":
            s["k_new"] = _rows(gen, off[-1], hk, d)
            s["v_new"] = _rows(gen, off[-1], hk, d)
        # the buffers that a serving loop reads rows into
        s["k_out"] = torch.empty(off[-1], hk, d, dtype=s["dtype"], device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
        return s
    t = n_seq * case["rows"]
    s["q"] = torch.randn(t, case["n_heads"], d, generator=gen, device="cuda")
    s["kv_len"] = torch.tensor(first, dtype=torch.int32, device="cuda")
    s["seq_of"] = torch.arange(t, dtype=torch.int32, device="cuda") // case["rows"]
    s["max_len"] = max(max(first), 1)
    s["scale"] = d ** -0.5
    s["window"], s["n_sink"] = case["window"], case["n_sink"]
    if case["op"] == "q4":
        s["kq"], s["ksc"] = _cache(gen, n_seq, hk, cap, d, 0)
        s["vq"], s["vsc"] = _cache(gen, n_seq, hk, cap, d, 0)
    else:
        s["k"] = _rows(gen, n_seq, cap, hk, d).half()
        s["v"] = _rows(gen, n_seq, cap, hk, d).half()
    # the output buffer and the zeroed workspace that a decode loop keeps
    s["out"] = torch.empty_like(s["q"])
    s["ws"] = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    return s


def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "append":
        return _plain_append(s) + [s["ksc"].view(torch.float8_e4m3fn),
                                   s["vsc"].view(torch.float8_e4m3fn)]
    if s["op"] == "read":
        return _plain_read(s)
    n = s["max_len"]
    if s["op"] == "q4":
        k = _values(s["kq"][:, :, :n], s["ksc"][:, :, :n], 0, s["table"])
        v = _values(s["vq"][:, :, :n], s["vsc"][:, :, :n], 0, s["table"])
    else:
        k = s["k"][:, :n].transpose(1, 2).float()
        v = s["v"][:, :n].transpose(1, 2).float()
    return _plain_decode(s, k, v)


def _run_own(s):
    from gqa_decode_attention_03_gb300 import gqa_decode as gd

    if s["op"] in ("append", "read"):
        cache = (s["kq"], s["vq"], s["ksc"], s["vsc"], s["row_off"], s["t0"])
        scales = dict(k_scale=2.0 ** s["k_exp"], v_scale=2.0 ** s["v_exp"])
        if s["op"] == "append":
            gd.kv_append_q4(s["k_new"], s["v_new"], *cache, **scales)
        k, v = gd.kv_read_q4(*cache, k_out=s["k_out"], v_out=s["v_out"], **scales)
        if s["op"] == "read":
            return [k, v]
        return [k, v, s["ksc"].view(torch.float8_e4m3fn), s["vsc"].view(torch.float8_e4m3fn)]
    common = dict(scale=s["scale"], seq_of=s["seq_of"], max_kv_len=s["max_len"], out=s["out"],
                  ws=s["ws"], n_sink=s["n_sink"])
    if s["op"] == "q4":
        return gd.attn_decode_q4(s["q"], s["kq"], s["vq"], s["ksc"], s["vsc"], s["kv_len"],
                                 window=s["window"] or None, **common)
    return gd.attn_decode_f16_window(s["q"], s["k"], s["v"], s["kv_len"], s["window"], **common)


# ------------------------------------------------------------------------------------ work

def work(case):
    hk, d = case["n_kv_heads"], case["head_dim"]
    first, _ = _ints(case)
    packed = d / 2 + d / 16  # bytes of a row of codes and scales
    if case["op"] in ("append", "read"):
        n = sum(first) * hk * 2  # rows of K and of V
        if case["op"] == "append":  # fp32 rows in, packed rows out, their values out
            return {"bytes": n * (4 * d + packed + 4 * d), "flops": n * d * 4}
        return {"bytes": n * (packed + d * (2 if case["half"] else 4)), "flops": n * d}
    r, w, ns = case["rows"], case["window"], case["n_sink"]

    def seen(n):
        return n if not w else min(n, w) + max(0, min(ns, n - w))

    total = 0
    for i in range(case["n_seq"]):  # rows of a sequence need each of its positions once
        rows = first[i * r:(i + 1) * r]
        hi = max(rows)
        lo = max(0, min(rows) - w) if w else 0
        total += hi - lo + min(ns, lo)
    per = 2 * packed if case["op"] == "q4" else 4 * d
    t, h = len(first), case["n_heads"]
    return {"bytes": total * hk * per + 8 * t * h * d,
            "flops": sum(seen(n) for n in first) * h * d * 4}


# ------------------------------------------------------------------------------------ 64 bits

def _exact_scales():
    """Every e4m3 value from 0 to 448, in the order of its code."""
    return torch.tensor([c * 2.0 ** -9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10)
                         for c in range(127)], dtype=torch.float64, device="cuda")


def _nearest(x, grid):
    """Index of the grid value nearest to x, the even index on a tie; x past the end: the last.
    The comparisons are with the exact midpoints, so nothing is rounded on the way."""
    mid = (grid[..., 1:] + grid[..., :-1]) / 2
    i = torch.searchsorted(mid, x.contiguous(), right=False)  # mid[i - 1] < x <= mid[i]
    at = mid.gather(-1, i.clamp(max=mid.shape[-1] - 1))
    return i + ((i < mid.shape[-1]) & (at == x) & (i % 2 == 1)).long()


def _exact_quantised(x, exp):
    """(values, scales) in 64 bits of fp32 rows x [..., D], by sorting into the midpoints between
    neighbouring values of each format."""
    scales = _exact_scales()
    y = torch.nan_to_num(x.double() / 2.0 ** exp, nan=0.0, posinf=1e300, neginf=-1e300)
    y = y.reshape(-1, 16)
    a = y.abs().max(1).values
    s = scales[_nearest(a, 6 * scales)]
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    mag = grid[_nearest(y.abs(), s[:, None] * grid)]
    mag = torch.where(s[:, None] > 0, mag * s[:, None], 0.0)
    val = torch.where(y < 0, -mag, mag) * 2.0 ** exp
    return val.reshape(x.shape), s.reshape(*x.shape[:-1], -1)


def _exact_rows(packed, scales, exp):
    """The values of packed rows, in 64 bits, from the bits of codes and scales."""
    c = torch.stack((packed % 16, packed // 16), -1).flatten(-2).long()
    e, m = (c // 2) % 4, c % 2
    mag = torch.where(e == 0, m * 0.5, (2.0 + m) * 2.0 ** (e.double() - 2))
    val = torch.where(c >= 8, -mag, mag).double()
    s = _exact_scales()[scales.long()].repeat_interleave(16, -1)
    return val * s * 2.0 ** exp


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("append", "read"):
        first, t0 = _ints(case)
        out, side = [], []
        for n in ("k", "v"):
            exp, packed, sc = s[n + "_exp"], s[n + "q"], s[n + "sc"]
            if case["op"] == "append":
                val, scale = _exact_quantised(s[n + "_new"], exp)
                whole = _exact_scales()[sc.long()]
                for i, (c, t) in enumerate(zip(first, t0)):
                    o = sum(first[:i])
                    whole[i, :, t:t + c] = scale[o:o + c].transpose(0, 1)
                side.append(whole)
            else:
                val = torch.cat([_exact_rows(packed[i, :, t:t + c], sc[i, :, t:t + c],
                                             exp).transpose(0, 1)
                                 for i, (c, t) in enumerate(zip(first, t0))])
            out.append(val)
        return out + side
    lengths, _ = _ints(case)
    h, hk, d = case["n_heads"], case["n_kv_heads"], case["head_dim"]
    g, r = h // hk, case["rows"]
    w, ns = case["window"], case["n_sink"]
    out = torch.zeros(len(lengths), h, d, dtype=torch.float64, device="cuda")
    for i in range(case["n_seq"]):
        n = max(lengths[i * r:(i + 1) * r])
        for kvh in range(hk):
            if case["op"] == "q4":
                k = _exact_rows(s["kq"][i, kvh, :n], s["ksc"][i, kvh, :n], 0)
                v = _exact_rows(s["vq"][i, kvh, :n], s["vsc"][i, kvh, :n], 0)
            else:
                k, v = s["k"][i, :n, kvh].double(), s["v"][i, :n, kvh].double()
            lens = torch.tensor(lengths[i * r:(i + 1) * r], device="cuda")[:, None, None]
            x = torch.einsum("rgd,nd->rgn", s["q"][i * r:(i + 1) * r,
                                                   kvh * g:(kvh + 1) * g].double(), k) * s["scale"]
            j = torch.arange(n, device="cuda")
            hide = j >= lens
            if w:
                hide = hide | ((j < lens - w) & (j >= ns))
            p = torch.softmax(x.masked_fill(hide, -math.inf), -1)
            p = torch.where(hide, 0.0, p)  # a row that sees nothing gives zeros
            out[i * r:(i + 1) * r, kvh * g:(kvh + 1) * g] = torch.einsum("rgn,nd->rgd", p, v)
    return out
