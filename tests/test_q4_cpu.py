"""CPU checks of the 4-bit cache and the window calls: the oracle against rational arithmetic, the
plans, and the refusals of the C entry points (nothing is launched)."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest

import oracle

E2M1 = [Fraction(x) for x in (0, Fraction(1, 2), 1, Fraction(3, 2), 2, 3, 4, 6)]
E4M3 = [Fraction(c, 512) if c < 8 else Fraction(8 + c % 8) * Fraction(2) ** (c // 8 - 10)
        for c in range(127)]


@pytest.fixture(scope="module")
def gd():
    from gqa_decode_attention_03_gb300 import gqa_decode
    return gqa_decode


def nearest(x, grid):
    best = min(range(len(grid)), key=lambda c: (abs(x - grid[c]), c % 2))
    return best


def group_by_fractions(x, scale):
    y = [Fraction(float(v)) / Fraction(scale) for v in x]
    sc = nearest(max(abs(v) for v in y) / 6, E4M3)
    codes = [nearest(abs(v) / E4M3[sc], E2M1) if sc else 0 for v in y]
    return [c | (8 if v < 0 and c else 0) for c, v in zip(codes, y)], sc


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -7, 2.0 ** 20])
def test_quantiser_against_rationals(scale):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((60, 16)) * 10.0 ** rng.uniform(-4, 4, (60, 1))).astype(np.float32)
    x[0] = 0
    x[1] = 1e-6                                       # scale rounds to 0 (at scale 1)
    x[2] = 1e9                                        # past 6 * 448
    # ties: amax / 6 between two e4m3 values, and every midpoint of the codes
    x[3] = 6 * float(E4M3[60] + E4M3[61]) / 2
    x[4] = 6 * float(E4M3[61] + E4M3[62]) / 2
    x[5] = np.float32([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5,
                       -5, -0.0])
    x[6] = np.nextafter(x[5], np.float32(9))
    x[7] = np.nextafter(x[5], np.float32(-9))
    x[3:8] *= np.float32(scale)
    packed, sc = oracle.quantize_q4(x, scale)
    for i in range(len(x)):
        codes, s = group_by_fractions(x[i], scale)
        assert s == sc[i, 0], i
        got = [int(b) >> (4 * k) & 15 for b in packed[i] for k in (0, 1)]
        assert got == codes, i
    want = [float((-1) ** (c >> 3) * E2M1[c & 7] * E4M3[s] * Fraction(scale))
            for c, s in ((c, group_by_fractions(x[9], scale)[1])
                         for c in group_by_fractions(x[9], scale)[0])]
    assert oracle.dequant_q4(packed[9], sc[9], scale).tolist() == want


def test_quantiser_special_values():
    x = np.zeros((3, 16), np.float32)
    x[0, :3] = [np.nan, 1.0, -6.0]
    x[1, :3] = [np.inf, -np.inf, 3.0]
    packed, sc = oracle.quantize_q4(x)
    v = oracle.dequant_q4(packed, sc)
    assert v[0, :3].tolist() == [0.0, 1.0, -6.0]
    assert v[1, :3].tolist() == [2688.0, -2688.0, 0.0] and sc[1, 0] == 126
    assert not packed[2].any() and sc[2, 0] == 0


def test_visible_positions():
    vis = oracle.visible_positions
    assert vis(0, 4, 2).tolist() == [] and vis(3).tolist() == [0, 1, 2]
    assert vis(10, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert vis(4, 3, 2).tolist() == [0, 1, 2, 3]      # sinks and window meet: each once
    assert vis(10, 3, 99).tolist() == list(range(10))
    assert vis(10, 99, 0).tolist() == list(range(10))
    assert vis(1, 1, 0).tolist() == [0]


def test_decode_over_everything_is_dense_decode():
    rng = np.random.default_rng(8)
    q = rng.standard_normal((2, 4, 64)).astype(np.float32)
    k, v = (rng.standard_normal((2, 20, 2, 64)).astype(np.float16) for _ in range(2))
    a = oracle.decode_f16_window(q, k, v, [20, 7], 0.2, 20)
    assert np.allclose(a, oracle.decode_f16(q, k, v, np.int32([20, 7]), 0.2), atol=1e-12)
    kq, ksc = oracle.quantize_q4(k.transpose(0, 2, 1, 3).astype(np.float32))
    vq, vsc = oracle.quantize_q4(v.transpose(0, 2, 1, 3).astype(np.float32))
    kd = oracle.dequant_q4(kq, ksc).transpose(0, 2, 1, 3).astype(np.float16)
    vd = oracle.dequant_q4(vq, vsc).transpose(0, 2, 1, 3).astype(np.float16)
    b = oracle.decode_q4(q, kq, vq, ksc, vsc, [20, 7], 0.2)
    assert np.allclose(b, oracle.decode_f16(q, kd, vd, np.int32([20, 7]), 0.2), atol=1e-12)


# ------------------------------------------------------------------------------------ refusals

P = ctypes.c_void_p
OK = P(1 << 20)


def append(gd, **kw):
    a = dict(k_new=OK, v_new=OK, n=4, hk=2, d=64, row_off=OK, t0=OK, ks=1.0, vs=1.0, kq=OK, vq=OK,
             ksc=OK, vsc=OK, n_seq=2, cap=32, err=None) | kw
    return gd.LIB.kv_append_q4(a["k_new"], a["v_new"], a["n"], a["hk"], a["d"], a["row_off"],
                               a["t0"], a["ks"], a["vs"], a["kq"], a["vq"], a["ksc"], a["vsc"],
                               a["n_seq"], a["cap"], a["err"], None)


def read(gd, **kw):
    a = dict(k_out=OK, v_out=OK, n=4, hk=2, d=64, row_off=OK, t0=OK, ks=1.0, vs=1.0, kq=OK, vq=OK,
             ksc=OK, vsc=OK, n_seq=2, cap=32, err=None) | kw
    return gd.LIB.kv_read_q4(a["kq"], a["vq"], a["ksc"], a["vsc"], a["n_seq"], a["cap"], a["n"],
                             a["hk"], a["d"], a["row_off"], a["t0"], a["ks"], a["vs"], a["k_out"],
                             a["v_out"], 0, a["err"], None)


ROWS_BAD = [dict(n=-1), dict(hk=0), dict(d=96), dict(d=32), dict(n_seq=0), dict(cap=0),
            dict(cap=24), dict(cap=-16), dict(ks=0.0), dict(ks=-1.0), dict(ks=3.0),
            dict(vs=float("nan")), dict(vs=float("inf")), dict(vs=2.0 ** 65), dict(ks=2.0 ** -65),
            dict(kq=None), dict(vq=None), dict(ksc=None), dict(vsc=None), dict(row_off=None),
            dict(t0=None), dict(kq=P((1 << 20) + 8)), dict(vsc=P((1 << 20) + 4)),
            dict(row_off=P((1 << 20) + 2)), dict(t0=P((1 << 20) + 1)), dict(err=P((1 << 20) + 2))]


@pytest.mark.parametrize("kw", ROWS_BAD + [dict(k_new=None), dict(v_new=P((1 << 20) + 4))], ids=str)
def test_append_refuses(gd, kw):
    assert append(gd, **kw) == gd.GQA_EINVAL and b"kv_append_q4" in gd.LIB.gqa_last_error()


@pytest.mark.parametrize("kw", ROWS_BAD + [dict(k_out=None), dict(v_out=P((1 << 20) + 4))], ids=str)
def test_read_refuses(gd, kw):
    assert read(gd, **kw) == gd.GQA_EINVAL and b"kv_read_q4" in gd.LIB.gqa_last_error()


def test_rows_of_too_many_heads(gd):
    for call in (append, read):
        assert call(gd, n=1 << 27, hk=16) == gd.GQA_EUNSUPPORTED
        assert b"n_rows * n_kv_heads" in gd.LIB.gqa_last_error()


def test_no_rows_is_no_work(gd):
    assert append(gd, n=0, k_new=None) == gd.GQA_OK and read(gd, n=0, k_out=None) == gd.GQA_OK


def q4(gd, **kw):
    a = dict(q=OK, kq=OK, vq=OK, ksc=OK, vsc=OK, ks=1.0, vs=1.0, window=0, n_sink=0, out=OK, len=OK,
             seq=None, T=1, n_seq=1, H=4, hk=1, d=64, cap=32, max=32, scale=0.1, gate=None, gs=0,
             err=None) | kw
    return gd.LIB.attn_decode_q4(a["q"], a["kq"], a["vq"], a["ksc"], a["vsc"], a["ks"], a["vs"],
                                 a["window"], a["n_sink"], a["out"], a["len"], a["seq"], a["T"],
                                 a["n_seq"], a["H"], a["hk"], a["d"], a["cap"], a["max"],
                                 a["scale"], a["gate"], a["gs"], None, 0, a["err"], None)


def f16w(gd, **kw):
    a = dict(q=OK, kq=OK, vq=OK, window=8, n_sink=0, out=OK, len=OK, seq=None, T=1, n_seq=1, H=4,
             hk=1, d=64, cap=32, max=32, scale=0.1, gate=None, gs=0, err=None) | kw
    return gd.LIB.attn_decode_f16_window(a["q"], a["kq"], a["vq"], a["window"], a["n_sink"],
                                         a["out"], a["len"], a["seq"], a["T"], a["n_seq"], a["H"],
                                         a["hk"], a["d"], a["cap"], a["max"], a["scale"],
                                         a["gate"], a["gs"], None, 0, a["err"], None)


DECODE_BAD = [dict(q=None), dict(kq=None), dict(vq=None), dict(out=None), dict(len=None),
              dict(q=P((1 << 20) + 4)), dict(kq=P((1 << 20) + 8)), dict(out=P((1 << 20) + 4)),
              dict(len=P((1 << 20) + 2)), dict(seq=P((1 << 20) + 2)), dict(err=P((1 << 20) + 1)),
              dict(T=-1), dict(T=65536), dict(n_seq=0), dict(H=5, hk=2), dict(hk=0), dict(d=96),
              dict(d=32), dict(cap=0), dict(max=-1), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(T=2), dict(window=-1), dict(window=8, n_sink=-1),
              dict(gate=OK, gs=63), dict(gate=P((1 << 20) + 2), gs=64)]


@pytest.mark.parametrize("kw", DECODE_BAD + [
    dict(ksc=None), dict(vsc=None), dict(vsc=P((1 << 20) + 8)), dict(cap=24), dict(ks=1.5),
    dict(vs=0.0)], ids=str)
def test_q4_decode_refuses(gd, kw):
    assert q4(gd, **kw) == gd.GQA_EINVAL and gd.LIB.gqa_last_error()


@pytest.mark.parametrize("kw", DECODE_BAD + [dict(window=0)], ids=str)
def test_f16_window_refuses(gd, kw):
    assert f16w(gd, **kw) == gd.GQA_EINVAL and gd.LIB.gqa_last_error()


def test_decode_unsupported_and_empty(gd):
    for call in (q4, f16w):
        assert call(gd, H=34, hk=2) == gd.GQA_EUNSUPPORTED             # group 17
        assert call(gd, cap=1 << 31, T=1) == gd.GQA_EUNSUPPORTED       # 2^31 rows
        assert call(gd, T=0, q=None, out=None) == gd.GQA_OK


def test_plans_check_their_sizes(gd):
    for kind in (gd.KIND_Q4, gd.KIND_F16_WINDOW):
        with pytest.raises(gd.GqaError, match="EINVAL"):
            gd.plan(1, 4, 1, 64, 10, 0, kind, num_sms=152)             # budget 0
        with pytest.raises(gd.GqaError, match="EINVAL"):
            gd.plan(1, 4, 1, 32, 10, 5, kind, num_sms=152)             # head_dim 32
        assert gd.plan(1, 4, 1, 64, 0, 5, kind, num_sms=152).merge == 0
        for n_tok, n_seq in ((0, 1), (1, 1), (300, 1), (300, 300)):
            p = gd.plan(n_tok, 32, 8, 128, 0, kind=kind, num_sms=152, n_seq=n_seq)
            assert p.merge == 0 and p.ws_bytes == 0


def test_q4_plans(gd):
    def plan(n_tok, H, Hk, D, n, budget=-1, n_seq=None):
        return gd.plan(n_tok, H, Hk, D, n, budget, gd.KIND_Q4, num_sms=152, n_seq=n_seq)

    # a ragged batch of long rows: one wave of three CTAs an SM with equal shares; counters, a
    # word a row and head, then two records of the group's 4 heads a CTA
    p = plan(16, 32, 8, 128, 32768)
    assert p.streamk == 1 and (p.grid_x, p.grid_y, p.grid_z) == (456, 1, 1)
    assert p.ws_bytes == 16 * 32 * 4 + 2 * 456 * 4 * 130 * 4
    # short lists, or more rows than the shares are found for: chunks of 2048 positions
    p = plan(200, 32, 8, 128, 1024)
    assert p.streamk == 0 and p.merge == 0 and (p.grid_x, p.grid_y, p.grid_z) == (1, 8, 200)
    p = plan(300, 32, 8, 128, 32768)
    assert p.streamk == 0 and p.chunk == 2048 and (p.grid_x, p.grid_y, p.grid_z) == (16, 8, 300)
    # one row: as many chunks as give every SM one CTA, at most 16
    p = plan(1, 48, 4, 256, 8191)
    assert p.n_split == 16 and p.grid_y == 8 and p.chunk == 512     # 12 heads: two CTAs of 6
    assert plan(1, 4, 1, 64, 256).merge == 0
    # rows that may share a sequence: two of four heads a CTA, 128 / 4 where there is work enough
    assert plan(32, 32, 8, 64, 8100, 2052, n_seq=2).row_group == 2
    p = plan(512, 32, 8, 128, 8000, n_seq=1)
    assert p.row_group == 32 and (p.grid_x, p.grid_y, p.grid_z) == (1, 8, 16) and p.merge == 0
    assert plan(64, 32, 8, 128, 8000, n_seq=1).n_split == 9
    assert plan(512, 32, 8, 256, 8000, n_seq=1).row_group == 2      # head_dim 256


def test_f16_window_plans(gd, monkeypatch):
    def plan(n_tok, H, Hk, D, n, budget, n_seq=None):
        return gd.plan(n_tok, H, Hk, D, n, budget, gd.KIND_F16_WINDOW, num_sms=152, n_seq=n_seq)

    # what a row sees sizes the grid: 1024 + 4 positions, in a cluster of up to 8 chunks
    p = plan(1, 32, 8, 64, 16001, 1028)
    assert p.tile == 128 and p.n_split == 6 and p.merge == 1
    # a chunk of a prompt: 128 pairs a CTA
    p = plan(512, 32, 8, 128, 6500, 2064, n_seq=1)
    assert p.row_group == 32 and p.grid_z == 16 and p.merge == 0
    monkeypatch.setenv("GQA_F16_ROWS", "off")
    assert plan(512, 32, 8, 128, 6500, 2064, n_seq=1).row_group == 1
