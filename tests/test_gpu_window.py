"""GPU tests of decode attention over the f16 cache through a sliding window with sinks, against
64-bit values.  Every position that a row does not see holds NaN or infinity."""

import numpy as np
import pytest
import torch

import oracle
from gpu_util import assert_close, dev, forced_chunk
from q4_util import TOL, hidden, rows

pytestmark = pytest.mark.gpu


def _gd():
    from gqa_decode_attention_03_gb300 import gqa_decode
    return gqa_decode


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def f16_cache(rng, n_seq, cap, Hk, D):
    return (rows(rng, n_seq, cap, Hk, D).astype(np.float16),
            rows(rng, n_seq, cap, Hk, D).astype(np.float16))


def bury(k, v, s, mask):
    """Positions under mask get values that no output may show."""
    k[s, :len(mask)][mask] = np.float16(np.nan)
    v[s, :len(mask)][mask] = np.float16(np.inf)


def run(q, k, v, lens, window, n_sink, seq_of=None, **kw):
    return _gd().attn_decode_f16_window(dev(q), dev(k), dev(v), i32(lens), window, n_sink,
                                        seq_of=None if seq_of is None else i32(seq_of), **kw)


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 500, 511, 520]


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (7, 4), (16, 0), (33, 20), (64, 16),
                                           (64, 64), (129, 1), (200, 300), (511, 5), (1000, 4),
                                           (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("chunk", [None, 64])
def test_window(D, window, n_sink, chunk):
    rng = np.random.default_rng(window % 9973 + D)
    cap, Hk, H = 520, 2, 8
    k, v = f16_cache(rng, len(LENS), cap, Hk, D)
    for s, n in enumerate(LENS):
        bury(k, v, s, np.concatenate([hidden(n, window, n_sink), np.ones(cap - n, bool)]))
    q = rows(rng, len(LENS), H, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    with forced_chunk(chunk):
        got = run(q, k, v, LENS, window, n_sink, err=err).cpu().numpy()
    ref = oracle.decode_f16_window(q, k, v, LENS, D ** -0.5, window, n_sink)
    assert_close(got, ref, TOL, f"window {window} sinks {n_sink} D {D}")
    assert (got[0] == 0).all() and int(err) == 0


@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 1), (8, 8), (12, 1), (16, 1), (10, 2), (22, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_heads(D, H, Hk):
    rng = np.random.default_rng(D + H)
    lens, window, n_sink = [300, 41, 0, 77], 50, 5
    k, v = f16_cache(rng, 4, 301, Hk, D)
    q = rows(rng, 4, H, D)
    for chunk in (None, 64):
        with forced_chunk(chunk):
            got = run(q, k, v, lens, window, n_sink).cpu().numpy()
        assert_close(got, oracle.decode_f16_window(q, k, v, lens, D ** -0.5, window, n_sink), TOL,
                     f"heads {H}/{Hk} D {D}")


def test_window_over_everything_is_dense():
    gd = _gd()
    rng = np.random.default_rng(3)
    lens = [900, 1, 513]
    k, v = f16_cache(rng, 3, 900, 2, 128)
    q = rows(rng, 3, 8, 128)
    a = run(q, k, v, lens, 900, 0).cpu().numpy()
    b = gd.attn_decode_f16(dev(q), dev(k), dev(v), i32(lens)).cpu().numpy()
    assert_close(a, b, 2 * TOL, "against attn_decode_f16")


@pytest.mark.parametrize("H,Hk,D", [(8, 2, 128), (4, 4, 64), (32, 2, 64), (12, 2, 256), (7, 1, 128),
                                    (16, 2, 128), (6, 3, 64)])
@pytest.mark.parametrize("window,n_sink", [(40, 3), (1, 0), (100, 80), (400, 1), (64, 0)])
def test_rows_sharing_sequences(H, Hk, D, window, n_sink):
    """Causal rows of three sequences in runs, rows out of order, one sequence in two runs, rows of
    very different lengths side by side, empty rows between."""
    rng = np.random.default_rng(H + D + window)
    seq = [2] * 40 + [0] * 3 + [1] * 8 + [2] * 5 + [0, 1, 0]
    lens = (list(range(381, 421)) + [5, 0, 1] + list(range(90, 98)) + [430, 2, 0, 300, 77]
            + [9, 64, 9])
    k, v = f16_cache(rng, 3, 432, Hk, D)
    for s in range(3):
        seen = np.zeros(432, bool)
        for t, n in zip(seq, lens):
            if t == s:
                seen[oracle.visible_positions(n, window, n_sink)] = True
        bury(k, v, s, ~seen)
    q = rows(rng, len(seq), H, D)
    ref = oracle.decode_f16_window(q, k, v, lens, D ** -0.5, window, n_sink, seq_of=seq)
    for chunk in (None, 64):
        with forced_chunk(chunk):
            got = run(q, k, v, lens, window, n_sink, seq).cpu().numpy()
        assert_close(got, ref, TOL, f"shared sequences, chunk {chunk}")


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_chunk(D):
    """A chunk of 150 causal rows of one sequence, from its first position on and further in; NaN
    between the sinks and the first window and behind the last row."""
    rng = np.random.default_rng(D)
    H, Hk, window, n_sink = 8, 2, 130, 4
    for first in (0, 700):
        lens = [first + 1 + r for r in range(150)]
        k, v = f16_cache(rng, 1, 900, Hk, D)
        seen = np.zeros(900, bool)
        for n in lens:
            seen[oracle.visible_positions(n, window, n_sink)] = True
        bury(k, v, 0, ~seen)
        q = rows(rng, 150, H, D)
        got = run(q, k, v, lens, window, n_sink, [0] * 150).cpu().numpy()
        ref = oracle.decode_f16_window(q, k, v, lens, D ** -0.5, window, n_sink, seq_of=[0] * 150)
        assert_close(got, ref, TOL, f"chunk at {first}")


@pytest.mark.parametrize("H,Hk,D,T", [(8, 2, 128, 150), (2, 2, 64, 200), (32, 2, 64, 40),
                                      (12, 1, 128, 33), (8, 2, 256, 20), (4, 2, 128, 5)])
def test_values_that_some_rows_see(H, Hk, D, T):
    """NaN and infinities in K and V at positions that some rows of a chunk see and others do not:
    the others' outputs are what they are without them."""
    rng = np.random.default_rng(T + D)
    window, n_sink, first = 60, 3, 240
    lens = [first + r for r in range(T)]
    k, v = f16_cache(rng, 1, first + T, Hk, D)
    q = rows(rng, T, H, D)
    odd = [(first + 2, 0, 5, np.inf), (first - 40, Hk - 1, D - 1, np.nan), (first + T // 2, 0, 9, -np.inf)]
    bad_k = first + T - 3                               # seen by the last rows only
    clean_k, clean_v = k.copy(), v.copy()
    for pos, g, d, x in odd:
        v[0, pos, g, d], clean_v[0, pos, g, d] = x, 0
    k[0, bad_k, :, 7] = np.nan
    got = run(q, k, v, lens, window, n_sink, [0] * T).cpu().numpy()
    ref = oracle.decode_f16_window(q, clean_k, clean_v, lens, D ** -0.5, window, n_sink,
                                   seq_of=[0] * T)
    G = H // Hk
    fine = np.ones(got.shape, bool)
    for t, n in enumerate(lens):
        see = set(oracle.visible_positions(n, window, n_sink).tolist())
        if bad_k in see:
            fine[t] = False
        for pos, g, d, _ in odd:
            if pos in see:
                fine[t, g * G:(g + 1) * G, d] = False
    assert not np.isfinite(got[~fine]).any() and np.isfinite(got[fine]).all()
    assert fine.any() and not fine.all()
    assert_close(np.where(fine, got, 0), np.where(fine, ref, 0), TOL, "rows that do not see them")


@pytest.mark.parametrize("H,Hk,D", [(2, 2, 64), (8, 2, 128), (32, 2, 128), (12, 2, 64)])
def test_many_rows_of_several_sequences(H, Hk, D):
    """300 rows in runs of 1 to 60 of five sequences, lengths from 0 on: several runs in a group, a
    run over several groups; a grid split over positions and one that is not."""
    rng = np.random.default_rng(D + H)
    seq, lens = [], []
    while len(seq) < 300:
        s, m, n0 = int(rng.integers(5)), int(rng.integers(1, 61)), int(rng.integers(0, 900))
        seq += [s] * m
        lens += [min(960, n0 + i) for i in range(m)]
    seq, lens = seq[:300], lens[:300]
    k, v = f16_cache(rng, 5, 960, Hk, D)
    q = rows(rng, 300, H, D)
    for window, n_sink in ((150, 4), (5000, 0), (33, 200)):
        for T in (300, 40):
            got = run(q[:T], k, v, lens[:T], window, n_sink, seq[:T]).cpu().numpy()
            ref = oracle.decode_f16_window(q[:T], k, v, lens[:T], D ** -0.5, window, n_sink,
                                           seq_of=seq[:T])
            assert_close(got, ref, TOL, f"window {window} rows {T}")


def test_large_scores_and_infinite_values_in_sight():
    """Scores of many thousands keep one position; an infinite V in sight leaves its dim without a
    finite value, one hidden does not.  (Which one is open: a weight w goes into the product as
    f16 hi + lo with lo of either sign or 0, and hi inf + lo inf is inf or NaN by that sign.)"""
    rng = np.random.default_rng(7)
    k, v = f16_cache(rng, 1, 64, 1, 64)
    q = rows(rng, 1, 4, 64) * np.float32(100)
    got = run(q, k, v, [60], 30, 2, scale=8.0).cpu().numpy()
    ref = oracle.decode_f16_window(q, k, v, [60], 8.0, 30, 2)
    # scores up to ~100 * 8 * 8 * 4 = 25000 carry 2^-22 of it: 6e-3 of a weight's exponent
    assert_close(got, ref, 2e-2, "large scores")
    v[0, 40, 0, 3] = np.inf
    v[0, 10] = np.inf
    got = run(q * np.float32(0.01), k, v, [60], 30, 2).cpu().numpy()
    assert not np.isfinite(got[0, :, 3]).any() and np.isfinite(np.delete(got, 3, 2)).all()


def test_tiny_caches_under_many_rows():
    rng = np.random.default_rng(15)
    for D in (64, 128):
        k, v = f16_cache(rng, 1, 9, 2, D)
        q = rows(rng, 200, 8, D)
        lens = [int(n) for n in rng.integers(0, 10, 200)]
        got = run(q, k, v, lens, 5, 2, [0] * 200).cpu().numpy()
        ref = oracle.decode_f16_window(q, k, v, lens, D ** -0.5, 5, 2, seq_of=[0] * 200)
        assert_close(got, ref, TOL, f"D {D}")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(q[:1], k, v, [0], 5, 2, max_kv_len=0, err=err)
    assert (got == 0).all() and int(err) == 0
    assert run(q[:0], k, v, [], 5, 2).shape == (0, 8, 128)


def test_bad_lengths_and_sequences():
    gd = _gd()
    rng = np.random.default_rng(5)
    k, v = f16_cache(rng, 2, 50, 1, 64)
    q = rows(rng, 5, 4, 64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(q, k, v, [-3, 51, 20, 20, 20], 9, 2, [0, 1, 2, -1, 1], err=err).cpu().numpy()
    assert int(err) == gd.ERR_KVLEN_RANGE | gd.ERR_SEQ_RANGE
    ref = oracle.decode_f16_window(q, k, v, [0, 50, 0, 0, 20], 0.125, 9, 2, seq_of=[0, 1, 0, 0, 1])
    assert_close(got, ref, TOL, "clamped rows")
    err.zero_()
    got = run(q[:1], k, v, [40], 9, 2, [0], err=err, max_kv_len=25).cpu().numpy()
    assert int(err) == gd.ERR_KVLEN_RANGE
    assert_close(got, oracle.decode_f16_window(q[:1], k, v, [25], 0.125, 9, 2), TOL, "max_kv_len")


@pytest.mark.parametrize("rows_per_seq", [1, 6])
def test_gate(rows_per_seq):
    rng = np.random.default_rng(6)
    lens = [0, 300, 37, 38, 39, 40]
    seq = [0] * 6 if rows_per_seq == 6 else list(range(6))
    k, v = f16_cache(rng, 6 // rows_per_seq, 304, 2, 128)
    q = rows(rng, 6, 8, 128)
    gate = rows(rng, 48 * 200)
    ref = oracle.decode_f16_window(q, k, v, lens, 128 ** -0.5, 70, 4, seq_of=seq)
    ref = oracle.output_gate(ref, gate.reshape(6, 8, 200)[..., :128])
    for chunk in (None, 64):
        with forced_chunk(chunk):
            got = run(q, k, v, lens, 70, 4, seq, gate=dev(gate), gate_stride=200).cpu().numpy()
        assert_close(got, ref, TOL, "gate")


@pytest.mark.parametrize("shared", [False, True])
def test_graphs_share_a_workspace(shared):
    """Two captured calls of different shapes on one workspace, replayed in turn with lengths that
    change between replays."""
    gd = _gd()
    rng = np.random.default_rng(8)
    T, H, Hk, D, cap = 6, 8, 2, 128, 1200
    k, v = f16_cache(rng, 1 if shared else T, cap, Hk, D)
    seq = [0] * T if shared else list(range(T))
    q = rows(rng, T, H, D)
    kd, vd, sd = dev(k), dev(v), i32(seq)
    lens = [i32([cap] * T), i32([cap] * 2)]
    outs = [torch.empty((T, H, D), device="cuda"), torch.empty((2, H, D), device="cuda")]
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda")
    qd = [dev(q), dev(q[:2])]

    def call(i):
        gd.attn_decode_f16_window(qd[i], kd, vd, lens[i], (600, 333)[i], 4, seq_of=sd[:len(qd[i])],
                                  out=outs[i], ws=ws)

    call(0)
    call(1)
    torch.cuda.synchronize()
    graphs = []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for it in range(3):
        n = [int(x) for x in rng.integers(0, cap + 1, T)]
        lens[0].copy_(i32(n))
        lens[1].copy_(i32(n[:2]))
        for i in (it % 2, 1 - it % 2):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i, w in ((0, 600), (1, 333)):
            ref = oracle.decode_f16_window(q[:len(qd[i])], k, v, n[:len(qd[i])], D ** -0.5, w, 4,
                                           seq_of=seq)
            assert_close(outs[i].cpu().numpy(), ref, TOL, f"graph {i} replay {it}")


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements a side; only its last positions and sinks are seen."""
    gd = _gd()
    cap, Hk, D = 150000, 64, 256
    k = torch.zeros((1, cap, Hk, D), dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    rng = np.random.default_rng(1)
    kn, vn = f16_cache(rng, 1, 80, Hk, D)
    for t, o in ((0, 0), (cap - 40, 40)):
        k[0, t:t + 40] = dev(kn[0, o:o + 40])
        v[0, t:t + 40] = dev(vn[0, o:o + 40])
    q = rows(rng, 2, Hk, D)
    got = gd.attn_decode_f16_window(dev(q), k, v, i32([cap, cap]), 40, 40,
                                    seq_of=i32([0, 0])).cpu().numpy()
    for t in range(2):
        for h in (0, 31, 63):
            ref = oracle.attend_positions(q[t, h:h + 1], kn[0, :, h], vn[0, :, h], D ** -0.5)
            assert_close(got[t, h:h + 1], ref, TOL, f"row {t} head {h}")


def test_binding_refuses():
    gd = _gd()
    rng = np.random.default_rng(2)
    k, v = map(dev, f16_cache(rng, 1, 16, 1, 64))
    q, n = dev(rows(rng, 1, 4, 64)), i32([16])
    bad = [lambda: gd.attn_decode_f16_window(q, k, v, n, None),
           lambda: gd.attn_decode_f16_window(q, k, v, n, 0),
           lambda: gd.attn_decode_f16_window(q, k, v, n, -1),
           lambda: gd.attn_decode_f16_window(q, k, v, n, 4, -1),
           lambda: gd.attn_decode_f16_window(q, k.float(), v, n, 4),
           lambda: gd.attn_decode_f16_window(q, k, v[:, :8], n, 4),
           lambda: gd.attn_decode_f16_window(q, k.cpu(), v, n, 4),
           lambda: gd.attn_decode_f16_window(q, k, v, n.long(), 4),
           lambda: gd.attn_decode_f16_window(q, k, v, n, 4, out=q),
           lambda: gd.attn_decode_f16_window(q, k, v, n, 4, err=torch.zeros(1, device="cuda")),
           lambda: gd.attn_decode_f16_window(q, k, v, n, 4, scale=float("nan"))]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, gd.GqaError)):
            call()
            pytest.fail(f"call {i} went through")
