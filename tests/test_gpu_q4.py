"""GPU tests of the 4-bit cache: appending (bit-exact against the oracle), reading (exact), and
decode attention over it, against 64-bit values."""

import numpy as np
import pytest
import torch

import oracle
from gpu_util import _env, assert_close, dev, forced_chunk, forced_ctas
from q4_util import TOL, hidden, q4_cache, rows

pytestmark = pytest.mark.gpu


def _gd():
    from gqa_decode_attention_03_gb300 import gqa_decode
    return gqa_decode


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def ragged(counts):
    return np.concatenate([[0], np.cumsum(counts)])


# ------------------------------------------------------------------------------------ rows

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hk", [1, 3, 8])
@pytest.mark.parametrize("k_scale,v_scale", [(1.0, 1.0), (2.0 ** -5, 4.0)])
def test_append_is_bit_exact(D, Hk, k_scale, v_scale):
    rng = np.random.default_rng(D + Hk)
    counts, t0, cap, pad = [5, 0, 1, 33, 0, 16, 2], [9, 0, 47, 3, 1, 32, 46], 48, 3
    n, n_seq = sum(counts), len(counts)
    x = rng.standard_normal((2, n + pad, Hk, D)) * 10.0 ** rng.uniform(-3, 3, (2, n + pad, Hk, 1))
    x = x.astype(np.float32)
    x[0, 1, 0, :16] = 0.0
    x[0, 2, 0, :16] = np.float32([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75,
                                  -2.5, -3.5, -5, -0.0]) * np.float32(k_scale)
    x[0, 3, 0, :16] = np.nextafter(x[0, 2, 0, :16], np.float32(99))
    x[0, 4, 0, :16] = np.nextafter(x[0, 2, 0, :16], np.float32(-99))
    x[1, 0, 0, :16] = 6 * 11.5 * v_scale                # amax / 6 between two scales
    x[1, 1, 0, :16] = 6 * 12.5 * v_scale
    x[1, 2, 0, :16] = np.nextafter(np.float32(6 * 12.5 * v_scale), np.float32(1e9))
    x[1, 3, 0, :4] = [np.nan, np.inf, -np.inf, 1.0]
    x[1, 4, 0, :16] = 1e-30
    old = rng.integers(0, 256, (4, n_seq, Hk, cap, D // 2), dtype=np.uint8)
    cache = [dev(old[0]), dev(old[1]), dev(old[2][..., :D // 16]), dev(old[3][..., :D // 16])]
    want = [c.cpu().numpy() for c in cache]
    off = ragged(counts)
    for side, scale in ((0, k_scale), (1, v_scale)):
        q, s = oracle.quantize_q4(x[side, :n], scale)
        for i, (c, t) in enumerate(zip(counts, t0)):
            want[side][i, :, t:t + c] = q[off[i]:off[i] + c].transpose(1, 0, 2)
            want[2 + side][i, :, t:t + c] = s[off[i]:off[i] + c].transpose(1, 0, 2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (*cache, i32(off), i32(t0))
    _gd().kv_append_q4(dev(x[0]), dev(x[1]), *args, k_scale=k_scale, v_scale=v_scale, err=err)
    for got, ref, name in zip(cache, want, ("kq", "vq", "ksc", "vsc")):
        assert np.array_equal(got.cpu().numpy(), ref), name
    for dtype in (torch.float32, torch.float16):
        k = torch.full((n + pad, Hk, D), 7.0, dtype=dtype, device="cuda")
        v = k.clone()
        _gd().kv_read_q4(*args, k_out=k, v_out=v, k_scale=k_scale, v_scale=v_scale, err=err)
        for got, side, scale in ((k, 0, k_scale), (v, 1, v_scale)):
            q, s = oracle.quantize_q4(x[side, :n], scale)
            ref = torch.from_numpy(oracle.dequant_q4(q, s, scale)).to(dtype).numpy()
            assert np.array_equal(got[:n].cpu().numpy(), ref)
            assert (got[n:] == 7.0).all()               # rows behind the last sequence
    assert int(err) == 0


@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (128, torch.float32),
                                     (128, torch.float16), (256, torch.float32),
                                     (256, torch.float16), (64, torch.float32)])
@pytest.mark.parametrize("Hk", [1, 3, 16])
def test_many_rows_of_ragged_sequences_read(D, dtype, Hk):
    """More than 2048 rows, sequences that end anywhere in a block of 16 rows; rows behind the last one
    keep what they held."""
    rng = np.random.default_rng(D)
    counts, cap, pad = [1003, 0, 1, 2, 0, 0, 17, 700, 400, 5, 1, 1, 0, 1, 1, 1], 1008, 9
    n, n_seq = sum(counts), len(counts)
    t0 = [int(rng.integers(0, cap - c + 1)) for c in counts]
    codes = rng.integers(0, 256, (2, n_seq, Hk, cap, D // 2), dtype=np.uint8)
    scales = rng.integers(40, 88, (2, n_seq, Hk, cap, D // 16), dtype=np.uint8)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.full((n + pad, Hk, D), 7.0, dtype=dtype, device="cuda")
    v = k.clone()
    _gd().kv_read_q4(dev(codes[0]), dev(codes[1]), dev(scales[0]), dev(scales[1]),
                     i32(ragged(counts)), i32(t0), k_out=k, v_out=v, v_scale=2.0, err=err)
    for got, side, scale in ((k, 0, 1.0), (v, 1, 2.0)):
        plane = oracle.dequant_q4(codes[side], scales[side], scale).transpose(0, 2, 1, 3)
        ref = np.concatenate([plane[s, t:t + c] for s, (c, t) in enumerate(zip(counts, t0))])
        assert np.array_equal(got[:n].cpu().numpy(), torch.from_numpy(ref).to(dtype).numpy())
        assert (got[n:] == 7.0).all()
    assert int(err) == 0


@pytest.mark.parametrize("n_seq", [1, 31, 32, 33, 1024, 1025, 5000])
def test_rows_find_their_sequence(n_seq):
    """One KV head of 64 dims, many sequences of 0 to 3 rows: reading back what was appended."""
    rng = np.random.default_rng(n_seq)
    counts = rng.integers(0, 4, n_seq)
    counts[-1] = 2
    cap, n = 16, int(counts.sum())
    t0 = rng.integers(0, cap - 3, n_seq)
    x = rng.integers(-3, 4, (n, 1, 64)).astype(np.float32) * 2
    x[:, :, ::16] = 6.0                                 # scale 1: every value is exact
    z = lambda w: torch.zeros((n_seq, 1, cap, w), dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = [z(32), z(32), z(4), z(4)]
    args = (*cache, i32(ragged(counts)), i32(t0))
    gd = _gd()
    gd.kv_append_q4(dev(x), dev(-x), *args)
    k, v = gd.kv_read_q4(*args, n_rows=n)
    assert torch.equal(k, dev(x)) and torch.equal(v, -dev(x))
    pos = i32(sum(([s] * c for s, c in enumerate(counts)), []))
    assert (cache[2].view(n_seq, -1).ne(0).sum(1) == 4 * i32(counts)).all() and len(pos) == n


def test_bad_rows_are_flagged_and_skipped():
    gd = _gd()
    n_seq, Hk, cap, D = 3, 2, 16, 64
    x = torch.ones((6, Hk, D), device="cuda")

    def run(off, t0, n=6):
        z = lambda w: torch.zeros((n_seq, Hk, cap, w), dtype=torch.uint8, device="cuda")  # noqa: E731
        cache = [z(D // 2), z(D // 2), z(D // 16), z(D // 16)]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        gd.kv_append_q4(x[:n], x[:n], *cache, i32(off), i32(t0), err=err)
        k = torch.full((n, Hk, D), 7.0, device="cuda")
        v = k.clone()
        err2 = torch.zeros_like(err)
        gd.kv_read_q4(*cache, i32(off), i32(t0), k_out=k, v_out=v, err=err2)
        assert int(err) == int(err2)
        written = cache[2][:, 0, :, 0].ne(0).cpu().numpy()
        return int(err), written, (k[:, 0, 0] != 7.0).cpu().tolist()

    e, w, r = run([0, 2, 4, 6], [15, -1, 2147483647])
    assert e == gd.ERR_KVLEN_RANGE and w.sum() == 2 and w[0, 15] and w[1, 0]
    assert r == [True, False, False, True, False, False]
    e, w, r = run([1, 2, 4, 6], [0, 0, 0])              # does not start at 0
    assert e == gd.ERR_SEQ_RANGE and w.sum() == 5 and r == [False] + [True] * 5
    e, w, _ = run([0, 5, 2, 6], [0, 0, 0])              # does not ascend
    assert e & ~gd.ERR_SEQ_RANGE == 0 and w.sum() <= 6
    e, w, r = run([0, 2, 4, 99], [0, 0, 0])             # more rows than the batch has
    assert e == 0 and w.sum() == 6 and all(r)
    e, w, r = run([0, 0, 0, 0], [0, 0, 0])              # nothing to append
    assert e == 0 and w.sum() == 0 and not any(r)


# ------------------------------------------------------------------------------------ decode

def run_q4(q, cache, lens, seq_of=None, err=None, stream=None, **kw):
    return _gd().attn_decode_q4(dev(q), *map(dev, cache), i32(lens),
                                seq_of=None if seq_of is None else i32(seq_of), err=err,
                                stream=stream, **kw)


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 127, 128, 129, 500, 511, 512]


@pytest.mark.parametrize("chunk", [None, 64])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 1), (8, 4), (12, 1), (16, 1), (10, 2), (22, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_dense(D, H, Hk, chunk):
    rng = np.random.default_rng(100 * D + H)
    cap = 512
    cache = q4_cache(rng, LENS, Hk, cap, D)
    q = rows(rng, len(LENS), H, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    with forced_chunk(chunk):
        got = run_q4(q, cache, LENS, err=err).cpu().numpy()
    ref = oracle.decode_q4(q, *cache, LENS, D ** -0.5)
    assert_close(got, ref, TOL, f"D {D} H {H}/{Hk}")
    assert (got[0] == 0).all() and int(err) == 0


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (7, 4), (16, 0), (33, 20), (64, 16),
                                           (129, 1), (200, 300), (511, 5), (1000, 4),
                                           (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("chunk", [None, 64])
def test_decode_window(D, window, n_sink, chunk):
    """Hidden positions hold garbage too: only what a row sees may reach its output."""
    rng = np.random.default_rng(window % 9973 + D)
    cap, Hk, H = 512, 2, 8
    cache = q4_cache(rng, LENS, Hk, cap, D)
    for s, n in enumerate(LENS):
        m = hidden(n, window, n_sink)
        for x in cache:
            x[s, :, :n][:, m] = 0xff
    q = rows(rng, len(LENS), H, D)
    with forced_chunk(chunk):
        got = run_q4(q, cache, LENS, window=window, n_sink=n_sink).cpu().numpy()
    ref = oracle.decode_q4(q, *cache, LENS, D ** -0.5, window=window, n_sink=n_sink)
    assert_close(got, ref, TOL, f"window {window} sinks {n_sink} D {D}")


@pytest.mark.parametrize("H,Hk,T", [(12, 1, 1), (48, 4, 1), (16, 4, 2), (32, 4, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L", [1300, 2040])
def test_decode_lists_of_many_pieces(H, Hk, T, D, L):
    """Lists of 9 to 16 pieces of eight warps: few lists merge in clusters, eight by the last CTA."""
    rng = np.random.default_rng(H + D + L)
    lens = [L] * T
    cache = q4_cache(rng, lens, Hk, 2048, D)
    q = rows(rng, T, H, D)
    with forced_chunk(128):
        got = _gd().attn_decode_q4(dev(q), *map(dev, cache), i32(lens))
    assert_close(got.cpu().numpy(), oracle.decode_q4(q, *cache, lens, D ** -0.5), TOL, "pieces")


@pytest.mark.parametrize("ctas", [1, 3, 7, 40, 500])
@pytest.mark.parametrize("H,Hk,D", [(4, 1, 128), (16, 2, 128), (3, 3, 64), (12, 1, 256)])
def test_decode_balanced(H, Hk, D, ctas):
    """One wave of CTAs with equal shares of all lists: shares that hold several lists, lists over
    many shares, empty rows, a workspace used twice."""
    rng = np.random.default_rng(D + ctas)
    lens = [0, 1, 2100, 63, 64, 65, 0, 700, 512, 513, 1030, 0]
    cache = q4_cache(rng, lens, Hk, 2112, D)
    q = rows(rng, len(lens), H, D)
    gate = rows(rng, len(lens) * H * D)
    with forced_ctas(ctas):
        assert _gd().plan(len(lens), H, Hk, D, 2112, kind=_gd().KIND_Q4).streamk == 1
        ws = _gd().alloc_workspace(len(lens), H, Hk, D, 2112, kind=_gd().KIND_Q4)
        for window, n_sink in ((None, 0), (600, 70), (None, 0)):
            got = run_q4(q, cache, lens, window=window, n_sink=n_sink, ws=ws).cpu().numpy()
            ref = oracle.decode_q4(q, *cache, lens, D ** -0.5, window=window, n_sink=n_sink)
            assert_close(got, ref, TOL, f"{ctas} CTAs, window {window}")
            got = run_q4(q, cache, lens, window=window, n_sink=n_sink, ws=ws,
                         gate=dev(gate)).cpu().numpy()
            assert_close(got, oracle.output_gate(ref, gate.reshape(ref.shape)), TOL, "gate")


@pytest.mark.parametrize("H,Hk,D", [(8, 2, 128), (4, 4, 64), (32, 2, 64), (12, 2, 256), (7, 1, 128),
                                     (18, 2, 64), (22, 2, 128), (13, 1, 256)])
@pytest.mark.parametrize("window", [None, 100])
def test_decode_rows_sharing_sequences(H, Hk, D, window):
    """Causal rows of three sequences in runs, rows out of order, one sequence named twice."""
    rng = np.random.default_rng(H + D)
    seq = [2] * 19 + [0] * 3 + [1] * 8 + [2] * 2 + [0, 1, 0]
    lens = list(range(401, 420)) + [5, 0, 1] + list(range(90, 98)) + [420, 300, 9, 64, 9]
    cache = q4_cache(rng, [16, 120, 430], Hk, 432, D)
    q = rows(rng, len(seq), H, D)
    ref = oracle.decode_q4(q, *cache, lens, D ** -0.5, seq_of=seq, window=window, n_sink=3)
    # the kernel for 128 pairs a CTA (not at D = 256) and the one for up to 8, split and not
    for rows_env, chunk in (("on", None), (None, None), ("off", 96)):
        with _env(GQA_Q4_ROWS=rows_env), forced_chunk(chunk):
            got = run_q4(q, cache, lens, seq, window=window, n_sink=3).cpu().numpy()
        assert_close(got, ref, TOL, f"shared sequences, {rows_env}, {chunk}")


@pytest.mark.parametrize("H,Hk,D", [(2, 2, 64), (8, 2, 128), (32, 2, 128), (12, 2, 64), (6, 2, 256)])
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
    last = [max([n for n, t in zip(lens, seq) if t == s] + [0]) for s in range(5)]
    cache = q4_cache(rng, last, Hk, 960, D, 0.5, 4.0)
    q = rows(rng, 300, H, D) * np.float32(3)
    gate = rows(rng, 300 * H * D)
    for window, n_sink, scale in ((None, 0, D ** -0.5), (150, 4, D ** -0.5), (33, 200, -0.1)):
        for T in (300, 40):
            with _env(GQA_Q4_ROWS="on"):
                got = run_q4(q[:T], cache, lens[:T], seq[:T], window=window, n_sink=n_sink,
                             scale=scale, k_scale=0.5, v_scale=4.0,
                             gate=dev(gate[:T * H * D])).cpu().numpy()
            ref = oracle.decode_q4(q[:T], *cache, lens[:T], scale, seq_of=seq[:T], window=window,
                                   n_sink=n_sink, k_scale=0.5, v_scale=4.0)
            ref = oracle.output_gate(ref, gate[:T * H * D].reshape(ref.shape))
            # values of v_scale 4: four times the error; scores of 3 q: three times
            assert_close(got / 4, ref / 4, 3 * TOL, f"window {window} rows {T}")


def test_prompt_chunk_scales_and_zero_scale():
    """A chunk of causal rows on the kernel for 128 pairs: queries and cache scales far from 1, a
    softmax scale of 0 (the mean of what is seen), a NaN query."""
    rng = np.random.default_rng(21)
    T, H, Hk, D = 40, 8, 2, 128
    lens = [100 + r for r in range(T)]
    cache = q4_cache(rng, [140], Hk, 144, D, 2.0 ** -20, 2.0 ** 30)
    q = rows(rng, T, H, D)
    for qmul, scale in ((2.0 ** 30, 2.0 ** -10 * D ** -0.5), (2.0 ** -30, 2.0 ** 50 * D ** -0.5),
                        (1.0, 0.0)):
        kw = dict(scale=scale, k_scale=2.0 ** -20, v_scale=2.0 ** 30)
        with _env(GQA_Q4_ROWS="on"):
            got = run_q4(q * np.float32(qmul), cache, lens, [0] * T, **kw).cpu().numpy()
        ref = oracle.decode_q4(q * np.float32(qmul), *cache, lens, seq_of=[0] * T, **kw)
        assert_close(got / 2.0 ** 30, ref / 2.0 ** 30, TOL, f"q times {qmul}")
    q[3, 2, 5] = np.nan
    with _env(GQA_Q4_ROWS="on"):
        got = run_q4(q, cache, lens, [0] * T, k_scale=2.0 ** -20, v_scale=2.0 ** 30).cpu().numpy()
    assert np.isnan(got[3, 2]).all()
    got[3, 2] = 0
    assert np.isfinite(got).all()


@pytest.mark.parametrize("k_scale,v_scale,scale,qmul", [
    (2.0 ** -12, 2.0 ** 9, 0.125 * 2 ** 12, 1.0), (2.0 ** 40, 1.0, 2.0 ** -43, 1.0),
    (1.0, 2.0 ** -30, 2.0 ** -20, 2.0 ** 17), (1.0, 1.0, 0.125 * 2 ** 30, 2.0 ** -30)])
def test_decode_scales(k_scale, v_scale, scale, qmul):
    """Scales and queries far from 1: the products keep their precision (the result divided by
    v_scale is the well-scaled problem's)."""
    rng = np.random.default_rng(4)
    cache = q4_cache(rng, [200, 77], 2, 208, 64, k_scale, v_scale)
    q = rows(rng, 2, 8, 64) * np.float32(qmul)
    got = run_q4(q, cache, [200, 77], scale=scale, k_scale=k_scale, v_scale=v_scale).cpu().numpy()
    ref = oracle.decode_q4(q, *cache, [200, 77], scale, k_scale=k_scale, v_scale=v_scale)
    assert_close(got / v_scale, ref / v_scale, TOL, "scales")


@pytest.mark.parametrize("chunk", [None, 64])
def test_decode_nan_query(chunk):
    """A row with a NaN in q comes out as NaN, the others as they are; an empty one as zeros."""
    rng = np.random.default_rng(14)
    lens = [300, 300, 0]
    cache = q4_cache(rng, lens, 2, 304, 128)
    q = rows(rng, 3, 8, 128)
    q[0, 1, 77] = q[2, 1, 3] = np.nan
    with forced_chunk(chunk):
        got = run_q4(q, cache, lens).cpu().numpy()
    assert np.isnan(got[0, 1]).all() and (got[2] == 0).all()
    ref = oracle.decode_q4(np.nan_to_num(q), *cache, lens, 128 ** -0.5)
    got[0, 1] = ref[0, 1]
    assert_close(got, ref, TOL, "NaN query")


def test_decode_over_nothing_and_tiny_caches():
    """max_kv_len 0, no rows, and caches of 16 positions under many rows."""
    rng = np.random.default_rng(15)
    cache = q4_cache(rng, [16], 2, 16, 128)
    q = rows(rng, 200, 8, 128)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_q4(q[:1], cache, [0], max_kv_len=0, err=err)
    assert (got == 0).all() and int(err) == 0
    assert run_q4(q[:0], cache, []).shape == (0, 8, 128)
    lens = [int(n) for n in rng.integers(0, 17, 200)]
    for env in ("on", "off"):
        with _env(GQA_Q4_ROWS=env):
            got = run_q4(q, cache, lens, [0] * 200, err=err).cpu().numpy()
        assert_close(got, oracle.decode_q4(q, *cache, lens, 128 ** -0.5, seq_of=[0] * 200), TOL, env)
    assert int(err) == 0


def test_first_call_is_captured():
    """A fresh process whose first call of each kernel is inside a capture."""
    import subprocess
    import sys
    code = """
import torch
from gqa_decode_attention_03_gb300 import gqa_decode as gd
z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
cache = [z(1, 8, 8192, 64), z(1, 8, 8192, 64), z(1, 8, 8192, 8), z(1, 8, 8192, 8)]
k = torch.ones(40, 8, 128, device="cuda")
q, out = torch.ones(40, 32, 128, device="cuda"), torch.zeros(40, 32, 128, device="cuda")
f = torch.ones(1, 8192, 8, 128, dtype=torch.float16, device="cuda")
off, t0, n, s = i(0, 40), i(0), i(*[40] * 40), i(*[0] * 40)
ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
outs = [torch.zeros_like(out) for _ in range(4)]
with torch.cuda.graph(g):
    gd.kv_append_q4(k, k, *cache, off, t0)
    gd.attn_decode_q4(q[:1], *cache, n[:1], out=outs[0][:1], ws=ws)
    gd.attn_decode_q4(q, *cache, n, seq_of=s, out=outs[1], ws=ws)
    gd.attn_decode_f16_window(q[:1], f, f, n[:1], 5000, 4, out=outs[2][:1], ws=ws)
    gd.attn_decode_f16_window(q, f, f, n, 30, 4, seq_of=s, out=outs[3], ws=ws)
g.replay()
torch.cuda.synchronize()
v = gd.kv_read_q4(*cache, off, t0, n_rows=40)[1][0, 0, 0].item()  # 1 = code x scale e4m3(1 / 6)
assert abs(v - 1) < 0.1
for o, rows, x in zip(outs, (1, 40, 1, 40), (v, v, 1, 1)):
    assert (o[:rows] - x).abs().max().item() < 1e-4, (rows, x)
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_decode_bad_lengths_and_sequences():
    gd = _gd()
    rng = np.random.default_rng(5)
    cache = q4_cache(rng, [48, 48], 1, 48, 64)
    q = rows(rng, 5, 4, 64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_q4(q, cache, [-3, 49, 20, 20, 20], [0, 1, 2, -1, 1], err=err).cpu().numpy()
    assert int(err) == gd.ERR_KVLEN_RANGE | gd.ERR_SEQ_RANGE
    ref = oracle.decode_q4(q, *cache, [0, 48, 0, 0, 20], 0.125, seq_of=[0, 1, 0, 0, 1])
    assert_close(got, ref, TOL, "clamped rows")
    err.zero_()
    got = run_q4(q[:1], cache, [40], [0], err=err, max_kv_len=24).cpu().numpy()
    assert int(err) == gd.ERR_KVLEN_RANGE
    assert_close(got, oracle.decode_q4(q[:1], *cache, [24], 0.125), TOL, "max_kv_len")


@pytest.mark.parametrize("stride", [None, 200])
def test_decode_gate(stride):
    rng = np.random.default_rng(6)
    lens = [0, 300, 37]
    cache = q4_cache(rng, lens, 2, 304, 128)
    q = rows(rng, 3, 8, 128)
    w = stride or 128
    gate = rows(rng, 24 * w)
    ref = oracle.decode_q4(q, *cache, lens, 128 ** -0.5)
    ref = oracle.output_gate(ref, gate.reshape(3, 8, w)[..., :128])
    for chunk in (None, 64):
        with forced_chunk(chunk):
            got = run_q4(q, cache, lens, gate=dev(gate), gate_stride=stride).cpu().numpy()
        assert_close(got, ref, TOL, "gate")


def test_serving_loop():
    """Prompts go into the cache, then every step appends a token per live sequence and attends
    through window and sinks, in a captured graph whose inputs change from step to step; the cache
    read back is what the oracle holds."""
    gd = _gd()
    rng = np.random.default_rng(12)
    n_seq, H, Hk, D, cap, window, n_sink = 5, 8, 2, 128, 160, 40, 4
    prompt = [100, 1, 63, 0, 17]
    z = lambda w: torch.zeros((n_seq, Hk, cap, w), dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = [z(D // 2), z(D // 2), z(D // 16), z(D // 16)]
    hold = [np.zeros((n_seq, Hk, cap, w), np.uint8) for w in (D // 2, D // 2, D // 16, D // 16)]

    def put(k, v, counts, t0):
        off = ragged(counts)
        for side, x in ((0, k), (1, v)):
            q, s = oracle.quantize_q4(x)
            for i, (c, t) in enumerate(zip(counts, t0)):
                hold[side][i, :, t:t + c] = q[off[i]:off[i] + c].transpose(1, 0, 2)
                hold[2 + side][i, :, t:t + c] = s[off[i]:off[i] + c].transpose(1, 0, 2)

    k, v = rows(rng, sum(prompt), Hk, D), rows(rng, sum(prompt), Hk, D)
    gd.kv_append_q4(dev(k), dev(v), *cache, i32(ragged(prompt)), i32([0] * n_seq))
    put(k, v, prompt, [0] * n_seq)
    # the step's buffers, its workspace and its graph
    k_new = torch.zeros((n_seq, Hk, D), device="cuda")
    v_new, q = torch.zeros_like(k_new), torch.zeros((n_seq, H, D), device="cuda")
    off, t0, lens = i32([0] * (n_seq + 1)), i32([0] * n_seq), i32([0] * n_seq)
    out = torch.empty_like(q)
    ws = gd.alloc_workspace(n_seq, H, Hk, D, cap, window + n_sink, gd.KIND_Q4)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        gd.kv_append_q4(k_new, v_new, *cache, off, t0, err=err)
        gd.attn_decode_q4(q, *cache, lens, window=window, n_sink=n_sink, out=out, ws=ws, err=err)

    step()                                              # warm up: no rows, no positions
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    n = list(prompt)
    for it in range(6):
        live = [int(s != it % n_seq) for s in range(n_seq)]
        c = sum(live)
        x = rows(rng, 3, n_seq, Hk, D)
        k_new.copy_(dev(x[0]))
        v_new.copy_(dev(x[1]))
        off.copy_(i32(ragged(live)))
        t0.copy_(i32(n))
        put(x[0, :c], x[1, :c], live, n)
        n = [a + b for a, b in zip(n, live)]
        lens.copy_(i32(n))
        qh = rows(rng, n_seq, H, D)
        q.copy_(dev(qh))
        graph.replay()
        ref = oracle.decode_q4(qh, *hold, n, D ** -0.5, window=window, n_sink=n_sink)
        assert_close(out.cpu().numpy(), ref, TOL, f"step {it}")
    assert int(err) == 0
    for got, ref in zip(cache, hold):
        assert np.array_equal(got.cpu().numpy(), ref)
    kk, vv = gd.kv_read_q4(*cache, i32(ragged(n)), i32([0] * n_seq), n_rows=sum(n),
                           dtype=torch.float16)
    for got, a, b in ((kk, hold[0], hold[2]), (vv, hold[1], hold[3])):
        ref = np.concatenate([oracle.dequant_q4(a[s, :, :n[s]], b[s, :, :n[s]]).transpose(1, 0, 2)
                              for s in range(n_seq)])
        assert np.array_equal(got.cpu().numpy(), ref.astype(np.float16))


def test_other_stream_and_shared_workspace():
    """Calls of different shapes on one workspace and one side stream, the first ones' outputs kept."""
    gd = _gd()
    rng = np.random.default_rng(9)
    side = torch.cuda.Stream()
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device="cuda")
    todo = []
    for H, Hk, D, lens in ((8, 2, 128, [700, 3]), (16, 1, 64, [650] * 4), (4, 2, 256, [1]),
                           (8, 2, 128, [5, 699])):
        cache = q4_cache(rng, lens, Hk, 704, D)
        q = rows(rng, len(lens), H, D)
        args = [dev(q), *map(dev, cache), i32(lens)]
        todo.append((args, oracle.decode_q4(q, *cache, lens, D ** -0.5)))
    torch.cuda.synchronize()
    with forced_chunk(128):
        got = [gd.attn_decode_q4(*a, ws=ws, stream=side) for a, _ in todo]
    side.synchronize()
    for g, (_, ref) in zip(got, todo):
        assert_close(g.cpu().numpy(), ref, TOL, "side stream")


def test_calls_of_every_kind_share_a_workspace():
    """Dense and windowed f16 layers, 4-bit ones, rows of one sequence, more rows and fewer: one after
    another on one workspace, each over what the ones before have left there."""
    gd = _gd()
    rng = np.random.default_rng(14)
    Hk, H, D, cap, T = 2, 8, 128, 1200, 48
    lens = [int(n) for n in rng.integers(0, cap + 1, T)]
    lens[:3] = [cap, 0, 1100]
    kv = [(rows(rng, T, cap, Hk, D)).astype(np.float16) for _ in range(2)]
    cache = q4_cache(rng, lens, Hk, cap, D)
    q = rows(rng, T, H, D)
    qd, kd, vd, cd = dev(q), dev(kv[0]), dev(kv[1]), list(map(dev, cache))
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    scale = D ** -0.5

    def dense(n):
        out = gd.attn_decode_f16(qd[:n], kd, vd, i32(lens[:n]), ws=ws)
        return out, oracle.decode_f16(q[:n], *kv, lens[:n], scale)

    def window(n):
        out = gd.attn_decode_f16_window(qd[:n], kd, vd, i32(lens[:n]), 700, 4, ws=ws)
        return out, oracle.decode_f16_window(q[:n], *kv, lens[:n], scale, 700, 4)

    def shared(n):
        seq, ln = [0] * n, list(range(cap - n + 1, cap + 1))
        with _env(GQA_F16_ROWS="on"):
            out = gd.attn_decode_f16_window(qd[:n], kd[:1], vd[:1], i32(ln), 700, 4, seq_of=i32(seq),
                                            ws=ws)
        return out, oracle.decode_f16_window(q[:n], *kv, ln, scale, 700, 4, seq_of=seq)

    def q4(n):
        out = gd.attn_decode_q4(qd[:n], *cd, i32(lens[:n]), ws=ws)
        return out, oracle.decode_q4(q[:n], *cache, lens[:n], scale)

    def q4_shares(n):
        with forced_ctas(40):
            return q4(n)

    def q4_shared(n):
        seq, ln = [0] * n, list(range(lens[2] - n + 1, lens[2] + 1))
        one = [x[2:3] for x in cd]
        with _env(GQA_Q4_ROWS="on"):
            out = gd.attn_decode_q4(qd[:n], *one, i32(ln), seq_of=i32(seq), ws=ws)
        return out, oracle.decode_q4(q[:n], *[x[2:3] for x in cache], ln, scale, seq_of=seq)

    # (a dense call counts on zeros where its counters lie, which partials of a call of fewer rows reach)
    want = [(f, n) for f in (dense, window, q4, shared, q4_shared) for n in (6, T)]
    want = [w for w in want if w != (dense, T)] + [(q4, 6), (dense, 6), (window, T), (q4, T)]
    order = [want[i % len(want)] for i in rng.permutation(2 * len(want))]
    for step, (f, n) in enumerate(order):
        with forced_chunk(128):
            got, ref = f(n)
        assert_close(got.cpu().numpy(), ref, TOL, f"step {step}: {f.__name__} of {n} rows")
        if step % 3 == 0:
            got, ref = q4_shares(n)
            assert_close(got.cpu().numpy(), ref, TOL, f"step {step}: shares of {n} rows")


def test_a_call_makes_its_tensors_on_its_own_stream():
    """No output, no workspace given: the current stream is busy while the side stream's call runs, and
    the memory held other bytes before."""
    gd = _gd()
    rng = np.random.default_rng(12)
    side, D, lens = torch.cuda.Stream(), 128, [700, 0, 90]
    cache = q4_cache(rng, lens, 2, 704, D)
    q = rows(rng, 3, 8, D)
    ref = oracle.decode_q4(q, *cache, lens, D ** -0.5)
    args = [dev(q), *map(dev, cache), i32(lens)]
    off, t0 = i32([0, 3, 3, 3]), i32([5, 0, 0])
    with torch.cuda.stream(side):
        poison = torch.full((4 << 20,), 255, dtype=torch.uint8, device="cuda")
        poison2 = torch.full((64 << 10,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del poison, poison2
    with forced_chunk(128):
        torch.cuda._sleep(20_000_000)
        got = gd.attn_decode_q4(*args, stream=side)
        k, _ = gd.kv_read_q4(*args[1:5], off, t0, n_rows=5, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        got, k = got.cpu().numpy(), k.cpu().numpy()
    assert_close(got, ref, TOL, "side stream")
    kd = oracle.dequant_q4(cache[0][0, :, 5:8], cache[2][0, :, 5:8]).transpose(1, 0, 2)
    assert np.array_equal(k, np.concatenate([kd, np.zeros((2, 2, D))]).astype(np.float32))


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes of codes a side; only the last head's last positions and its
    first ones are seen."""
    gd = _gd()
    Hk, D, cap = 72, 256, 1 << 19                       # 72 x 2^19 x 128 bytes = 4.8 GB a side
    z = lambda w: torch.zeros((1, Hk, cap, w), dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = [z(D // 2), z(D // 2), z(D // 16), z(D // 16)]
    rng = np.random.default_rng(1)
    n = 40
    x = rows(rng, 2, n, Hk, D)
    for t0 in (0, cap - n):
        gd.kv_append_q4(dev(x[0]), dev(x[1]), *cache, i32([0, n]), i32([t0]))
        k, v = gd.kv_read_q4(*cache, i32([0, n]), i32([t0]), n_rows=n)
        for got, side in ((k, 0), (v, 1)):
            assert np.array_equal(got.cpu().numpy(),
                                  oracle.dequant_q4(*oracle.quantize_q4(x[side])))
    q = rows(rng, 1, Hk, D)
    got = gd.attn_decode_q4(dev(q), *cache, i32([cap]), window=n, n_sink=n).cpu().numpy()
    kd = oracle.dequant_q4(*oracle.quantize_q4(x[0])).transpose(1, 0, 2)
    vd = oracle.dequant_q4(*oracle.quantize_q4(x[1])).transpose(1, 0, 2)
    for h in (0, 35, 71):
        ref = oracle.attend_positions(q[0, h:h + 1], np.concatenate([kd[h], kd[h]]),
                                      np.concatenate([vd[h], vd[h]]), D ** -0.5)
        assert_close(got[0, h:h + 1], ref, TOL, f"head {h}")


def test_binding_refuses():
    gd = _gd()
    rng = np.random.default_rng(2)
    kq, vq, ksc, vsc = map(dev, q4_cache(rng, [16], 1, 16, 64))
    q, n = dev(rows(rng, 1, 4, 64)), i32([16])
    x = dev(rows(rng, 1, 1, 64))
    off, t0 = i32([0, 1]), i32([0])
    bad = [lambda: gd.attn_decode_q4(q.half(), kq, vq, ksc, vsc, n),
           lambda: gd.attn_decode_q4(q, kq.cpu(), vq, ksc, vsc, n),
           lambda: gd.attn_decode_q4(q, kq, vq, ksc[..., :2], vsc, n),
           lambda: gd.attn_decode_q4(q, kq, vq, ksc, vsc, i32([1, 2])),
           lambda: gd.attn_decode_q4(q, kq, vq, ksc, vsc, n, seq_of=i32([0, 0])),
           lambda: gd.attn_decode_q4(q, kq, vq, ksc, vsc, n, out=q),
           lambda: gd.attn_decode_q4(q, kq, vq, ksc, vsc, n, out=torch.empty_like(q)[:, :2]),
           lambda: gd.attn_decode_q4(q, kq, vq, ksc, vsc, n, window=-4),
           lambda: gd.attn_decode_q4(q, kq, vq, ksc, vsc, n, window=1 << 31),
           lambda: gd.attn_decode_q4(q, kq, vq, ksc, vsc, n, k_scale=0.3),
           lambda: gd.attn_decode_q4(q, kq, vq, ksc, vsc, n, gate=q[..., :32].contiguous()),
           lambda: gd.attn_decode_q4(q[..., :32].contiguous(), kq, vq, ksc, vsc, n),
           lambda: gd.kv_append_q4(x.double(), x, kq, vq, ksc, vsc, off, t0),
           lambda: gd.kv_append_q4(x, x[:, :, :32], kq, vq, ksc, vsc, off, t0),
           lambda: gd.kv_append_q4(x, x, kq, vq, ksc, vsc, off[:1], t0),
           lambda: gd.kv_append_q4(x, x, kq, vq, ksc, vsc, off, off),
           lambda: gd.kv_append_q4(x, x, kq, vq, ksc, vsc, off.long(), t0),
           lambda: gd.kv_append_q4(x, x, kq, vq, ksc, vsc, off, t0, v_scale=-1.0),
           lambda: gd.kv_read_q4(kq, vq, ksc, vsc, off, t0),
           lambda: gd.kv_read_q4(kq, vq, ksc, vsc, off, t0, k_out=x),
           lambda: gd.kv_read_q4(kq, vq, ksc, vsc, off, t0, n_rows=1, dtype=torch.bfloat16),
           lambda: gd.kv_read_q4(kq, vq, ksc, vsc, off, t0, k_out=x, v_out=x.half())]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, gd.GqaError)):
            call()
            pytest.fail(f"call {i} went through")
