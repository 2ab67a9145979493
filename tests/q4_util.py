"""Inputs of the 4-bit cache and window tests: host arrays, seeded, with garbage in every place that
no row sees."""

import numpy as np

import oracle

# Tolerance of the windowed and 4-bit decode calls, |gpu - ref| <= TOL * max(1, |ref|).  Both sides
# hold the same cache values exactly; q and the softmax weights go through the matrix products as
# f16 hi + lo pairs (2^-22 of each), the sums are fp32.  A score is a sum of D <= 256 products that
# add up to at most ~40 in log2 units here (q, k ~ N(0, 1), scale <= 1/8), accumulated in steps of
# 16: its error stays below (256 / 16 + 16) 2^-24 40 < 1e-4 in the worst case and near 1e-6 as the
# roundings fall; a weight's relative error is ln 2 times that and the output a mean of values of
# size ~1 under those weights.
TOL = 1e-4


def rows(rng, *shape):
    return rng.standard_normal(shape).astype(np.float32)


def q4_cache(rng, lens, Hk, cap, D, k_scale=1.0, v_scale=1.0):
    """A quantised cache [n_seq][Hk][cap] whose positions past each sequence's length hold garbage
    (every byte value, the scale codes that the format does not use among them)."""
    n_seq = len(lens)
    kq, ksc = oracle.quantize_q4(rows(rng, n_seq, Hk, cap, D) * k_scale, k_scale)
    vq, vsc = oracle.quantize_q4(rows(rng, n_seq, Hk, cap, D) * v_scale, v_scale)
    for s, n in enumerate(lens):
        for x in (kq, ksc, vq, vsc):
            x[s, :, n:] = rng.integers(0, 256, x[s, :, n:].shape, dtype=np.uint8)
        ksc[s, :, n:, 0] = 0x7f
        vsc[s, :, n:, 0] = 0xff
    return kq, vq, ksc, vsc


def hidden(n, window, n_sink):
    """Mask of the positions below n that a row of length n does not see."""
    see = np.zeros(n, bool)
    see[oracle.visible_positions(n, window, n_sink)] = True
    return ~see
