"""Shared pieces of the cache operators' GPU tests: 4-bit pools, and tolerances worked out from the arithmetic.

Tolerances.  A logit x = scale * sum_d q_d k_d comes of exact products added up in fp32, D terms at most half a step
(2^-24, doubled for an adder that truncates) of the running sum each, which sum_d |q_d k_d| bounds; the scaling adds
two roundings:  dx = (D + 4) 2^-23 scale sum_d |q_d k_d|.  exp turns that into a relative error, once in the weight
and once in the denominator, beside a few units of 2^-22 for exp2 and the division: dw = 2 dx + 2^-19.
An output sum_t w v adds the rounding of the weights to the product's type and of the result to bf16, each half a
step, finfo.eps / 2 (`p_step`: bf16, whose steps are 2^-7 of a value, 2^-8; f16, whose steps are 2^-10, 2^-11):
(dw + p_step) sum_t w |v| + 2^-8 |out|.  The 4-bit decode multiplies in f16 while V's scales stay within eight powers
of two, and in bf16 where they do not, blocks of zeros (scale byte 0) among them.  Halves below 2^-14 have fewer bits:
that adds n 2^-32 6 2^(window's top - 127) to an output's error (test_gpu_mx4_light_tokens.py derives it), which these
tolerances leave out: rows whose heavy tokens have ordinary values stay far below it.
"""
import numpy as np
import torch

from oracle import cache_ops as C

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2
F16_HALF = torch.finfo(torch.float16).eps / 2


def logit_error(D, scale, size):
    """dx of the worst token, per query head (size: the largest sum_d |q_d k_d|)."""
    return (D + 4) * 2.0 ** -23 * scale * size


def weight_tolerance(D, scale, size):
    return 2 * logit_error(D, scale, size) + 2.0 ** -19


def check_out(got, want, reach, size, D, scale, p_step, what=""):
    """got, want [H_q][D] of one row."""
    tol = (weight_tolerance(D, scale, size)[:, None] + p_step) * reach + BF16_HALF * np.abs(want) + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - want).max()), float(tol.min()))


def check_scores(got, before, weights, size, D, scale, what=""):
    """got, before, weights [H_kv][N] of one row: before + weights, with the relative error of every weight and one
    rounding of the sum (and one per added head)."""
    tol = weight_tolerance(D, scale, size.max() if size.size else 0.0) * weights + 2.0 ** -22 * (np.abs(before) + weights)
    bad = ~(np.abs(got - (before + weights)) <= tol + 1e-37)
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - before - weights).max()))


def scattered_table(rng, lens, max_pages, spare=3):
    """(block_table int32 [B][max_pages], pages): every row's pages scattered; entries past a row's last page are
    out of range, so reading one would show."""
    pages = sum(-(-n // 16) for n in lens) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), max_pages), 2 ** 30, np.int32)
    at = 0
    for i, n in enumerate(lens):
        k = -(-n // 16)
        table[i, :k] = order[at:at + k]
        at += k
    return table, pages


def mx4_pool(rng, pages, H, D, spread=0, zeros=0.0):
    """uint8 [pages][H][17 D] of random codes; scale bytes near 127, or uniform over 127 +- spread; a share `zeros` of
    the scale blocks holds zeros (scale byte 0)."""
    pool = rng.integers(0, 256, (pages, H, 17 * D)).astype(np.uint8)
    scales = 125 + rng.integers(0, 3, (pages, H, D)) if not spread else \
        127 + rng.integers(-spread, spread + 1, (pages, H, D))
    pool[:, :, 16 * D:] = np.where(rng.random((pages, H, D)) < zeros, 0, scales)
    return pool


def poison_tails(pool, table, lens):
    """NaN scales in every slot past a row's last token and in every page no row uses."""
    pages, H, R = pool.shape
    D = R // 17
    live = np.zeros((pages, 16), bool)
    for i, n in enumerate(lens):
        for t in range(n):
            live[table[i, t // 16], t % 16] = True
    scales = pool[:, :, 16 * D:].reshape(pages, H, 2, 16, D // 32)
    scales[np.broadcast_to(~live[:, None, None, :, None], scales.shape)] = 255


def mx4_rows(pool, table, lens, i):
    """float64 K and V [H][N][D] of row i."""
    H = pool.shape[1]
    n = lens[i]
    return tuple(np.stack([C.row_values(pool, table[i], n, h, is_v) for h in range(H)]) for is_v in (False, True))
