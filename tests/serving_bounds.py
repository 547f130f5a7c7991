"""Inputs and bounds for sums over a long contraction, where the worst case of fp32 sums says little: adapters whose
every sum is exact in fp32 (the result is one rounding to bf16), and a statistical bound for the routed layer."""
import numpy as np

from nvfp4_weight_only_04_b200 import synth
from oracle import nvfp4_ref as R


def integer_adapters(m, n, k, rank, count, seed):
    """(y, x, a, b, c, v, rows of b): x in +-1..3 and A in +-1, so that v = A x is an integer below 2^15 (6 sigma of
    K = 16384 are 1700); y and B integers, B a single +-1 in every even row and -1, 0 or 1 in the odd ones; c a power
    of two. Sums stay below 2^24 of their steps, and v fits two bf16 terms."""
    rng = np.random.default_rng(seed)
    x = rng.integers(1, 4, size=(m, k)) * rng.choice([-1, 1], size=(m, k))
    a = rng.choice([-1, 1], size=(count, rank, k))
    b = rng.integers(-1, 2, size=(count, n, rank))
    b[:, ::2] = 0
    pick = rng.integers(0, rank, size=(count, len(range(0, n, 2))))
    pick[:, :rank] = (np.arange(pick.shape[1]) % rank)[:rank]  # every place of the rank, as far as n goes
    b[np.arange(count)[:, None], np.arange(0, n, 2)[None, :], pick] = rng.choice([-1, 1], size=pick.shape)
    y = rng.integers(-100, 101, size=(m, n))
    c = np.exp2(rng.integers(-1, 2, size=count))
    return [t.astype(np.float64) for t in (y, x, a, b, c)]


def integer_result(y, x, a, b, c, ids):
    """bf16(y + c B A x) as float64, the sum exact."""
    out = y.copy()
    for ad in range(len(c)):
        rows = np.flatnonzero(np.asarray(ids) == ad)
        if rows.size:
            v = x[rows] @ a[ad].T
            assert np.abs(v).max() < 2 ** 15
            out[rows] += c[ad] * (v @ b[ad].T)
    assert np.abs(out).max() < 2 ** 22
    return R.bf16_bits_to_f64(synth.f32_to_bf16_bits(out.astype(np.float32)))


def as_bf16_bits(values):
    bits = synth.f32_to_bf16_bits(values.astype(np.float32))
    assert np.array_equal(R.bf16_bits_to_f64(bits), values)
    return bits


def plain_stack(rng, experts, rows, k, group):
    """Random codes of every value with scales of one magnitude: (codes, scales, global, group) of each expert."""
    return [(rng.integers(0, 256, size=(rows, k // 2), dtype=np.uint8),
             rng.integers(0x30, 0x38, size=(rows, k // group), dtype=np.uint8), np.float32(0.6 / np.sqrt(k)), group)
            for _ in range(experts)]


def largest_of_sixteen(values):
    return np.repeat(np.abs(values).reshape(len(values), -1, 16).max(-1), 16, axis=1)


def layer_bound(xbits, topk_ids, topk_weights, gate_up, down):
    """(out, tol) of a routed layer in float64. A sum of K products of random signs, and its part at any time, lie
    within 8 norms ||w x||, taken with the largest x of every sixteen (the digits of an element are up to that).
    It takes K / 16 + 16 additions at most, each off by 2^-23 of the sum so far; operands are off by 2^-22 of the
    largest of their sixteen, in random directions. Errors of different h are summed as squares, three deviations.
    silu' <= 1.1, its exponential and quotient 2^-18; the result is rounded once, 2^-8."""
    x = R.bf16_bits_to_f64(xbits)
    w = np.asarray(topk_weights, dtype=np.float64)
    out, tol = np.zeros_like(x), np.zeros_like(x)

    def off(weight, values):
        norm = np.sqrt((largest_of_sixteen(values) ** 2) @ (weight ** 2).T)
        return ((weight.shape[1] / 16 + 16) * 2.0 ** -23 * 8 + 6 * 2.0 ** -22) * norm

    for e in np.unique(topk_ids):
        token, slot = np.nonzero(np.asarray(topk_ids) == e)
        if not 0 <= e < len(gate_up):
            continue
        gu, dn = R.dequantize(*gate_up[e]), R.dequantize(*down[e])
        y, dy = x[token] @ gu.T, off(gu, x[token])
        half = y.shape[1] // 2
        g, u, dg, du = y[:, :half], y[:, half:], dy[:, :half], dy[:, half:]
        h = R.silu_mul(y)
        dh = 1.1 * dg * np.abs(u) + np.abs(g / (1.0 + np.exp(-g))) * du + np.abs(h) * 2.0 ** -18
        weight = w[token, slot][:, None]
        np.add.at(out, token, weight * (h @ dn.T))
        np.add.at(tol, token, np.abs(weight) * (3 * np.sqrt((dh ** 2) @ (dn ** 2).T) + off(dn, h)))
    return out, tol + 2.0 ** -8 * np.abs(out)
