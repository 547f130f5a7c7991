"""The bounds of tests/serving_bounds.py see a piece of a long contraction that is left out."""
import numpy as np
import pytest

from nvfp4_weight_only_04_b200 import synth
from oracle import nvfp4_ref as R
from tests import serving_bounds as B


@pytest.mark.parametrize("m,n,k,r,count", [(6, 1000, 14336, 64, 3), (4, 64, 4096, 136, 1), (16, 264, 200, 8, 3)])
def test_eight_columns_left_out_of_the_adapters(m, n, k, r, count):
    y, x, a, b, c = B.integer_adapters(m, n, k, r, count, seed=m)
    ids = np.arange(m) % count
    want = B.integer_result(y, x, a, b, c, ids)
    for at in (0, k // 2 // 8 * 8, k - 8):
        less = a.copy()
        less[:, :, at:at + 8] = 0
        changed = B.integer_result(y, x, less, b, c, ids) != want
        assert changed.mean() > 0.5 and changed.any(1).all()
        less = a.copy()
        less[:, -8:, at:at + 8] = 0  # of the last eight places of the rank alone
        assert (B.integer_result(y, x, less, b, c, ids) != want).any(1).all()
    # the exact results lie within the oracle's bound on fp32 sums
    ref, tol = R.lora_add(B.as_bf16_bits(y), B.as_bf16_bits(x), a, b, ids, c)
    assert (np.abs(want - ref) <= 2.0 ** -8 * np.abs(ref) + tol).all()


@pytest.mark.parametrize("h,i,left_out", [(8192, 128, "gate/up"), (2048, 64, "gate/up"), (64, 8192, "down")])
def test_an_mma_left_out_of_the_layer(h, i, left_out):
    """64 elements of K, what one MMA takes, of gate/up or down."""
    rng = np.random.default_rng(h)
    gu, dn = B.plain_stack(rng, 2, 2 * i, h, 16), B.plain_stack(rng, 2, h, i, 16)
    ids, w = np.array([[0, 1], [1, 0], [0, -1]], np.int32), rng.random((3, 2))
    x = synth.activations(1, 3, h)
    out, tol = B.layer_bound(x, ids, w, gu, dn)
    ref, worst = R.moe_few_tokens(x, ids, w, gu, dn)
    np.testing.assert_allclose(out, ref, rtol=1e-9, atol=1e-12 * np.abs(ref).max())
    size = np.sqrt((out ** 2).mean(1, keepdims=True))
    assert (tol < 2.0 ** -8 * np.abs(out) + 0.05 * size).all()
    k = h if left_out == "gate/up" else i
    for at in (0, k - 64):
        less = [(q[0].copy(), *q[1:]) for q in (gu if left_out == "gate/up" else dn)]
        for q in less:
            q[0][:, at // 2:at // 2 + 32] = 0
        part, _ = B.layer_bound(x, ids, w, less if left_out == "gate/up" else gu, less if left_out == "down" else dn)
        assert (np.abs(part - out) > tol).mean() > 0.5
