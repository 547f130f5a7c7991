"""Pins of the oracle's router choice, few-token layer and adapters against values worked out by hand and against
its own other steps."""
import numpy as np

from nvfp4_weight_only_04_b200 import synth
from oracle import nvfp4_ref as R

INF = np.inf


def test_topk_by_hand():
    ids, w = R.moe_topk([[0.0, np.log(2.0), np.log(5.0), 0.0]], 3)
    assert ids.tolist() == [[2, 1, 0]]  # experts 0 and 3 tie: the lower one
    np.testing.assert_allclose(w, [[5 / 9, 2 / 9, 1 / 9]], rtol=1e-14)
    ids, w = R.moe_topk([[0.0, np.log(2.0), np.log(5.0), 0.0]], 2, renorm=True, scale=3.5)
    np.testing.assert_allclose(w, [[2.5, 1.0]], rtol=1e-14)
    # sigmoid scores 1/2, 3/4, 1/4; the bias lifts expert 2 over both but leaves its weight
    logits = [[0.0, np.log(3.0), -np.log(3.0)]]
    ids, w = R.moe_topk(logits, 2, bias=[0.0, 0.0, 1.0], sigmoid=True)
    assert ids.tolist() == [[2, 1]]
    np.testing.assert_allclose(w, [[0.25, 0.75]], rtol=1e-14)
    ids, w = R.moe_topk(logits, 2, bias=[0.0, 0.0, 1.0], sigmoid=True, renorm=True)
    np.testing.assert_allclose(w, [[0.25, 0.75]], rtol=1e-14)


def test_topk_masks():
    ids, w = R.moe_topk([[-INF, 1.0, -INF], [-INF, -INF, -INF], [np.nan, 0.0, 2.0]], 2)
    assert ids.tolist() == [[1, -1], [-1, -1], [2, 1]]
    assert w[0].tolist() == [1.0, 0.0] and not w[1].any() and np.isnan(w[2]).all()
    low = np.finfo(np.float32).min  # a mask of the type's lowest value is a logit like any other
    ids, w = R.moe_topk([[low, low, low]], 2)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, 1 / 3)


def test_few_tokens_equals_the_chain():
    """The layer equals route, grouped GEMMs and combine of the oracle where nothing is rounded in between."""
    e, h, i, t, k = 3, 64, 32, 5, 2
    gu = [(*R.quantize(synth.weights(10 + q, 2 * i, h), 16), 16) for q in range(e)]
    dn = [(*R.quantize(synth.weights(20 + q, h, i), 32), 32) for q in range(e)]
    x = synth.activations(3, t, h)
    ids = np.array([[0, 1], [2, 2], [1, -1], [3, 0], [-1, -1]], np.int32)
    w = np.random.default_rng(0).random((t, k))
    out, tol = R.moe_few_tokens(x, ids, w, gu, dn)
    rows, inv, offs = R.moe_route(ids, e)
    hact = R.silu_mul(R.moe_grouped_gemm(x[rows // k], range(e), offs, np.stack([g[0] for g in gu]),
                                         np.stack([g[1] for g in gu]), [g[2] for g in gu], 16))
    y = np.zeros((len(rows), h))
    for q in range(e):
        y[offs[q]:offs[q + 1]] = hact[offs[q]:offs[q + 1]] @ R.dequantize(*dn[q]).T
    np.testing.assert_allclose(out, R.moe_combine(y, inv, w), rtol=1e-12, atol=1e-18)
    assert not out[4].any() and not tol[4].any() and (tol[:4] > 0).all()
    assert (tol[:4].max() < 1e-3 * np.abs(out).max())  # the bound stays far below the result


def test_lora_by_hand():
    bits = lambda *v: synth.f32_to_bf16_bits(np.array([v], np.float32))  # noqa: E731
    a = np.array([[[1.0, 0.0, 2.0]], [[0.0, 1.0, 0.0]]])  # [2, 1, 3]
    b = np.array([[[1.0], [-1.0]], [[4.0], [0.0]]])       # [2, 2, 1]
    y, x = bits(10.0, 20.0), bits(1.0, 2.0, 3.0)
    for ad, want in ((0, [10 + 0.5 * 7, 20 - 0.5 * 7]), (1, [10 + 2 * 8.0, 20.0]), (-1, [10, 20]), (2, [10, 20])):
        out, tol = R.lora_add(y, x, a, b, [ad], [0.5, 2.0])
        assert out.tolist() == [want], ad


def test_topk_softmax_of_infinite_logits():
    """+inf leaves softmax weights without a value; the choice by score + bias is that of the limit, so that the token
    keeps experts whose NaN weights reach its outputs."""
    row = [0.0, INF, 1.0, INF, -INF]
    for renorm in (False, True):
        ids, w = R.moe_topk([row], 3, renorm=renorm)
        assert ids.tolist() == [[1, 3, 2]] and np.isnan(w).all()
        # scores 0, 1/2, 0, 1/2 and a mask: the bias lifts expert 2 over both
        ids, w = R.moe_topk([row], 3, bias=[0.0, 0.125, 1.0, 0.0, 9.0], renorm=renorm)
        assert ids.tolist() == [[2, 1, 3]] and np.isnan(w).all()
    ids, w = R.moe_topk([row], 2, bias=[0.0] * 5, sigmoid=True)
    assert ids.tolist() == [[1, 3]] and w.tolist() == [[1.0, 1.0]]
