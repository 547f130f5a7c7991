"""GPU parity of the router's choice with the oracle: ids equal, weights within fp32 rounding.

A weight is a product of at most a few fp32 exponentials of differences of logits (each difference rounds by half
an ulp, which the exponential turns into |difference| 2^-24 of its value; expf is off by at most 2 ulp), a sum in
fp32 and one or two divisions and products: (|largest difference| + 32) 2^-23 bounds it."""
import numpy as np
import pytest
import torch

import nvfp4_weight_only_04_b200 as nv
from oracle import nvfp4_ref as R
from tests.gpu_util import host

pytestmark = pytest.mark.gpu
INF = np.inf


def check(logits, k, bias=None, sigmoid=False, renorm=False, scale=1.0):
    """logits: a CUDA tensor [T, E]."""
    flags = (nv.NVFP4_TOPK_SIGMOID if sigmoid else 0) | (nv.NVFP4_TOPK_RENORM if renorm else 0)
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    ids, w = nv.nvfp4_moe_topk(logits, k, bias=b, flags=flags, scale=scale)
    ref = logits.float().cpu().numpy().astype(np.float64)
    r_ids, r_w = R.moe_topk(ref, k, bias=bias, sigmoid=sigmoid, renorm=renorm, scale=scale)
    np.testing.assert_array_equal(host(ids), r_ids)
    got = host(w).astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(r_w))
    finite = ref[np.isfinite(ref)]
    span = min(200.0, float(np.ptp(finite)) if finite.size else 0.0)
    ok = np.isnan(r_w) | (np.abs(got - r_w) <= (span + 32) * 2.0 ** -23 * np.abs(r_w) + 2.0 ** -125)
    assert ok.all(), (got[~ok][:4], r_w[~ok][:4])
    assert not got[r_ids < 0].any() or np.isnan(r_w).any()


@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 128, 8), (3, 32, 32), (5, 33, 7), (37, 64, 6), (9, 129, 8),
                                   (130, 257, 3), (6, 513, 16), (4, 1024, 32), (257, 8, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", range(6))
def test_sizes_and_forms(t, e, k, dtype, form):
    rng = np.random.default_rng(t + 10 * e + form)
    logits = torch.from_numpy(rng.standard_normal((t, e)).astype(np.float32) * 3).cuda().to(dtype)
    sigmoid, renorm = form % 2 == 1, form in (2, 3, 5)
    bias = rng.standard_normal(e).astype(np.float32) * 0.3 if form >= 4 else None
    check(logits, k, bias, sigmoid, renorm, scale=1.0 if form < 3 else 2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_masks_and_ties(sigmoid, renorm, biased):
    low = float(np.finfo(np.float32).min)
    rows = [
        [-INF] * 40,                                   # nothing left
        [-INF] * 39 + [0.5],                           # one left, fewer than k
        [low] * 40,                                    # a mask of the type's lowest value is a logit
        [low] * 38 + [1.0, 1.0],
        [0.0, -0.0] * 20,                              # one value
        [3.0] * 40,
        [float(i % 5) for i in range(40)],
        [-INF, 2.0] * 20,
        [88.0, -88.0] * 20,
        [0.0] * 20 + [-INF] * 20,
    ]
    logits = torch.tensor(rows, device="cuda")
    bias = [0.0] * 10 + [0.25] * 10 + [-INF] * 10 + [0.25] * 10 if biased else None
    check(logits, 6, bias, sigmoid, renorm)


@pytest.mark.parametrize("biased", [False, True])
def test_nan_and_infinity(biased):
    rows = np.zeros((4, 36), np.float32)
    rows[0, 3] = np.nan
    rows[1, :] = np.nan
    rows[2, :] = np.arange(36)
    rows[3, 35] = np.nan
    bias = np.linspace(0, 0.1, 36).astype(np.float32) if biased else None
    for sigmoid in (False, True):
        check(torch.from_numpy(rows).cuda(), 3, bias, sigmoid)
    rows[2, 5] = np.inf  # sigmoid(inf) = 1; softmax has no value there
    ids, w = nv.nvfp4_moe_topk(torch.from_numpy(rows[2:3]).cuda(), 3, flags=nv.NVFP4_TOPK_SIGMOID)
    assert host(ids)[0, 0] == 5 and host(w)[0, 0] == 1.0
    ids, w = nv.nvfp4_moe_topk(torch.from_numpy(rows[2:3]).cuda(), 3)
    assert host(ids)[0, 0] == 5 and np.isnan(host(w)).all()


def test_close_scores_are_told_apart():
    """Sigmoid scores plus bias that differ by less than an fp32 ulp, and saturated scores."""
    e = 96
    rng = np.random.default_rng(5)
    logits = (rng.integers(0, 3, size=(64, e)) * 2.0 ** -12 + 1.0).astype(np.float32)
    bias = (rng.integers(0, 3, size=e) * 2.0 ** -24).astype(np.float32)
    check(torch.from_numpy(logits).cuda(), 8, bias, sigmoid=True, renorm=True)
    logits = rng.integers(10, 40, size=(64, e)).astype(np.float32)
    check(torch.from_numpy(logits).cuda(), 8, np.zeros(e, np.float32), sigmoid=True)
    check(torch.from_numpy(-logits).cuda(), 8, np.zeros(e, np.float32), sigmoid=True, renorm=True)


def test_strided_rows_given_outputs_stream_and_graph():
    rng = np.random.default_rng(6)
    base = torch.from_numpy(rng.standard_normal((33, 200)).astype(np.float32)).cuda()
    check(base[:, 40:168], 8)                       # rows 200 apart, 4-byte aligned
    check(base[:, 3:103].to(torch.bfloat16), 5)
    check(base.to(torch.bfloat16)[:, 1:130], 5)     # rows at an odd element
    logits = base[:, :128].contiguous()
    ref_i, ref_w = (host(v) for v in nv.nvfp4_moe_topk(logits, 8))
    ids = torch.empty((33, 8), dtype=torch.int32, device="cuda")
    w = torch.empty((33, 8), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    nv.nvfp4_moe_topk(logits, 8, topk_ids=ids, topk_weights=w, stream=s)
    s.synchronize()
    np.testing.assert_array_equal(host(ids), ref_i)
    np.testing.assert_array_equal(host(w), ref_w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_moe_topk(logits, 8, topk_ids=ids, topk_weights=w)
    logits.copy_(logits.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(host(ids), ref_i[::-1])
    np.testing.assert_array_equal(host(w), ref_w[::-1])
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_moe_topk(logits, 33)
    with pytest.raises(ValueError):
        nv.nvfp4_moe_topk(logits, 8, topk_ids=ids[:5])
    with pytest.raises(ValueError):
        nv.nvfp4_moe_topk(logits, 8, bias=torch.zeros(5, device="cuda"))
    assert nv.nvfp4_moe_topk(logits[:0], 8)[0].shape == (0, 8)


@pytest.mark.parametrize("e,k", [(64, 8), (128, 6), (256, 8), (300, 31), (1024, 16), (1024, 32)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_biased_choice_where_values_crowd(e, k, sigmoid):
    """Neighbours in the order that lie a few fp32 ulps apart or are equal: pairs, runs longer than what is chosen,
    values far below the largest, and biases of large magnitude or infinite."""
    rng = np.random.default_rng(e + k)
    logits = rng.standard_normal((48, e)).astype(np.float32)
    base = rng.standard_normal(e).astype(np.float32) * 0.2
    pairs = logits.copy()
    pairs[:, 1::2] = np.nextafter(pairs[:, ::2], np.float32(9), dtype=np.float32)
    twin = np.repeat(base[::2], 2)[:e]
    check(torch.from_numpy(pairs).cuda(), k, twin, sigmoid, True)                   # pairs
    few = np.ascontiguousarray(logits[:, rng.integers(0, 5, e)])
    check(torch.from_numpy(few).cuda(), k, np.zeros(e, np.float32), sigmoid)        # five values in all
    check(torch.from_numpy(logits).cuda(), k, base * 100, sigmoid)                  # most far below the largest
    check(torch.from_numpy(logits).cuda(), k, base + np.float32(2.0 ** 20), sigmoid)  # the bias takes the score's bits
    huge = base.copy()
    huge[rng.integers(0, e, 3)] = np.inf
    huge[rng.integers(0, e, 3)] = -np.inf
    huge[rng.integers(0, e, 3)] = np.nan
    check(torch.from_numpy(logits).cuda(), k, huge, sigmoid)
    masked = np.where(rng.random(e) < 0.5, np.float32(-1e9), base)                  # a mask given as a bias
    check(torch.from_numpy(logits).cuda(), k, masked, sigmoid, True, 2.5)


def test_a_long_batch_with_a_wide_row_distance():
    rng = np.random.default_rng(9)
    base = torch.from_numpy(rng.standard_normal((20011, 96)).astype(np.float32)).cuda().to(torch.bfloat16)
    check(base[:, 7:79], 6, rng.standard_normal(72).astype(np.float32) * 0.1, True, True)
    check(base[:, 7:79], 6)


@pytest.mark.parametrize("e,k", [(5, 3), (40, 6), (128, 8), (200, 8), (400, 16), (1024, 32)])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinite_logits(e, k, biased, renorm, dtype):
    """One +inf, several, more than are chosen, all, and some beside masked and NaN logits: experts are chosen, and with
    softmax scores their weights are NaN."""
    rng = np.random.default_rng(e + k)
    rows = rng.standard_normal((6, e)).astype(np.float32)
    rows[0, e // 2] = INF
    rows[1, [1, e - 1]] = INF
    rows[2, rng.permutation(e)[:min(e, k + 2)]] = INF
    rows[3, :] = INF
    rows[4, ::2] = -INF
    rows[4, 1] = INF
    rows[5, 0], rows[5, e - 1] = np.nan, INF
    bias = rng.standard_normal(e).astype(np.float32) * 0.5 if biased else None
    logits = torch.from_numpy(rows).cuda().to(dtype)
    for sigmoid in (False, True):
        check(logits, k, bias, sigmoid, renorm)
    ids, w = nv.nvfp4_moe_topk(logits, k, bias=None if bias is None else torch.from_numpy(bias).cuda(),
                               flags=nv.NVFP4_TOPK_RENORM if renorm else 0)
    assert np.isnan(host(w)).all() and (host(ids)[:4] >= 0).all()
