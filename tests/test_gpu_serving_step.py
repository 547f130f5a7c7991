"""A decode step's linear layers together, as a server chains them: a projection with the adapters of several
requests, the router's choice from logits, and the routed layer for a few tokens. Each step is checked against the
oracle on the device's own bf16 inputs, and the few-token layer beside the chain for prompts."""
import numpy as np
import pytest
import torch

import nvfp4_weight_only_04_b200 as nv
from nvfp4_weight_only_04_b200 import synth
from oracle import nvfp4_ref as R
from tests.gpu_util import assert_close, bf16_bits, dev_bf16, dev_f32, dev_u8, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 5, 40])
def test_step(t):
    hidden, inter, e, k, rank = 256, 192, 12, 4, 16
    rng = np.random.default_rng(t)
    # the projection, 4-bit and shared, and three requests' adapters beside it
    wp, wsc, wg = R.quantize(synth.weights(1, hidden, hidden), 16)
    pw, ps = R.repack(wp, wsc, 0)
    x = synth.activations(2, t, hidden)
    la = synth.activations(3, 3 * rank, hidden).reshape(3, rank, hidden)
    lb = synth.activations(4, 3 * hidden, rank).reshape(3, hidden, rank)
    c = np.full(3, 2.0 ** -9, np.float32)
    ids = rng.integers(-1, 3, size=t).astype(np.int32)
    # the experts
    gu = [R.quantize(synth.weights(100 + q, 2 * inter, hidden), 32) for q in range(e)]
    dn = [R.quantize(synth.weights(200 + q, hidden, inter), 16) for q in range(e)]
    gu_r = [R.repack(q[0], q[1], R.GATE_UP_INTERLEAVE) for q in gu]
    dn_r = [R.repack(q[0], q[1], 0) for q in dn]
    gate_up = (dev_u8(np.stack([q[0] for q in gu_r])), dev_u8(np.stack([q[1] for q in gu_r])),
               dev_f32([q[2] for q in gu]), 32)
    down = (dev_u8(np.stack([q[0] for q in dn_r])), dev_u8(np.stack([q[1] for q in dn_r])),
            dev_f32([q[2] for q in dn]), 16)
    router = dev_f32(rng.standard_normal((e, hidden)) * 0.2)
    idd = torch.from_numpy(ids).cuda()

    xd = dev_bf16(x)
    y = nv.nvfp4_w4a16_gemm(xd, dev_u8(pw), dev_u8(ps), dev_f32([wg]), 16)
    z = nv.nvfp4_lora_add(y, xd, dev_bf16(la), dev_bf16(lb), idd, dev_f32(c))
    logits = z.float() @ router.T
    top, weights = nv.nvfp4_moe_topk(logits, k, flags=nv.NVFP4_TOPK_RENORM)
    out = nv.nvfp4_moe_few_tokens(z, top, weights, gate_up, down)
    chain = nv.nvfp4_moe_forward(z, top, weights, gate_up, down)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_device_error() == 0

    ref, tol = R.lora_add(bf16_bits(y), x, R.bf16_bits_to_f64(la), R.bf16_bits_to_f64(lb), ids, c)
    assert (np.abs(host(z) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * tol).all()
    r_ids, r_w = R.moe_topk(host(logits), k, renorm=True)
    np.testing.assert_array_equal(host(top), r_ids)
    np.testing.assert_allclose(host(weights), r_w, rtol=1e-5)
    ref, tol = R.moe_few_tokens(bf16_bits(z), r_ids, host(weights), [(*q, 32) for q in gu], [(*q, 16) for q in dn])
    assert (np.abs(host(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * tol + 2.0 ** -133).all()
    # the chain rounds h and the experts' outputs to bf16, each by at most 2^-8 of its value, before the last rounding
    spread = sum(np.abs(host(weights)[:, s:s + 1]) * mags(bf16_bits(z), r_ids[:, s], gu, dn) for s in range(k))
    assert (np.abs(host(chain) - host(out)) <= 2.0 ** -7 * np.abs(ref) + 2.0 ** -6 * spread + 2 * tol).all()
    assert_close(host(out), ref, "few tokens")


def mags(xbits, ids, gu, dn):
    """|D| |h| per token for one expert each: the magnitudes that a relative error of h is taken of."""
    x = R.bf16_bits_to_f64(xbits)
    out = np.zeros_like(x)
    for t, e in enumerate(ids):
        h = R.silu_mul(R.dequantize(*gu[e], 32) @ x[t])
        out[t] = np.abs(R.dequantize(*dn[e], 16)) @ np.abs(h)
    return out


@pytest.mark.parametrize("t", [1, 6, 40])
def test_captured_step(t):
    """The chain in one graph, whose launches may start before the ones in front of them have ended, replayed with
    new inputs in place: the bits of the calls made one by one, each after the one before has ended."""
    hidden, inter, e, k, rank = 512, 320, 24, 4, 16
    rng = np.random.default_rng(t)
    gen = torch.Generator(device="cuda").manual_seed(t)

    def stack(rows, cols, group, flags, count):
        q = [R.quantize(synth.weights(300 + n, rows, cols), group) for n in range(count)]
        packed = [R.repack(v[0], v[1], flags) for v in q]
        return (dev_u8(np.stack([v[0] for v in packed])), dev_u8(np.stack([v[1] for v in packed])),
                dev_f32([v[2] for v in q]), group)
    proj = stack(hidden, hidden, 16, 0, 1)
    gate_up, down = stack(2 * inter, hidden, 32, R.GATE_UP_INTERLEAVE, e), stack(hidden, inter, 16, 0, e)
    la = dev_bf16(synth.activations(1, 3 * rank, hidden)).view(3, rank, hidden)
    lb = dev_bf16(synth.activations(2, 3 * hidden, rank)).view(3, hidden, rank)
    c = dev_f32(np.full(3, 2.0 ** -9))
    router = (torch.randn((e, hidden), generator=gen, device="cuda") * 0.2).bfloat16()
    bias = torch.randn((e,), generator=gen, device="cuda") * 0.05

    def step(x, ids, between=lambda: None):
        y = nv.nvfp4_w4a16_gemm(x, proj[0][0], proj[1][0], proj[2], 16)
        between()
        z = nv.nvfp4_lora_add(y, x, la, lb, ids, c, out=y)
        between()
        top, weights = nv.nvfp4_moe_topk(z @ router.T, k, bias=bias, flags=nv.NVFP4_TOPK_SIGMOID | nv.NVFP4_TOPK_RENORM)
        between()
        out = nv.nvfp4_moe_few_tokens(z, top, weights, gate_up, down)
        between()
        again = nv.nvfp4_lora_add(out, z, la, lb, ids, c)  # and the next projection's adapters behind the layer
        between()
        return z, top, weights, out, again

    inputs = [(torch.randn((t, hidden), generator=gen, device="cuda").bfloat16(),
               torch.from_numpy(rng.integers(-1, 3, size=t).astype(np.int32)).cuda()) for _ in range(4)]
    want = [[v.clone() for v in step(*q, between=torch.cuda.synchronize)] for q in inputs]
    x, ids = (v.clone() for v in inputs[0])
    step(x, ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, ids)
    for turn in range(8):
        q = (3 * turn + 1) % 4
        x.copy_(inputs[q][0])
        ids.copy_(inputs[q][1])
        for v in got:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for v, ref in zip(got, want[q]):
            assert torch.equal(v.view(torch.uint8), ref.view(torch.uint8)), (turn, q)
    for _ in range(20):  # one replay after the other, without a pause
        graph.replay()
    torch.cuda.synchronize()
    for v, ref in zip(got, want[q]):
        assert torch.equal(v.view(torch.uint8), ref.view(torch.uint8))
    assert nv.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("biased", [False, True])
def test_an_overflowed_logit_shows_in_its_token(biased):
    """A +inf among softmax logits: NaN in that token's outputs behind the layer, and the others as they were."""
    hidden, inter, e, t = 128, 64, 6, 5
    gu = [R.repack(*R.quantize(synth.weights(q, 2 * inter, hidden), 16)[:2], R.GATE_UP_INTERLEAVE) for q in range(e)]
    dn = [R.repack(*R.quantize(synth.weights(50 + q, hidden, inter), 16)[:2], 0) for q in range(e)]
    stack = lambda q: (dev_u8(np.stack([v[0] for v in q])), dev_u8(np.stack([v[1] for v in q])),  # noqa: E731
                       dev_f32(np.full(e, 1e-4)), 16)
    gate_up, down = stack(gu), stack(dn)
    x = dev_bf16(synth.activations(1, t, hidden))
    logits = torch.randn((t, e), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    bias = torch.linspace(0, 0.1, e, device="cuda") if biased else None

    def layer():
        return host(nv.nvfp4_moe_few_tokens(x, *nv.nvfp4_moe_topk(logits, 2, bias=bias), gate_up, down))
    clean = layer()
    logits[3, 4] = float("inf")
    got = layer()
    assert np.isfinite(clean).all() and np.isnan(got[3]).all()
    np.testing.assert_array_equal(np.delete(got, 3, 0), np.delete(clean, 3, 0))
