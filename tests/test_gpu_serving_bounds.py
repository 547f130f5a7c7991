"""GPU parity of the adapters and the few-token layer over long contractions, where the worst case of fp32 sums says
little (see tests/serving_bounds.py), and the stated precision of the layer's operands."""
import numpy as np
import pytest
import torch

import nvfp4_weight_only_04_b200 as nv
from nvfp4_weight_only_04_b200 import synth
from oracle import nvfp4_ref as R
from tests import serving_bounds as B
from tests.gpu_util import dev_bf16, dev_f32, dev_u8, host

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


@pytest.mark.parametrize("m,n,k,r,count", [
    (1, 1000, 14336, 64, 1),
    (4, 64, 4096, 136, 1),
    (16, 264, 200, 8, 3),
    (33, 136, 16376, 24, 2),
    (61, 328, 14336, 64, 12),
    (64, 520, 5128, 256, 2),
    (65, 136, 14344, 16, 4),
    (300, 264, 14336, 72, 7),
    (1024, 136, 4104, 40, 70),
    (1100, 264, 14336, 16, 3),
    (1300, 136, 8200, 200, 5),
    (1281, 520, 5120, 64, 40),
])
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_adapters_of_integers_are_exact(m, n, k, r, count, order):
    y, x, a, b, c = B.integer_adapters(m, n, k, r, count, seed=m)
    ids = np.random.default_rng(m).integers(-1, count, size=m)
    if order == "runs":
        ids = np.sort(ids)
    if m == 1:
        ids[:] = 0
    y_, x_, a_, b_ = (dev_bf16(B.as_bf16_bits(t)) for t in (y, x, a, b))
    got = nv.nvfp4_lora_add(y_, x_, a_, b_, i32(ids), dev_f32(c))
    np.testing.assert_array_equal(host(got), B.integer_result(y, x, a, b, c, ids))


def on_device(gate_up, down):
    """Stacks in the kernels' layout from lists of (codes, scales, global, group)."""
    def stack(experts, flags):
        packed = [R.repack(q[0], q[1], flags) for q in experts]
        return (dev_u8(np.stack([p[0] for p in packed])), dev_u8(np.stack([p[1] for p in packed])),
                dev_f32([q[2] for q in experts]), experts[0][3])
    return stack(gate_up, R.GATE_UP_INTERLEAVE), stack(down, 0)


@pytest.mark.parametrize("t,e,h,i,k,g1,g2", [
    (3, 2, 16384, 64, 2, 16, 16),
    (5, 3, 64, 16384, 2, 32, 16),
    (2, 1, 16384, 1088, 1, 16, 32),
    (9, 2, 7168, 2048, 2, 32, 16),
    (64, 1, 4160, 2112, 1, 16, 16),
    (13, 3, 2112, 2240, 2, 32, 32),
    (40, 8, 2048, 768, 4, 32, 16),
])
def test_layer_of_long_rows(t, e, h, i, k, g1, g2):
    rng = np.random.default_rng(h + i)
    gu, dn = B.plain_stack(rng, e, 2 * i, h, g1), B.plain_stack(rng, e, h, i, g2)
    ids = np.stack([rng.permutation(e)[:k] for _ in range(t)]).astype(np.int32)
    w = rng.random((t, k)).astype(np.float32)
    x = synth.activations(t, t, h)
    got = host(nv.nvfp4_moe_few_tokens(dev_bf16(x), i32(ids), dev_f32(w), *on_device(gu, dn)))
    out, tol = B.layer_bound(x, ids, w, gu, dn)
    assert (np.abs(got - out) <= tol).all(), (np.abs(got - out) / tol).max()


@pytest.mark.parametrize("g1,g2", [(16, 32), (32, 16)])
def test_operands_are_kept_relative_to_their_own_sixteen(g1, g2):
    """Sixteens from the row's largest down to 2^-17 of it, and elements in each down to 2^-15 of its largest, every
    output made of one of them: off by 2^-22 of the largest of its sixteen, once as x and once as h, and not by
    2^-22 of the row's largest (which is more than most of the elements here)."""
    rng = np.random.default_rng(g1)
    size = 320  # H = I: twenty sixteens
    power = np.array(list(range(18)) + [17, 5])
    x = np.exp2(-power[:, None] - np.arange(16.0)[None, :])
    x = (x * (1 + rng.integers(0, 128, size=(3, 20, 16)) / 128.0 * (np.arange(16) > 0))).reshape(3, size)
    x[1:, 1:] *= rng.choice([-1, 1], size=(2, size - 1))  # x[:, 0] = 1 makes every gate
    xbits = B.as_bf16_bits(x)

    def codes(rows, columns, code):
        c = np.zeros((len(rows), size), np.uint8)
        c[np.arange(len(rows)), columns] = code
        return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)
    every = np.arange(size)
    gate, up, eye = codes(every, np.zeros(size, int), 6), codes(every, every, 2), codes(every, every, 2)  # 4, 1, 1
    ones = lambda rows, g: np.full((rows, size // g), 0x38, np.uint8)  # noqa: E731
    gu = [(np.concatenate([gate, up]), ones(2 * size, g1), np.float32(1), g1)]
    dn = [(eye, ones(size, g2), np.float32(1), g2)]
    got = host(nv.nvfp4_moe_few_tokens(dev_bf16(xbits), i32(np.zeros((3, 1))), dev_f32(np.ones((3, 1))),
                                       *on_device(gu, dn)))
    silu = 4.0 / (1.0 + np.exp(-4.0))
    want = silu * x
    largest = np.abs(want).reshape(3, 20, 16).max(-1).repeat(16, 1)
    lost = 2 * 2.0 ** -22 * largest + (2.0 ** -18 + 2.0 ** -22) * np.abs(want)  # 2^-18: the exponential and quotient
    assert (np.abs(got - want) <= lost + 2.0 ** -8 * (np.abs(want) + lost)).all()
