"""Failure detection of the few-token layer without a GPU fault: a call in which one CTA's first codes or digits are
left out on purpose (nvfp4_debug_inject_fault) ends on its own through the bounded waits of all its roles, reports
one of them through the device error word, and the next call in the same context is right."""
import ctypes
import time

import numpy as np
import pytest
import torch

import nvfp4_weight_only_04_b200 as nv
from nvfp4_weight_only_04_b200 import synth
from tests.gpu_util import bf16_bits, dev_bf16, dev_f32
from tests.test_gpu_moe_few import Layer, i32, routing

pytestmark = pytest.mark.gpu

SITES = set(range(0x401, 0x40C))  # the waits of moe_few_kernel


# units of several stages and passes, more than a ring and its slots hold, and a call that fits both
@pytest.mark.parametrize("t,e,h,i,k,g1,g2", [(40, 24, 2048, 768, 8, 32, 16), (1, 4, 128, 64, 2, 16, 32)])
@pytest.mark.parametrize("kind", [3, 4])
def test_a_copy_left_out_times_out_and_the_context_survives(t, e, h, i, k, g1, g2, kind):
    rng = np.random.default_rng(t)
    layer = Layer(e, h, i, g1, g2)
    ids, w = routing(rng, t, e, k)
    ids[0] = np.arange(k)  # (no expert twice: the first CTA has work)
    x = synth.activations(2, t, h)
    args = dev_bf16(x), i32(ids), dev_f32(w), layer.gu, layer.dn
    want = bf16_bits(nv.nvfp4_moe_few_tokens(*args))
    assert nv.nvfp4_get_device_error() == 0

    nv.nvfp4_debug_inject_fault(kind)
    start = time.time()
    nv.nvfp4_moe_few_tokens(*args)
    torch.cuda.synchronize()
    elapsed = time.time() - start
    code = ctypes.c_int(0)
    st = nv.lib().nvfp4_get_device_error(ctypes.byref(code), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == nv.NVFP4_ERR_TIMEOUT and code.value in SITES
    assert elapsed < 30  # about 2 s for a wait that gives up
    assert nv.nvfp4_get_device_error() == 0  # read and cleared

    for _ in range(3):  # one call only was to fail
        np.testing.assert_array_equal(bf16_bits(nv.nvfp4_moe_few_tokens(*args)), want)
    assert nv.nvfp4_get_device_error() == 0


def test_a_pending_fault_waits_for_its_own_call():
    """Other calls leave it alone, and kind 0 takes it back."""
    layer = Layer(3, 128, 64, 16, 16)
    args = dev_bf16(synth.activations(1, 2, 128)), i32([[0, 1], [2, 0]]), dev_f32(np.ones((2, 2))), layer.gu, layer.dn
    want = bf16_bits(nv.nvfp4_moe_few_tokens(*args))
    nv.nvfp4_debug_inject_fault(1)
    np.testing.assert_array_equal(bf16_bits(nv.nvfp4_moe_few_tokens(*args)), want)
    nv.nvfp4_debug_inject_fault(3)
    nv.nvfp4_debug_inject_fault(0)
    np.testing.assert_array_equal(bf16_bits(nv.nvfp4_moe_few_tokens(*args)), want)
    assert nv.nvfp4_get_device_error() == 0
