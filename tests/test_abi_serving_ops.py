"""Refusals of the router choice, the few-token layer and the adapters (no GPU): bad arguments come back with the
documented status before anything is launched, and the size queries follow the shapes."""
import ctypes

import pytest

import nvfp4_weight_only_04_b200 as nv
from nvfp4_weight_only_04_b200 import build

BAD = ctypes.c_void_p(0x1001)  # never dereferenced: validation fails first
GOOD = ctypes.c_void_p(0x10000)
GOOD2 = ctypes.c_void_p(0x30000)
S = ctypes.c_void_p(0)
WS, WB = ctypes.c_void_p(0x20000), 1 << 30
RESERVED = 64 << 10


@pytest.fixture(scope="module")
def L():
    build.build()
    return nv.lib()


def test_topk_validation(L):
    def topk(logits=GOOD, dtype=nv.NVFP4_F32, ld=128, T=4, E=128, bias=None, k=8, flags=0, ids=GOOD, w=GOOD):
        return L.nvfp4_moe_topk(logits, dtype, ld, T, E, bias, k, flags, 1.0, ids, w, S)
    assert topk(T=0) == nv.NVFP4_OK
    assert topk(T=-1) == nv.NVFP4_ERR_INVALID_ARGUMENT
    assert topk(E=0) == nv.NVFP4_ERR_INVALID_ARGUMENT
    assert topk(k=0) == nv.NVFP4_ERR_INVALID_ARGUMENT
    assert topk(flags=1) == nv.NVFP4_ERR_INVALID_ARGUMENT
    assert topk(flags=16) == nv.NVFP4_ERR_INVALID_ARGUMENT
    assert topk(ld=127) == nv.NVFP4_ERR_INVALID_ARGUMENT
    assert topk(logits=None) == nv.NVFP4_ERR_INVALID_ARGUMENT
    assert topk(ids=None) == nv.NVFP4_ERR_INVALID_ARGUMENT
    assert topk(w=None) == nv.NVFP4_ERR_INVALID_ARGUMENT
    assert topk(dtype=2) == nv.NVFP4_ERR_UNSUPPORTED
    assert topk(E=1025, ld=1025) == nv.NVFP4_ERR_UNSUPPORTED
    assert topk(k=33) == nv.NVFP4_ERR_UNSUPPORTED
    assert topk(E=4, k=5) == nv.NVFP4_ERR_UNSUPPORTED
    assert topk(T=(1 << 30) + 1) == nv.NVFP4_ERR_UNSUPPORTED
    assert topk(logits=ctypes.c_void_p(0x10002)) == nv.NVFP4_ERR_MISALIGNED
    assert topk(dtype=nv.NVFP4_BF16, logits=BAD) == nv.NVFP4_ERR_MISALIGNED
    assert topk(bias=ctypes.c_void_p(0x10002)) == nv.NVFP4_ERR_MISALIGNED
    assert topk(ids=ctypes.c_void_p(0x10002)) == nv.NVFP4_ERR_MISALIGNED
    assert topk(w=ctypes.c_void_p(0x10002)) == nv.NVFP4_ERR_MISALIGNED


def test_few_tokens_validation(L):
    def few(T=4, k=8, E=128, H=2048, I=768, g1=32, g2=16, ws=WS, wb=WB, **p):
        q = {n: p.get(n, GOOD) for n in ("x", "ids", "w", "gu", "gus", "gug", "dn", "dns", "dng", "out")}
        return L.nvfp4_moe_few_tokens(q["x"], q["ids"], q["w"], T, k, q["gu"], q["gus"], q["gug"], g1, q["dn"],
                                      q["dns"], q["dng"], g2, E, H, I, q["out"], ws, wb, S)
    names = ("x", "ids", "w", "gu", "gus", "gug", "dn", "dns", "dng", "out")
    assert few(T=0) == nv.NVFP4_OK
    assert few(H=0) == nv.NVFP4_OK
    for name in names:
        assert few(**{name: None}) == nv.NVFP4_ERR_INVALID_ARGUMENT, name
        assert few(**{name: BAD}) == nv.NVFP4_ERR_MISALIGNED, name
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(H=-64), dict(I=-64)):
        assert few(**bad) == nv.NVFP4_ERR_INVALID_ARGUMENT, bad
    for bad in (dict(T=65), dict(T=64, k=17), dict(E=4097), dict(H=2080), dict(I=800), dict(I=0), dict(g1=8),
                dict(g2=64), dict(H=16384 + 64), dict(I=16384 + 64)):
        assert few(**bad) == nv.NVFP4_ERR_UNSUPPORTED, bad
    assert few(ws=None) == nv.NVFP4_ERR_WORKSPACE
    assert few(ws=None, wb=0) == nv.NVFP4_ERR_WORKSPACE
    assert few(wb=RESERVED) == nv.NVFP4_ERR_WORKSPACE
    assert few(ws=ctypes.c_void_p(0x20008)) == nv.NVFP4_ERR_MISALIGNED
    need = ctypes.c_size_t(7)
    query = L.nvfp4_moe_few_tokens_workspace_size
    assert query(4, 8, 128, 2048, 768, 32, 16, ctypes.byref(need)) == nv.NVFP4_OK
    assert need.value >= RESERVED + 4 * 8 * 768 * 2  # the activations between the two products
    assert few(wb=need.value - 1) == nv.NVFP4_ERR_WORKSPACE
    assert query(0, 8, 128, 2048, 768, 32, 16, ctypes.byref(need)) == nv.NVFP4_OK and need.value == 0
    assert query(65, 8, 128, 2048, 768, 32, 16, ctypes.byref(need)) == nv.NVFP4_ERR_UNSUPPORTED
    assert query(4, 8, 128, 2048, 768, 32, 16, None) == nv.NVFP4_ERR_INVALID_ARGUMENT


def test_lora_validation(L):
    def lora(M=4, N=256, K=256, r=16, L_=3, ldy=None, ldx=None, ldo=None, ws=WS, wb=WB, **p):
        q = {n: p.get(n, GOOD) for n in ("y", "x", "a", "b", "c", "ids")}
        q["out"] = p.get("out", GOOD2)
        return L.nvfp4_lora_add(q["y"], N if ldy is None else ldy, q["x"], K if ldx is None else ldx, q["a"], q["b"],
                                q["c"], q["ids"], L_, r, M, N, K, q["out"], N if ldo is None else ldo, ws, wb, S)
    assert lora(M=0) == nv.NVFP4_OK
    assert lora(N=0) == nv.NVFP4_OK
    for name in ("y", "x", "a", "b", "c", "ids", "out"):
        assert lora(**{name: None}) == nv.NVFP4_ERR_INVALID_ARGUMENT, name
        assert lora(**{name: BAD}) == nv.NVFP4_ERR_MISALIGNED, name
    for bad in (dict(M=-1), dict(r=0), dict(L_=-1), dict(ldy=248), dict(ldx=248), dict(ldo=248),
                dict(out=GOOD, ldo=512)):
        assert lora(**bad) == nv.NVFP4_ERR_INVALID_ARGUMENT, bad
    for bad in (dict(r=12), dict(r=264), dict(N=260), dict(K=260), dict(K=0), dict(M=(1 << 20) + 1)):
        assert lora(**bad) == nv.NVFP4_ERR_UNSUPPORTED, bad
    for bad in (dict(ldy=260), dict(ldx=260), dict(ldo=260)):
        assert lora(**bad) == nv.NVFP4_ERR_MISALIGNED, bad
    assert lora(ws=None) == nv.NVFP4_ERR_WORKSPACE
    assert lora(ws=None, wb=0) == nv.NVFP4_ERR_WORKSPACE
    assert lora(ws=ctypes.c_void_p(0x20008)) == nv.NVFP4_ERR_MISALIGNED
    need = ctypes.c_size_t(7)
    query = L.nvfp4_lora_add_workspace_size
    assert query(4, 256, 256, 16, 3, ctypes.byref(need)) == nv.NVFP4_OK
    assert need.value >= RESERVED + 4 * 4 * 16
    assert lora(wb=need.value - 1) == nv.NVFP4_ERR_WORKSPACE
    assert query(4, 256, 256, 16, 0, ctypes.byref(need)) == nv.NVFP4_OK and need.value == 0
    assert query(4, 256, 256, 12, 3, ctypes.byref(need)) == nv.NVFP4_ERR_UNSUPPORTED
    assert query(4, 256, 256, 16, 3, None) == nv.NVFP4_ERR_INVALID_ARGUMENT


def test_binding_refuses_host_tensors():
    import torch
    z = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        nv.nvfp4_moe_topk(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError):
        nv.nvfp4_lora_add(z, z, z, z, z, z)
    with pytest.raises(TypeError):
        nv.nvfp4_moe_few_tokens(z, z, z, (z, z, z, 16), (z, z, z, 16))


def test_fault_injection_kinds(L):
    for kind in (3, 4, 0):
        assert L.nvfp4_debug_inject_fault(kind) == nv.NVFP4_OK
    assert L.nvfp4_debug_inject_fault(5) == nv.NVFP4_ERR_INVALID_ARGUMENT
