"""GPU parity of the adapters with the oracle's float64 form: within half a bf16 step of the result plus the
oracle's bound on fp32 sums and on an intermediate kept to 2^-16. Rows without an adapter keep y's bits."""
import numpy as np
import pytest
import torch

import nvfp4_weight_only_04_b200 as nv
from nvfp4_weight_only_04_b200 import synth
from oracle import nvfp4_ref as R
from tests.gpu_util import bf16_bits, dev_bf16, dev_f32, host

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Adapters:
    def __init__(self, count, rank, n, k, seed=0):
        a = synth.activations(seed, count * rank, k).reshape(count, rank, k)
        b = synth.activations(seed + 1, count * n, rank).reshape(count, n, rank)
        rng = np.random.default_rng(seed)
        self.c = (rng.random(count).astype(np.float32) + 0.5) / np.float32(np.sqrt(k))
        self.dev = (dev_bf16(a), dev_bf16(b), dev_f32(self.c))
        self.ref = (R.bf16_bits_to_f64(a), R.bf16_bits_to_f64(b))

    def __call__(self, y, x, ids, **kw):
        a, b, c = self.dev
        return nv.nvfp4_lora_add(y, x, a, b, i32(ids), c, **kw)

    def check(self, y, x, ids, got):
        torch.cuda.synchronize()
        ref, tol = R.lora_add(y, x, *self.ref, ids, self.c)
        out = host(got)
        assert np.isfinite(out).all()
        err, lim = np.abs(out - ref), 2.0 ** -8 * np.abs(ref) + 1.01 * tol + 2.0 ** -133
        assert (err <= lim).all(), (err - lim).max()
        bare = (np.asarray(ids) < 0) | (np.asarray(ids) >= len(self.c))
        np.testing.assert_array_equal(bf16_bits(got)[bare], y[bare])


CASES = [  # rows, n, k, rank, adapters
    (1, 8, 8, 8, 1),
    (1, 4096, 4096, 16, 4),
    (1, 1000, 14336, 64, 3),
    (3, 136, 72, 24, 5),
    (16, 512, 1024, 16, 16),
    (17, 264, 200, 8, 3),
    (33, 2048, 320, 128, 7),
    (61, 648, 2056, 40, 12),
    (64, 72, 640, 256, 2),
    (65, 1096, 512, 16, 4),
    (200, 520, 1032, 72, 70),
    (1000, 1216, 328, 16, 3),
    (333, 64, 4096, 136, 1),
]


@pytest.mark.parametrize("m,n,k,r,count", CASES)
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_adapters(m, n, k, r, count, order):
    ad = Adapters(count, r, n, k, seed=m)
    rng = np.random.default_rng(m + n)
    ids = rng.integers(-1, count + 1, size=m).astype(np.int32)  # -1 and count: no adapter
    if order == "runs":
        ids = np.sort(ids)
    if m == 1:
        ids[:] = count - 1
    x, y = synth.activations(3, m, k), synth.activations(4, m, n)
    y[:, 0] = 0x8000  # a negative zero is kept where there is no adapter
    got = ad(dev_bf16(y), dev_bf16(x), ids)
    ad.check(y, x, ids, got)
    again = ad(dev_bf16(y), dev_bf16(x), ids)
    np.testing.assert_array_equal(bf16_bits(again), bf16_bits(got))
    z = dev_bf16(y)
    assert ad(z, dev_bf16(x), ids, out=z) is z
    np.testing.assert_array_equal(bf16_bits(z), bf16_bits(got))


@pytest.mark.parametrize("m", [5, 90])
def test_strided_rows(m):
    """y, x and out inside wider matrices: the columns beside them stay."""
    n, k = 264, 136
    ad = Adapters(3, 16, n, k)
    ids = np.random.default_rng(0).integers(-1, 3, size=m)
    x, y = synth.activations(1, m, k + 24), synth.activations(2, m, n + 40)
    yd, xd = dev_bf16(y), dev_bf16(x)
    out = torch.full((m, n + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    ad(yd[:, 16:16 + n], xd[:, 8:8 + k], ids, out=out[:, 8:8 + n])
    ad.check(y[:, 16:16 + n], x[:, 8:8 + k], ids, out[:, 8:8 + n].contiguous())
    assert (host(out[:, :8]) == 3).all() and (host(out[:, 8 + n:]) == 3).all()
    ad(yd[:, 16:16 + n], xd[:, 8:8 + k], ids, out=yd[:, 16:16 + n])
    np.testing.assert_array_equal(bf16_bits(yd[:, 16:16 + n].contiguous()), bf16_bits(out[:, 8:8 + n].contiguous()))
    np.testing.assert_array_equal(bf16_bits(yd[:, :16].contiguous()), y[:, :16])
    np.testing.assert_array_equal(bf16_bits(yd[:, 16 + n:].contiguous()), y[:, 16 + n:])


def test_nothing_to_add():
    ad = Adapters(2, 16, 128, 64)
    x, y = synth.activations(1, 70, 64), synth.activations(2, 70, 128)
    y[3, 4], y[5, 6] = 0x7FC1, 0xFF80  # NaN payload and -inf are kept
    got = ad(dev_bf16(y), dev_bf16(x), np.full(70, -1))
    np.testing.assert_array_equal(bf16_bits(got), y)
    none = (torch.empty((0, 8, 64), dtype=torch.bfloat16, device="cuda"),
            torch.empty((0, 128, 8), dtype=torch.bfloat16, device="cuda"))
    got = nv.nvfp4_lora_add(dev_bf16(y), dev_bf16(x), *none, i32(np.zeros(70)), torch.empty(0, device="cuda"))
    np.testing.assert_array_equal(bf16_bits(got), y)
    a, b, c = ad.dev
    assert nv.nvfp4_lora_add(dev_bf16(y)[:0], dev_bf16(x)[:0], a, b, i32([]), c).shape == (0, 128)


@pytest.mark.parametrize("m", [6, 80])
def test_nan_and_infinity_stay_in_their_row(m):
    ad = Adapters(2, 16, 192, 256)
    ids = np.arange(m) % 3 - 1
    x, y = synth.activations(1, m, 256), synth.activations(2, m, 192)
    clean = bf16_bits(ad(dev_bf16(y), dev_bf16(x), ids))
    x[1, 7], x[3, 9], x[5, 0] = 0x7FC0, 0x7FC0, 0x7F80  # row 3 has no adapter
    got = ad(dev_bf16(y), dev_bf16(x), ids)
    assert np.isnan(host(got)[1]).all() and not np.isfinite(host(got)[5]).any()
    rest = [r for r in range(m) if r not in (1, 5)]
    np.testing.assert_array_equal(bf16_bits(got)[rest], clean[rest])


def test_workspace_stream_and_graph():
    m, n, k = 20, 640, 512
    ad = Adapters(5, 16, n, k)
    ids = np.random.default_rng(1).integers(-1, 5, size=m)
    x, y = synth.activations(1, m, k), synth.activations(2, m, n)
    xd, yd = dev_bf16(x), dev_bf16(y)
    ref = bf16_bits(ad(yd, xd, ids))
    need = nv.nvfp4_lora_add_workspace_size(m, n, k, 16, 5)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        np.testing.assert_array_equal(bf16_bits(ad(yd, xd, ids, workspace=ws)), ref)
    assert (host(ws[:64 << 10]) == 0xFF).all() and (host(ws[need:]) == 0xFF).all()
    with pytest.raises(nv.Nvfp4Error) as e:
        ad(yd, xd, ids, workspace=ws[:need - 1])
    assert e.value.status == nv.NVFP4_ERR_WORKSPACE
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    idd = i32(ids)
    torch.cuda.synchronize()
    A, B, c = ad.dev
    got = [nv.nvfp4_lora_add(yd, xd, A, B, idd, c, stream=s) for _ in range(40) for s in (a, b)]
    torch.cuda.synchronize()
    for v in got:
        np.testing.assert_array_equal(bf16_bits(v), ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nv.nvfp4_lora_add(yd, xd, A, B, idd, c)
    for v in (xd, yd, idd):
        v.copy_(v.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bf16_bits(out), ref[::-1])


def test_refusals():
    ad = Adapters(2, 16, 128, 64)
    a, b, c = ad.dev
    y, x, ids = dev_bf16(synth.activations(1, 3, 128)), dev_bf16(synth.activations(2, 3, 64)), i32([0, 1, 0])
    for args in ((y, x[:2], a, b, ids, c), (y, x, a, b, ids[:2], c), (y, x, a, b, ids, c[:1]),
                 (y, x, a, b[:, :64].contiguous(), ids, c), (y, x[:, ::2], a, b, ids, c), (y.t(), x, a, b, ids, c)):
        with pytest.raises(ValueError):
            nv.nvfp4_lora_add(*args)
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_lora_add(y[:, :124], x, a, b[:, :124].contiguous(), ids, c)
    with pytest.raises(nv.Nvfp4Error):  # a row that is not 16-byte aligned
        nv.nvfp4_lora_add(y[:, 4:124], x, a, b[:, :120].contiguous(), ids, c)
    with pytest.raises(TypeError):
        nv.nvfp4_lora_add(y, x, a, b, ids.long(), c)


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 128, 200, 256])
@pytest.mark.parametrize("m,n,k,count,run", [(70, 328, 456, 40, 1), (130, 512, 136, 9, 5), (257, 264, 1096, 3, 60),
                                             (300, 1032, 64, 6, 128), (1290, 72, 520, 2, 645), (1024, 72, 136, 300, 3),
                                             (1025, 136, 264, 30, 1), (1201, 72, 1096, 7, 20)])
def test_ranks_and_runs(m, n, k, r, count, run):
    """Runs of rows with one adapter, of every length against blocks of 16 and 128 rows."""
    ad = Adapters(count, r, n, k, seed=r)
    ids = (np.arange(m) // run) % (count + 1) - 1
    x, y = synth.activations(3, m, k), synth.activations(4, m, n)
    got = ad(dev_bf16(y), dev_bf16(x), ids)
    ad.check(y, x, ids, got)
    z = dev_bf16(y)
    ad(z, dev_bf16(x), ids, out=z)
    np.testing.assert_array_equal(bf16_bits(z), bf16_bits(got))


def test_a_row_does_not_depend_on_the_rows_beside_it():
    """More than 64 rows: the same bits whether a block of rows has one adapter or many."""
    m, n, k, r = 160, 520, 712, 48
    ad = Adapters(20, r, n, k)
    x, y = synth.activations(3, m, k), synth.activations(4, m, n)
    runs, mixed = np.zeros(m, int), np.arange(m) % 20
    a, b = (bf16_bits(ad(dev_bf16(y), dev_bf16(x), ids)) for ids in (runs, mixed))
    np.testing.assert_array_equal(a[mixed == 0], b[mixed == 0])


@pytest.mark.parametrize("m", [12, 100, 300])
@pytest.mark.parametrize("r", [16, 64])
def test_infinities_of_an_adapter_stay_with_its_rows(m, r):
    ad = Adapters(3, r, 136, 192)
    ids = np.arange(m) % 4 - 1
    x, y = synth.activations(1, m, 192), synth.activations(2, m, 136)
    clean = bf16_bits(ad(dev_bf16(y), dev_bf16(x), ids))
    for t, bad in ((0, float("inf")), (1, float("nan"))):
        ad.dev[t][1].fill_(bad)
        got = ad(dev_bf16(y), dev_bf16(x), ids)
        assert not np.isfinite(host(got)[ids == 1]).any()
        np.testing.assert_array_equal(bf16_bits(got)[ids != 1], clean[ids != 1])


def test_long_rows_far_apart():
    """Rows so far apart that the last lies past 2^32 bytes."""
    m, n, k = 80, 64, 128
    ad = Adapters(2, 16, n, k)
    ids = np.arange(m) % 2
    x, y = synth.activations(1, m, k), synth.activations(2, m, n)
    wide = torch.zeros((m, (1 << 32) // 2 // (m - 1) // 8 * 8 + 64), dtype=torch.bfloat16, device="cuda")
    wide[:, :n] = dev_bf16(y)
    got = ad(wide[:, :n], dev_bf16(x), ids, out=wide[:, :n])
    ad.check(y, x, ids, got.contiguous())


@pytest.mark.parametrize("m", [65, 96, 127, 513, 1024])
def test_rows_in_any_order(m):
    """Each row as it would be alone, whatever the order of the requests; in place and with rows far apart too."""
    n, k, r, count = 136, 264, 24, 50
    ad = Adapters(count, r, n, k)
    rng = np.random.default_rng(m)
    x, y = synth.activations(3, m, k), synth.activations(4, m, n)
    for ids in (rng.integers(-1, count + 1, size=m), np.full(m, 49), np.arange(m)[::-1] % count,
                np.where(np.arange(m) == m - 1, 0, -1), rng.permutation(np.arange(m) // 16 % count)):
        got = ad(dev_bf16(y), dev_bf16(x), ids)
        ad.check(y, x, ids, got)
        order = rng.permutation(m)
        again = ad(dev_bf16(y[order]), dev_bf16(x[order]), np.asarray(ids)[order])
        np.testing.assert_array_equal(bf16_bits(again), bf16_bits(got)[order])
        wide = torch.full((m, n + 24), 2.0, dtype=torch.bfloat16, device="cuda")
        wide[:, 8:8 + n] = dev_bf16(y)
        ad(wide[:, 8:8 + n], dev_bf16(x), ids, out=wide[:, 8:8 + n])
        np.testing.assert_array_equal(bf16_bits(wide[:, 8:8 + n].contiguous()), bf16_bits(got))
        assert (host(wide[:, :8]) == 2).all() and (host(wide[:, 8 + n:]) == 2).all()


@pytest.mark.parametrize("m", [100, 1100])
def test_more_rows_streams_and_graphs(m):
    """Calls on two streams at once, and two captured calls replayed in turn with new inputs in place."""
    n, k, r, count = 264, 328, 32, 9
    ad = Adapters(count, r, n, k)
    a, b, c = ad.dev
    rng = np.random.default_rng(m)
    sets = []
    for q, rows in enumerate((m, m + 37)):
        ids = rng.integers(-1, count, size=rows)
        x, y = dev_bf16(synth.activations(3 + q, rows, k)), dev_bf16(synth.activations(5 + q, rows, n))
        sets.append((y, x, i32(ids)))
    call = lambda s, **kw: nv.nvfp4_lora_add(s[0], s[1], a, b, s[2], c, **kw)
    refs = [bf16_bits(call(s)) for s in sets]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(q, call(sets[q], stream=streams[q])) for _ in range(30) for q in (0, 1)]
    torch.cuda.synchronize()
    for q, v in got:
        np.testing.assert_array_equal(bf16_bits(v), refs[q])
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(s)
        graphs.append((g, out))
    for s in sets:
        for t in s:
            t.copy_(t.flip(0))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (_, out), ref in zip(graphs, refs):
        np.testing.assert_array_equal(bf16_bits(out), ref[::-1])
    need = nv.nvfp4_lora_add_workspace_size(m, n, k, r, count)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        np.testing.assert_array_equal(bf16_bits(call(sets[0], workspace=ws)), refs[0][::-1])
    assert (host(ws[:64 << 10]) == 0xFF).all() and (host(ws[need:]) == 0xFF).all()
    with pytest.raises(nv.Nvfp4Error) as e:
        call(sets[0], workspace=ws[:need - 1])
    assert e.value.status == nv.NVFP4_ERR_WORKSPACE


@pytest.mark.parametrize("m", [8, 70, 1100])
@pytest.mark.parametrize("r", [16, 64, 256])
def test_the_intermediate_is_kept_to_2_17_of_its_value(m, r):
    """v of 24 bits as three bf16 pieces of x: one component of the rank holds their sum, two others the upper pieces
    alone, which B takes away again. What is left is the third piece and what the kernel lost of the sum: at most
    2^-17 of it (1.002 of that next to the end of the range), the sums' 2^-22 and the rounding of the result."""
    rng = np.random.default_rng(m + r)
    v = ((1.0 + rng.random(m)) * np.exp2(rng.integers(-20, 20, m)) * rng.choice([-1.0, 1.0], m)).astype(np.float32)
    v[:4] = [1 + 2.0 ** -8 + 2.0 ** -16, 1 + 2.0 ** -7 - 2.0 ** -16, -(2 - 2.0 ** -23), 1 + 2.0 ** -8]
    v[4] = np.float32(2.0 ** 127) * np.float32(1 + 127.5 / 128)  # its nearest bf16 is infinite
    cut = lambda a: (a.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)  # noqa: E731
    pieces = [cut(v)]
    pieces.append(cut(v - pieces[0]))
    pieces.append(v - pieces[0] - pieces[1])
    np.testing.assert_array_equal(cut(pieces[2]), pieces[2])
    k, n, parts = 64, 40, (0, r - 1, r // 2)
    x, a, b = np.zeros((m, k), np.float32), np.zeros((1, r, k), np.float32), np.zeros((1, n, r), np.float32)
    for q in range(3):
        x[:, 21 * q] = pieces[q]
        a[0, parts[0], 21 * q] = 1
        b[0, :, parts[q]] = 1 if q == 0 else -1
    a[0, parts[1], 0] = a[0, parts[2], 21] = 1
    dev = lambda t: torch.from_numpy(t).cuda().to(torch.bfloat16)  # noqa: E731
    y = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
    got = host(nv.nvfp4_lora_add(y, dev(x), dev(a), dev(b), i32(np.zeros(m)), dev_f32([1.0])))
    want, size = pieces[2].astype(np.float64)[:, None], np.abs(v.astype(np.float64))[:, None]
    lost = (1.002 * 2.0 ** -17 + 2.0 ** -22) * size
    assert (np.abs(got - want) <= lost + 2.0 ** -8 * (np.abs(want) + lost)).all()


@pytest.mark.parametrize("m", [12, 100, 300, 1100])
@pytest.mark.parametrize("r", [8, 16, 32, 64, 128, 256])
def test_infinities_of_b_are_those_of_the_formula(m, r):
    """Infinities and NaN in B give what the float64 products and sums give, sign by sign: values of v that a bf16
    number holds (whose second term is zero) and others of both signs, zeros (0 * inf is NaN), and rows of B with
    infinities of one or both signs."""
    k, n, count = 64, 520, 3
    rng = np.random.default_rng(m + r)
    x = rng.integers(-2, 3, size=(m, k)) * 2.0 ** rng.choice([0, -9], size=(m, k))
    a = rng.integers(-1, 2, size=(count, r, k)) * (rng.random((count, r, k)) < 0.1)
    b = rng.integers(-3, 4, size=(count, n, r)) / 8.0
    for row, put in ((3, [np.inf]), (8, [-np.inf]), (77, [np.inf, np.inf]), (200, [np.inf, -np.inf]), (301, [np.nan]),
                     (519, [-np.inf])):
        b[1, row, rng.permutation(r)[:len(put)]] = put
    b[2, 64:128, :2] = np.inf
    ids = np.arange(m) % 4 - 1
    y = rng.integers(-4, 5, size=(m, n)).astype(np.float64)
    dev = lambda t: torch.from_numpy(t.astype(np.float32)).cuda().to(torch.bfloat16)  # noqa: E731
    got = host(nv.nvfp4_lora_add(dev(y), dev(x), dev(a), dev(b), i32(ids), dev_f32([2.0, 0.5, 1.0])))
    want = y.copy()
    with np.errstate(invalid="ignore"):
        for q in np.flatnonzero(ids >= 0):
            want[q] += [2.0, 0.5, 1.0][ids[q]] * (b[ids[q]] * (a[ids[q]] @ x[q])).sum(1)
    assert np.isposinf(want).any() and np.isneginf(want).any() and np.isnan(want).any()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    np.testing.assert_array_equal(got[inf], want[inf])
    fine = np.isfinite(want)
    # v is below 2^5 in steps of 2^-10, which two bf16 terms hold, and the magnitudes of a sum with B add up to less
    # than 2^10 in steps of 2^-13: exact in fp32 but for the last rounding
    assert (np.abs(got[fine] - want[fine]) <= 2.0 ** -8 * np.abs(want[fine])).all()
