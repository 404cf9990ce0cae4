"""The entry points around the packed product without a GPU: struct layout,
the refusals, which come before anything is enqueued, and whose memory a
workspace comes from."""
import contextlib
import ctypes
import types

import pytest
import torch

A, B, C = 0x100000, 0x200000, 0x300000        # device addresses that are never followed
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    return _pq


def norm_args(pq):
    return [pq.PQ_BF16, 3, 64, A, 64, B, 64, C, 64, A, pq.PQ_F32, 1e-6, B, 64, None, 0, None, A, None]


@pytest.mark.parametrize("at,value,status", [
    (0, 3, 3), (0, -1, 3), (1, -1, 2), (1, 1 << 31, 2), (2, 0, 2), (2, 32769, 2), (3, None, 1), (3, A + 1, 4), (5, B + 1, 4),
    (7, None, 1), (5, None, 7), (7, C + 1, 4), (9, None, 1), (9, A + 2, 4), (10, 3, 3), (11, 0.0, 7), (11, -1.0, 7), (11, NAN, 7),
    (11, INF, 7), (11, 1e-60, 7), (12, None, 7), (12, B + 1, 4), (14, C, 1), (17, A + 2, 4), (1, 0, 0)])
def test_norm_refusals(pq, at, value, status):
    a = norm_args(pq)
    a[at] = value
    assert pq.lib.pq_rmsnorm(*a) == status


def test_norm_overlaps(pq):
    def with_(**over):
        a = norm_args(pq)
        for k, v in over.items():
            a[int(k[1:])] = v
        return pq.lib.pq_rmsnorm(*a)
    assert with_(_7=A, _8=128) == 7                       # sum is x, another stride
    assert with_(_7=B, _8=128) == 7                       # sum is the residual, another stride
    assert with_(_12=A, _13=128) == 7                     # y is x, another stride
    assert with_(_12=A, _7=A) == 7                        # y and sum both x
    assert with_(_14=C, _15=64, _16=A) == 7               # both outputs
    assert with_(_12=C) == 7                              # y is sum
    assert with_(_12=None, _14=C, _15=64, _16=A + 2) == 4


def bwd_args(pq):
    return [pq.PQ_BF16, 3, 64, A, 64, A, pq.PQ_F32, A, B, 64, C, 64, B, 64, A, C, 1 << 20, None]


@pytest.mark.parametrize("at,value,status", [
    (0, 3, 3), (1, -1, 2), (1, 1 << 31, 2), (2, 0, 2), (2, 32769, 2), (3, None, 1), (3, A + 1, 4), (5, None, 1), (6, 5, 3),
    (7, None, 1), (7, A + 2, 4), (8, None, 1), (8, B + 1, 4), (10, C + 1, 4), (12, None, 1), (12, B + 1, 4), (13, 128, 7),
    (12, A, 7), (14, A + 2, 4), (15, None, 1), (15, C + 4, 4), (16, 16, 7)])
def test_norm_bwd_refusals(pq, at, value, status):
    a = bwd_args(pq)
    a[at] = value
    assert pq.lib.pq_rmsnorm_bwd(*a) == status


def test_norm_bwd_empty(pq):
    a = bwd_args(pq)
    a[1], a[14] = 0, None
    assert pq.lib.pq_rmsnorm_bwd(*a) == 0
    w = pq.pq_rmsnorm_bwd_workspace_bytes
    assert w(-1, 64) == -1 and w(3, 0) == -1 and w(3, 32769) == -1 and w(0, 64) == 0 and w(3, 64) % 16 == 0
    assert w(100000, 4096) >= 4096 * 4


@pytest.mark.parametrize("at,value,status", [
    (0, 3, 3), (1, -1, 2), (1, 1 << 31, 2), (2, 0, 2), (2, 65537, 2), (3, None, 1), (3, A + 1, 4), (5, None, 1), (7, None, 1),
    (7, B + 2, 4), (1, 0, 0)])
def test_rows_refusals(pq, at, value, status):
    a = [pq.PQ_BF16, 3, 100, A, 100, C, 100, B, None]
    a[at] = value
    assert pq.lib.pq_quantize_rows(*a) == status


def gemm_args(pq, e=None):
    return [pq.PQ_W2_SEQ, 5, 48, 128, A, 128, A, B, A, pq.PQ_BF16, ctypes.addressof(e) if e else None, pq.PQ_BF16, C, 48, B,
            1 << 30, None]


@pytest.mark.parametrize("at,value,status", [
    (0, 7, 3), (0, -1, 3), (1, -1, 2), (1, (1 << 24) + 1, 2), (2, -1, 2), (2, (1 << 24) + 1, 2), (3, 0, 2), (3, 96, 2),
    (3, 1 << 17, 2), (4, None, 1), (4, A + 8, 4), (5, 64, 2), (5, 136, 2), (6, None, 1), (6, A + 2, 4), (7, None, 1),
    (7, B + 8, 4), (8, None, 1), (8, A + 1, 4), (9, 2, 3), (11, 3, 3), (12, None, 1), (12, C + 1, 4), (15, -1, 7), (1, 0, 0),
    (2, 0, 0)])
def test_gemm_refusals(pq, at, value, status):
    a = gemm_args(pq)
    a[at] = value
    assert pq.lib.pq_gemm_a8(*a) == status


def test_gemm_refuses_more_tiles_than_a_launch(pq):
    a = gemm_args(pq)
    a[1] = a[2] = a[13] = 1 << 24
    assert pq.lib.pq_gemm_a8(*a) == 2
    a = gemm_args(pq)
    a[5] = (1 << 23) + 16
    assert pq.lib.pq_gemm_a8(*a) == 2


@pytest.mark.parametrize("over,status", [
    ({"activation": 5}, 3), ({"activation": -1}, 3), ({"combine": 2}, 3), ({"bias": A, "bias_dtype": 3}, 3),
    ({"bias": A + 2, "bias_dtype": 0}, 4), ({"other": C + 1}, 4), ({"other": C, "other_stride": 64}, 7), ({"reserved": 1}, 7)])
def test_epilogue_refusals(pq, over, status):
    e = pq.pq_epilogue()
    for k, v in over.items():
        setattr(e, k, v)
    assert pq.lib.pq_gemm_a8(*gemm_args(pq, e)) == status
    assert ctypes.sizeof(pq.pq_epilogue) == 40 and pq.pq_epilogue.bias_dtype.offset == 24


def test_gemm_workspace(pq):
    for m, n, k in ((0, 1, 64), (4, 17, 8256), (2, 640, 192)):        # what the binding takes pq_packed_bytes to be
        assert pq.pq_packed_bytes(m, n, k) == (k * pq.CODE_BITS[m] + 511) // 512 * ((n + 15) // 16) * 1024
    w = pq.pq_gemm_a8_workspace_bytes
    assert w(9, 1, 1, 64) == -1 and w(2, -1, 1, 64) == -1 and w(2, 1, 1, 65) == -1 and w(2, 1, 1, 1 << 17) == -1
    assert w(2, 0, 0, 64) == 0 and w(2, 1, 16, 64) % 16 == 0
    for m, n, k in ((100, 64, 16384), (64, 576, 1536), (333, 1600, 4352)):
        need = w(2, m, n, k)
        assert need >= 0 and need % 16 == 0
        if need:
            a = gemm_args(pq)
            a[1], a[2], a[3], a[5], a[13] = m, n, k, k, n
            a[15] = need - 1
            assert pq.lib.pq_gemm_a8(*a) == 7
            a[14] = None
            assert pq.lib.pq_gemm_a8(*a) == 1
            a[14], a[15] = B + 4, need
            assert pq.lib.pq_gemm_a8(*a) == 4


def distill_args(pq):
    return [pq.PQ_BF16, 3, 100, A, 100, 8, A, B, pq.PQ_F32, 2.0, A, B, C, 1.0, C, 100, None]


COMMON = [(0, 3, 3), (1, -1, 2), (1, 1 << 31, 2), (2, 0, 2), (2, (1 << 30) + 1, 2), (3, None, 1), (3, A + 1, 4), (5, 0, 2),
          (5, 1025, 2), (6, None, 1), (6, A + 2, 4), (7, None, 1), (7, B + 2, 4), (8, 3, 3), (9, 0.0, 7), (9, -1.0, 7),
          (9, NAN, 7), (9, INF, 7), (9, 1e-45, 7), (9, 1e45, 7), (10, A + 2, 4), (1, 0, 0)]


@pytest.mark.parametrize("at,value,status", COMMON + [(11, B + 2, 4), (12, C + 2, 4), (13, NAN, 7), (13, INF, 7), (14, C + 1, 4)])
def test_distill_refusals(pq, at, value, status):
    a = distill_args(pq)
    a[at] = value
    assert pq.lib.pq_distill(*a) == status


def test_distill_outputs_and_overlap(pq):
    a = distill_args(pq)
    a[11] = a[12] = a[14] = None
    assert pq.lib.pq_distill(*a) == 1
    a[14], a[15] = A, 128
    assert pq.lib.pq_distill(*a) == 7


@pytest.mark.parametrize("at,value,status", COMMON + [(11, None, 1), (11, B + 2, 4), (12, None, 1), (12, C + 2, 4), (13, None, 1),
                                                      (13, C + 1, 4)])
def test_distill_bwd_refusals(pq, at, value, status):
    a = [pq.PQ_BF16, 3, 100, A, 100, 8, A, B, pq.PQ_F32, 2.0, A, B, C, C, 100, None]
    a[at] = value
    assert pq.lib.pq_distill_bwd(*a) == status


# ------------------------------------------------------------- the binding

@pytest.fixture
def world(monkeypatch, pq):
    """The binding with a library that only notes its calls, CPU tensors standing for the current GPU's."""
    w = types.SimpleNamespace(pq=pq, current="the caller's", made=[], calls=[])

    @contextlib.contextmanager
    def on(s):
        before, w.current = w.current, s
        yield
        w.current = before
    empty = torch.empty

    def spy(*shape, device=None, **kw):
        w.made.append(w.current)
        return empty(*shape, **kw)

    def call(*args):
        w.calls.append(args)
        return 0
    def gemm(*args):
        w.calls.append(args)
        return 1 if args[-3] is None else 0         # a shape that needs a workspace
    monkeypatch.setattr(pq, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(pq, "_current_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    monkeypatch.setattr(pq, "lib", types.SimpleNamespace(
        pq_rmsnorm=call, pq_rmsnorm_bwd=call, pq_quantize_rows=call, pq_gemm_a8=gemm, pq_distill=call, pq_distill_bwd=call,
        pq_rmsnorm_bwd_workspace_bytes=lambda *a: 64, pq_gemm_a8_workspace_bytes=lambda *a: 64))
    w.spy = lambda: monkeypatch.setattr(torch, "empty", spy)
    return w


def test_workspaces_come_from_the_launch_stream(world):
    pq = world.pq
    h, y = torch.zeros(4, 64), torch.zeros(4, 16)
    dw, r, x8 = torch.zeros(64), torch.zeros(4), torch.zeros(4, 64, dtype=torch.int8)
    packed = torch.zeros(1024, dtype=torch.uint8)
    world.spy()
    pq.pq_rmsnorm_bwd(h, dw, r, h, torch.zeros(4, 64), dweight=dw, stream=77)
    pq.pq_gemm_a8(2, x8, r, packed, torch.zeros(16), y, stream=77)
    assert world.made == [("external", 77)] * 2 and [c[-1] for c in world.calls] == [77, 77, 77]
    assert [c[-2] for c in world.calls] == [64, 0, 64]      # the product is tried without one first
    pq.pq_gemm_a8(2, x8, r, packed, torch.zeros(16), y, stream=77, workspace=torch.zeros(64, dtype=torch.uint8))
    assert len(world.made) == 2


def test_binding_refuses_other_tensors(world, monkeypatch):
    pq = world.pq
    x, w, q, s = torch.zeros(4, 64), torch.zeros(64), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    packed, y = torch.zeros(1024, dtype=torch.uint8), torch.zeros(4, 16)
    z, ix, t = torch.zeros(4, 50), torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, 3)
    good = [lambda: pq.pq_rmsnorm(x, w, y=torch.zeros(4, 64)), lambda: pq.pq_quantize_rows(x, q, s),
            lambda: pq.pq_gemm_a8(2, q, s, packed, torch.zeros(16), y, stream=1), lambda: pq.pq_distill(z, ix, t, s, stream=1)]
    for f in good:
        f()
    bad = [lambda: pq.pq_rmsnorm(x[0], w, y=x), lambda: pq.pq_rmsnorm(x, w[:63], y=x), lambda: pq.pq_rmsnorm(x, w, y=x[:3]),
           lambda: pq.pq_rmsnorm(x, w, y=x.double()), lambda: pq.pq_rmsnorm(x, w, q=x, scale=s),
           lambda: pq.pq_rmsnorm(x, w, q=q, scale=s[:3]), lambda: pq.pq_rmsnorm(x.t(), s, y=torch.zeros(64, 4)),
           lambda: pq.pq_rmsnorm(x, w, y=x, residual=x.half(), sum=x), lambda: pq.pq_rmsnorm(x, w, y=x, rstd=s.double()),
           lambda: pq.pq_rmsnorm_bwd(x, w, s, x[:, :63], x), lambda: pq.pq_rmsnorm_bwd(x, w, s[:1], x, x),
           lambda: pq.pq_rmsnorm_bwd(x, w, s, x, x, dweight=s), lambda: pq.pq_quantize_rows(x, q.to(torch.uint8), s),
           lambda: pq.pq_gemm_a8(2, x, s, packed, torch.zeros(16), y), lambda: pq.pq_gemm_a8(2, q, s, packed[:1023], torch.zeros(16), y),
           lambda: pq.pq_gemm_a8(2, q, s, packed, torch.zeros(15), y), lambda: pq.pq_gemm_a8(2, q, s, packed, torch.zeros(16), y[:3]),
           lambda: pq.pq_gemm_a8(2, q, s, packed, torch.zeros(16), y, other=y.half()),
           lambda: pq.pq_gemm_a8(2, q, s, packed, torch.zeros(16), y, bias=s),
           lambda: pq.pq_distill(z, ix.long(), t, s), lambda: pq.pq_distill(z, ix, t[:, :2], s),
           lambda: pq.pq_distill(z, ix, t, torch.zeros(5)), lambda: pq.pq_distill(z, ix[:3], t[:3], s),
           lambda: pq.pq_distill_bwd(z, ix, t, s, s, z)]
    n = len(world.calls)
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("taken:", i)
    assert len(world.calls) == n
    with pytest.raises(TypeError):
        pq.pq_rmsnorm(x.double(), w, y=x.double())


def test_binding_refuses_tensors_of_another_device(world, monkeypatch):
    pq = world.pq
    monkeypatch.setattr(pq, "_current_device", lambda: 1)
    x, w = torch.zeros(4, 64), torch.zeros(64)
    for f in (lambda: pq.pq_rmsnorm(x, w, y=x), lambda: pq.pq_quantize_rows(x, x.to(torch.int8), torch.zeros(4)),
              lambda: pq.pq_distill(x, torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, 1), torch.zeros(4))):
        with pytest.raises(ValueError, match="current GPU"):
            f()
    monkeypatch.setattr(pq, "_current_device", lambda: 0)
    for where in (-1, 1):                       # the others: host memory, another GPU
        other, out = torch.zeros(4, 64), torch.zeros(64)
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: where if t is other or t is out else 0)
        for f in (lambda: pq.pq_rmsnorm(x, w, y=other), lambda: pq.pq_rmsnorm(x, out, y=x), lambda: pq.pq_rmsnorm(other, w, y=x)):
            with pytest.raises(ValueError, match="device|GPU"):
                f()
    assert not world.calls
