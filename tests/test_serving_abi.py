"""The serving entry points without a GPU: struct layouts and the refusals,
which come before anything is enqueued."""
import ctypes

import pytest
import torch

A, B, MIS = 0x100000, 0x200000, 0x100004        # device addresses that are never followed


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    return _pq


def cache(pq, **over):
    c = pq.pq_kv_cache(A, B, A, B, 10, 4 * 64 * 64, 64 * 64, 64, pq.PQ_KV_8, 0, 64, 4, 64, 0)
    for k, v in over.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [({"format": 3}, 3), ({"format": 0, "dtype": 0}, 3), ({"dim": 72}, 2), ({"dim": 0}, 2), ({"dim": 272}, 2),
              ({"heads": 0}, 2), ({"page_size": 8}, 2), ({"page_size": 48}, 2), ({"page_size": 65536}, 2),
              ({"num_pages": 0}, 2), ({"page_stride": -8}, 2), ({"token_stride": 68}, 2), ({"token_stride": 56}, 2),
              ({"token_stride": 1 << 26}, 2), ({"head_stride": 12}, 2), ({"k": None}, 1), ({"v": None}, 1),
              ({"v": MIS}, 4), ({"k_param": None}, 1), ({"v_param": MIS}, 4), ({"reserved": 1}, 7)]


def append_args(pq, c):
    return [ctypes.addressof(c), pq.PQ_BF16, 3, A, 256, 64, B, 256, 64, A, A, A, 100, 64, 0, A, 8, 512, 64, B, 512, 64, None]


def load_args(pq, c):
    return [ctypes.addressof(c), pq.PQ_BF16, 2, 5, A, 4, 4, A, A, A, 256, 64, B, 256, 64, None]


def attn_args(pq, c):
    return [ctypes.addressof(c), pq.PQ_BF16, 2, 8, A, 512, 64, A, 4, 4, A, 0.125, 0, 0, B, 512, 64, A, B, 1 << 30, None]


def test_struct_layout(pq):
    assert ctypes.sizeof(pq.pq_kv_cache) == 88 and pq.pq_kv_cache.format.offset == 64
    assert ctypes.sizeof(pq.pq_rope_scaling) == 40 and pq.pq_rope_scaling.factor.offset == 8


def test_row_bytes(pq):
    assert [pq.pq_kv_row_bytes(f, 80) for f in range(4)] == [160, 80, 40, -1]
    assert pq.pq_kv_row_bytes(1, 72) == -1 and pq.pq_kv_row_bytes(1, 272) == -1


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_cache_descriptor(pq, over, status):
    c = cache(pq, **over)
    assert pq.lib.pq_kv_append(*append_args(pq, c)) == status
    assert pq.lib.pq_kv_load(*load_args(pq, c)) == status
    assert pq.lib.pq_attn_decode(*attn_args(pq, c)) == status
    assert pq.lib.pq_attn_decode_workspace_bytes(ctypes.addressof(c), 2, 8) == -1


def test_null_cache(pq):
    c = cache(pq)
    for fn, args in ((pq.lib.pq_kv_append, append_args), (pq.lib.pq_kv_load, load_args), (pq.lib.pq_attn_decode, attn_args)):
        a = args(pq, c)
        a[0] = None
        assert fn(*a) == 1


@pytest.mark.parametrize("at,value,status", [
    (1, 3, 3), (2, -1, 2), (3, None, 1), (3, MIS, 4), (4, 4, 2), (6, None, 1), (8, 12, 2), (9, None, 1), (9, MIS + 8, 4),
    (10, None, 1), (11, MIS, 4), (12, -1, 2), (13, 63, 2), (13, 66, 2), (14, 2, 3), (15, None, 1), (15, MIS, 4), (16, -1, 2),
    (17, 4, 2), (19, None, 1), (20, 4, 2), (11, None, 7), (2, 0, 0)])
def test_append_refusals(pq, at, value, status):
    c = cache(pq)
    a = append_args(pq, c)
    a[at] = value
    if at == 9 and value:
        a[at] = MIS
    assert pq.lib.pq_kv_append(*a) == status


def test_append_in_place_needs_equal_strides(pq):
    c = cache(pq)
    a = append_args(pq, c)
    a[19], a[20] = A, 1024
    assert pq.lib.pq_kv_append(*a) == 7


@pytest.mark.parametrize("at,value,status", [
    (1, 3, 3), (2, -1, 2), (2, 0, 7), (3, -1, 2), (4, None, 1), (4, MIS - 2, 4), (5, -1, 2), (6, -1, 2), (8, None, 1), (9, None, 1),
    (9, MIS, 4), (10, 4, 2), (12, None, 1), (3, 0, 0)])
def test_load_refusals(pq, at, value, status):
    c = cache(pq)
    a = load_args(pq, c)
    a[at] = value
    assert pq.lib.pq_kv_load(*a) == status


@pytest.mark.parametrize("at,value,status", [
    (1, 0, 3), (1, 3, 3), (2, -1, 2), (3, 0, 2), (3, 6, 2), (3, 65540, 2), (4, None, 1), (4, MIS, 4), (5, 4, 2), (7, None, 1),
    (7, MIS - 2, 4), (8, -1, 2), (9, -1, 2), (9, 1 << 30, 2), (10, None, 1), (11, float("nan"), 7), (12, -1, 7), (13, -1, 7),
    (14, None, 1), (15, 12, 2), (17, MIS - 2, 4), (18, None, 1), (18, MIS, 4), (19, 64, 7), (2, 0, 0)])
def test_attn_refusals(pq, at, value, status):
    c = cache(pq)
    a = attn_args(pq, c)
    a[at] = value
    assert pq.lib.pq_attn_decode(*a) == status


def test_attn_16_bit_types_agree(pq):
    c = cache(pq, format=0, dtype=2, token_stride=128, head_stride=128 * 64)
    assert pq.lib.pq_attn_decode(*attn_args(pq, c)) == 3


def test_workspace_size(pq):
    c = cache(pq)
    q = lambda b, h: pq.lib.pq_attn_decode_workspace_bytes(ctypes.addressof(c), b, h)  # noqa: E731
    assert q(0, 8) == 0 and q(1, 6) == -1 and q(-1, 8) == -1 and q(1, 0) == -1
    assert q(64, 8) >= q(1, 8) > 0 and q(1, 8) % 16 == 0
    a = attn_args(pq, c)
    a[19] = q(2, 8) - 16
    assert pq.lib.pq_attn_decode(*a) == 7


def test_rope_refusals(pq):
    ok = [pq.PQ_BF16, 3, 2, 64, 64, 0, 0, A, 128, 64, A, A, 100, B, 128, 64, None]
    for at, value, status in ((0, 3, 3), (5, 2, 3), (1, -1, 2), (2, -1, 2), (3, 0, 2), (3, 1025, 2), (4, 66, 2), (4, 7, 2),
                              (12, -1, 2), (7, None, 1), (13, None, 1), (10, None, 1), (11, None, 1), (7, A + 1, 4),
                              (10, A + 2, 4), (11, MIS, 4), (1, 0, 0), (2, 0, 0)):
        a = list(ok)
        a[at] = value
        assert pq.lib.pq_rope(*a) == status, (at, value)
    a = list(ok)
    a[13], a[14] = A, 256
    assert pq.lib.pq_rope(*a) == 7                  # in place with other strides


def test_rope_table_refusals(pq):
    def rc(max_pos=10, rot=64, base=1e4, s=None, table=A):
        return pq.lib.pq_rope_table(max_pos, rot, base, ctypes.addressof(s) if s else None, table, None)
    assert rc(max_pos=-1) == 2 and rc(rot=63) == 2 and rc(rot=0) == 2 and rc(rot=1026) == 2
    assert rc(base=1.0) == 7 and rc(base=float("inf")) == 7 and rc(table=None) == 1 and rc(table=MIS) == 4
    assert rc(max_pos=0, table=None) == 0
    assert rc(s=pq.rope_scaling(5, 2.0)) == 3 and rc(s=pq.rope_scaling(pq.PQ_ROPE_LINEAR, 0.5)) == 7
    assert rc(rot=2, s=pq.rope_scaling(pq.PQ_ROPE_NTK, 2.0)) == 2
    assert rc(s=pq.rope_scaling(pq.PQ_ROPE_YARN, 2.0)) == 7                          # no trained length
    assert rc(s=pq.rope_scaling(pq.PQ_ROPE_BANDS, 2.0, 8192, 1.0, 1.0)) == 7         # no band


def test_binding_checks(pq):
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    pos, table = torch.zeros(2, dtype=torch.int32), torch.zeros(4, 32, 2)
    with pytest.raises(ValueError):
        pq.pq_rope(x[0], pos, table, stream=0)
    with pytest.raises(ValueError):
        pq.pq_rope(x.transpose(1, 2), pos, table, stream=0)
    with pytest.raises(ValueError):
        pq.pq_rope(x, pos.long(), table, stream=0)
    with pytest.raises(TypeError):
        pq.pq_rope(x.double(), pos, table, stream=0)
    with pytest.raises(ValueError):
        pq.pq_rope(x, pos, table.double(), stream=0)
    with pytest.raises(ValueError):
        pq.KVCache(pq.PQ_KV_8, 16, torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 16, 64))
    with pytest.raises(ValueError):
        pq.KVCache(pq.PQ_KV_16, 32, x[None, :, :2], x[None, :, :2])
    with pytest.raises(pq.PQError):
        k = torch.zeros(2, 1, 16, 72, dtype=torch.bfloat16)
        c = pq.KVCache(pq.PQ_KV_16, 16, k, k)
        pq.attn_workspace(c, 1, 1, device="cpu")


def test_launch_failure_reports_pq_err_hip(pq):
    """Without a device the launch fails and says so.  Runs only where no GPU is visible."""
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible: this check needs a host without one")
    c = cache(pq)
    assert pq.lib.pq_kv_append(*append_args(pq, c)) == 6
    assert pq.lib.pq_kv_load(*load_args(pq, c)) == 6
    assert pq.lib.pq_attn_decode(*attn_args(pq, c)) == 6
    assert pq.lib.pq_rope(pq.PQ_BF16, 3, 2, 64, 64, 0, 0, A, 128, 64, A, A, 100, B, 128, 64, None) == 6
    assert pq.lib.pq_rope_table(10, 64, 1e4, None, A, None) == 6


def test_sizes_past_a_launch_are_refused(pq):
    """A grid's threads are counted in 32 bits, and the rotation's heads too."""
    rope = [pq.PQ_BF16, 3, 2, 64, 64, 0, 0, A, 128, 64, A, A, 100, B, 128, 64, None]
    for at, value in ((1, 2 ** 26 - 3), (1, 2 ** 40), (2, 2 ** 31 - 1), (2, 2 ** 30 + 1), (2, 2 ** 40)):
        a = list(rope)
        a[at] = value
        assert pq.lib.pq_rope(*a) == 2, (at, value)
    c = cache(pq)
    a = append_args(pq, c)
    a[2] = 2 ** 26 - 3
    assert pq.lib.pq_kv_append(*a) == 2
    a = load_args(pq, c)
    a[3] = 2 ** 28 - 15
    assert pq.lib.pq_kv_load(*a) == 2
    assert pq.lib.pq_rope_table(2 ** 27, 64, 1e4, None, A, None) == 2
    assert pq.pq_attn_decode_workspace_bytes(type("C", (), {"ptr": ctypes.addressof(c)}), 1, 65536) == -1
