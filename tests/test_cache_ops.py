"""The operators around the paged attention without a GPU: pins of their oracle, and refusals.

Every refused call returns before any launch, so the pointers are never dereferenced.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle


@pytest.fixture(scope="module")
def b():
    from paged_kv_attention_28_gb300 import build
    build.build(quiet=True)
    from paged_kv_attention_28_gb300 import binding
    return binding


P = ctypes.c_void_p(1 << 20)
P2 = ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 4)
P2, P3 = ctypes.c_void_p(1 << 21), ctypes.c_void_p(1 << 22)
ODD1 = ctypes.c_void_p((1 << 20) + 1)


# ------------------------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_a_rotation(inter):
    r = np.random.default_rng(0)
    x, t = r.standard_normal((3, 8)), r.standard_normal(3)
    y = oracle.rotate(x, t, inter)
    assert np.allclose(oracle.rotate(y, -t, inter), x) and np.array_equal(y[:, 6:], x[:, 6:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    quarter = oracle.rotate(np.array([[1.0, 2.0]]), np.array([math.pi / 2]), inter)
    assert np.allclose(quarter, [[-2.0, 1.0]])


def test_dot_products_of_rotated_rows_go_by_the_distance():
    r = np.random.default_rng(1)
    q, k, f = r.standard_normal(16), r.standard_normal(16), 0.3 ** np.arange(8)
    dots = [oracle.rotate(q, f * (p + 7), False) @ oracle.rotate(k, f * p, False) for p in (0, 5, 1000)]
    assert np.allclose(dots, dots[0])


def test_norm_by_hand():
    assert np.allclose(oracle.rms_norm([3.0, 4.0], [1.0, 2.0], 0.0), np.array([3.0, 8.0]) / math.sqrt(12.5))


def test_key_weights_sum_to_the_queries():
    r = np.random.default_rng(2)
    q, kp = r.standard_normal((1, 3, 4, 8)), r.standard_normal((4, 2, 16, 8))
    table, lens = np.array([[2, 0]]), np.array([20])
    keys = kp[table[0]].transpose(1, 0, 2, 3).reshape(2, 32, 8)
    lse = np.array([[[math.log(np.exp(0.3 * keys[h // 2, :21 + i] @ q[0, i, h]).sum()) for i in range(3)] for h in range(4)]])
    w = oracle.key_weights(q, kp, table, lens, lse, 0.3)
    assert np.isnan(w[0, :, 23:]).all() and np.allclose(w[0, :, :23].sum(-1), [6.0, 6.0])
    one = oracle.key_weights(q, kp, table, lens, lse, 0.3, first=[2], last=[3])
    assert np.allclose(one[0, :, :23].sum(-1), [2.0, 2.0])


def test_evict_by_hand():
    kept, lens, sums = oracle.evict([6, 3], np.array([[[9, 1, 5, 5, 0, 2.0]], [[1, 2, 3, 7, 7, 7.0]]]), 4, 1, 1)
    assert kept == [[0, 2, 3, 5], [0, 1, 2]] and lens == [4, 3] and sums == [[9, 5, 5, 2], [1, 2, 3]]
    kept, _, _ = oracle.evict([4], np.array([[[0.0, float("nan"), 1.0, -0.0]]]), 2, 0, 0)
    assert kept == [[1, 2]]


def test_linear_by_hand():
    y = oracle.linear([[1.0, 2.0]], [[3.0, 4.0], [-1.0, 0.0]], [1.0, 0.5], "relu", [[0.25, 0.5]])
    assert np.allclose(y, [[12.25, 0.5]])
    assert np.allclose(oracle.linear([[0.0]], [[1.0]], None, "silu"), 0.0)


# ------------------------------------------------------------------------------------ refusals

def append_args(b, **kw):
    a = dict(q=P, k=P, v=P, qs=8 * 64, ks=2 * 64, vs=2 * 64, qn=None, kn=None, eps=1e-6, fr=P, rot=64, inter=0, pos=None,
             axes=1, pa=None, bt=P, pl=P, cl=None, out=P2, kp=P, vp=P, batch=1, chunk=1, mb=4, np=4, hq=8, hkv=2, d=64,
             page=16, dt=b.PKV_BF16)
    a.update(kw)
    return list(a.values()) + [None, None]


@pytest.mark.parametrize("bad,want", [
    (dict(q=None), -1), (dict(v=None), -1), (dict(out=None), -1), (dict(kp=None), -1), (dict(bt=None), -1),
    (dict(pl=None), -1), (dict(fr=None), -1), (dict(batch=-1), -1), (dict(chunk=-1), -1), (dict(mb=0), -1),
    (dict(hq=0), -1), (dict(dt=2), -1), (dict(rot=-8), -1), (dict(rot=72), -1), (dict(inter=2), -1), (dict(axes=0), -1),
    (dict(qs=8 * 64 - 4), -1), (dict(ks=64), -1), (dict(vs=130), -1), (dict(q=ODD), -1), (dict(k=ODD), -1),
    (dict(kp=ODD), -1), (dict(vp=ctypes.c_void_p((1 << 20) + 8)), -1), (dict(qn=P, eps=float("nan")), -1),
    (dict(qn=P, eps=-1.0), -1), (dict(qn=ODD), -1), (dict(q=P2, qs=1024), -1), (dict(k=P2), -1), (dict(v=P2), -1), (dict(kp=P2), -1), (dict(vp=P2), -1), (dict(out=P), -1), (dict(mb=1 << 28), -1),
    (dict(d=96, qs=8 * 96, ks=192, vs=192), -2), (dict(page=32), -2), (dict(rot=12), -2), (dict(axes=5), -2),
    (dict(batch=1 << 17), -2), (dict(batch=0), 0), (dict(chunk=0, q=None), 0),
])
def test_append_refuses(b, bad, want):
    assert b.lib.attn_qk_norm_rope_append(*append_args(b, **bad)) == want


@pytest.mark.parametrize("name", ["k", "v", "qn", "kn", "fr", "pos", "pa", "bt", "pl", "cl", "kp", "vp"])
def test_append_refuses_an_output_at_an_input(b, name):
    other = dict(vp=P3) if name != "vp" else dict(kp=P3)
    assert b.lib.attn_qk_norm_rope_append(*append_args(b, **{name: P2, **other})) == -1


def test_append_refuses_one_pool_for_keys_and_values(b):
    assert b.lib.attn_qk_norm_rope_append(*append_args(b)) == -1


def weights_args(b, **kw):
    a = dict(q=P, kp=P, vp=P, bt=P, ln=P, out=P, lse=None, si=P, so=P, batch=1, mb=4, np=4, hq=8, hkv=2, d=128, page=16,
             scale=0.1, decay=1.0, splits=0, dt=b.PKV_BF16, ws=P, wsz=1 << 30)
    a.update(kw)
    return list(a.values()) + [None, None]


@pytest.mark.parametrize("bad,want", [
    (dict(si=None), -1), (dict(so=None), -1), (dict(si=ODD), -1), (dict(so=ODD), -1), (dict(decay=float("inf")), -1),
    (dict(q=None), -1), (dict(hq=9), -1), (dict(scale=float("nan")), -1), (dict(dt=2), -1), (dict(splits=-1), -1),
    (dict(d=96), -2), (dict(hq=6), -2), (dict(page=8), -2), (dict(ws=None), -3), (dict(wsz=100), -3),
    (dict(ws=ctypes.c_void_p((1 << 20) + 16)), -3), (dict(batch=0, si=None, q=None), 0),
])
def test_decode_weights_refuses(b, bad, want):
    assert b.lib.attn_decode_paged_weights(*weights_args(b, **bad)) == want


def test_decode_weights_workspace(b):
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    for dt in (b.PKV_F32, b.PKV_BF16):
        got = b.decode_weights_workspace_size(3, 20, 8, 2, 128, 16, 4, dt)
        assert got == b.decode_workspace_size(3, 20, 8, 2, 128, 16, 4, dt) + up(3 * 8 * 320 * 4) + up(3 * 8 * 4)
    for bad in ((1, 0, 8, 8, 64, 16), (1, 4, 6, 4, 64, 16)):
        with pytest.raises(b.AttnError):
            b.decode_weights_workspace_size(*bad)
    with pytest.raises(b.AttnError):
        b.decode_weights_workspace_size(1, 4, 8, 8, 64, 16, 0, b.PKV_FP8_E4M3)


def evict_args(b, **kw):
    a = dict(kp=P, vp=P, bt=P, ln=P, s=P, nt=P, kept=P3, nl=P3, ns=P3, batch=1, mb=8, nb=2, np=16, hkv=2, d=64, page=16,
             budget=32, sink=4, recent=8, dt=b.PKV_BF16)
    a.update(kw)
    return list(a.values()) + [None, None]


@pytest.mark.parametrize("bad,want", [
    (dict(kp=None), -1), (dict(kept=None), -1), (dict(ns=None), -1), (dict(nt=None), -1), (dict(kp=ODD), -1), (dict(s=ODD), -1),
    (dict(budget=0), -1), (dict(budget=33), -1), (dict(sink=-1), -1), (dict(recent=-1), -1), (dict(sink=25), -1),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), -1), (dict(batch=-1), -1), (dict(mb=0), -1), (dict(nb=0), -1),
    (dict(dt=5), -1), (dict(mb=1 << 28), -1), (dict(mb=(1 << 26) + 1), -2), (dict(nl=P2, ln=P2), -1), (dict(s=P2, ns=P2), -1),
    (dict(kept=P2, nt=P2), -1), (dict(kept=P2, bt=P2), -1), (dict(d=96), -2), (dict(page=32, budget=64), -2), (dict(batch=70000), -2),
    (dict(batch=0, kp=None), 0),
])
def test_evict_refuses(b, bad, want):
    assert b.lib.attn_cache_evict(*evict_args(b, **bad)) == want


@pytest.mark.parametrize("out", ["kept", "nl", "ns"])
@pytest.mark.parametrize("name", ["kp", "vp", "bt", "ln", "s", "nt"])
def test_evict_refuses_an_output_at_an_input(b, out, name):
    own = dict(kept=ctypes.c_void_p(1 << 23), nl=ctypes.c_void_p(1 << 24), ns=ctypes.c_void_p(1 << 25), **{name: P2})
    own[out] = P2
    assert b.lib.attn_cache_evict(*evict_args(b, **own)) == -1


@pytest.mark.parametrize("one,two", [("kept", "nl"), ("kept", "ns"), ("nl", "ns")])
def test_evict_refuses_two_outputs_at_one_address(b, one, two):
    own = dict(kept=ctypes.c_void_p(1 << 23), nl=ctypes.c_void_p(1 << 24), ns=ctypes.c_void_p(1 << 25))
    own[one] = own[two]
    assert b.lib.attn_cache_evict(*evict_args(b, **own)) == -1


def chunk_args(b, **kw):
    a = dict(q=P, kp=P, bt=P, pl=P, cl=None, lse=P, si=P, so=P, batch=1, chunk=8, window=0, mb=4, np=4, hq=8, hkv=2,
             d=128, page=16, scale=0.1, decay=1.0, dt=b.PKV_BF16)
    a.update(kw)
    return list(a.values()) + [None, None]


@pytest.mark.parametrize("bad,want", [
    (dict(q=None), -1), (dict(lse=None), -1), (dict(si=None), -1), (dict(so=None), -1), (dict(kp=None), -1),
    (dict(q=ODD), -1), (dict(kp=ODD), -1), (dict(window=-1), -1), (dict(chunk=-1), -1), (dict(chunk=65), -1),
    (dict(scale=float("inf")), -1), (dict(decay=float("nan")), -1), (dict(hq=9), -1), (dict(dt=7), -1), (dict(mb=0), -1),
    (dict(dt=0), -2), (dict(d=64), -2), (dict(page=8, mb=8), -2), (dict(hq=6), -2), (dict(mb=(1 << 26) + 1), -2),
    (dict(batch=0, q=None), 0),
    (dict(chunk=0, q=None), 0),
])
def test_chunk_weights_refuses(b, bad, want):
    assert b.lib.attn_chunk_weights(*chunk_args(b, **bad)) == want


def linear_args(b, **kw):
    a = dict(x=P, w=P, bias=None, res=None, y=P2, m=4, n=8, k=64, act=0, dt=b.PKV_BF16)
    a.update(kw)
    return list(a.values()) + [None, None]


@pytest.mark.parametrize("bad,want", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(x=ODD), -1), (dict(w=ODD), -1), (dict(m=-1), -1),
    (dict(n=-1), -1), (dict(k=0), -1), (dict(act=5), -1), (dict(act=-1), -1), (dict(dt=3), -1),
    (dict(y=ctypes.c_void_p((1 << 20) + 1)), -1), (dict(x=P2), -1), (dict(w=P2), -1), (dict(bias=P2), -1), (dict(bias=ctypes.c_void_p((1 << 20) + 1)), -1),
    (dict(k=12), -2), (dict(dt=0), -2), (dict(m=0, x=None), 0), (dict(n=0, w=None), 0),
])
def test_linear_refuses(b, bad, want):
    assert b.lib.attn_linear(*linear_args(b, **bad)) == want


def test_binding_refuses_host_tensors_and_wrong_shapes(b):
    q = torch.zeros(1, 1, 8, 64)
    kp = torch.zeros(4, 2, 16, 64)
    i = torch.zeros(1, 4, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        b.qk_norm_rope_append(q, q[:, :, :2], q[:, :, :2], kp, kp, i, n)
    with pytest.raises(ValueError):
        b.decode_paged_weights(q[:, 0], kp, kp, i, n, torch.zeros(1, 2, 64), 0.1)
    with pytest.raises(ValueError):
        b.chunk_weights(q, kp, i, n, torch.zeros(1, 8, 1), torch.zeros(1, 2, 64), 0.1)
    with pytest.raises(ValueError):
        b.linear(q[0, 0], q[0, 0])
    with pytest.raises(ValueError):
        b.linear(q[0, 0], q[0, 0], activation="tanh")
    with pytest.raises(ValueError):
        b.cache_evict(kp, kp, i, n, torch.zeros(1, 2, 64), i, 16)


def test_native_calls_check_their_arguments(b):
    """What stands before any use of a device: argument counts, types, dimensions."""
    from paged_kv_attention_28_gb300 import _pycall
    x = torch.zeros(2, 3)
    for name in ("qk_norm_rope_append", "decode_paged_weights", "chunk_weights", "cache_evict", "linear"):
        with pytest.raises(TypeError, match="takes"):
            getattr(_pycall, name)(x)
    for bad in (None, 3, "x", [1.0]):
        with pytest.raises(TypeError, match="must be a tensor"):
            _pycall.linear(bad, x, None, None, x, 0, None, None)
    with pytest.raises(ValueError, match="x must have 2 dimensions, has 1"):
        _pycall.linear(x[0], x, None, None, x, 0, None, None)
    with pytest.raises(ValueError, match="w must have 2 dimensions"):
        b.linear(x, x[None])
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        b.linear(x, x)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        _pycall.linear(x.to("meta"), x, None, None, x, 0, None, None)
    kp = torch.zeros(4, 2, 16, 64)
    with pytest.raises(ValueError, match="k_pages has head_dim 64, q has 128"):
        b.chunk_weights(torch.zeros(1, 1, 8, 128), kp, x, x, x, x, 0.1)
    with pytest.raises(ValueError, match="k_pages must have 4 dimensions"):
        b.cache_evict(x, x, x, x, x, x, 1, kept=x, new_lens=x, new_sums=x)


def test_need_checks_a_tensor(b):
    from paged_kv_attention_28_gb300 import _pycall
    class T:
        dtype, shape = torch.int32, torch.Size((2, 3))
        get_device = staticmethod(lambda: 0)
        is_contiguous = staticmethod(lambda: True)
        data_ptr = staticmethod(lambda: 4096)
    assert _pycall.need(T, "t", 0, torch.int32, (2, 3)) == 4096 and _pycall.need(T, "t", 0, None, None) == 4096
    for bad in ((1, torch.int32, (2, 3)), (0, torch.int64, (2, 3)), (0, torch.int32, (3, 2)), (0, torch.int32, (2,))):
        with pytest.raises(ValueError):
            _pycall.need(T, "t", *bad)
    with pytest.raises(ValueError, match="t must be a CUDA tensor"):
        _pycall.need(torch.zeros(2), "t", 0, None, None)
    T.is_contiguous = staticmethod(lambda: False)
    with pytest.raises(ValueError, match="contiguous"):
        _pycall.need(T, "t", 0, None, None)
    with pytest.raises(ValueError, match="t must be a CUDA tensor"):
        _pycall.need(torch.zeros(2, device="meta"), "t", 0, None, None)
    with pytest.raises(AttributeError):
        _pycall.need(None, "t", 0, None, None)
