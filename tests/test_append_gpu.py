"""Norm, rotation and page write of new tokens (``attn_qk_norm_rope_append``) against the fp64 oracle.

Bars. With A = |y_a| + |y_b| of the element's pair after the norm (A = |y| where nothing turns),
the fp32 arithmetic is off by less than 2^-19 A: the sum of squares (128 terms, pairwise over
lanes and 8 in a row: 2^-20), its reciprocal root (2^-22), the phase's and sincospi's roundings
(2^-22 of a turn's slope each, times A) and six products and sums (6 x 2^-24). A bf16 output
adds half a step, 2^-8 of the value. Values are copied exactly.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_28_gb300 import build
    build.build(quiet=True)
    from paged_kv_attention_28_gb300 import binding
    return binding


class Case:
    def __init__(self, seed, batch, chunk, hq, hkv, d, dtype, lens, rot, axes=1, inter=False, norm=True, packed=False,
                 chunk_lens=None, far=0, spare=3):
        g = torch.Generator().manual_seed(seed)
        t = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dtype, self.inter, self.d = dtype, inter, d
        blocks = max(1, (max(lens) + chunk + 15) // 16)
        pages = batch * blocks + spare
        order = torch.randperm(pages, generator=g).to(torch.int32)
        self.table = order[:batch * blocks].view(batch, blocks).contiguous()
        self.k_pages = torch.randn(pages, hkv, 16, d, generator=g).to(t)
        self.v_pages = torch.randn(pages, hkv, 16, d, generator=g).to(t)
        x = (2 * torch.randn(batch, chunk, hq + 2 * hkv, d, generator=g)).to(t)
        self.x = x
        self.hq, self.hkv, self.packed = hq, hkv, packed
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.chunk_lens = None if chunk_lens is None else torch.tensor(chunk_lens, dtype=torch.int32)
        self.q_norm = (1 + 0.3 * torch.randn(d, generator=g)).to(t) if norm else None
        self.k_norm = (1 + 0.3 * torch.randn(d, generator=g)).to(t) if norm else None
        self.inv_freq = (1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)).float() if rot else None
        self.pair_axis = torch.randint(0, axes, (rot // 2,), generator=g).to(torch.int32) if axes > 1 else None
        self.pos = None
        if axes > 1 or far:
            self.pos = (torch.randint(-50, 5000, (axes, batch, chunk), generator=g) + far).to(torch.int32)
        self.q_out = torch.randn(batch, chunk, hq, d, generator=g).to(t)

    def parts(self, x):
        p = x[:, :, :self.hq], x[:, :, self.hq:self.hq + self.hkv], x[:, :, self.hq + self.hkv:]
        return p if self.packed else tuple(t.contiguous() for t in p)

    def call(self, b, **kw):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        kp, vp, out, err = c(self.k_pages), c(self.v_pages), c(self.q_out), torch.zeros(1, dtype=torch.int32, device="cuda")
        q, k, v = self.parts(c(self.x))
        b.qk_norm_rope_append(q, k, v, kp, vp, c(self.table), c(self.lens), chunk_lens=c(self.chunk_lens),
                              positions=c(self.pos), inv_freq=c(self.inv_freq), pair_axis=c(self.pair_axis),
                              q_norm=c(self.q_norm), k_norm=c(self.k_norm), eps=1e-5, interleaved=self.inter, out=out,
                              err_flag=err, **kw)
        torch.cuda.synchronize()
        return out.cpu(), kp.cpu(), vp.cpu(), int(err)

    def want(self):
        n = lambda t: None if t is None else t.double().numpy() if t.is_floating_point() else t.numpy()  # noqa: E731
        B, C = self.x.shape[:2]
        pos = self.pos if self.pos is not None else (self.lens[:, None] + torch.arange(C))[None]
        q, k, v = (n(t) for t in self.parts(self.x))
        args = (n(self.table), n(self.lens), n(self.chunk_lens), n(pos), n(self.inv_freq), n(self.pair_axis),
                n(self.q_norm), n(self.k_norm), 1e-5, self.inter)
        got = oracle.append(q, k, v, n(self.k_pages), n(self.v_pages), *args, n(self.q_out))
        # A of each element: |y| turned by no angle, summed over the pair
        zero = [None if t is None else np.zeros_like(t) for t in (n(pos),)][0]
        flat = oracle.append(q, k, v, n(self.k_pages), n(self.v_pages), n(self.table), n(self.lens), n(self.chunk_lens),
                             zero, n(self.inv_freq), n(self.pair_axis), n(self.q_norm), n(self.k_norm), 1e-5,
                             self.inter, n(self.q_out))
        return got, [self.pair_sum(np.abs(t)) for t in flat[:2]]

    def pair_sum(self, y):
        if self.inv_freq is None:
            return y
        n = len(self.inv_freq)
        lo, hi = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if self.inter else (slice(0, n), slice(n, 2 * n))
        s = y[..., lo] + y[..., hi]
        out = y.copy()
        out[..., lo] = s
        out[..., hi] = s
        return out


def check(case, got):
    (wq, wk, wv), (aq, ak) = case.want()
    half = 2.0 ** -8 if case.dtype == "bf16" else 2.0 ** -24
    for g, w, a, what in ((got[0], wq, aq, "q"), (got[1], wk, ak, "k")):
        g = g.double().numpy()
        bar = half * np.abs(w) + 2.0 ** -19 * a
        worst = np.max(np.abs(g - w) - bar)
        assert np.isfinite(g).all() and worst <= 0, (what, worst)
    assert np.array_equal(got[2].double().numpy(), wv)


@pytest.mark.parametrize("case", [
    dict(batch=1, chunk=1, hq=8, hkv=8, d=64, dtype="f32", lens=[0], rot=64),
    dict(batch=5, chunk=1, hq=32, hkv=8, d=128, dtype="bf16", lens=[0, 15, 16, 31, 200], rot=128, packed=True),
    dict(batch=2, chunk=33, hq=14, hkv=2, d=128, dtype="bf16", lens=[7, 0], rot=32, inter=True),
    dict(batch=3, chunk=20, hq=8, hkv=2, d=64, dtype="bf16", lens=[3, 16, 100], rot=64, axes=3, packed=True,
         chunk_lens=[20, 0, 11]),
    dict(batch=2, chunk=17, hq=4, hkv=1, d=128, dtype="f32", lens=[0, 40], rot=64, axes=2, inter=True, packed=True),
    dict(batch=1, chunk=1100, hq=2, hkv=1, d=128, dtype="bf16", lens=[5], rot=128, axes=4, chunk_lens=[1099]),
    dict(batch=1, chunk=1027, hq=3, hkv=3, d=64, dtype="f32", lens=[9], rot=8, norm=False),
    dict(batch=2, chunk=5, hq=8, hkv=8, d=64, dtype="bf16", lens=[30, 2], rot=0, norm=True),
    dict(batch=2, chunk=5, hq=8, hkv=4, d=128, dtype="bf16", lens=[30, 2], rot=0, norm=False, packed=True),
    dict(batch=2, chunk=9, hq=8, hkv=4, d=128, dtype="f32", lens=[30, 2], rot=128, far=2 ** 31 - 6000),
    dict(batch=2, chunk=9, hq=8, hkv=4, d=128, dtype="f32", lens=[30, 2], rot=128, far=-2 ** 31 + 50),
])
def test_append_matches_the_oracle(b, case):
    c = Case(11, **case)
    got = c.call(b)
    assert got[3] == 0
    check(c, got)


def test_queries_may_be_written_in_place(b):
    c = Case(12, 2, 9, 8, 4, 128, "bf16", [3, 20], 128, packed=False)
    q, k, v = (t.cuda() for t in c.parts(c.x))
    kp, vp = c.k_pages.cuda(), c.v_pages.cuda()
    b.qk_norm_rope_append(q, k, v, kp, vp, c.table.cuda(), c.lens.cuda(), inv_freq=c.inv_freq.cuda(),
                          q_norm=c.q_norm.cuda(), k_norm=c.k_norm.cuda(), eps=1e-5, out=q)
    torch.cuda.synchronize()
    check(c, (q.cpu(), kp.cpu(), vp.cpu()))


def test_bad_lengths_pages_and_axes_touch_only_their_rows(b):
    c = Case(13, 4, 6, 8, 4, 128, "bf16", [3, 20, 10, 30], 128, axes=2)
    c.lens[1] = -1
    c.table[2, 0] = 10 ** 6
    blocks = c.table.shape[1]
    c.lens[3] = blocks * 16 - 5  # 6 tokens do not fit
    c.pair_axis[7] = 2
    out, kp, vp, err = c.call(b)
    assert err == b.PKV_DEVERR_BAD_LEN | b.PKV_DEVERR_BAD_PAGE | b.PKV_DEVERR_BAD_AXIS
    assert torch.isnan(out[1]).all() and torch.isnan(out[2]).all() and torch.isnan(out[3]).all()
    pair = [7, 7 + 64]
    assert torch.isnan(out[0][..., pair]).all()
    rest = [i for i in range(128) if i not in pair]
    good = Case(13, 4, 6, 8, 4, 128, "bf16", [3, 20, 10, 30], 128, axes=2)
    o2, k2, _, e2 = good.call(b)
    assert e2 == 0 and torch.equal(out[0][..., rest], o2[0][..., rest])
    # only sequence 0's six slots changed in the pools
    changed = (vp != c.v_pages).any(-1)
    slots = {(int(c.table[0, 0]), s) for s in range(3, 9)}
    assert {(int(p), int(s)) for p, _, s in changed.nonzero()} <= slots
    assert not torch.isnan(vp).any()


def test_append_in_a_graph_on_another_stream(b):
    c = Case(14, 3, 1, 8, 4, 128, "bf16", [3, 20, 10], 128)
    q, k, v = (t.cuda() for t in c.parts(c.x))
    kp, vp, out, tab, lens = c.k_pages.cuda(), c.v_pages.cuda(), c.q_out.cuda(), c.table.cuda(), c.lens.cuda()
    fr, qn, kn = c.inv_freq.cuda(), c.q_norm.cuda(), c.k_norm.cuda()
    call = lambda: b.qk_norm_rope_append(q, k, v, kp, vp, tab, lens, inv_freq=fr, q_norm=qn, k_norm=kn, eps=1e-5, out=out)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    fresh = Case(15, 3, 1, 8, 4, 128, "bf16", [3, 20, 10], 128)
    fresh.lens += 1
    fresh.table, fresh.k_pages, fresh.v_pages = c.table, kp.cpu(), vp.cpu()
    fresh.q_norm, fresh.k_norm = c.q_norm, c.k_norm
    for dst, src in zip((q, k, v), fresh.parts(fresh.x)):
        dst.copy_(src)
    lens += 1
    g.replay()
    torch.cuda.synchronize()
    check(fresh, (out.cpu(), kp.cpu(), vp.cpu()))


def test_empty_calls_do_nothing(b):
    c = Case(16, 2, 4, 8, 4, 64, "f32", [3, 20], 64, chunk_lens=[0, 0])
    out, kp, vp, err = c.call(b)
    assert err == 0 and torch.equal(out, c.q_out) and torch.equal(kp, c.k_pages) and torch.equal(vp, c.v_pages)


def test_native_checks_of_real_tensors(b):
    """The call's quick look at its tensors, and what it says of those that are not in order."""
    from paged_kv_attention_28_gb300 import _pycall
    bf, dev = torch.bfloat16, "cuda"
    x, w = torch.randn(4, 64, dtype=bf, device=dev), torch.randn(16, 64, dtype=bf, device=dev)
    y, bias = torch.empty(4, 16, dtype=bf, device=dev), torch.zeros(16, dtype=bf, device=dev)
    flag = torch.zeros(1, dtype=torch.int32, device=dev)
    good = [x, w, bias, y, y, 0, flag, None]
    assert _pycall.linear(*good) == 0 and _pycall.linear(x, w, None, None, y, 0, None, torch.cuda.current_stream()) == 0
    for at, bad in ((0, x.float()), (0, x[:, ::2]), (0, x.T), (0, x.cpu()), (1, w.float()), (1, w[:, :32]), (1, w.cpu()),
                    (1, w.T.contiguous().T), (2, bias[:8]), (2, bias.float()), (2, bias[None]), (3, y.T), (3, y[:2]), (4, y.cpu()),
                    (4, y.half()), (4, y[:, :8]), (6, flag.float()), (6, flag.cpu())):
        with pytest.raises(ValueError):
            _pycall.linear(*good[:at], bad, *good[at + 1:])
    for at, bad in ((0, None), (4, None), (5, "relu"), (5, None), (6, 3), (7, 3)):
        with pytest.raises((TypeError, ValueError, AttributeError)):
            _pycall.linear(*good[:at], bad, *good[at + 1:])
    assert _pycall.linear(*good[:5], (1 << 32) + 1, flag, None) == b.PKV_ERR_INVALID_ARG  # does not wrap
    for t, d, s in ((x, bf, (4, 64)), (x, None, None), (x[:0], bf, (0, 64)), (x[1:], bf, x[1:].shape)):
        assert _pycall.need(t, "x", 0, d, s) == t.data_ptr()
    for t, d, s in ((x, torch.float16, None), (x, bf, (64, 4)), (x, bf, (4, 1 << 70)), (x[:, ::2], bf, None)):
        with pytest.raises(ValueError):
            _pycall.need(t, "x", 0, d, s)
    with pytest.raises(ValueError, match="current device"):
        _pycall.need(x, "x", 1, bf, None)
