"""Linear layer with its epilogue (``attn_linear``) against the fp64 oracle.

Bars. The fp32 accumulation of k exact products is off by at most (k + 2) 2^-23 S, S = sum |x w|;
every activation's slope is below 1.13, and its own arithmetic and the residual's add stay below
2^-20 (|pre| + |result|); the one rounding to bf16 is half a step, 2^-8 of the result.
On average the accumulation's roundings add up like a random walk: sqrt(k) 2^-23 S.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_28_gb300 import build
    build.build(quiet=True)
    from paged_kv_attention_28_gb300 import binding
    return binding


def make(seed, m, n, k, bias, res, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (std * torch.randn(m, k, generator=g)).bfloat16()
    w = (torch.randn(n, k, generator=g) / k ** 0.5).bfloat16()
    return (x, w, torch.randn(n, generator=g).bfloat16() if bias else None,
            torch.randn(m, n, generator=g).bfloat16() if res else None)


def check(got, x, w, bias, act, res):
    d = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    k = x.shape[1]
    pre = oracle.linear(d(x), d(w), d(bias))
    want = oracle.linear(d(x), d(w), d(bias), act, d(res))
    S = np.abs(d(x)) @ np.abs(d(w)).T
    g = got.double().cpu().numpy()
    small = 2.0 ** -20 * (np.abs(pre) + np.abs(want) + (np.abs(d(res)) if res is not None else 0))
    bar = 2.0 ** -8 * np.abs(want) + 1.13 * (k + 2) * 2.0 ** -23 * S + small
    off = np.abs(g - want)
    assert (off <= bar).all(), float(np.max(off / bar))
    mean = 2.0 ** -8 * np.abs(want).mean() + (1.13 * k ** 0.5 * 2.0 ** -23 * S + small).mean()
    assert off.mean() <= mean


@pytest.mark.parametrize("m,n,k", [
    (1, 1, 8), (1, 130, 72), (8, 256, 512), (16, 1000, 200), (17, 96, 264), (33, 384, 128), (64, 4097, 64),
    (65, 64, 64), (65, 1, 8), (66, 33, 72), (129, 257, 192), (200, 1000, 136), (128, 256, 1024), (700, 640, 320),
    (1111, 1111, 88), (300, 20000, 64), (2500, 4104, 128),
])
@pytest.mark.parametrize("act,bias,res", [("none", False, False), ("gelu_tanh", True, True), ("silu", False, True)])
def test_linear_matches_the_oracle(b, m, n, k, act, bias, res):
    x, w, bi, re = make(m + n + k, m, n, k, bias, res)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = b.linear(c(x), c(w), bias=c(bi), activation=act, residual=c(re), err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(got, x, w, bi, act, re)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [5, 100])
def test_activations_over_a_wide_range(b, act, m):
    x, w, bi, re = make(3, m, 200, 64, True, False, std=8.0)
    got = b.linear(x.cuda(), w.cuda(), bias=bi.cuda(), activation=act)
    check(got, x, w, bi, act, re)


@pytest.mark.parametrize("m", [3, 90])
@pytest.mark.parametrize("act", ACTS)
def test_infinities_and_nan(b, act, m):
    x = torch.zeros(m, 64).bfloat16()
    w = torch.zeros(16, 64).bfloat16()
    x[:, 0] = 1.0
    w[:4, 0] = torch.tensor([float("inf"), float("nan"), -100.0, 100.0]).bfloat16()
    got = b.linear(x.cuda(), w.cuda(), activation=act).float().cpu()[:, :4]
    assert torch.isinf(got[:, 0]).all() and torch.isnan(got[:, 1]).all()
    assert (got[:, 2].abs() <= (0 if act != "none" else 100)).all() and (got[:, 3] == 100).all()


@pytest.mark.parametrize("m,n", [(7, 64), (100, 64), (100, 33)])
def test_residual_in_place_and_nothing_beyond(b, m, n):
    x, w, bi, re = make(4, m, n, 128, True, True)
    buf = torch.full((m * n + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    y = buf[:m * n].view(m, n)
    y.copy_(re)
    got = b.linear(x.cuda(), w.cuda(), bias=bi.cuda(), activation="relu", residual=y, out=y)
    check(got, x, w, bi, "relu", re)
    assert bool((buf[m * n:] == 3.0).all())


def test_rows_that_are_not_aligned(b):
    """y, the residual and the bias two bytes off a 16-byte boundary."""
    x, w, bi, re = make(5, 140, 320, 128, True, True)
    shift = lambda t: torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)  # noqa: E731
    y = torch.empty(140 * 320 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(140, 320)
    got = b.linear(x.cuda(), w.cuda(), bias=shift(bi), activation="gelu", residual=shift(re), out=y)
    check(got, x, w, bi, "gelu", re)
    got = b.linear(x.cuda(), w.cuda(), bias=shift(bi), activation="gelu", residual=re.cuda())
    check(got, x, w, bi, "gelu", re)


@pytest.mark.parametrize("m", [8, 300])
def test_linear_in_a_graph(b, m):
    x, w, bi, re = make(6, m, 512, 256, True, True)
    xs, ws, bs, rs = (t.cuda() for t in (x, w, bi, re))
    y = torch.empty_like(rs)
    call = lambda: b.linear(xs, ws, bias=bs, activation="silu", residual=rs, out=y)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    x2 = make(7, m, 512, 256, False, False)[0]
    xs.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    check(y, x2, w, bi, "silu", re)


@pytest.mark.parametrize("m", [1, 32, 33, 64, 65])
@pytest.mark.parametrize("n,k", [(1024, 128), (1024, 136), (1000, 1024), (1000, 1032), (2064, 1032), (2062, 1032), (33, 72), (4097, 200)])
def test_linear_on_both_sides_of_the_choice_of_kernel(b, m, n, k):
    """Sizes beside the bounds at which another kernel takes over, with rows of every alignment and a residual in place."""
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    x, w = (torch.randn(*s, device="cuda", generator=g).bfloat16() for s in ((m, k), (n, k)))
    bias, y = (torch.randn(*s, device="cuda", generator=g).bfloat16() for s in ((n,), (m, n)))
    res = y.clone()
    b.linear(x, w, bias, "relu", y, out=y)
    z = x.double() @ w.double().T + bias.double()
    want = z.clamp(min=0) + res.double()
    # k products added in fp32 (each sum at most S, k roundings), bias and residual; one rounding to bf16
    size = x.double().abs() @ w.double().abs().T + bias.double().abs() + res.double().abs()
    bar = (k + 4) * 2.0 ** -24 * size + 2.0 ** -8 * want.abs()
    assert bool(((y.double() - want).abs() <= bar).all())
