"""Calls at the edge of what the operators around the paged attention take: empty and padded chunks, infinite
values, results near the smallest numbers, more features than one kernel's grid holds, tables of many pages.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_kv_attention_28_gb300 import workloads
from tests.test_chunk_weights_gpu import make as make_chunk
from tests.test_weights_evict_gpu import check_evict

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_28_gb300 import build
    build.build(quiet=True)
    from paged_kv_attention_28_gb300 import binding
    return binding


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------ linear

@pytest.mark.parametrize("m,act", [(1, "none"), (3, "relu")])
def test_linear_with_more_features_than_the_few_token_kernel_has_tiles(b, m, act):
    """65535 tiles of 128 features are its grid's limit. One feature more; the weights are 2.3 GB."""
    n, k = 65535 * 128 + 1, 136
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
    w = torch.randn(4096, k, generator=g, device="cuda").bfloat16().repeat((n + 4095) // 4096, 1)[:n].contiguous()
    bias = torch.randn(n, generator=g, device="cuda").bfloat16()
    err = i32(0)
    got = b.linear(x, w, bias=bias, activation=act, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    z = (x.double() @ w[:4096].double().T).repeat(1, (n + 4095) // 4096)[:, :n] + bias.double()
    size = (x.double().abs() @ w[:4096].double().abs().T).repeat(1, (n + 4095) // 4096)[:, :n] + bias.double().abs()
    want = z.clamp(min=0) if act == "relu" else z
    # k products added in fp32 and the bias, one rounding each at most S; one rounding to bf16
    bar = (k + 2) * 2.0 ** -24 * size + 2.0 ** -8 * want.abs()
    assert bool(((got.double() - want).abs() <= bar).all())


@pytest.mark.parametrize("m,k", [(3, 8), (3, 512), (90, 8)])  # the tiled kernel, that of few tokens, the tiled one
def test_small_results_of_silu_and_gelu(b, m, k):
    """Results of 1e-36 and less, which bf16 still holds. y / (1 + 2^t) with |t| <= 136: t is off by 2^-24 of itself
    for each of at most five roundings (constants, y^2, fma, product), so 2^t by 136 * 5 * 2^-24 ln 2 < 2^-14 of
    itself, numbers below fp32's smallest normal by 2^-16 more at 2^-133; then half a step of bf16, or of its
    smallest numbers (2^-133)."""
    y = torch.tensor([-60.0, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -92.0, -1e-30, 1e-30, 90.0, 3e38, -3e38]).bfloat16()
    z = torch.tensor([-8.0, -9.875, -9.9375, -10.0, -10.0625, -10.125, -1e-30, 1e-30, 11.0, 3e38, -3e38]).bfloat16()
    for act, v in (("silu", y), ("gelu_tanh", z)):
        x, w = torch.zeros(m, k).bfloat16(), torch.zeros(len(v), k).bfloat16()
        x[:, 0] = 1.0
        w[:, 0] = v
        got = b.linear(x.cuda(), w.cuda(), activation=act).double().cpu()
        d = [float(t) for t in v]
        t = d if act == "silu" else [2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3) for a in d]
        want = torch.tensor([a / (1 + math.exp(-s)) if s > -700 else 0.0 for a, s in zip(d, t)], dtype=torch.float64)
        off = (got - want).abs()
        bar = (2.0 ** -8 + 2.0 ** -14 + 2.0 ** -16) * want.abs() + 2.0 ** -134
        assert bool((off <= bar).all()), (act, got[0], want)


@pytest.mark.parametrize("m,k", [(3, 8), (3, 512), (90, 8)])
def test_gelu_keeps_the_precision_of_small_results(b, m, k):
    """y Phi(y) from -13.5, where bf16's smallest numbers are, to 20. exp(-y^2 / 2) has an argument of at most 92, off by
    three roundings of 2^-24 each: 92 * 3 * 2^-24 < 2^-15 of the result, with the polynomial's 2^-20 less than 2^-14;
    numbers below fp32's smallest normal by 2^-149 / 2^-137 more. Then half a step of bf16, or of its smallest."""
    y = torch.cat((torch.arange(-13.5, 0, 0.125), torch.arange(0, 20, 0.25), torch.tensor([-1e-30, 1e-30, -3e-38, 0.01, -0.01,
                   -20.0, 3e38, -3e38]))).bfloat16()
    x, w = torch.zeros(m, k).bfloat16(), torch.zeros(len(y), k).bfloat16()
    x[:, 0] = 1.0
    w[:, 0] = y
    got = b.linear(x.cuda(), w.cuda(), activation="gelu").double().cpu()
    want = torch.tensor([0.5 * v * math.erfc(-v / math.sqrt(2)) for v in y.double().tolist()], dtype=torch.float64)
    bar = (2.0 ** -8 + 2.0 ** -14 + 2.0 ** -12 * (want.abs() < 2.0 ** -126)) * want.abs() + 2.0 ** -134
    off = (got - want).abs()
    assert bool((off <= bar).all()), (y[(off > bar).any(0)], got[:, (off > bar).any(0)])


# ------------------------------------------------------------------------------------ cache write

def test_append_flags_a_bad_length_without_new_tokens(b):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(4, 3, 4, 64, generator=g, device="cuda")
    kp, vp = torch.zeros(9, 2, 16, 64, device="cuda"), torch.zeros(9, 2, 16, 64, device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    out = torch.full_like(x, 7.0)
    for lens, news, flag in (((0, 32, 5, 9), (0, 0, 0, 0), 0), ((0, 33, 5, 9), (0, 0, 0, 0), 2), ((0, 3, -1, 9), (0, 0, 0, 0), 2),
                             ((0, 3, -1, 9), (0, 3, 0, 2), 2)):
        err = i32(0)
        b.qk_norm_rope_append(x, x[:, :, :2].contiguous(), x[:, :, 2:].contiguous(), kp, vp, table, i32(*lens),
                              chunk_lens=i32(*news), out=out, err_flag=err)
        assert int(err) == flag, (lens, news)
        for j, n in enumerate(news):
            assert torch.equal(out[j, :n], x[j, :n]) and bool((out[j, n:] == 7.0).all())
        out.fill_(7.0)


# ------------------------------------------------------------------------------------ weights over a chunk

@pytest.mark.parametrize("in_place,decay", [(True, 0.5), (False, 0.5), (False, 1.0), (True, 1.0)])
@pytest.mark.parametrize("window", [0, 32])
def test_an_empty_chunk_decays_the_sums(b, in_place, decay, window):
    """chunk_len 0, and the same said by chunk_lens."""
    lens, cap = [0, 1, 40, 640, 300], 640
    g = torch.Generator(device="cuda").manual_seed(3)
    kp = torch.randn(200, 2, 16, 128, generator=g, device="cuda").bfloat16()
    table = torch.arange(200, dtype=torch.int32, device="cuda").view(5, 40)
    sums = torch.rand(5, 2, cap, generator=g, device="cuda")
    want = sums * decay  # one rounding, as the call's
    for chunk in (0, 3):
        s = sums.clone()
        o = s if in_place else torch.full_like(s, 7.0)
        before = o.clone()
        err = i32(0)
        b.chunk_weights(torch.full((5, chunk, 8, 128), float("nan"), device="cuda").bfloat16(), kp, table, i32(*lens),
                        torch.full((5, 8, chunk), float("nan"), device="cuda"), s, 0.1, sums_out=o, decay=decay, window=window,
                        chunk_lens=i32(0, 0, 0, 0, 0) if chunk else None, err_flag=err)
        assert int(err) == 0
        for j, n in enumerate(lens):
            assert torch.equal(o[j, :, :n], want[j, :, :n]) and torch.equal(o[j, :, n:], before[j, :, n:])


def test_an_empty_chunk_flags_bad_lengths_and_pages(b):
    kp = torch.randn(8, 2, 16, 128, device="cuda").bfloat16()
    table = i32(*range(8)).view(4, 2).contiguous()
    table[1, 1] = 99
    sums = torch.ones(4, 2, 32, device="cuda")
    out, err = torch.full_like(sums, 7.0), i32(0)
    b.chunk_weights(torch.zeros(4, 0, 8, 128, device="cuda").bfloat16(), kp, table, i32(32, 20, 33, -1),
                    torch.zeros(4, 8, 0, device="cuda"), sums, 0.1, sums_out=out, decay=0.25, err_flag=err)
    assert int(err) == b.PKV_DEVERR_BAD_LEN | b.PKV_DEVERR_BAD_PAGE
    assert bool((out[0] == 0.25).all()) and bool((out[1, :, :16] == 0.25).all()) and bool(out[1, :, 16:20].isnan().all())
    assert bool((out[1, :, 20:] == 7.0).all()) and bool((out[2:] == 7.0).all())


@pytest.mark.parametrize("prefix,n,pad,window", [([3, 0], [10, 16], 40, 0), ([0, 200], [30, 7], 600, 0), ([5, 9], [20, 0], 100, 8)])
def test_a_chunk_padded_past_the_table(b, prefix, n, pad, window):
    """Padding may be wider than the table; the new tokens that count fit."""
    q, kp, table, pl, lse, sums, _ = make_chunk(11, prefix, max(n), 8, 2, n, extra=0)
    B, hq, scale = len(prefix), 8, 128 ** -0.5
    used = max(p + x for p, x in zip(prefix, n))
    blocks = (used + 15) // 16
    assert pad > blocks * 16
    table, sums = table[:, :blocks].contiguous(), sums[:, :, :blocks * 16].contiguous()
    qp = torch.full((B, pad, hq, 128), float("nan")).bfloat16()
    qp[:, :max(n)] = q
    lp = torch.full((B, hq, pad), float("nan"))
    lp[:, :, :max(n)] = lse
    err = i32(0)
    got = b.chunk_weights(qp.cuda(), kp.cuda(), table.cuda(), pl.cuda(), lp.cuda(), sums.cuda(), scale, window=window,
                          chunk_lens=torch.tensor(n, dtype=torch.int32).cuda(), err_flag=err).cpu()
    assert int(err) == 0
    first = [max(0, x - window) if window else 0 for x in n]
    w = oracle.key_weights(q.nan_to_num(0).double().numpy(), kp.double().numpy(), table.numpy(), pl.numpy(),
                           lse.nan_to_num(0).double().numpy(), scale, first=first, last=n)
    # a weight's logit is off by 2^-23 (128 S + 4 (S + |lse|)); n weights add n + 8 roundings; the old sum one more
    S = scale * float(q.nan_to_num(0).double().abs().amax() * kp.nan_to_num(0).double().abs().sum(-1).amax())
    e = 2.0 ** -23 * (128 * S + 4 * (S + float(lse.nan_to_num(0).abs().max())))
    for j in range(B):
        end = prefix[j] + n[j]
        old = sums[j, :, :end].double().numpy()
        want = w[j, :, :end] + old
        bar = w[j, :, :end] * (2 * e + 2.0 ** -20 + (4 * max(n) + 8) * 2.0 ** -24) + (want + old) * 2.0 ** -23
        assert (np.abs(got[j, :, :end].double().numpy() - want) <= bar).all()
        assert torch.equal(got[j, :, end:], sums[j, :, end:])


def test_unwritten_slots_of_a_padded_chunk_may_hold_any_finite_value(b):
    """Cache write and chunked prefill of ragged chunks: the prefill's padding queries read the slots behind a
    sequence, which the cache write has left as they were. The queries that count come out the same,
    bit for bit, whatever finite values are there."""
    g = torch.Generator(device="cuda").manual_seed(7)
    B, C, hq, hkv, n, prefix = 3, 90, 8, 2, (90, 1, 61), i32(0, 37, 100)
    x = torch.randn(B, C, hq + 2 * hkv, 128, generator=g, device="cuda").bfloat16()
    table = torch.randperm(60, generator=g, device="cuda")[:36].to(torch.int32).view(B, 12).contiguous()
    old = torch.randn(60, hkv, 16, 128, generator=g, device="cuda").bfloat16()
    got = []
    for junk in (0.0, 1.0, 1e30, -3e38):
        kp, vp = (torch.full((60, hkv, 16, 128), junk, device="cuda").bfloat16() for _ in range(2))
        for j in range(B):  # the prefix's tokens
            for t in range(int(prefix[j])):
                p = int(table[j, t // 16])
                kp[p, :, t % 16], vp[p, :, t % 16] = old[p, :, t % 16], old[p, :, 15 - t % 16]
        q = b.qk_norm_rope_append(x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], kp, vp, table, prefix,
                                  chunk_lens=i32(*n), out=torch.zeros(B, C, hq, 128, device="cuda").bfloat16())
        err = i32(0)
        out, lse = b.prefill_paged_chunk(q, kp, vp, table, prefix, 128 ** -0.5, err_flag=err)
        s = b.chunk_weights(q, kp, table, prefix, lse, torch.zeros(B, hkv, 192, device="cuda"), 128 ** -0.5,
                            chunk_lens=i32(*n), err_flag=err)
        assert int(err) == 0
        got.append([out[j, :n[j]] for j in range(B)] + [lse[j, :, :n[j]] for j in range(B)] + [s])
    for other in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], other))
    assert all(bool(t.isfinite().all()) for t in got[0])
    count = torch.tensor([hq // hkv * float(x) for x in n], device="cuda")
    assert bool(((got[0][-1].sum(-1) - count[:, None]).abs() < 1e-3 * count[:, None]).all())


# ------------------------------------------------------------------------------------ decode with weights

@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 2, 128), (8, 8, 128), (8, 4, 64)])
def test_infinite_values_reach_the_output_as_infinities(b, hq, hkv, d, splits):
    """An infinite element of V makes its output element infinite, as the plain decode does, since every weight is
    above 0; of both signs, or a NaN, it makes it NaN. The other elements and the sums do not change."""
    lens = [200, 40]
    c = workloads.make_paged_decode(31, 2, hq, hkv, d, 16, lens, num_pages=20, dtype="bf16")
    dev = [t.cuda() for t in (c.q, c.k_pages, c.v_pages, c.block_table, c.kv_lens)]
    sums = torch.zeros(2, hkv, c.block_table.shape[1] * 16, device="cuda")
    clean, _, s0 = b.decode_paged_weights(*dev, sums.clone(), c.scale, num_splits=splits)
    at = [(int(t), int(e)) for t, e in zip(torch.arange(0, 200, 3), torch.arange(200) % (d - 5))]  # (token, element) of sequence 0
    want = clean.clone()
    for t, e in at:
        dev[2][int(c.block_table[0, t // 16]), :, t % 16, e] = float("inf")
        want[0, :, e] = float("inf")
    page = lambda t: int(c.block_table[1, t // 16])  # noqa: E731
    inf = float("inf")
    for t, e, x in ((0, 0, -inf), (39, 1, -inf), (5, 2, inf), (20, 2, -inf), (7, d - 1, float("nan"))):
        dev[2][page(t), :, t % 16, e] = x
        want[1, :, e] = x if e < 2 else float("nan")
    got, _, s1 = b.decode_paged_weights(*dev, sums.clone(), c.scale, num_splits=splits)
    plain, _ = b.decode_paged(*dev, c.scale, num_splits=splits)
    assert torch.equal(s0, s1)
    for y in (got, plain):
        assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.isinf(), want.isinf())
        assert torch.equal(y[want.isinf()], want[want.isinf()])
    assert torch.equal(got[want.isfinite()], want[want.isfinite()])


# ------------------------------------------------------------------------------------ eviction

@pytest.mark.parametrize("kind", ["mixed", "equal", "odd", "close"])
@pytest.mark.parametrize("lens,budget,sink,recent,blocks", [
    ([53249, 30], 4000, 4, 64, None), ([60001], 59990, 0, 1, None), ([70000, 65536], 1, 0, 0, None),
    ([2000, 1, 0, 57], 56, 2, 9, 3400), ([66000], 300, 150, 150, None),
])
def test_evict_from_tables_past_the_rows_kept_in_shared_memory(b, kind, lens, budget, sink, recent, blocks):
    """Rows of more than 53248 tokens, and short sequences in tables that could hold as many."""
    check_evict(b, lens, 1, 64, "bf16", budget, sink, recent, kind=kind, blocks=blocks)


def test_evict_reads_no_further_than_the_length_in_a_wide_table(b):
    n, blocks, budget = 1500, 4000, 100
    g = torch.Generator().manual_seed(3)
    order = torch.randperm(110, generator=g).to(torch.int32)
    table = torch.full((1, blocks), -1, dtype=torch.int32)
    table[0, :94] = order[:94]
    s = torch.full((1, 1, blocks * 16), float("nan"))
    s[0, 0, :n] = torch.rand(n, generator=g)
    kp = torch.randn(110, 1, 16, 64, generator=g).cuda()
    err = i32(0)
    kept, nl, _ = b.cache_evict(kp, kp.clone(), table.cuda(), i32(n), s.cuda(), order[94:101].view(1, 7).cuda(), budget, 1, 4,
                                err_flag=err)
    wk, _, _ = oracle.evict([n], s.numpy(), budget, 1, 4)
    assert int(err) == 0 and int(nl) == budget and kept[0, 0].tolist() == wk[0]
