"""Weights that keys receive from a chunk's queries (``attn_chunk_weights``) against the fp64 oracle.

Bars. A weight is exp(s - lse) for the lse given. The product of 128 bf16 pairs accumulates in
fp32, one unit in the last place (2^-23) of at most S = scale sum |q k| per addition; scaling to
base 2 and subtracting the lse round at most 4 times at magnitude S + |lse|. So s - lse is off by
e = 2^-23 (128 S + 4 (S + |lse|)), the weight by w (2 e + 2^-20) with the exponential, and the sum of n
weights adds n + 8 roundings: (n + 8) 2^-24 of the sum. decay * sums_in rounds once (2^-24).
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


def make(seed, prefix, chunk, hq, hkv, chunk_lens=None, extra=1, std=1.0):
    """Pages whose slots past a sequence's end are NaN, as are padding queries and their lse."""
    g = torch.Generator().manual_seed(seed)
    B = len(prefix)
    n = [chunk] * B if chunk_lens is None else chunk_lens
    blocks = (max(prefix) + chunk + 15) // 16 + extra
    order = torch.randperm(B * blocks + 2, generator=g).to(torch.int32)
    table = order[:B * blocks].view(B, blocks).contiguous()
    kp = torch.randn(B * blocks + 2, hkv, 16, 128, generator=g).bfloat16()
    q = (std * torch.randn(B, chunk, hq, 128, generator=g)).bfloat16()
    lse = torch.full((B, hq, chunk), float("nan"))
    for i in range(B):
        used = (prefix[i] + n[i] + 15) // 16
        kp[table[i, used:].long()] = float("nan")
        if (prefix[i] + n[i]) % 16:
            kp[table[i, used - 1].long(), :, (prefix[i] + n[i]) % 16:] = float("nan")
        table[i, used:] = -1
        q[i, n[i]:] = float("nan")
        keys = kp[table[i, :used].long()].double().permute(1, 0, 2, 3).reshape(hkv, -1, 128)
        for j in range(n[i]):
            z = 128 ** -0.5 * torch.einsum("hgd,htd->hgt", q[i, j].double().view(hkv, hq // hkv, 128), keys[:, :prefix[i] + j + 1])
            lse[i, :, j] = z.logsumexp(-1).flatten().float()
    sums = torch.rand(B, hkv, blocks * 16, generator=g)
    for i in range(B):
        sums[i, :, prefix[i] + n[i]:] = 5.0
    return q, kp, table, torch.tensor(prefix, dtype=torch.int32), lse, sums, n


def check(b, prefix, chunk, hq, hkv, window=0, chunk_lens=None, decay=1.0, in_place=True, std=1.0):
    q, kp, table, pl, lse, sums, n = make(1000 + chunk + hq, prefix, chunk, hq, hkv, chunk_lens, std=std)
    scale = 128 ** -0.5
    first = [max(0, x - window) if window else 0 for x in n]
    w = oracle.key_weights(q.nan_to_num(0).double().numpy(), kp.double().numpy(), table.numpy(), pl.numpy(),
                           lse.nan_to_num(0).double().numpy(), scale, first=first, last=n)
    S = scale * float(q.nan_to_num(0).double().abs().amax() * kp.nan_to_num(0).double().abs().sum(-1).amax())
    e = 2.0 ** -23 * (128 * S + 4 * (S + float(lse.nan_to_num(0).abs().max())))
    cols = max([x - f for x, f in zip(n, first)] + [0]) * (hq // hkv)
    s = sums.cuda()
    o = s if in_place else torch.full_like(s, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cl = None if chunk_lens is None else torch.tensor(chunk_lens, dtype=torch.int32).cuda()
    b.chunk_weights(q.cuda(), kp.cuda(), table.cuda(), pl.cuda(), lse.cuda(), s, scale, sums_out=o, decay=decay,
                    window=window, chunk_lens=cl, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    got = o.cpu()
    before = sums if in_place else torch.full_like(sums, 7.0)
    for i in range(len(prefix)):
        end = prefix[i] + n[i]
        assert torch.equal(got[i, :, end:], before[i, :, end:])
        old = decay * sums[i, :, :end].double().numpy()
        want = w[i, :, :end] + old
        bar = w[i, :, :end] * (2 * e + 2.0 ** -20 + (cols + 8) * 2.0 ** -24) + (want + old) * 2.0 ** -23
        off = np.abs(got[i, :, :end].double().numpy() - want)
        assert (off <= bar).all(), (i, float(np.max(off / bar)))


@pytest.mark.parametrize("prefix,chunk,hq,hkv,kw", [
    ([0], 1, 1, 1, {}), ([0], 1, 8, 2, {}), ([255], 1, 8, 2, {}), ([256, 0], 1, 8, 8, {}), ([300, 17], 33, 8, 2, dict(decay=0.5)),
    ([0, 100], 129, 16, 2, dict(in_place=False)), ([40, 700], 70, 8, 1, dict(window=32)), ([5], 300, 4, 4, dict(window=1)),
    ([300, 20, 0], 64, 32, 2, dict(chunk_lens=[64, 0, 13], window=20)), ([511, 513], 20, 16, 4, dict(chunk_lens=[1, 20])),
    ([1000], 40, 128, 1, {}), ([30, 2], 90, 2, 1, dict(window=500)), ([128], 130, 8, 2, dict(std=6.0)),
    ([0, 0], 600, 4, 2, dict(decay=-0.5)),
])
def test_chunk_weights_match_the_oracle(b, prefix, chunk, hq, hkv, kw):
    check(b, prefix, chunk, hq, hkv, **kw)


def test_many_items_per_cta(b):
    check(b, [37 * i % 1500 for i in range(48)], 24, 16, 8)


def test_more_sequences_than_lengths_kept_in_shared_memory(b):
    check(b, [(7 * i) % 23 for i in range(2100)], 2, 1, 1)


def test_bad_lengths_and_pages(b):
    q, kp, table, pl, lse, sums, n = make(5, [100, 200, 300], 40, 8, 2)
    clean = b.chunk_weights(q.cuda(), kp.cuda(), table.cuda(), pl.cuda(), lse.cuda(), sums.cuda(), 0.1).cpu()
    pl[0] = -7
    table[1, 3] = 10 ** 6
    cl = torch.tensor([40, 40, 41], dtype=torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = b.chunk_weights(q.cuda(), kp.cuda(), table.cuda(), pl.cuda(), lse.cuda(), sums.cuda(), 0.1,
                          chunk_lens=cl.cuda(), err_flag=err).cpu()
    assert int(err) == b.PKV_DEVERR_BAD_LEN | b.PKV_DEVERR_BAD_PAGE
    assert torch.equal(got[0], sums[0]) and torch.equal(got[2], sums[2])
    bad = torch.zeros(got.shape[2], dtype=torch.bool)
    bad[48:64] = True
    assert torch.isnan(got[1][:, bad]).all() and torch.equal(got[1][:, ~bad], clean[1][:, ~bad])


def test_after_the_chunked_prefill_the_weights_sum_to_the_queries(b):
    """The lse of the chunked prefill on the same inputs: every query spreads a weight of 1."""
    g = torch.Generator().manual_seed(8)
    kp, vp = (torch.randn(80, 4, 16, 128, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.randperm(80, generator=g)[:72].to(torch.int32).view(2, 36).cuda()
    pl = torch.tensor([0, 301], dtype=torch.int32).cuda()
    q = torch.randn(2, 256, 16, 128, generator=g).bfloat16().cuda()
    _, lse = b.prefill_paged_chunk(q, kp, vp, table, pl, 128 ** -0.5)
    for window, count in ((0, 256), (32, 32)):
        sums = torch.zeros(2, 4, 36 * 16, device="cuda")
        b.chunk_weights(q, kp, table, pl, lse, sums, 128 ** -0.5, window=window)
        total = sums.double().sum(-1).cpu()
        # per weight the bar above is 2 e with S < 30; the sum's own rounding is smaller
        assert ((total / (4 * count) - 1).abs() < 2 * 2.0 ** -23 * 132 * 30 + 2.0 ** -18).all()


def test_chunk_weights_in_a_graph(b):
    q, kp, table, pl, lse, sums, _ = (t.cuda() if torch.is_tensor(t) else t for t in make(6, [100, 30], 40, 8, 2))
    out = torch.zeros_like(sums)
    call = lambda: b.chunk_weights(q, kp, table, pl, lse, sums, 0.1, sums_out=out)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    sums.mul_(3)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, call())


def test_dozens_of_items_per_cta_from_cold_memory(b):
    """Long caches under a short window: a CTA's rings of tiles turn over many times while pages come late and out of
    order. Every call gives the same bits, and they are right."""
    B, prefix, chunk, hq, hkv, scale = 16, 8192, 40, 32, 8, 128 ** -0.5
    g = torch.Generator(device="cuda").manual_seed(5)
    blocks = (prefix + chunk + 15) // 16
    table = torch.randperm(B * blocks, device="cuda", generator=g).to(torch.int32).view(B, blocks)
    kp = torch.randn(B * blocks, hkv, 16, 128, device="cuda", generator=g, dtype=torch.bfloat16)
    q = torch.randn(B, chunk, hq, 128, device="cuda", generator=g, dtype=torch.bfloat16)
    pl = torch.tensor([prefix - 100 * i for i in range(B)], dtype=torch.int32, device="cuda")
    lse = 9.0 + torch.rand(B, hq, chunk, device="cuda", generator=g)
    sums = torch.rand(B, hkv, blocks * 16, device="cuda", generator=g)
    flush = torch.zeros(192 << 20, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for window in (1, 32):
        got = []
        for _ in range(6):
            flush.zero_()
            got.append(b.chunk_weights(q, kp, table, pl, lse, sums, scale, sums_out=torch.full_like(sums, 7.0), window=window,
                                       err_flag=err))
        assert int(err) == 0
        assert all(torch.equal(got[0], x) for x in got[1:])
        for i in range(B):
            n = int(pl[i]) + chunk
            keys = kp[table[i].long()].permute(1, 0, 2, 3).reshape(hkv, -1, 128)[:, :n].double()
            z = torch.einsum("qhgd,htd->hqgt", q[i, chunk - window:].double().view(window, hkv, hq // hkv, 128), keys) * scale
            seen = torch.arange(n, device="cuda") <= n - window + torch.arange(window, device="cuda")[:, None]
            w = (z - lse[i, :, chunk - window:].double().view(hkv, hq // hkv, window).permute(0, 2, 1)[..., None]).exp()
            w = (w * seen[None, :, None]).sum((1, 2))
            # the product's 128 additions, the exponent's roundings, the sum over the columns, the final addition
            top = scale * float(q[i].double().abs().amax() * keys.abs().sum(-1).amax())
            e = 2.0 ** -23 * (128 * top + 4 * (top + 10.0))
            want = w + sums[i, :, :n].double()
            bar = w * (2 * e + 2.0 ** -20 + (window * hq // hkv + 8) * 2.0 ** -24) + (want + sums[i, :, :n].double()) * 2.0 ** -23
            off = (got[0][i, :, :n].double() - want).abs()
            assert bool((off <= bar).all()), (window, i, float((off / bar).max()))
            assert bool((got[0][i, :, n:] == 7.0).all())


def test_more_items_than_the_list_of_one_cta_per_sm(b):
    """5000 sequences of a page with 16 KV heads: 80000 items, which take more CTAs than the device has SMs."""
    B, h, scale = 5000, 16, 128 ** -0.5
    g = torch.Generator(device="cuda").manual_seed(8)
    table = torch.randperm(B, device="cuda", generator=g).to(torch.int32).view(B, 1)
    kp = torch.randn(B, h, 16, 128, device="cuda", generator=g, dtype=torch.bfloat16)
    q = torch.randn(B, 1, h, 128, device="cuda", generator=g, dtype=torch.bfloat16)
    pl = (torch.arange(B, device="cuda") % 16).to(torch.int32)
    lse = 3.0 + torch.rand(B, h, 1, device="cuda", generator=g)
    sums = torch.rand(B, h, 16, device="cuda", generator=g)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = b.chunk_weights(q, kp, table, pl, lse, sums, scale, sums_out=torch.full_like(sums, 7.0), err_flag=err)
    assert int(err) == 0
    keys = kp[table[:, 0].long()].double()
    w = (torch.einsum("bhd,bhtd->bht", q[:, 0].double(), keys) * scale - lse.double()).exp()
    top = scale * float(q.double().abs().amax() * keys.abs().sum(-1).amax())
    bar = w * (2.0 ** -22 * (128 * top + 4 * (top + 4.0)) + 2.0 ** -20) + (w + 2 * sums.double()) * 2.0 ** -23
    live = (torch.arange(16, device="cuda") <= pl[:, None])[:, None].expand_as(w)
    off = (got.double() - (w + sums.double())).abs()
    assert bool((off <= bar)[live].all()) and bool((got[~live] == 7.0).all())


@pytest.mark.parametrize("prefix,chunk,hq,hkv,kw", [
    ([40, 25], 500, 32, 4, {}), ([40, 25], 500, 32, 4, dict(chunk_lens=[500, 3])), ([0], 700, 32, 8, dict(in_place=False)),
    ([900, 1, 300], 130, 64, 16, dict(window=129)), ([0, 0, 0, 0], 200, 16, 16, dict(chunk_lens=[200, 1, 0, 199])),
])
def test_items_shared_by_more_clusters_than_fit_at_once(b, prefix, chunk, hq, hkv, kw):
    check(b, prefix, chunk, hq, hkv, **kw)
