"""Decode with accumulated weights, and eviction, against the fp64 oracle.

Bars for the sums. A weight is exp(s - lse) with s = scale q . k. The dot product of D terms in
fp32 (at most D + 2 roundings of partial sums no larger than S = scale sum |q k|), the rounding
of logits in base 2 and of lse move s - lse by at most e = (D + 10) 2^-24 (S_max + |lse| + 4);
the exponential and its argument's rounding add 2^-20. A group's sum is then off by
sum_h w_h (2 e + 2^-20), and decay * sums_in by 2^-23 of itself.
"""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_attention_28_gb300 import workloads
from tests._compare import assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_28_gb300 import build
    build.build(quiet=True)
    from paged_kv_attention_28_gb300 import binding
    return binding


def logit_bar(c, lse, d):
    q, k = c.q.double().abs(), c.k_pages.double().abs().nan_to_num(0.0)
    s_max = float(c.scale * (q.amax(-1).amax(-1).amax() * k.sum(-1).amax()))
    return (d + 10) * 2.0 ** -24 * (s_max + float(np.abs(lse[np.isfinite(lse)]).max(initial=0.0)) + 4)


def sums_bar(c, lse, w, d):
    return np.abs(w) * (2 * logit_bar(c, lse, d) + 2.0 ** -20)


def run_decode(b, c, sums, decay=1.0, splits=0, in_place=True, err=None):
    dev = [t.cuda() for t in (c.q, c.k_pages, c.v_pages, c.block_table, c.kv_lens)]
    s = sums.cuda()
    o = s if in_place else torch.full_like(s, 7.0)
    out, lse, got = b.decode_paged_weights(*dev, s, c.scale, sums_out=o, decay=decay, num_splits=splits, err_flag=err)
    torch.cuda.synchronize()
    assert got.data_ptr() == o.data_ptr()
    return out.float().cpu().numpy(), lse.cpu().numpy(), got.cpu()


CASES = [
    (1, 8, 8, 64, "f32", [256], 0), (1, 1, 1, 64, "bf16", [1], 0), (3, 16, 8, 128, "f32", [17, 100, 0], 3),
    (2, 8, 8, 128, "bf16", [333, 16], 0), (4, 16, 8, 128, "bf16", [1, 129, 640, 15], 4),
    (3, 32, 8, 128, "bf16", [700, 33, 0], 5), (2, 32, 4, 128, "bf16", [1000, 128], 0),
    (2, 16, 2, 64, "bf16", [77, 300], 2), (2, 8, 2, 64, "f32", [31, 500], 0), (2, 8, 1, 128, "f32", [40, 90], 0),
    (70, 8, 2, 128, "bf16", [1 + 13 * i for i in range(70)], 1),
]


@pytest.mark.parametrize("batch,hq,hkv,d,dtype,lens,splits", CASES)
@pytest.mark.parametrize("decay,in_place", [(1.0, True), (0.75, False)])
def test_weights_match_the_oracle(b, batch, hq, hkv, d, dtype, lens, splits, decay, in_place):
    c = workloads.make_paged_decode(500 + batch + hq, batch, hq, hkv, d, 16, lens, num_pages=sum((n + 15) // 16 for n in lens) + 5,
                                    dtype=dtype)
    cap = c.block_table.shape[1] * 16
    sums = torch.rand(batch, hkv, cap, generator=torch.Generator().manual_seed(3))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse, got = run_decode(b, c, sums, decay, splits, in_place, err)
    assert int(err) == 0
    wo, wl = oracle.decode_paged(c.q.double().numpy(), c.k_pages.double().numpy(), c.v_pages.double().numpy(),
                                 c.block_table.numpy(), c.kv_lens.numpy(), c.scale)
    assert_close(out, wo, dtype, "out")
    assert_close(lse, wl, dtype, "lse")
    # a decode step is a chunk of one query whose own key is the last one
    lens_before = c.kv_lens.numpy() - 1
    has = np.array([n > 0 for n in lens])
    w = oracle.key_weights(c.q[:, None].double().numpy()[has], c.k_pages.double().numpy(), c.block_table.numpy()[has],
                           lens_before[has], wl[has][:, :, None], c.scale)
    bar = sums_bar(c, wl, w, d) + decay * 2.0 ** -23 * sums.double().numpy()[has]
    want = w + decay * sums.double().numpy()[has]
    live = ~np.isnan(w)
    g = got.double().numpy()[has]
    assert (np.abs(g - want)[live] <= bar[live]).all(), np.nanmax((np.abs(g - want) / bar)[live])
    # slots past the length are left as they were, also of empty sequences
    before = sums if in_place else torch.full_like(sums, 7.0)
    for i, n in enumerate(lens):
        assert torch.equal(got[i, :, n:], before[i, :, n:])
    # the plain decode's lse is the same; so is its output, but where the tensor cores take the
    # weights as one bf16 part there and as two here: then half a bf16 step of the weights (they sum
    # to 1, so at most of the largest value) and two roundings of the output lie between them
    dev = [t.cuda() for t in (c.q, c.k_pages, c.v_pages, c.block_table, c.kv_lens)]
    o2, l2 = b.decode_paged(*dev, c.scale, num_splits=splits)
    assert np.array_equal(l2.cpu().numpy(), lse)
    o2 = o2.float().cpu().numpy()
    if dtype == "bf16" and d == 128 and hq // hkv in (4, 8):
        top = float(c.v_pages.nan_to_num(0).double().abs().max())
        assert (np.abs(o2 - out) <= 2.0 ** -8 * (top + np.abs(o2) + np.abs(out))).all()
        # and the output here is off by its rounding, half a bf16 step, and by its weights: 2 e each
        # from the logits and the sum, 2^-16 for the two parts and the fp32 sums
        assert (np.abs(out - wo) <= 2.0 ** -8 * np.abs(wo) + (4 * logit_bar(c, wl, d) + 2.0 ** -16) * top).all()
    else:
        assert np.array_equal(o2, out)


@pytest.mark.parametrize("hq,hkv,dtype", [(8, 8, "f32"), (32, 8, "bf16")])
def test_bad_pages_and_lengths_do_not_spread(b, hq, hkv, dtype):
    lens = [200, 40, 60, 90]
    c = workloads.make_paged_decode(77, 4, hq, hkv, 128, 16, lens, num_pages=64, dtype=dtype)
    sums = torch.rand(4, hkv, c.block_table.shape[1] * 16, generator=torch.Generator().manual_seed(3))
    clean = run_decode(b, c, sums)
    c.block_table[1, 1] = -5
    c.kv_lens[2] = 10 ** 6
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse, got = run_decode(b, c, sums, err=err)
    assert int(err) == b.PKV_DEVERR_BAD_PAGE | b.PKV_DEVERR_BAD_LEN
    assert np.isnan(out[1]).all() and torch.isnan(got[1, :, :40]).all() and torch.equal(got[1, :, 40:], sums[1, :, 40:])
    assert np.isnan(out[2]).all() and torch.equal(got[2], sums[2])
    for i in (0, 3):
        assert np.array_equal(out[i], clean[0][i]) and torch.equal(got[i], clean[2][i])


def test_weights_without_lse_and_workspace_bounds(b):
    import ctypes
    c = workloads.make_paged_decode(78, 2, 8, 2, 128, 16, [50, 70], num_pages=16, dtype="bf16")
    q, kp, vp, bt, ln = (t.cuda() for t in (c.q, c.k_pages, c.v_pages, c.block_table, c.kv_lens))
    sums = torch.zeros(2, 2, bt.shape[1] * 16, device="cuda")
    _, _, want = b.decode_paged_weights(q, kp, vp, bt, ln, sums.clone(), c.scale)
    need = b.decode_weights_workspace_size(2, bt.shape[1], 8, 2, 128, 16)
    ws = torch.full((need + 512,), 170, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    args = [p(q), p(kp), p(vp), p(bt), p(ln), p(out), None, p(sums), p(sums), 2, bt.shape[1], kp.shape[0], 8, 2, 128,
            16, c.scale, 1.0, 0, b.PKV_BF16]
    assert b.lib.attn_decode_paged_weights(*args, p(ws), need - 1, None, None) == b.PKV_ERR_WORKSPACE
    assert b.lib.attn_decode_paged_weights(*args, p(ws), need, None, None) == b.PKV_OK
    torch.cuda.synchronize()
    assert torch.equal(sums, want) and bool((ws[need:] == 170).all())


def pools(g, pages, hkv, d, t):
    return torch.randn(pages, hkv, 16, d, generator=g).to(t), torch.randn(pages, hkv, 16, d, generator=g).to(t)


def make_evict(seed, lens, hkv, d, dtype, budget, blocks=None, kind="mixed"):
    g = torch.Generator().manual_seed(seed)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    B = len(lens)
    blocks = blocks or max(1, (max(lens) + 15) // 16)
    nb = (budget + 15) // 16
    pages = B * (blocks + nb) + 2
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table, new = order[:B * blocks].view(B, blocks).contiguous(), order[B * blocks:B * (blocks + nb)].view(B, nb).contiguous()
    kp, vp = pools(g, pages, hkv, d, t)
    s = torch.rand(B, hkv, blocks * 16, generator=g)
    if kind == "mixed":
        s = torch.where(s < 0.3, torch.zeros_like(s), (s * 8).round() * s.lt(0.7) + s.pow(6) * 40 * s.ge(0.7))
    elif kind == "equal":
        s = torch.full_like(s, 0.125)
    elif kind == "odd":  # infinities, NaN, negative, both zeros, subnormals, the type's lowest value
        pick = torch.tensor([float("inf"), float("nan"), -float("inf"), 0.0, -0.0, 1e-42, -1e-42, -3.4028234663852886e38,
                             3.4028234663852886e38, 1.0, -1.0, 0.5])
        s = pick[torch.randint(0, len(pick), s.shape, generator=g)]
    elif kind == "close":  # neighbouring floats
        s = (torch.full_like(s, 1.0).view(torch.int32) + torch.randint(0, 40, s.shape, generator=g, dtype=torch.int32)).view(torch.float32)
    return table, new, kp, vp, s, torch.tensor(lens, dtype=torch.int32)


def check_evict(b, lens, hkv, d, dtype, budget, sink, recent, kind="mixed", blocks=None, seed=5):
    table, new, kp, vp, s, ln = make_evict(seed, lens, hkv, d, dtype, budget, blocks, kind)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k2, v2 = kp.cuda(), vp.cuda()
    kept, nl, ns = b.cache_evict(k2, v2, table.cuda(), ln.cuda(), s.cuda(), new.cuda(), budget, sink, recent, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    kept, nl, ns, k2, v2 = kept.cpu(), nl.cpu(), ns.cpu(), k2.cpu(), v2.cpu()
    wk, wl, wn = oracle.evict(ln.numpy(), s.numpy(), budget, sink, recent)
    assert nl.tolist() == wl
    want_k, want_v = kp.clone(), vp.clone()
    for i in range(len(lens)):
        for h in range(hkv):
            keep = wk[i * hkv + h]
            assert kept[i, h].tolist() == keep + [-1] * (budget - len(keep)), (i, h)
            assert np.array_equal(ns[i, h, :len(keep)].numpy(), np.array(wn[i * hkv + h], dtype=np.float32), equal_nan=True)
            assert not ns[i, h, len(keep):].any()
            at, j = torch.tensor(keep, dtype=torch.long), torch.arange(len(keep))
            src, dst = table[i].long()[at // 16], new[i].long()[j // 16]
            want_k[dst, h, j % 16] = kp[src, h, at % 16]
            want_v[dst, h, j % 16] = vp[src, h, at % 16]
    # the kept rows moved, every other slot is as it was
    assert torch.equal(k2, want_k) and torch.equal(v2, want_v)


@pytest.mark.parametrize("lens,hkv,d,dtype,budget,sink,recent", [
    ([1], 1, 64, "bf16", 1, 0, 0), ([2], 1, 64, "f32", 1, 0, 0), ([2], 1, 64, "f32", 1, 1, 0), ([2], 3, 64, "f32", 1, 0, 1),
    ([0, 5, 40, 100], 2, 128, "bf16", 33, 2, 7), ([33, 34], 2, 128, "f32", 33, 0, 0), ([100, 64], 4, 64, "bf16", 48, 48, 0),
    ([100, 99], 1, 128, "bf16", 47, 20, 27), ([1025, 1024, 1023], 2, 64, "bf16", 1000, 4, 64), ([2300, 2048], 2, 128, "bf16", 2048, 4, 256),
    ([9000, 8200], 1, 64, "bf16", 500, 4, 32), ([33000, 20], 1, 64, "bf16", 1111, 4, 32), ([40000], 2, 64, "bf16", 30000, 0, 1),
])
def test_evict_matches_the_oracle(b, lens, hkv, d, dtype, budget, sink, recent):
    check_evict(b, lens, hkv, d, dtype, budget, sink, recent)


@pytest.mark.parametrize("kind", ["equal", "odd", "close"])
@pytest.mark.parametrize("lens,budget", [([500, 77], 76), ([9001], 3333), ([33333], 5000)])
def test_evict_orders_ties_and_odd_values(b, kind, lens, budget):
    check_evict(b, lens, 2, 64, "bf16", budget, 3, 11, kind=kind)


@pytest.mark.parametrize("top", [0x3f81, 0xff7f, 0x8000])  # 1.0078 ..., the most negative numbers, -0 and below
@pytest.mark.parametrize("few", [1, 2, 127, 128, 129, 300])
@pytest.mark.parametrize("n", [900, 5000])
def test_evict_among_keys_that_share_their_leading_digits(b, top, few, n):
    """`few` sums share 16 bits, some of them all 32; the budget ends among them, at every place."""
    g = torch.Generator().manual_seed(few)
    order = torch.randperm(n, generator=g)
    bits = torch.full((n,), 0x40000000, dtype=torch.int64) + torch.arange(n) * 4096  # above: 2 and more
    bits[n // 2:] = 0xff7fffff if top != 0xff7f else 0xff800000  # below: the lowest number, -infinity
    bits[n // 4:n // 4 + few] = (top << 16) + torch.randint(0, max(2, few // 2), (few,), generator=g) * 97
    row = (bits - (bits >= 1 << 31) * (1 << 32)).to(torch.int32).view(torch.float32)[order]
    sums = row.repeat(1, 1, 1)
    pad = (n + 15) // 16 * 16 - n
    sums = torch.cat((sums, torch.full((1, 1, pad), float("nan"))), -1).cuda()
    blocks = (n + 15) // 16
    kp = torch.zeros(blocks, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").view(1, -1)
    above = int((row > (torch.tensor([top << 16 if top < 0x8000 else (top << 16) - (1 << 32)], dtype=torch.int64)
                        .to(torch.int32).view(torch.float32))).sum())
    for budget in sorted({max(1, above - few), max(1, above - 1), above + 1, above + few // 2, above + few, n // 2 + few}):
        if budget >= n:
            continue
        nb = (budget + 15) // 16
        new = torch.arange(nb, dtype=torch.int32, device="cuda").view(1, -1)  # (what moves is not looked at)
        spare = torch.zeros(nb, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
        pool = torch.cat((kp, spare))
        kept, _, ns = b.cache_evict(pool, pool.clone(), table, torch.tensor([n], dtype=torch.int32, device="cuda"), sums,
                                    new + blocks, budget)
        wk, _, wn = oracle.evict(np.array([n]), sums.cpu().numpy(), budget, 0, 0)
        assert kept[0, 0].tolist() == wk[0], budget
        assert np.array_equal(ns[0, 0, :budget].cpu().numpy(), np.array(wn[0], dtype=np.float32))


@pytest.mark.parametrize("sink,recent,budget", [(16, 32, 48), (0, 48, 48), (48, 0, 48), (16, 31, 48), (0, 0, 48)])
def test_evict_when_sinks_and_recents_fill_the_budget(b, sink, recent, budget):
    check_evict(b, [700, 49, 5000], 2, 64, "bf16", budget, sink, recent, kind="odd")


def test_evict_reads_no_further_than_the_length(b):
    # a table wider than the sequences: entries and sums past the length are poison
    table, new, kp, vp, s, ln = make_evict(6, [40, 70], 2, 64, "bf16", 32, blocks=40)
    for i, n in enumerate([40, 70]):
        s[i, :, n:] = float("nan")
        table[i, (n + 15) // 16:] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, nl, _ = b.cache_evict(kp.cuda(), vp.cuda(), table.cuda(), ln.cuda(), s.cuda(), new.cuda(), 32, 1, 4, err_flag=err)
    wk, wl, _ = oracle.evict(ln.numpy(), s.numpy(), 32, 1, 4)
    assert int(err) == 0 and nl.tolist() == wl and kept.cpu().flatten(0, 1).tolist() == wk


def test_evict_flags_bad_lengths_and_pages(b):
    table, new, kp, vp, s, ln = make_evict(7, [64, 64, 64, 64], 1, 64, "bf16", 32)
    ln[0], ln[1] = -3, 10 ** 6
    table[2] = 10 ** 6  # bad source pages
    new[3, 1] = -1      # a bad target page
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k2, v2 = kp.cuda(), vp.cuda()
    kept, nl, ns = b.cache_evict(k2, v2, table.cuda(), ln.cuda(), s.cuda(), new.cuda(), 32, 0, 4, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == b.PKV_DEVERR_BAD_PAGE | b.PKV_DEVERR_BAD_LEN
    assert nl.tolist() == [0, 0, 32, 32] and bool((kept[:2] == -1).all()) and not bool(ns[:2].any())
    k2 = k2.cpu()
    assert torch.isnan(k2[new[2].long()]).all()
    src = kept[3, 0].cpu().long()
    assert torch.equal(k2[new[3, 0].long(), 0], kp[table[3].long()[src[:16] // 16], 0, src[:16] % 16])
    untouched = [p for p in range(kp.shape[0]) if p not in new.flatten().tolist()]
    assert torch.equal(k2[untouched], kp[untouched])


def test_evict_of_shared_pages_leaves_them_whole(b):
    table, new, kp, vp, s, ln = make_evict(8, [64, 64], 2, 64, "bf16", 20)
    table[1] = table[0]
    k2, v2 = kp.cuda(), vp.cuda()
    kept, _, _ = b.cache_evict(k2, v2, table.cuda(), ln.cuda(), s.cuda(), new.cuda(), 20, 2, 2)
    kept, k2 = kept.cpu().long(), k2.cpu()
    assert torch.equal(k2[table[0].long()], kp[table[0].long()])
    for i in range(2):
        for h in range(2):
            at, j = kept[i, h], torch.arange(20)
            assert torch.equal(k2[new[i].long()[j // 16], h, j % 16], kp[table[i].long()[at // 16], h, at % 16])


def test_decode_and_evict_in_graphs(b):
    lens, budget = [60, 75], 48
    table, new, kp, vp, s, ln = (t.cuda() for t in make_evict(9, lens, 2, 128, "bf16", budget, blocks=5))
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    sums = s.clone()
    ws = b.alloc_workspace(b.decode_weights_workspace_size(2, 5, 8, 2, 128, 16), "cuda")
    out, lse = torch.empty_like(q), torch.empty(2, 8, device="cuda")
    kept = torch.empty(2, 2, budget, dtype=torch.int32, device="cuda")
    nl, ns = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(2, 2, 48, device="cuda")

    def step():
        b.decode_paged_weights(q, kp, vp, table, ln, sums, 0.1, out=out, lse=lse, workspace=ws)
        b.cache_evict(kp, vp, table, ln, sums, new, budget, 2, 8, kept=kept, new_lens=nl, new_sums=ns)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    sums.copy_(s)
    q.copy_(torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(2)).bfloat16())
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (out, lse, sums, kept, nl, ns, kp, vp)]
    sums.copy_(s)
    step()
    torch.cuda.synchronize()
    for x, y in zip(got, (out, lse, sums, kept, nl, ns, kp, vp)):
        assert torch.equal(x, y)
