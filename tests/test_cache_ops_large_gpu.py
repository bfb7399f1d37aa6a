"""The operators around the paged attention where offsets pass 32 bits, and on two streams at once."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_attention_28_gb300 import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_28_gb300 import build
    build.build(quiet=True)
    from paged_kv_attention_28_gb300 import binding
    return binding


def test_pages_past_four_gigabytes(b):
    """Pools of 135000 pages (8 heads, head_dim 128, bf16: 4.4 GB each), the work at their end, gives
    what it gives in a small pool."""
    g = torch.Generator(device="cuda").manual_seed(1)
    hkv, hq, n_pages = 8, 32, 135000
    small = [torch.randn(24, hkv, 16, 128, generator=g, device="cuda").bfloat16() for _ in range(2)]
    big = [torch.empty(n_pages, hkv, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for s, l in zip(small, big):
        l[n_pages - 24:] = s
    table = torch.randperm(24, generator=g, device="cuda").to(torch.int32).view(2, 12)
    tab, new = table[:, :7].contiguous(), table[:, 7:].contiguous()
    shift = n_pages - 24
    x = torch.randn(2, 3, hq + 2 * hkv, 128, generator=g, device="cuda").bfloat16()
    freq = (1e4 ** (-torch.arange(64, device="cuda") / 64)).float()
    lens = torch.tensor([50, 90], dtype=torch.int32, device="cuda")
    sums0 = torch.rand(2, hkv, 7 * 16, generator=g, device="cuda")
    got = []
    for pools, t, n in ((small, tab, new), (big, tab + shift, new + shift)):
        q = b.qk_norm_rope_append(x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], *pools, t, lens, inv_freq=freq)
        end = lens + 3
        _, lse = b.prefill_paged_chunk(q, *pools, t, lens, 128 ** -0.5)
        sums = b.chunk_weights(q, pools[0], t, lens, lse, sums0.clone(), 128 ** -0.5)
        o, l, sums = b.decode_paged_weights(q[:, 2].contiguous(), *pools, t, end, sums, 128 ** -0.5, num_splits=3)
        kept, nl, ns = b.cache_evict(*pools, t, end, sums, n, 40, 2, 8)
        torch.cuda.synchronize()
        got.append([q, lse, o, l, sums[:, :, :53], kept, nl, ns] + [p[n.long()][:, :2] for p in pools] + [p[t.long()] for p in pools])
    for s, l in zip(*got):
        assert torch.equal(s, l)


@pytest.mark.parametrize("hq,hkv,dtype", [(64, 8, "bf16"), (64, 32, "f32")])
def test_logits_past_two_billion(b, hq, hkv, dtype):
    """A table of 2^20 pages per sequence: the scratch and the sums are indexed past 2^31."""
    lens = [70, 0, 33]
    c = workloads.make_paged_decode(9, 3, hq, hkv, 128, 16, lens, num_pages=12, dtype=dtype)
    blocks = 1 << 20
    table = torch.full((3, blocks), -1, dtype=torch.int32)
    table[:, :c.block_table.shape[1]] = c.block_table
    q, kp, vp, ln = (t.cuda() for t in (c.q, c.k_pages, c.v_pages, c.kv_lens))
    narrow = torch.zeros(3, hkv, c.block_table.shape[1] * 16, device="cuda")
    o1, l1, s1 = b.decode_paged_weights(q, kp, vp, c.block_table.cuda(), ln, narrow, c.scale, num_splits=1)
    wide = torch.zeros(3, hkv, blocks * 16, device="cuda")
    o2, l2, s2 = b.decode_paged_weights(q, kp, vp, table.cuda(), ln, wide, c.scale, num_splits=1)
    torch.cuda.synchronize()
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    for i, n in enumerate(lens):
        assert torch.equal(s1[i, :, :n], s2[i, :, :n])
    assert int((s2 != 0).sum()) <= sum(lens) * hkv
    del wide, s2
    torch.cuda.empty_cache()


def test_two_streams_at_once(b):
    """The same calls on two streams, each with its own outputs and workspace, interleaved."""
    g = torch.Generator(device="cuda").manual_seed(2)
    kp, vp = (torch.randn(200, 8, 16, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    order = torch.randperm(200, generator=g, device="cuda").to(torch.int32)
    w = (torch.randn(512, 1024, generator=g, device="cuda") / 32).bfloat16()
    sets = []
    for i in range(2):
        t, n = order[100 * i:100 * i + 60].view(2, 30).contiguous(), order[100 * i + 60:100 * i + 80].view(2, 10).contiguous()
        sets.append(dict(t=t, n=n, lens=torch.tensor([470, 300], dtype=torch.int32, device="cuda"),
                         q=torch.randn(2, 32, 128, generator=g, device="cuda").bfloat16(),
                         x=torch.randn(200, 1024, generator=g, device="cuda").bfloat16(),
                         sums=torch.rand(2, 8, 480, generator=g, device="cuda"),
                         ws=b.alloc_workspace(b.decode_weights_workspace_size(2, 30, 32, 8, 128, 16), "cuda")))

    def run(s):
        o, l, sums = b.decode_paged_weights(s["q"], kp, vp, s["t"], s["lens"], s["sums"].clone(), 0.1, workspace=s["ws"])
        kept, nl, ns = b.cache_evict(kp, vp, s["t"], s["lens"], sums, s["n"], 160, 2, 8)
        y = b.linear(s["x"], w, activation="silu")
        z = b.linear(s["x"][:5], w, activation="gelu")
        return [o, l, sums, kept, ns, y, z]
    want = [[t.clone() for t in run(s)] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(run(s))
        torch.cuda.synchronize()
        for a, c in zip(want, got):
            for x, y in zip(a, c):
                assert torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0))


def test_a_stalled_decode_makes_its_sums_nan(b):
    c = workloads.make_paged_decode(5, 2, 8, 8, 64, 16, [200, 40], num_pages=20, dtype="f32")
    q, kp, vp, bt, ln = (t.cuda() for t in (c.q, c.k_pages, c.v_pages, c.block_table, c.kv_lens))
    sums = torch.zeros(2, 8, bt.shape[1] * 16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.debug_decode_stall(4, 20_000_000)  # page 4 of a split: only the first sequence has one
    try:
        _, lse, got = b.decode_paged_weights(q, kp, vp, bt, ln, sums, c.scale, num_splits=1, err_flag=err)
        torch.cuda.synchronize()
    finally:
        b.debug_decode_stall(-1)
    assert int(err) & b.PKV_DEVERR_TIMEOUT
    assert torch.isnan(got[0, :, :200]).all() and not got[0, :, 200:].any()
    w = oracle.key_weights(c.q[1:, None].double().numpy(), c.k_pages.nan_to_num(0).double().numpy(), c.block_table.numpy()[1:],
                           c.kv_lens.numpy()[1:] - 1, lse[1:, :, None].cpu().double().numpy(), c.scale)
    np.testing.assert_allclose(got[1, :, :40].cpu().numpy(), w[0, :, :40], rtol=1e-4)


def test_chunk_weights_far_back(b):
    """A key 2^24 and more tokens behind the query, with 128 heads on a KV head: the causal bound in columns is past
    32 bits. All blocks are one of three pages, so the answer repeats."""
    blocks, hq, scale = (1 << 21) + 8, 128, 128 ** -0.5
    g = torch.Generator(device="cuda").manual_seed(3)
    kp = torch.randn(3, 1, 16, 128, device="cuda", generator=g, dtype=torch.bfloat16)
    q = torch.randn(1, 2, hq, 128, device="cuda", generator=g, dtype=torch.bfloat16)
    table = (torch.arange(blocks, device="cuda") % 3).to(torch.int32).view(1, blocks)
    n = blocks * 16
    lse = torch.full((1, hq, 2), 12.0, device="cuda")
    sums = torch.zeros(1, 1, n, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pl = torch.tensor([n - 2], dtype=torch.int32, device="cuda")
    got = b.chunk_weights(q, kp, table, pl, lse, sums, scale, err_flag=err)
    assert int(err) == 0
    w = (torch.einsum("qhd,ptd->qhpt", q[0].double(), kp[:, 0].double()) * scale - 12.0).exp().sum(1).reshape(2, 48)
    want = (w[0] + w[1]).repeat(n // 48 + 1)[:n]
    want[n - 1] = w[1][(n - 1) % 48]  # the last key is seen by the last query alone
    top = scale * float(q.double().abs().amax() * kp.double().abs().sum(-1).amax())
    bar = 2.0 ** -22 * (128 * top + 4 * (top + 12.0)) + 2.0 ** -20 + 2 * (hq + 8) * 2.0 ** -24 + 2.0 ** -23
    assert float(((got[0, 0].double() - want).abs() / want).max()) <= bar
