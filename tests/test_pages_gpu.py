"""Page reservation and compaction on the GPU against the oracle, bit for bit, and a serving loop on 4-bit pages."""
import numpy as np
import pytest
import torch

from oracle import pages as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_28_gb300 import build
    build.build(quiet=True)
    from paged_kv_attention_28_gb300 import binding
    return binding


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def some_state(r, batch, blocks, pages, page, shared, held):
    """Rows of pages, some of which are taken over from another row up to a block."""
    order = r.permutation(max(pages, batch * blocks))[:batch * blocks] % pages
    table = order.reshape(batch, blocks)
    lens = r.integers(0, blocks * page + 1, batch)
    for b in range(1, batch):
        if r.random() < shared:
            a = r.integers(0, b)
            n = r.integers(0, blocks + 1)
            table[b, :n] = table[a, :n]
            lens[b] = min(lens[b], n * page)
            if r.random() < 0.5:  # a fork: the same length
                table[b], lens[b] = table[a], lens[a]
    return table, lens, (r.random(pages) < held).astype(np.uint8)


def some_pools(r, pages, sizes):
    return [torch.tensor(r.integers(0, 256, (pages, n), dtype=np.uint8)).cuda() for n in sizes]


CASES = [  # batch, blocks, pages, page, pools' bytes
    (1, 1, 1, 16, [16]),
    (3, 4, 40, 16, [64, 4, 1152]),
    (17, 9, 300, 16, [8192, 20]),
    (40, 33, 2000, 1, [4100]),
    (8, 50, 1000, 7, []),
    (300, 40, 20000, 16, [32]),
    (70, 400, 40001, 16, [48, 12]),
    (2048, 4, 28672, 16, [16]),   # the largest problem of one CTA, and one past each of its limits
    (2049, 3, 28672, 16, [16]),
    (1, 8193, 9000, 16, [16]),
    (5, 7, 28673, 2, [16]),
    (2048, 40, 28672, 16, [16]),
    (1, 8192, 9000, 16, [16]),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"b{c[0]}n{c[2]}p{c[3]}")
def test_reserve(b, case, in_place):
    batch, blocks, pages, page, sizes = case
    r = np.random.default_rng(batch + in_place)
    for held in (0.0, 0.05):
        table, lens, mask = some_state(r, batch, blocks, pages, page, 0.5, held)
        lens = np.minimum(lens, blocks * page // 2 + 1)
        new_lens = np.minimum(blocks * page, lens + r.integers(-2, 3 * page + 2, batch))
        pools = some_pools(r, pages, sizes)
        before = [p.clone() for p in pools]
        t = i32(table)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, n_free = b.cache_reserve(t, i32(lens), i32(new_lens), pools, num_pages=pages, page_size=page,
                                      held=torch.tensor(mask).cuda() if held else None, out=t if in_place else None, err_flag=err)
        new, left, copies = O.reserve(table, lens, new_lens, mask if held else None, pages, page)
        assert int(n_free) == left and (out.cpu().numpy() == new).all()
        assert int(err) == (b.PKV_DEVERR_NO_PAGES if left < 0 else 0)
        assert in_place or (t.cpu().numpy() == table).all()
        for p, old in zip(pools, before):
            for s, d in copies:
                old[d] = old[s]
            assert torch.equal(p, old)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"b{c[0]}n{c[2]}p{c[3]}")
def test_compact(b, case, in_place):
    batch, blocks, pages, page, sizes = case
    r = np.random.default_rng(batch + 50 + in_place)
    for held in (0.0, 0.05):
        table, lens, mask = some_state(r, batch, blocks, pages, page, 0.3, held)
        pools = some_pools(r, pages, sizes)
        before = [p.clone() for p in pools]
        t = i32(table)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, page_map, n_used = b.cache_compact(t, i32(lens), pools, num_pages=pages, page_size=page,
                                                held=torch.tensor(mask).cuda() if held else None, out=t if in_place else None,
                                                err_flag=err)
        new, want_map, n, moves = O.compact(table, lens, mask if held else None, pages, page)
        assert int(err) == 0 and int(n_used) == n
        assert (out.cpu().numpy() == new).all() and (page_map.cpu().numpy() == want_map).all()
        for p, old in zip(pools, before):
            for s, d in moves:
                old[d] = old[s]
            assert torch.equal(p, old)


def test_nothing_to_do(b):
    """No sequences, none that grows, all of length 0, a full pool without a free page."""
    pool = torch.arange(64, device="cuda", dtype=torch.int32).view(8, 8)
    keep = pool.clone()
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    out, left = b.cache_reserve(none, i32([]), i32([]), [pool])
    assert out.shape == (0, 3) and int(left) == 8
    out, page_map, n = b.cache_compact(none, i32([]), [pool])
    assert int(n) == 0 and (page_map == -1).all()
    table = i32([[3, 1], [9, -4]])  # (entries past the length are not looked at)
    out, left = b.cache_reserve(table, i32([32, 0]), i32([5, -3]), [pool])
    assert torch.equal(out, table) and int(left) == 6
    out, page_map, n = b.cache_compact(table, i32([0, 0]), [pool])
    assert torch.equal(out, table) and int(n) == 0
    full = i32([[0, 1, 2, 3, 4, 5, 6, 7]])
    out, page_map, n = b.cache_compact(full, i32([128]), [pool])
    assert torch.equal(out, full) and int(n) == 8
    out, left = b.cache_reserve(full, i32([120]), i32([128]), [pool])
    assert torch.equal(out, full) and int(left) == 0
    assert torch.equal(pool, keep)


@pytest.mark.parametrize("pages", [64, 20000])
def test_too_few_pages_changes_nothing(b, pages):
    r = np.random.default_rng(3)
    table = r.permutation(pages)[:60].reshape(4, 15)
    lens, want = [100, 200, 33, 16], [240, 240, 240, 240]
    held = np.ones(pages, dtype=np.uint8)
    held[r.permutation(pages)[:20]] = 0
    pools = some_pools(r, pages, [64])
    before = pools[0].clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, left = b.cache_reserve(i32(table), i32(lens), i32(want), pools, held=torch.tensor(held).cuda(), err_flag=err)
    new, missing, _ = O.reserve(table, lens, want, held, pages, 16)
    assert missing < 0 and int(left) == missing and int(err) == b.PKV_DEVERR_NO_PAGES
    assert (out.cpu().numpy() == table).all() and torch.equal(pools[0], before)


@pytest.mark.parametrize("pages", [64, 20000])
def test_bad_lengths_and_entries(b, pages):
    table = np.arange(12).reshape(3, 4)
    pool = torch.zeros(pages, 16, dtype=torch.uint8, device="cuda")
    for lens, want in (([20, -1, 30], [40, 40, 40]), ([20, 65, 30], [40, 66, 40]), ([20, 10, 30], [40, 65, 40]),
                       ([20, 1 << 30, 30], [40, 40, 40])):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, left = b.cache_reserve(i32(table), i32(lens), i32(want), [pool], err_flag=err)
        counts = [20, 0 if lens[1] < 0 else min(lens[1], 64), 30]  # what it holds stays its own
        new, free, _ = O.reserve(table, counts, [40, counts[1], 40], None, pages, 16)
        assert int(err) == b.PKV_DEVERR_BAD_LEN and (out.cpu().numpy() == new).all() and int(left) == free
        err.zero_()
        out, page_map, n = b.cache_compact(i32(table), i32(lens), [pool], err_flag=err)
        bad = lens[1] < 0 or lens[1] > 64
        new, want_map, used, _ = O.compact(table, counts, None, pages, 16)
        assert int(err) == (b.PKV_DEVERR_BAD_LEN if bad else 0) and (out.cpu().numpy() == new).all() and int(n) == used
    for entry in (-1, pages, 1 << 30):
        broken = table.copy()
        broken[1, 0] = entry
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, left = b.cache_reserve(i32(broken), i32([20, 10, 30]), i32([40, 40, 40]), [pool], err_flag=err)
        new, free, _ = O.reserve(broken, [20, 10, 30], [40, 40, 40], None, pages, 16)
        assert int(err) == b.PKV_DEVERR_BAD_PAGE and (out.cpu().numpy() == new).all() and int(left) == free
        err.zero_()
        out, page_map, n = b.cache_compact(i32(broken), i32([20, 10, 30]), [pool], err_flag=err)
        new, want_map, used, _ = O.compact(broken, [20, 10, 30], None, pages, 16)
        assert int(err) == b.PKV_DEVERR_BAD_PAGE and (out.cpu().numpy() == new).all() and int(n) == used


def test_pools_past_32_bits(b):
    """Copies at byte offsets past 2^32, in pools of several sizes."""
    pages = 140000
    big = torch.zeros(pages, 8192, dtype=torch.int32, device="cuda")  # 4.6 GB
    small = torch.zeros(pages, 1, dtype=torch.int32, device="cuda")
    big[pages - 1] = torch.arange(8192, device="cuda", dtype=torch.int32)
    small[pages - 1] = 7
    table = i32([[pages - 1, 0], [pages - 1, 0]])
    held = torch.ones(pages, dtype=torch.uint8, device="cuda")
    held[[pages - 1, pages - 2]] = 0
    out, left = b.cache_reserve(table, i32([5, 5]), i32([6, 6]), [big, small], held=held)
    assert int(left) == 0 and out[:, 0].tolist() == [pages - 1, pages - 2]
    assert torch.equal(big[pages - 2], big[pages - 1]) and int(small[pages - 2]) == 7
    out, page_map, n = b.cache_compact(out, i32([5, 5]), [big, small])
    assert out[:, 0].tolist() == [1, 0] and torch.equal(big[0], big[pages - 1]) and torch.equal(big[1], big[0])


def test_captured_and_replayed(b):
    r = np.random.default_rng(9)
    table, lens, _ = some_state(r, 9, 20, 260, 16, 0.5, 0)
    lens = np.minimum(lens, 200)
    pools = some_pools(r, 260, [256])
    t, n, m = i32(table), i32(lens), i32(lens + 40)
    first = b.cache_reserve(t, n, m, pools)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.cache_reserve(t, n, m, pools), b.cache_compact(t, n, pools)
    for shift in (0, 5, 11):
        n.copy_(i32(np.maximum(lens - shift, 0)))
        graph.replay()
        torch.cuda.synchronize()
        new, left, _ = O.reserve(table, np.maximum(lens - shift, 0), lens + 40, None, 260, 16)
        assert (got[0][0].cpu().numpy() == new).all() and int(got[0][1]) == left
        new, page_map, used, _ = O.compact(table, np.maximum(lens - shift, 0), None, 260, 16)
        assert (got[1][0].cpu().numpy() == new).all() and int(got[1][2]) == used
    assert first[0].shape == t.shape


@pytest.mark.parametrize("pages", [260, 30000])
def test_two_streams_at_once(b, pages):
    """Calls on two streams that make their own buffers, against the oracle."""
    r = np.random.default_rng(10)
    jobs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for _ in streams:
        table, lens, _ = some_state(r, 9, 20, pages, 16, 0.5, 0)
        jobs.append((table, np.minimum(lens, 200), some_pools(r, pages, [256])[0]))
    tensors = [(i32(t), i32(n), i32(n + 40)) for t, n, _ in jobs]
    before = [p.clone() for _, _, p in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (t, n, m) in enumerate(tensors):
            got[i].append(b.cache_reserve(t, n, m, [jobs[i][2]], stream=streams[i]) + b.cache_compact(t, n, [], num_pages=pages, stream=streams[i]))
    torch.cuda.synchronize()
    for i, (table, lens, pool) in enumerate(jobs):
        new, left, copies = O.reserve(table, lens, lens + 40, None, pages, 16)
        small, page_map, used, _ = O.compact(table, lens, None, pages, 16)
        for s, d in copies:
            before[i][d] = before[i][s]
        assert torch.equal(pool, before[i])
        for out, n_free, packed, where, n_used in got[i]:
            assert (out.cpu().numpy() == new).all() and int(n_free) == left
            assert (packed.cpu().numpy() == small).all() and (where.cpu().numpy() == page_map).all() and int(n_used) == used


def test_the_largest_batch_page_and_number_of_pools(b):
    """65535 sequences, pages of 32767 tokens, 256 pools of different widths; 257 pools are refused."""
    r = np.random.default_rng(12)
    batch, pages = 65535, 60000
    table = r.integers(0, 200, (batch, 2))
    lens = r.choice([0, 1, 32766, 32767, 32768, 65534], batch, p=[0.9, 0.02, 0.02, 0.02, 0.02, 0.02])
    want = np.minimum(lens + r.integers(0, 3, batch), 65534)
    out, left = b.cache_reserve(i32(table), i32(lens), i32(want), [], num_pages=pages, page_size=32767)
    new, free, copies = O.reserve(table, lens, want, None, pages, 32767)
    assert free >= 0 and len(copies) > 100 and int(left) == free and (out.cpu().numpy() == new).all()
    out, page_map, n = b.cache_compact(i32(new), i32(want), [], num_pages=pages, page_size=32767)
    new, where, used, _ = O.compact(new, want, None, pages, 32767)
    assert int(n) == used and (out.cpu().numpy() == new).all() and (page_map.cpu().numpy() == where).all()
    # every pool its own number of words; page 5 is in the middle of two sequences
    pools = some_pools(r, 8, [4 * (1 + i % 5) + 4096 * (i % 3 == 0) for i in range(256)])
    before = [p.clone() for p in pools]
    out, left = b.cache_reserve(i32([[5], [5]]), i32([9, 9]), i32([10, 10]), pools)
    assert out.flatten().tolist() == [5, 0] and int(left) == 6
    for p, old in zip(pools, before):
        old[0] = old[5]
        assert torch.equal(p, old)
    with pytest.raises(ValueError, match="pools"):
        b.cache_reserve(i32([[5], [5]]), i32([9, 9]), i32([10, 10]), pools + some_pools(r, 8, [4]))


@pytest.mark.parametrize("pages", [20000, 40000])
def test_a_row_of_more_than_2_to_the_30_blocks(b, pages):
    """Pages of one token, and a row so long that what is given lies past its 2^30-th entry: in the tables of a cluster and
    in those of the workspace. The row lists the pages from 1 on, over and over."""
    blocks, used = (1 << 30) + 70000, pages - 100
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").remainder_(used).add_(1).view(1, blocks)
    n = blocks - 50
    want = table[0, -1000:].clone()
    pool = torch.arange(pages, dtype=torch.int32, device="cuda").view(pages, 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, left = b.cache_reserve(table, i32([n]), i32([n + 10]), [pool], page_size=1, out=table, err_flag=err)
    want[-50:-40] = i32([0] + list(range(used + 1, used + 10)))  # (the free ones: 0 and those behind the row's)
    assert int(err) == 0 and int(left) == 90 and torch.equal(out[0, -1000:], want)
    assert torch.equal(out[0, :1 << 20], torch.arange(1 << 20, dtype=torch.int32, device="cuda").remainder_(used).add_(1))
    assert torch.equal(pool[:, 0], torch.arange(pages, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("n_pools", [16, 17])
@pytest.mark.parametrize("batch,blocks,pages", [(20, 40, 900), (300, 40, 15000), (40, 40, 30000)])
def test_many_pools_forks_and_too_few_pages(b, n_pools, batch, blocks, pages):
    """All three places of the marks: forks that copy in every pool, compaction, and a demand that cannot be met."""
    r = np.random.default_rng(13)
    table, lens, _ = some_state(r, batch, blocks, pages, 16, 0.5, 0)
    lens = np.minimum(lens, blocks * 16 - 40)
    pools = some_pools(r, pages, [16 + 4 * (i % 3) for i in range(n_pools)])
    before = [p.clone() for p in pools]
    held = np.ones(pages, dtype=np.uint8)
    held[r.permutation(pages)[:batch // 4]] = 0
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, n, m = i32(table), i32(lens), i32(lens + 40)
    out, left = b.cache_reserve(t, n, m, pools, held=torch.tensor(held).cuda(), err_flag=err)
    assert int(left) < 0 and int(err) == b.PKV_DEVERR_NO_PAGES and torch.equal(out, t)
    assert int(left) == O.reserve(table, lens, lens + 40, held, pages, 16)[1]
    assert all(torch.equal(p, old) for p, old in zip(pools, before))
    out, left = b.cache_reserve(t, n, m, pools, out=t)
    new, free, copies = O.reserve(table, lens, lens + 40, None, pages, 16)
    assert len(copies) and int(left) == free and (t.cpu().numpy() == new).all()
    packed, page_map, used = b.cache_compact(t, m, pools)
    last, where, count, moves = O.compact(new, lens + 40, None, pages, 16)
    assert int(used) == count and (packed.cpu().numpy() == last).all() and (page_map.cpu().numpy() == where).all()
    for p, old in zip(pools, before):
        for s, d in copies + moves:
            old[d] = old[s]
        assert torch.equal(p, old)


def test_serving_loop_on_4_bit_pages(b):
    """Prompts packed after their prefill, forked, grown token by token with pages as they are needed, compacted, and
    continued by a chunk over the unpacked prefix; each attention against the dequantised tokens kept aside."""
    torch.manual_seed(5)
    H, Hq, D, B, pages, blocks, scale = 2, 8, 128, 4, 64, 12, 0.09
    k4, v4 = (torch.zeros(pages, H, 9 * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((H,), 0.004, device="cuda") for _ in range(2))
    table = torch.zeros(B, blocks, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    freq = 1e4 ** (-torch.arange(D // 2, device="cuda") / (D // 2))
    stage_k, stage_v = (torch.zeros(B * blocks, H, 16, D, device="cuda").bfloat16() for _ in range(2))
    stage = torch.arange(B * blocks, dtype=torch.int32, device="cuda").view(B, blocks)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    kept = [[], []]  # per sequence [T, H, D] of what the cache holds

    def put(counts, chunk):
        """New tokens through the norm and rotation call, into the staging pages, and packed."""
        q, k, v = (torch.randn(B, chunk, h, D, device="cuda").bfloat16() for h in (Hq, H, H))
        n = i32(counts)
        new = lens + n
        nonlocal table
        table, left = b.cache_reserve(table, lens, new, [k4, v4], out=table, err_flag=err)
        assert int(left) >= 0
        pos = (lens[:, None] + torch.arange(chunk, device="cuda")).to(torch.int32)[None].contiguous()
        q = b.qk_norm_rope_append(q, k, v, stage_k, stage_v, stage, zero, chunk_lens=n, positions=pos, inv_freq=freq, err_flag=err)
        b.cache_pack_fp4(stage_k, stage_v, stage, k4, v4, table, n, first=lens, k_scale=ks, v_scale=vs, err_flag=err)
        for x, src, s in ((kept[0], stage_k, ks), (kept[1], stage_v, vs)):
            rows = src.view(B, blocks, H, 16, D).transpose(2, 3).reshape(B, -1, H, D).float().cpu().numpy()
            for i in range(B):
                got = np.stack([O.values(*O.quantise(rows[i, :counts[i], h], float(s[h])), float(s[h])) for h in range(H)], 1)
                if len(x) <= i:
                    x.append(got)
                else:
                    x[i] = np.concatenate([x[i], got])
        lens.copy_(new)
        return q

    def check(out, q):
        for i in range(B):
            for h in range(Hq):
                kk, vv = (x[i][:, h * H // Hq].astype(np.float64) for x in kept)
                w = np.exp(scale * (kk @ q[i, h].double().cpu().numpy()))
                want = (w[:, None] * vv).sum(0) / w.sum()
                # the bf16 rounding of the output, the weights' f16 rounding, and fp32's shares (logits up to 2^5)
                tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 136 * 2.0 ** -18) * (w[:, None] * np.abs(vv)).sum(0) / w.sum() + 1e-6
                assert (np.abs(out[i, h].double().cpu().numpy() - want) <= tol).all()

    q = put([37, 50, 16, 1], 50)
    # sequence 3 becomes a continuation of sequence 1: its old page is free then
    table[3], lens[3] = table[1], lens[1]
    for x in kept:
        x[3] = x[1].copy()
    for step in range(20):
        q = put([1, 1, 1, 1], 1)
        out, _ = b.decode_paged_fp4(q[:, 0].contiguous(), k4, v4, table, lens, scale, ks, vs, err_flag=err)
        check(out, q[:, 0].float())
        if step == 9:
            table, page_map, used = b.cache_compact(table, lens, [k4, v4], out=table, err_flag=err)
            live = {int(p) for i in range(B) for p in table[i, :(int(lens[i]) + 15) // 16]}
            assert live == set(range(int(used)))
    # a chunk over the prefix: unpacked into ordinary pages, the chunk's tokens behind it as they are
    wide_k, wide_v = (torch.zeros(B * blocks, H, 16, D, device="cuda").bfloat16() for _ in range(2))
    b.cache_unpack_fp4(k4, v4, table, wide_k, wide_v, stage, lens, k_scale=ks, v_scale=vs, err_flag=err)
    chunk = 24
    qc, kc, vc = (torch.randn(B, chunk, h, D, device="cuda").bfloat16() for h in (Hq, H, H))
    qc = b.qk_norm_rope_append(qc, kc, vc, wide_k, wide_v, stage, lens, inv_freq=freq, err_flag=err)
    out, _ = b.prefill_paged_chunk(qc, wide_k, wide_v, stage, lens, scale, err_flag=err)
    for i in range(B):
        n = int(lens[i])
        for x, src in zip(kept, (wide_k, wide_v)):
            rows = src.view(B, blocks, H, 16, D).transpose(2, 3).reshape(B, -1, H, D)[i, :n + chunk].float().cpu().numpy()
            assert np.array_equal(rows[:n], torch.tensor(x[i]).bfloat16().float().numpy())
            x[i] = rows
    last = torch.stack([out[:, -1]]).squeeze(0)
    for i in range(B):
        for h in range(Hq):
            kk, vv = (x[i][:, h * H // Hq].astype(np.float64) for x in kept)
            w = np.exp(scale * (kk @ qc[i, -1, h].double().cpu().numpy()))
            want = (w[:, None] * vv).sum(0) / w.sum()
            # weights rounded to bf16 there: 2^-8 each, and the output
            tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 136 * 2.0 ** -18) * (w[:, None] * np.abs(vv)).sum(0) / w.sum() + 1e-6
            assert (np.abs(last[i, h].double().cpu().numpy() - want) <= 2 * tol).all()
    assert int(err) == 0
