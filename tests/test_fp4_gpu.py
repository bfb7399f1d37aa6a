"""4-bit pages on the GPU against the oracle: codes bit for bit, attention within its roundings.

Bound of a decode output element: one rounding to bf16 (2^-8 of it), the weights' rounding to f16 (2^-11 of each, or
2^-25 below f16's normal range, against a largest weight of at least 1), and what fp32 does to a logit (a sum of D
products: D 2^-24 of their magnitudes, its scaling and the exponential: 2^-20) twice, in the weight and in the sum of
weights, and to sums over n keys (n 2^-24).
"""
import math

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


def gpu(x):
    return torch.tensor(np.asarray(x)).cuda()


def some_pool(r, pages, heads, d):
    """Random codes; scales of all sizes up to 8 (codes to 0x50), no NaN."""
    pool = r.integers(0, 256, (pages, heads, 9 * d), dtype=np.uint8)
    pool[..., 8 * d:] = r.integers(0, 0x50, (pages, heads, d))
    return pool


# ------------------------------------------------------------------------------------ pack and unpack

COPIES = [  # heads, d, dtype, first, counts, from, blocks of either table
    (1, 64, "bf16", [0], [1], [0], 1, 1),
    (2, 128, "bf16", [15, 0, 7], [1, 16, 40], [3, 0, 9], 4, 5),
    (3, 64, "f32", [1, 33, 14], [17, 0, 35], [0, 5, 31], 5, 5),
    (8, 128, "f32", [16, 2], [48, 30], [0, 15], 4, 4),
    (5, 128, "bf16", None, [31, 64, 5], None, 4, 4),
]


def setup_copy(case, seed):
    heads, d, dtype, first, counts, start, src_blocks, blocks = case
    r = np.random.default_rng(seed)
    B = len(counts)
    rows = [r.standard_normal((B * src_blocks + 1, heads, 16, d)).astype(np.float32) * r.choice([1e-3, 1, 30], (1, heads, 1, 1))
            for _ in range(2)]
    rows = [torch.tensor(x).to(torch.bfloat16 if dtype == "bf16" else torch.float32) for x in rows]
    src_table = r.permutation(B * src_blocks).reshape(B, src_blocks)
    table = r.permutation(B * blocks).reshape(B, blocks)
    pools = [some_pool(r, B * blocks + 1, heads, d) for _ in range(2)]
    hs = [(0.001 + r.random(heads)).astype(np.float32) for _ in range(2)]
    zero = [0] * B
    return rows, src_table, start or zero, pools, table, first or zero, counts, hs, start, first


@pytest.mark.parametrize("scaled", [True, False])
@pytest.mark.parametrize("case", COPIES, ids=lambda c: f"h{c[0]}d{c[1]}{c[2]}")
def test_pack_is_exact(b, case, scaled):
    rows, src_table, start, pools, table, first, counts, hs, start_arg, first_arg = setup_copy(case, 5)
    want = [O.pack(x.float().numpy(), src_table, start, p, table, first, counts, s if scaled else None)
            for x, p, s in zip(rows, pools, hs)]
    k, v = gpu(pools[0]), gpu(pools[1])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ks, vs = (gpu(hs[0]), gpu(hs[1])) if scaled else (None, None)
    b.cache_pack_fp4(rows[0].cuda(), rows[1].cuda(), i32(src_table), k, v, i32(table), i32(counts),
                     first=None if first_arg is None else i32(first), src_first=None if start_arg is None else i32(start),
                     k_scale=ks, v_scale=vs, err_flag=err)
    assert int(err) == 0
    assert (k.cpu().numpy() == want[0]).all() and (v.cpu().numpy() == want[1]).all()


@pytest.mark.parametrize("case", COPIES, ids=lambda c: f"h{c[0]}d{c[1]}{c[2]}")
def test_unpack_is_exact(b, case):
    rows, src_table, start, pools, table, first, counts, hs, start_arg, first_arg = setup_copy(case, 6)
    t = rows[0].dtype
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = rows[0].cuda(), rows[1].cuda()
    b.cache_unpack_fp4(gpu(pools[0]), gpu(pools[1]), i32(table), k, v, i32(src_table), i32(counts),
                       first=None if first_arg is None else i32(first), dst_first=None if start_arg is None else i32(start),
                       k_scale=gpu(hs[0]), v_scale=gpu(hs[1]), err_flag=err, max_count=max(counts))
    assert int(err) == 0
    for got, x, p, s in ((k, rows[0], pools[0], hs[0]), (v, rows[1], pools[1], hs[1])):
        want = torch.tensor(O.unpack(p, table, first, x.float().numpy(), src_table, start, counts, s)).to(t)
        assert torch.equal(got.cpu(), want)


def test_pack_special_values(b):
    """Groups of zeros, of numbers too small or too large for a scale, with NaN and infinities; ties of codes and scales."""
    d, r = 64, np.random.default_rng(7)
    x = np.zeros((1, 1, 16, d), dtype=np.float32)
    x[0, 0, 1, :16] = 1e-6
    x[0, 0, 2, :16] = 3e38 * r.choice([-1, 1], 16)
    x[0, 0, 3, 4], x[0, 0, 3, 20], x[0, 0, 3, 40] = np.nan, np.inf, -np.inf
    x[0, 0, 4, :16] = [6, 0.25, -0.25, 0.75, 1.25, -1.75, 2.5, 3.5, 5, -5, -0.0, 0.1, 5.000001, 4.999999, 0.24999999, -6]
    x[0, 0, 5, 0:64:16] = 6 * O.E4M3[[9, 50, 100, 126]] * (1 + 1 / 32)   # near halves of steps
    x[0, 0, 6, :] = 1e-38  # fp32 numbers at the edge of the normal range
    x[0, 0, 7, :] = r.standard_normal(d) * 1e-3
    x[0, 0, 8, 0:64:16] = 6 * (O.E4M3[[10, 51, 101, 3]] + O.E4M3[[11, 52, 102, 4]]) / 2
    pool = np.zeros((1, 1, 9 * d), dtype=np.uint8)
    for hs in (None, np.array([1e30], dtype=np.float32), np.array([1e-20], dtype=np.float32)):
        want = O.pack(x, [[0]], [0], pool, [[0]], [0], [16], hs)
        k, v = gpu(pool), gpu(pool)
        s = None if hs is None else gpu(hs)
        b.cache_pack_fp4(gpu(x), gpu(x), i32([[0]]), k, v, i32([[0]]), i32([16]), k_scale=s, v_scale=s)
        assert (k.cpu().numpy() == want).all() and (v.cpu().numpy() == want).all()
        back = torch.empty(1, 1, 16, d, device="cuda")
        b.cache_unpack_fp4(k, v, i32([[0]]), back, torch.empty_like(back), i32([[0]]), i32([16]), k_scale=s, v_scale=s)
        want = O.unpack(want, [[0]], [0], np.zeros((1, 1, 16, d)), [[0]], [0], [16], hs)
        assert np.array_equal(back.cpu().numpy(), want, equal_nan=True)


def test_copy_bad_lengths_and_pages(b):
    d, r = 128, np.random.default_rng(8)
    rows = [torch.randn(8, 2, 16, d) for _ in range(2)]
    pools = [some_pool(r, 8, 2, d) for _ in range(2)]
    table, src = np.arange(8).reshape(4, 2), np.arange(8).reshape(4, 2)
    for first, start, counts, which in (([0, 30, 0, 0], [0] * 4, [3, 3, 4, 5], 1), ([0] * 4, [0, 0, -1, 0], [3, 3, 4, 5], 2),
                                        ([0] * 4, [0] * 4, [3, -3, 4, 5], 1), ([0] * 4, [0] * 4, [3, 3, 4, 33], 3),
                                        ([-1, 0, 0, 0], [0] * 4, [3, 3, 4, 5], 0), ([0] * 4, [0] * 4, [3, 21, 4, 5], 1)):
        good = [0 if i == which else c for i, c in enumerate(counts)]
        for pack in (True, False):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            k, v = gpu(pools[0]), gpu(pools[1])
            kr, vr = rows[0].cuda(), rows[1].cuda()
            f = [max(x, 0) for x in first]
            s = [max(x, 0) for x in start]
            if pack:
                b.cache_pack_fp4(kr, vr, i32(src), k, v, i32(table), i32(counts), first=i32(first), src_first=i32(start),
                                 max_count=20, err_flag=err)
                want = O.pack(rows[0].numpy(), src, s, pools[0], table, f, good, None)
                assert (k.cpu().numpy() == want).all()
            else:
                b.cache_unpack_fp4(k, v, i32(table), kr, vr, i32(src), i32(counts), first=i32(first), dst_first=i32(start),
                                   max_count=20, err_flag=err)
                want = O.unpack(pools[0], table, f, rows[0].numpy(), src, s, good, None)
                assert np.array_equal(kr.cpu().numpy(), want)
            assert int(err) == b.PKV_DEVERR_BAD_LEN
    # bad entries: of the side that is written, of the side that is read
    for pack in (True, False):
        for entry in (-1, -2, 8, 1 << 30, -(1 << 31)):
            for bad_rows in (True, False):
                bad_src, bad_table = src.copy(), table.copy()
                (bad_src if bad_rows else bad_table)[1, 1] = entry
                counts = [20, 32, 17, 1]
                good = [20, 16, 17, 1]
                err = torch.zeros(1, dtype=torch.int32, device="cuda")
                k, v = gpu(pools[0]), gpu(pools[1])
                kr, vr = rows[0].cuda(), rows[1].cuda()
                if pack:
                    b.cache_pack_fp4(kr, vr, i32(bad_src), k, v, i32(bad_table), i32(counts), err_flag=err)
                    want = O.pack(rows[0].numpy(), src, [0] * 4, pools[0], table, [0] * 4, good, None)
                    assert (k.cpu().numpy() == want).all()
                else:
                    b.cache_unpack_fp4(k, v, i32(bad_table), kr, vr, i32(bad_src), i32(counts), err_flag=err)
                    want = O.unpack(pools[0], table, [0] * 4, rows[0].numpy(), src, [0] * 4, good, None)
                    if not bad_rows:
                        want[src[1, 1]] = np.nan
                    assert np.array_equal(kr.cpu().numpy(), want, equal_nan=True)
                assert int(err) == b.PKV_DEVERR_BAD_PAGE


# ------------------------------------------------------------------------------------ decode

def close(got, lse, want, want_lse, size, mass, lens, D, v_most):
    """The bound above, element by element; `v_most` is the largest |v|."""
    n = np.array(lens, dtype=np.float64)[:, None]
    e = (D + 8) * 2.0 ** -24 * mass + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * e + n * 2.0 ** -24)[..., None] * size + (n * 2.0 ** -25)[..., None] * v_most
    err = np.abs(got.astype(np.float64) - want)
    assert (err <= tol * (1 + 1e-6) + 1e-30).all(), float((err - tol).max())
    dead = np.isinf(want_lse)
    assert (np.isneginf(lse) == dead).all() and (got[dead] == 0).all()
    tol = e + n * 2.0 ** -24 + 2.0 ** -21 * np.abs(np.where(dead, 0, want_lse))
    assert (np.abs(np.where(dead, 0, lse) - np.where(dead, 0, want_lse)) <= tol).all()


def make_decode(r, lens, Hq, Hkv, D, extra_blocks=1, poison=True):
    B, blocks = len(lens), max(1, -(-max(lens) // 16)) + extra_blocks
    table = r.permutation(B * blocks).reshape(B, blocks)
    pools = [some_pool(r, B * blocks, Hkv, D) for _ in range(2)]
    if poison:  # everything that no token owns: codes of any kind, scales NaN
        for pool in pools:
            seen = np.zeros((B * blocks, 16), dtype=bool)
            for i, n in enumerate(lens):
                for j in range(-(-n // 16)):
                    seen[table[i, j], :min(16, n - 16 * j)] = True
            scales = pool[..., 8 * D:].reshape(B * blocks, Hkv, D // 16, 16)
            scales[np.broadcast_to(~seen[:, None, None, :], scales.shape)] = 0x7f
    bad = table.copy()
    for i, n in enumerate(lens):
        bad[i, -(-n // 16):] = -7
    q = (2 * r.standard_normal((B, Hq, D))).astype(np.float32)
    q = torch.tensor(q).bfloat16()
    hs = [(0.05 + 0.2 * r.random(Hkv)).astype(np.float32) for _ in range(2)]
    return q, pools, table, bad, hs


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (3, 1), (8, 2), (5, 1), (6, 1), (14, 2), (8, 1), (8, 8)])
@pytest.mark.parametrize("splits,extra", [(1, 1), (3, 1), (0, 1), (0, 60)])
def test_decode_matches_oracle(b, D, Hq, Hkv, splits, extra):
    """One CTA a sequence and KV head, splits, and the library's choice, also for a table much wider than the lengths."""
    r = np.random.default_rng(D + 10 * Hq + Hkv)
    lens = [0, 1, 15, 16, 17, 64, 65, 130, 333]
    q, pools, table, bad, hs = make_decode(r, lens, Hq, Hkv, D, extra_blocks=extra)
    want = O.decode(q.float().numpy(), *pools, *hs, table, lens, 0.11)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = b.decode_paged_fp4(q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), 0.11, k_scale=gpu(hs[0]),
                                  v_scale=gpu(hs[1]), num_splits=splits, err_flag=err)
    assert int(err) == 0
    close(out.float().cpu().numpy(), lse.cpu().numpy(), *want, lens, D, 6 * O.E4M3[0x4f] * hs[1].max())


def test_decode_long_and_many_pages_of_a_warp(b):
    """More than 32 pages of one warp (a second load of table entries), and splits that end anywhere."""
    r = np.random.default_rng(11)
    lens = [5000, 4097, 2111]
    q, pools, table, bad, hs = make_decode(r, lens, 4, 1, 64)
    want = O.decode(q.float().numpy(), *pools, *hs, table, lens, 0.05)
    for splits in (1, 2, 7, 100, 0):
        out, lse = b.decode_paged_fp4(q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), 0.05, k_scale=gpu(hs[0]),
                                      v_scale=gpu(hs[1]), num_splits=splits)
        close(out.float().cpu().numpy(), lse.cpu().numpy(), *want, lens, 64, 6 * O.E4M3[0x4f] * hs[1].max())


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (6, 2)])
def test_decode_long_at_head_dim_128(b, Hq, Hkv):
    """More than 32 pages of one warp where its ring has two steps; the same entries as one CTA's and as many splits'."""
    r = np.random.default_rng(30)
    D, lens = 128, [5000, 2065, 4111]
    q, pools, table, bad, hs = make_decode(r, lens, Hq, Hkv, D)
    want = O.decode(q.float().numpy(), *pools, *hs, table, lens, 0.04)
    for splits in (1, 2, 5, 0):
        out, lse = b.decode_paged_fp4(q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), 0.04, k_scale=gpu(hs[0]),
                                      v_scale=gpu(hs[1]), num_splits=splits)
        close(out.float().cpu().numpy(), lse.cpu().numpy(), *want, lens, D, 6 * O.E4M3[0x4f] * hs[1].max())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("block", [127, 128, 200, 257, 312])
def test_decode_bad_page_far_into_a_row(b, D, block):
    """A bad entry that a warp meets in its first load of table entries (block 127) and in later ones."""
    r = np.random.default_rng(31)
    lens = [300, 5000, 4900]
    q, pools, table, bad, hs = make_decode(r, lens, 2, 1, D, poison=False)
    args = q.cuda(), gpu(pools[0]), gpu(pools[1])
    for splits in (1, 2):
        clean, clean_lse = b.decode_paged_fp4(*args, i32(bad), i32(lens), 0.1, num_splits=splits)
        for entry in (-1, len(pools[0]), 1 << 30):
            broken = bad.copy()
            broken[1, block] = entry
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            out, lse = b.decode_paged_fp4(*args, i32(broken), i32(lens), 0.1, num_splits=splits, err_flag=err)
            assert int(err) == b.PKV_DEVERR_BAD_PAGE and out[1].isnan().all() and lse[1].isnan().all()
            assert torch.equal(out[[0, 2]], clean[[0, 2]]) and torch.equal(lse[[0, 2]], clean_lse[[0, 2]])


@pytest.mark.parametrize("B,Hkv,D,most", [(3, 2, 64, 4000), (40, 8, 64, 700), (129, 2, 128, 60), (300, 3, 64, 90), (1000, 1, 64, 20)])
def test_decode_many_sequences(b, B, Hkv, D, most):
    """Ragged batches with sequences without tokens at any place; the library's splits against one."""
    r = np.random.default_rng(B)
    lens = r.integers(0, most + 1, B)
    lens[r.random(B) < 0.2] = 0
    lens[[0, -1]] = [0, most]
    if B == 40:
        lens[5:30] = 0
    pools = [some_pool(r, 4 * most // 16 + 8, Hkv, D) for _ in range(2)]
    blocks = max(33, -(-most // 16) + 1)
    table = r.integers(0, len(pools[0]), (B, blocks))  # (pages may be shared)
    q = torch.tensor(2 * r.standard_normal((B, 2 * Hkv, D))).bfloat16().cuda()
    args = q, gpu(pools[0]), gpu(pools[1]), i32(table), i32(lens), 0.05
    out, lse = b.decode_paged_fp4(*args)
    want, want_lse = b.decode_paged_fp4(*args, num_splits=1)
    picked = sorted({0, B - 1, int(np.argmax(lens)), *r.integers(0, B, 12).tolist()})
    exact = O.decode(q.float().cpu().numpy()[picked], *pools, None, None, table[picked], lens[picked], 0.05)
    close(out.float().cpu().numpy()[picked], lse.cpu().numpy()[picked], *exact, lens[picked], D, 6 * O.E4M3[0x4f])
    # the others: both are within the bound, so within twice its largest
    n = int(lens.max())
    tol = 2 * (2.0 ** -8 + 2.0 ** -9 + n * 2.0 ** -23)
    live = torch.tensor(lens > 0).cuda()
    top = 6 * float(O.E4M3[0x4f])
    assert ((out.float() - want.float()).abs() <= tol * top).all() and (out[~live] == 0).all()
    assert torch.equal(lse[~live], want_lse[~live]) and (lse[live] - want_lse[live]).abs().max() < 1e-3
    # bad lengths and pages among them
    lens[1], lens[B // 2] = -1, blocks * 16 + 1
    which = int(np.argmax(np.where(lens <= blocks * 16, lens, 0)))
    table[which, int(lens[which] - 1) // 16] = len(pools[0])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, got_lse = b.decode_paged_fp4(*args[:3], i32(table), i32(lens), 0.05, err_flag=err)
    assert int(err) == b.PKV_DEVERR_BAD_LEN | b.PKV_DEVERR_BAD_PAGE
    nan = torch.zeros(B, dtype=torch.bool, device="cuda")
    nan[[1, B // 2, which]] = True
    assert got[nan].isnan().all() and got_lse[nan].isnan().all() and not got[~nan].isnan().any()
    assert ((got[~nan].float() - want[~nan].float()).abs() <= tol * top).all()
    # nothing at all
    out, lse = b.decode_paged_fp4(*args[:4], i32(np.zeros(B)), 0.05)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_decode_rising_logits(b):
    """Every page's logits pass the reference value, and by up to several hundred powers of two; then they fall."""
    r = np.random.default_rng(12)
    D, lens = 128, [640, 637]
    q, pools, table, bad, hs = make_decode(r, lens, 2, 1, D)
    for i, n in enumerate(lens):
        for j in range(-(-n // 16)):
            up = j if i == 0 else 39 - j
            pools[0][table[i, j], 0, 8 * D:] = np.where(pools[0][table[i, j], 0, 8 * D:] == 0x7f, 0x7f, 0x20 + up)
    want = O.decode(q.float().numpy(), *pools, *hs, table, lens, 0.3)
    assert np.ptp(want[1]) > 0
    for splits in (1, 5, 0):
        out, lse = b.decode_paged_fp4(q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), 0.3, k_scale=gpu(hs[0]),
                                      v_scale=gpu(hs[1]), num_splits=splits)
        close(out.float().cpu().numpy(), lse.cpu().numpy(), *want, lens, D, 6 * O.E4M3[0x4f] * hs[1].max())


@pytest.mark.parametrize("q_size,scale", [(1.0, 0.0), (1.0, -0.11), (1e-38, 0.1), (1e-30, 1e-20), (0.0, 1.0)])
def test_decode_scales_of_any_size(b, q_size, scale):
    """No scale, a negative one, negative scales of a head, logits far below fp32's smallest numbers; pages that are not full."""
    r = np.random.default_rng(20)
    D, lens = 128, [1, 17, 90]
    q, pools, table, bad, hs = make_decode(r, lens, 4, 2, D)
    hs[0][1] *= -1
    hs[1][0] *= -1
    q = (q.float() * q_size).bfloat16()
    want = O.decode(q.float().numpy(), *pools, *hs, table, lens, scale)
    want = want[:3] + (np.abs(want[3]),)
    out, lse = b.decode_paged_fp4(q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), scale, k_scale=gpu(hs[0]),
                                  v_scale=gpu(hs[1]))
    close(out.float().cpu().numpy(), lse.cpu().numpy(), *want, lens, D, 6 * O.E4M3[0x4f] * np.abs(hs[1]).max())


@pytest.mark.parametrize("D", [64, 128])
def test_decode_keeps_small_weights(b, D):
    """Tails of keys whose weights are 2^-13, 2^-19 and 2^-26 of the largest one's, which each warp meets in its first
    step and whose value is 0: what comes out is the tails'. A weight is held in f16 at 2^7 of what it is relative to the first
    step's largest, so it is off by 2^-11 of itself or, below f16's normal range, by 2^-32 of that one."""
    r = np.random.default_rng(27)
    pages, lens = 48, [768, 761, 750]
    codes_at, scale = 8 * D, 1.07 / math.log2(math.e)
    k, v = (np.zeros((3 * pages, 1, 9 * D), dtype=np.uint8) for _ in range(2))
    k[..., 0] = 0x07  # element 0 is 6 times its scale, the rest 0
    s = {x: int(np.flatnonzero(O.E4M3 == x)[0]) for x in (12, 13, 14, 16)}
    for i, tail in enumerate((14, 13, 12)):  # 12.8, 19.3 and 25.7 powers of two below the largest
        k[i * pages:(i + 1) * pages, 0, codes_at:codes_at + 16] = s[tail]
        v[i * pages:(i + 1) * pages, 0, :codes_at] = 0x22 + r.integers(0, 6, (pages, codes_at)) * 0x11 % 0x66
        v[i * pages:(i + 1) * pages, 0, codes_at:] = r.integers(0x38, 0x50, (pages, D))
        for w in range(4):  # a warp's first step: two pages
            k[i * pages + 2 * w, 0, codes_at] = s[16]
            v[i * pages + 2 * w, 0, codes_at::16] = 0
    table = np.arange(3 * pages).reshape(3, pages)
    q = torch.zeros(3, 2, D)
    q[:, 0, 0], q[:, 1, 0] = 1.0, 0.984375
    q = q.bfloat16()
    out, lse = b.decode_paged_fp4(q.cuda(), gpu(k), gpu(v), i32(table), i32(lens), scale, num_splits=1)
    want, want_lse, size, mass = O.decode(q.double().numpy(), k, v, None, None, table, lens, scale)
    n = np.array(lens, dtype=np.float64)[:, None]
    e = (D + 8) * 2.0 ** -24 * mass + 2.0 ** -20
    top = np.exp(scale * 96 * q[:, :, 0].double().numpy() - want_lse)  # the largest weight
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * e + n * 2.0 ** -24)[..., None] * size + (n * 2.0 ** -32 * top)[..., None] * 48
    got = out.double().cpu().numpy()
    assert (want > 0).any((1, 2)).all() and (np.abs(got - want) <= tol).all()
    assert (np.abs(lse.cpu().numpy() - want_lse) <= e + n * 2.0 ** -24 + 2.0 ** -21 * np.abs(want_lse)).all()


@pytest.mark.parametrize("most", [2.0 ** 8, 2.0 ** 17, 2.0 ** 20, 2.0 ** 23])
def test_decode_large_logits(b, most):
    """Logits up to 2^23, whose steps there are as wide as a factor of two of a weight: results are means of V."""
    r = np.random.default_rng(29)
    D, lens = 64, [900, 200]
    q, pools, table, bad, hs = make_decode(r, lens, 4, 2, D)
    scale = most / O.decode(q.double().numpy(), *pools, *hs, table, lens, 1.0)[3].max()  # (of the sums of magnitudes)
    scale = float(np.float32(scale))
    want, want_lse, size, mass = O.decode(q.double().numpy(), *pools, *hs, table, lens, scale)
    for splits in (1, 3):
        out, lse = b.decode_paged_fp4(q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), scale, k_scale=gpu(hs[0]),
                                      v_scale=gpu(hs[1]), num_splits=splits)
        got = out.double().cpu().numpy()
        # a logit's error makes other weights of the same sum: still a mean
        assert np.isfinite(got).all() and (np.abs(got).max((1, 2)) <= 6 * O.E4M3[0x4f] * hs[1].max() * (1 + 2.0 ** -7)).all()
        e = (D + 8) * 2.0 ** -24 * mass + 2.0 ** -20
        assert (np.abs(lse.cpu().numpy() - want_lse) <= e + 900 * 2.0 ** -24 + 2.0 ** -21 * np.abs(want_lse)).all()
        if most < 1000:
            close(out.float().cpu().numpy(), lse.cpu().numpy(), want, want_lse, size, mass, lens, D, 6 * O.E4M3[0x4f] * hs[1].max())


@pytest.mark.parametrize("scale,head,q_at", [(2.0 ** 100, 2.0 ** 29, -133), (2.0 ** -70, 2.0 ** -70, 122), (2.0 ** -120, 2.0 ** 20, 97),
                                             (-2.0 ** 64, 2.0 ** 64, -128), (2.0 ** -140, 2.0 ** 35, 100)])
def test_decode_scale_times_head_scale_outside_fp32(b, scale, head, q_at):
    """A scale and head scales whose product is no normal fp32 number, with queries of the opposite size: ordinary logits."""
    r = np.random.default_rng(28)
    D, lens = 128, [1, 40, 90]
    q, pools, table, bad, hs = make_decode(r, lens, 4, 2, D)
    for pool in pools:
        live = pool[..., 8 * D:]
        if q_at == 122:
            live[live < 0x50] += 0x2e  # (products of 2^-140 need large keys)
    hs[0] = (head * (1 + r.random(2))).astype(np.float32)
    x = r.integers(-8, 9, (3, 4, D)).astype(np.float64) * 2.0 ** q_at
    q = torch.tensor(x).to(torch.bfloat16)
    assert (q.double().numpy() == x).all()
    want = O.decode(x, *pools, *hs, table, lens, scale)
    want = want[:3] + (np.abs(want[3]),)
    out, lse = b.decode_paged_fp4(q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), scale, k_scale=gpu(hs[0]),
                                  v_scale=gpu(hs[1]))
    close(out.float().cpu().numpy(), lse.cpu().numpy(), *want, lens, D, 6 * 448 * hs[1].max())


@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_decode_queries_outside_f16(b, size):
    r = np.random.default_rng(13)
    D, lens = 64, [100]
    q, pools, table, bad, hs = make_decode(r, lens, 4, 2, D)
    q = (q.float() * size).bfloat16()
    scale = 0.2 / size
    want = O.decode(q.float().numpy(), *pools, *hs, table, lens, scale)
    out, lse = b.decode_paged_fp4(q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), scale, k_scale=gpu(hs[0]),
                                  v_scale=gpu(hs[1]))
    close(out.float().cpu().numpy(), lse.cpu().numpy(), *want, lens, D, 6 * O.E4M3[0x4f] * hs[1].max())


def test_decode_without_head_scales_or_lse_and_strided_heads(b):
    r = np.random.default_rng(14)
    D, lens = 128, [40, 3]
    q, pools, table, bad, _ = make_decode(r, lens, 4, 2, D)
    want = O.decode(q.float().numpy(), *pools, None, None, table, lens, 0.02)
    args = q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), 0.02
    out, lse = b.decode_paged_fp4(*args)
    close(out.float().cpu().numpy(), lse.cpu().numpy(), *want, lens, D, 6 * O.E4M3[0x4f])
    with pytest.raises(ValueError, match="contiguous"):
        b.decode_paged_fp4(q.cuda().transpose(0, 1).contiguous().transpose(0, 1), *args[1:])


def test_decode_nan_and_infinity_stay_in_their_rows(b):
    r = np.random.default_rng(15)
    D, lens = 64, [50, 33, 20]
    q, pools, table, bad, hs = make_decode(r, lens, 4, 2, D)
    clean, clean_lse = b.decode_paged_fp4(q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), 0.1, gpu(hs[0]), gpu(hs[1]))
    # a NaN scale of a live K: the row's queries of that KV head; of a live V: 16 columns of them
    pools[0][table[1, 0], 1, 8 * D + 2] = 0x7f
    pools[1][table[2, 0], 0, 8 * D + 16 + 3] = 0x7f
    q[0, 1, 5] = math.nan
    out, lse = b.decode_paged_fp4(q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), 0.1, gpu(hs[0]), gpu(hs[1]))
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[1, 2:4] = True
    nan[2, 0:2, 16:32] = True
    nan[0, 1] = True
    assert torch.equal(out.isnan(), nan)
    assert torch.equal(out[~nan], clean[~nan])
    assert torch.equal(lse.isnan(), torch.tensor([[False, True, False, False], [False, False, True, True], [False] * 4]).cuda())
    assert torch.equal(lse[~lse.isnan()], clean_lse[~lse.isnan()])


@pytest.mark.parametrize("splits,extra", [(1, 1), (2, 1), (0, 1), (0, 40)])
def test_decode_bad_pages_and_lengths(b, splits, extra):
    r = np.random.default_rng(16)
    D, lens = 128, [60, 70, 80]
    q, pools, table, bad, hs = make_decode(r, lens, 4, 2, D, extra_blocks=extra)
    args = [q.cuda(), gpu(pools[0]), gpu(pools[1])]
    clean, _ = b.decode_paged_fp4(*args, i32(bad), i32(lens), 0.1, num_splits=splits)
    for entry in (-1, len(pools[0]), 1 << 30, -(1 << 31)):
        broken = bad.copy()
        broken[1, 3] = entry
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = b.decode_paged_fp4(*args, i32(broken), i32(lens), 0.1, num_splits=splits, err_flag=err)
        assert int(err) == b.PKV_DEVERR_BAD_PAGE
        assert out[1].isnan().all() and lse[1].isnan().all()
        assert torch.equal(out[[0, 2]], clean[[0, 2]])
    for n in (-1, table.shape[1] * 16 + 1, 1 << 30):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = b.decode_paged_fp4(*args, i32(bad), i32([60, n, 80]), 0.1, num_splits=splits, err_flag=err)
        assert int(err) == b.PKV_DEVERR_BAD_LEN
        assert out[1].isnan().all() and lse[1].isnan().all()
        assert torch.equal(out[[0, 2]], clean[[0, 2]])


def test_offsets_past_32_bits(b):
    """Pools of more than 2^32 bytes: pack, decode and unpack at their last pages."""
    D, heads = 128, 8
    pages = (1 << 32) // (heads * 9 * D) + 40
    k, v = (torch.zeros(pages, heads, 9 * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    r = np.random.default_rng(17)
    rows = [torch.randn(3, heads, 16, D, device="cuda").bfloat16() for _ in range(2)]
    src, table = i32([[2, 0, 1]]), i32([[pages - 1, pages - 30, pages - 2]])
    b.cache_pack_fp4(*rows, src, k, v, table, i32([45]))
    small = [torch.stack([x[pages - 1], x[pages - 30], x[pages - 2]]) for x in (k, v)]
    want = O.pack(rows[0].float().cpu().numpy(), [[2, 0, 1]], [0], np.zeros((3, heads, 9 * D), dtype=np.uint8), [[0, 1, 2]], [0], [45], None)
    assert (small[0].cpu().numpy() == want).all()
    q = torch.tensor(r.standard_normal((1, 16, D))).bfloat16().cuda()
    for x, y in zip(b.decode_paged_fp4(q, k, v, table, i32([45]), 0.1),
                    b.decode_paged_fp4(q, *small, i32([[0, 1, 2]]), i32([45]), 0.1)):
        assert torch.equal(x, y)
    back = [torch.zeros(3, heads, 16, D, device="cuda").bfloat16() for _ in range(4)]
    b.cache_unpack_fp4(k, v, table, *back[:2], src, i32([45]))
    b.cache_unpack_fp4(*small, i32([[0, 1, 2]]), *back[2:], src, i32([45]))
    assert torch.equal(back[0], back[2]) and torch.equal(back[1], back[3]) and back[0].abs().max() > 1


def test_captured_and_replayed(b):
    """A step (pack, decode, unpack) captured once and replayed on new contents; two captures keep their own workspaces."""
    r = np.random.default_rng(18)
    D, lens = 128, [100, 250]
    q, pools, table, bad, hs = make_decode(r, lens, 8, 2, D, poison=False)
    k, v, t, n = gpu(pools[0]), gpu(pools[1]), i32(table), i32(lens)
    qs, new = q.cuda(), torch.randn(2, 2, 16, D, device="cuda").bfloat16()
    src, one, first = i32([[0], [1]]), i32([1, 1]), i32([99, 249])
    back = torch.zeros(table.size, 2, 16, D, device="cuda").bfloat16()

    def step():
        b.cache_pack_fp4(new, new, src, k, v, t, one, first=first, max_count=1)
        out, lse = b.decode_paged_fp4(qs, k, v, t, n, 0.1, num_splits=3)
        b.cache_unpack_fp4(k, v, t, back, torch.empty_like(back), t, n)
        return out, lse

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for seed in range(3):
        new.copy_(torch.randn(2, 2, 16, D, generator=torch.Generator("cuda").manual_seed(seed), device="cuda"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs[0]], [x.clone() for x in outs[1]], back.clone()
        want = step()
        for a in got[:2]:
            assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
        assert torch.equal(got[2], back)


def test_a_head_scale_that_is_nan_or_infinite(b):
    r = np.random.default_rng(21)
    D, lens = 64, [40]
    q, pools, table, bad, hs = make_decode(r, lens, 4, 4, D)
    for which in (0, 1):
        for value in (math.nan, math.inf):
            scales = [x.copy() for x in hs]
            scales[which][2] = value
            out, lse = b.decode_paged_fp4(q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), 0.1, gpu(scales[0]), gpu(scales[1]))
            assert not out[0, 2].isfinite().any() and out[0, [0, 1, 3]].isfinite().all()
    k = gpu(pools[0])
    rows = torch.randn(1, 4, 16, D, device="cuda")
    scales = gpu(np.array([1, 0, math.nan, math.inf], dtype=np.float32))
    b.cache_pack_fp4(rows, rows, i32([[0]]), k, k.clone(), i32([[0]]), i32([16]), k_scale=scales, v_scale=scales)
    back = torch.zeros_like(rows)
    b.cache_unpack_fp4(k, k, i32([[0]]), back, back.clone(), i32([[0]]), i32([16]))
    # a scale of 0 or NaN has nothing to say; by an infinite one everything is 0
    assert back[0, 0].isfinite().all() and back[0, 1:3].isnan().all() and (back[0, 3] == 0).all()


def test_two_streams_at_once(b):
    """Calls on two streams with buffers of their own, many at a time, against the same calls one after another."""
    r = np.random.default_rng(22)
    jobs = []
    for i in range(2):
        lens = [700 - 100 * i, 90]
        q, pools, table, bad, hs = make_decode(r, lens, 8, 2, 128, poison=False)
        jobs.append(((q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32(lens), 0.1), torch.randn(2, 2, 16, 128, device="cuda")))
    src, one = i32([[0], [1]]), i32([16, 9])
    want = []
    for args, rows in jobs:
        pools = args[1].clone(), args[2].clone()
        b.cache_pack_fp4(rows, rows, src, *pools, args[3], one)
        want.append(b.decode_paged_fp4(args[0], *pools, *args[3:], num_splits=5) + pools)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in jobs], [[], []]
    pools = [(a[1].clone(), a[2].clone()) for a, _ in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (args, rows) in enumerate(jobs):
            b.cache_pack_fp4(rows, rows, src, *pools[i], args[3], one, stream=streams[i])
            got[i].append(b.decode_paged_fp4(args[0], *pools[i], *args[3:], num_splits=5, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(pools[i][0], want[i][2]) and torch.equal(pools[i][1], want[i][3])
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_another_stream(b):
    """stream= with no buffers given, against the same call on the current stream."""
    r = np.random.default_rng(19)
    q, pools, table, bad, hs = make_decode(r, [200, 90], 4, 1, 64)
    args = q.cuda(), gpu(pools[0]), gpu(pools[1]), i32(bad), i32([200, 90]), 0.1
    want = b.decode_paged_fp4(*args, num_splits=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = b.decode_paged_fp4(*args, num_splits=2, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("B,Hkv,G,D,blocks,splits", [(130, 8, 1, 128, 250, 1), (20, 32, 1, 64, 280, 2), (700, 1, 7, 64, 80, 1),
                                                     (256, 4, 4, 128, 120, 1), (24, 8, 2, 128, 800, 6)])
def test_decode_batches_that_are_put_in_order(b, B, Hkv, G, D, blocks, splits):
    """More CTAs than fit, in order of their lengths: the same bits as the sequences a few at a time, with rows that are empty,
    full or bad among them; also captured, and replayed with other lengths."""
    r = np.random.default_rng(26)
    pages = 700
    k, v = (gpu(some_pool(r, pages, Hkv, D)) for _ in range(2))
    table = r.integers(0, pages, (B, blocks))
    lens = r.integers(1, blocks * 16 + 1, B)
    lens[r.random(B) < 0.3] //= 20
    lens[[0, 3, 7, 11]] = [0, blocks * 16, -1, blocks * 16 + 1]
    table[5, 0], lens[5] = pages, 40
    q = torch.tensor((2 * r.standard_normal((B, Hkv * G, D))).astype(np.float32)).bfloat16().cuda()
    t, n = i32(table), i32(lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def apart():
        some = [b.decode_paged_fp4(q[i:i + 4].contiguous(), k, v, t[i:i + 4].contiguous(), n[i:i + 4].contiguous(), 0.1,
                                   num_splits=splits) for i in range(0, B, 4)]
        return [torch.cat(x) for x in zip(*some)]

    def same(got, lens):
        for x, y in zip(got, apart()):
            assert torch.equal(torch.nan_to_num(x, nan=7.5), torch.nan_to_num(y, nan=7.5))
        bad = (lens < 0) | (lens > blocks * 16) | (np.arange(B) == 5)
        assert (got[0].isnan().flatten(1).all(1).cpu().numpy() == bad).all() and (got[0][0] == 0).all()

    same(b.decode_paged_fp4(q, k, v, t, n, 0.1, num_splits=splits, err_flag=err), lens)
    assert int(err) == b.PKV_DEVERR_BAD_PAGE | b.PKV_DEVERR_BAD_LEN
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.decode_paged_fp4(q, k, v, t, n, 0.1, num_splits=splits)
    lens = np.concatenate([[0], r.integers(1, blocks * 16 + 1, B - 1)])
    lens[5] = 40
    n.copy_(i32(lens))
    graph.replay()
    torch.cuda.synchronize()
    same(got, lens)


def test_pack_with_a_negative_head_scale(b):
    """Scales stay positive and the codes' signs turn, also where a group's scale is rounded to 0."""
    r = np.random.default_rng(23)
    for d, t in ((64, torch.float32), (128, torch.bfloat16)):
        x = torch.tensor((r.standard_normal((1, 2, 16, d)) * r.choice([1e-8, 1e-3, 1, 100], (1, 2, 16, 1))).astype(np.float32)).to(t)
        hs = np.array([-0.01, -3.0], dtype=np.float32)
        pool = np.zeros((1, 2, 9 * d), dtype=np.uint8)
        want = O.pack(x.float().numpy(), [[0]], [0], pool, [[0]], [0], [16], hs)
        k, v = gpu(pool), gpu(pool)
        b.cache_pack_fp4(x.cuda(), x.cuda(), i32([[0]]), k, v, i32([[0]]), i32([16]), k_scale=gpu(hs), v_scale=gpu(hs))
        assert (k.cpu().numpy() == want).all() and (v.cpu().numpy() == want).all()
        assert (want[..., 8 * d:] == 0).any() and (want[..., 8 * d:] < 128).all()


def test_the_largest_batch(b):
    """65535 sequences of 0, 1 or 2 tokens, all in the same two pages: packed, attended, read back."""
    r = np.random.default_rng(24)
    B, d = 65535, 64
    pool = [some_pool(r, 2, 1, d) for _ in range(2)]
    k, v = gpu(pool[0]), gpu(pool[1])
    lens = np.arange(B) % 3
    table = i32(np.stack([np.arange(B) % 2], 1))
    q = torch.tensor(r.standard_normal((2, 1, d)).astype(np.float32)).bfloat16().cuda()
    out, lse = b.decode_paged_fp4(q[torch.arange(B, device="cuda") % 2].contiguous(), k, v, table, i32(lens), 0.1)
    few, few_lse = b.decode_paged_fp4(q[[0, 1, 0, 1, 0, 1]].contiguous(), k, v, table[:6].contiguous(), i32(lens[:6]), 0.1)
    at = torch.arange(B, device="cuda") % 6
    assert torch.equal(out, few[at]) and torch.equal(lse, few_lse[at])
    want, want_lse, size, mass = O.decode(q.double().cpu().numpy()[[0, 1, 0, 1, 0, 1]], *pool, None, None, [[0], [1]] * 3,
                                          lens[:6], 0.1)
    close(few.double().cpu().numpy(), few_lse.double().cpu().numpy(), want, want_lse, size, mass, lens[:6], d, 48.0)
    # each into a slot of its own: token i of block j, sequence 16 j + i
    rows = torch.tensor(r.standard_normal((2, 1, 16, d)).astype(np.float32)).cuda()
    blocks = (B + 15) // 16
    wide = [torch.zeros(blocks, 1, 9 * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    own, one = i32(np.arange(B)[:, None] // 16), i32(np.ones(B))
    slot = i32(np.arange(B) % 16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.cache_pack_fp4(rows, rows, table, *wide, own, one, first=slot, src_first=slot, max_count=1, err_flag=err)
    back = [torch.zeros(blocks, 1, 16, d, device="cuda") for _ in range(2)]
    b.cache_unpack_fp4(*wide, own, *back, own, one, first=slot, dst_first=slot, max_count=1, err_flag=err)
    codes, scales = O.quantise(rows.cpu().numpy())
    want = torch.tensor(O.values(codes, scales)).cuda()  # [2, 1, 16, d]
    i = torch.arange(B, device="cuda")
    assert int(err) == 0 and all(torch.equal(x[i // 16, 0, i % 16], want[i % 2, 0, i % 16]) for x in back)
    assert all((x[-1, 0, 15] == 0).all() for x in back)  # (the slot of no sequence)


@pytest.mark.parametrize("batch,pages", [(40, 2000), (600, 26000), (600, 40000)])
def test_tables_changed_and_read_back_to_back(b, batch, pages):
    """A table that grows in place each step, with forks, and the calls that read it right behind: one CTA's tables, a
    cluster's, and those in the workspace, against the same steps with a pause after each call."""
    r = np.random.default_rng(25)
    H, d, blocks = 1, 64, 40
    lens = np.repeat(r.integers(0, 500, batch // 2), 2)
    rows = torch.randn(batch, H, 16, d, device="cuda").bfloat16()
    src, q = i32(np.arange(batch)[:, None]), torch.randn(batch, 4, d, device="cuda").bfloat16()
    results = []
    for pause in (True, False):
        k, v = (torch.full((pages, H, 9 * d), 0x22, dtype=torch.uint8, device="cuda") for _ in range(2))
        table, n, one = i32(np.zeros((batch, blocks))), i32(np.zeros(batch)), i32(np.ones(batch) * 7)
        err, got = torch.zeros(1, dtype=torch.int32, device="cuda"), []
        grown = [i32(lens + 7 * s) for s in range(18)]
        torch.cuda.synchronize()
        for s in range(17):
            if s == 6:  # every other sequence becomes a fork of the one before it
                table[1::2] = table[0::2]
            b.cache_reserve(table, n if s == 0 else grown[s], grown[s + 1], [k, v], out=table, err_flag=err)
            if pause:
                torch.cuda.synchronize()
            b.cache_pack_fp4(rows, rows, src, k, v, table, one, first=grown[s], max_count=7, err_flag=err)
            if pause:
                torch.cuda.synchronize()
            got.append(b.decode_paged_fp4(q, k, v, table, grown[s + 1], 0.1, err_flag=err)[0])
            if pause:
                torch.cuda.synchronize()
            if s % 5 == 4:
                b.cache_compact(table, grown[s + 1], [k, v], out=table, err_flag=err)
                if pause:
                    torch.cuda.synchronize()
                got.append(b.decode_paged_fp4(q, k, v, table, grown[s + 1], 0.1, err_flag=err)[0])
        torch.cuda.synchronize()
        assert int(err) == 0
        results.append(got + [table, k, v])
    assert all(torch.equal(x, y) for x, y in zip(*results)) and results[0][0].isfinite().all()


def test_no_sequences(b):
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    k = torch.zeros(2, 1, 9 * 64, dtype=torch.uint8, device="cuda")
    rows = torch.ones(2, 1, 16, 64, device="cuda")
    out, lse = b.decode_paged_fp4(torch.empty(0, 4, 64, device="cuda").bfloat16(), k, k.clone(), none, none[:, 0].contiguous(), 0.1)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    b.cache_pack_fp4(rows, rows.clone(), none, k, k.clone(), none, none[:, 0].contiguous())
    b.cache_unpack_fp4(k, k.clone(), none, rows, rows.clone(), none, none[:, 0].contiguous())
    assert (k == 0).all() and (rows == 1).all()
