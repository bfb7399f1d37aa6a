"""One layer's serving steps through the operators together: projection, norm, rotation and page
write, chunked prefill with its weights, output projection with the residual, eviction, and
decode steps on what was kept. Every stage is checked in fp64 on the inputs that the GPU gave it;
the bars are the operators' own (their test files derive them), the bf16 one for the attention.
"""
import numpy as np
import pytest
import torch

import oracle
from tests._compare import assert_close
from tests.test_linear_gpu import check as check_linear

pytestmark = pytest.mark.gpu

HQ, HKV, D, HIDDEN = 8, 2, 128, 256


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_28_gb300 import build
    build.build(quiet=True)
    from paged_kv_attention_28_gb300 import binding
    return binding


def test_prompt_eviction_and_decode(b):
    g = torch.Generator().manual_seed(21)
    B, C, budget, steps = 2, 90, 48, 3
    scale = D ** -0.5
    w_qkv = (torch.randn((HQ + 2 * HKV) * D, HIDDEN, generator=g) / HIDDEN ** 0.5).bfloat16()
    b_qkv = (0.1 * torch.randn(w_qkv.shape[0], generator=g)).bfloat16()
    w_o = (torch.randn(HIDDEN, HQ * D, generator=g) / (HQ * D) ** 0.5).bfloat16()
    qn, kn = ((1 + 0.1 * torch.randn(D, generator=g)).bfloat16() for _ in range(2))
    freq = (1e4 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)).float()
    dev = {k: v.cuda() for k, v in dict(w_qkv=w_qkv, b_qkv=b_qkv, w_o=w_o, qn=qn, kn=kn, freq=freq).items()}
    blocks, kept_blocks = 6, 4
    order = torch.randperm(32, generator=g).to(torch.int32)
    table = order[:B * blocks].view(B, blocks).contiguous().cuda()
    new_table = order[12:12 + B * kept_blocks].view(B, kept_blocks).contiguous().cuda()
    kp, vp = (torch.full((32, HKV, 16, D), float("nan")).bfloat16().cuda() for _ in range(2))
    sums = torch.zeros(B, HKV, blocks * 16, device="cuda")
    chunk_lens = torch.tensor([90, 61], dtype=torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def project_and_append(h, table, lens, positions, n_new):
        bb, c = h.shape[:2]
        qkv = b.linear(h.view(bb * c, HIDDEN), dev["w_qkv"], bias=dev["b_qkv"], err_flag=err)
        check_linear(qkv, h.view(bb * c, HIDDEN).cpu(), w_qkv, b_qkv, "none", None)
        x = qkv.view(bb, c, HQ + 2 * HKV, D)
        before = kp.cpu().double().numpy(), vp.cpu().double().numpy()
        q = torch.zeros(bb, c, HQ, D, dtype=torch.bfloat16, device="cuda")
        b.qk_norm_rope_append(x[:, :, :HQ], x[:, :, HQ:HQ + HKV], x[:, :, HQ + HKV:], kp, vp, table, lens.cuda(),
                              chunk_lens=n_new.cuda(), positions=positions.cuda(), inv_freq=dev["freq"],
                              q_norm=dev["qn"], k_norm=dev["kn"], out=q, err_flag=err)
        xs = x.cpu().double().numpy()
        wq, wk, wv = oracle.append(xs[:, :, :HQ], xs[:, :, HQ:HQ + HKV], xs[:, :, HQ + HKV:], *before, table.cpu().numpy(),
                                   lens.numpy(), n_new.numpy(), positions[None].numpy(), freq.numpy(), None,
                                   qn.double().numpy(), kn.double().numpy(), 1e-6, False, np.zeros(q.shape))
        # |y_a| + |y_b| <= 16 (a normed row has |y| <= sqrt(128) * 1.4 in all)
        for got, want in ((q, wq), (kp, wk)):
            got = got.cpu().double().numpy()
            assert np.array_equal(np.isnan(got), np.isnan(want))
            assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * 32)[~np.isnan(want)].all()
        assert np.array_equal(vp.cpu().double().numpy(), wv, equal_nan=True)
        return q

    # the prompt: a padded chunk
    h = torch.randn(B, C, HIDDEN, generator=g).bfloat16().cuda()
    lens = torch.zeros(B, dtype=torch.int32)
    pos = torch.arange(C, dtype=torch.int32).expand(B, C).contiguous()
    q = project_and_append(h, table, lens, pos, chunk_lens)
    out, lse = b.prefill_paged_chunk(q, kp.nan_to_num(0), vp.nan_to_num(0), table, lens.cuda(), scale)
    b.chunk_weights(q, kp, table, lens.cuda(), lse, sums, scale, chunk_lens=chunk_lens.cuda(), err_flag=err)
    w = oracle.key_weights(q.cpu().double().numpy(), kp.cpu().double().numpy(), table.cpu().numpy(), lens.numpy(),
                           lse.cpu().double().numpy(), scale, last=chunk_lens.numpy())
    for i in range(B):
        n = int(chunk_lens[i])
        np.testing.assert_allclose(sums[i, :, :n].cpu().numpy(), w[i, :, :n], rtol=2.0 ** -23 * 132 * 30 * 2 + 2.0 ** -16)
        assert not sums[i, :, n:].any()
    y = b.linear(out.view(B * C, HQ * D), dev["w_o"], residual=h.view(B * C, HIDDEN), err_flag=err)
    check_linear(y, out.view(B * C, HQ * D).cpu(), w_o, None, "none", h.view(B * C, HIDDEN).cpu())

    # eviction to new pages
    kept, lens_d, sums = b.cache_evict(kp, vp, table, chunk_lens.cuda(), sums, new_table, budget, 2, 16, err_flag=err)
    wk, wl, _ = oracle.evict(chunk_lens.numpy(), w, budget, 2, 16)
    assert lens_d.tolist() == wl
    assert kept.shape == (B, HKV, budget) and bool((kept[:, :, 1:] > kept[:, :, :-1]).all())

    # decode goes on: token positions run ahead of the cache slots
    lens, at = lens_d.cpu(), chunk_lens.clone()
    for _ in range(steps):
        h = torch.randn(B, 1, HIDDEN, generator=g).bfloat16().cuda()
        q = project_and_append(h, new_table, lens, at[:, None].contiguous(), torch.ones(B, dtype=torch.int32))
        lens, at = lens + 1, at + 1
        before = sums.clone()
        o, l, sums = b.decode_paged_weights(q[:, 0].contiguous(), kp, vp, new_table, lens.cuda(), sums, scale, decay=0.9,
                                            err_flag=err)
        args = (q[:, 0].cpu().double().numpy(), kp.cpu().double().numpy())
        wo, wl = oracle.decode_paged(*args, vp.cpu().double().numpy(), new_table.cpu().numpy(), lens.numpy(), scale)
        assert_close(o.float().cpu().numpy(), wo, "bf16", "out")
        assert_close(l.cpu().numpy(), wl, "bf16", "lse")
        w = oracle.key_weights(args[0][:, None], args[1], new_table.cpu().numpy(), lens.numpy() - 1, wl[:, :, None], scale)
        for i in range(B):
            n = int(lens[i])
            np.testing.assert_allclose(sums[i, :, :n].cpu().numpy(), w[i, :, :n] + 0.9 * before[i, :, :n].cpu().numpy(),
                                       rtol=2.0 ** -23 * 132 * 30 * 2 + 2.0 ** -16)
            assert not sums[i, :, n:].any()
        y = b.linear(o.view(B, HQ * D), dev["w_o"], residual=h.view(B, HIDDEN), err_flag=err)
        check_linear(y, o.view(B, HQ * D).cpu(), w_o, None, "none", h.view(B, HIDDEN).cpu())
    assert int(err) == 0
