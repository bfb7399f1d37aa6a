"""Calls at the edge of what the operators around the paged attention take: empty and padded chunks, infinite
values, results near the smallest numbers, more features than one kernel's grid holds, tables of many pages.
"""
import pytest
import torch

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
