"""Calls of the binding with ``stream=``, another stream than the current one, and no buffers given: what a
call allocates for itself belongs to the stream it runs on. Each call is compared with itself on the current
stream, bit for bit.
"""
import pytest
import torch

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


def calls(b):
    """name -> f(**kw), each with its inputs on the device and no buffer given; f() is the same on every call."""
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kp, vp = r(64, 2, 16, 128), r(64, 2, 16, 128)
    order = torch.randperm(64, generator=g, device="cuda").to(torch.int32)
    table, new, suffix = (t.contiguous() for t in (order[:40].view(2, 20), order[40:48].view(2, 4), order[48:56].view(2, 4)))
    prefix = table[0, :8].contiguous()
    q, qc, lens, start, tails = r(2, 8, 128), r(2, 40, 8, 128), i(300, 170), i(9, 77), i(60, 33)
    sums, to = torch.rand(2, 2, 320, generator=g, device="cuda"), torch.zeros(2, 2, 320, device="cuda")
    x, w, k, v = r(200, 256), r(320, 256), r(2, 40, 2, 128), r(2, 40, 2, 128)
    part, plse = torch.randn(2, 6, 128, generator=g, device="cuda"), torch.randn(2, 6, generator=g, device="cuda")
    f = workloads.make_paged_decode_fp8(3, 2, 8, 2, 128, 16, [40, 60], num_pages=12)
    f8 = [t.cuda() for t in (f.q, f.k_codes, f.v_codes, f.k_scale, f.v_scale, f.block_table, f.kv_lens)]
    pools = kp.clone(), vp.clone()
    return {
        "decode_paged": lambda **kw: b.decode_paged(q, kp, vp, table, lens, 0.1, num_splits=3, **kw),
        "decode_paged_fp8": lambda **kw: b.decode_paged_fp8(*f8, 0.1, num_splits=2, **kw),
        "merge_states": lambda **kw: b.merge_states(part[0], plse[0], part[1], plse[1], **kw),
        "prefill_causal": lambda **kw: b.prefill_causal(qc, k, v, 0.1, **kw),
        "prefill_paged_chunk": lambda **kw: b.prefill_paged_chunk(qc, kp, vp, table, start, 0.1, **kw),
        "decode_cascade": lambda **kw: b.decode_cascade(q, kp, vp, prefix, 128, suffix, tails, 0.1, **kw),
        "flat_gemm": lambda **kw: b.flat_gemm(x[:7], w, **kw),
        "qk_norm_rope_append": lambda **kw: b.qk_norm_rope_append(qc, k, v, *pools, table, start, **kw),
        "decode_paged_weights": lambda **kw: b.decode_paged_weights(q, kp, vp, table, lens, sums, 0.1, sums_out=to,
                                                                    num_splits=3, **kw),
        "cache_evict": lambda **kw: b.cache_evict(kp, vp, table, lens, sums, new, 60, 2, 8, **kw),
        "linear": lambda **kw: b.linear(x, w, activation="silu", **kw),
    }


NAMES = ["decode_paged", "decode_paged_fp8", "merge_states", "prefill_causal", "prefill_paged_chunk", "decode_cascade",
         "flat_gemm", "qk_norm_rope_append", "decode_paged_weights", "cache_evict", "linear"]


def outputs(x):
    return list(x) if isinstance(x, tuple) else [x]


def same(got, want):
    return all(torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0)) for x, y in zip(got, want))


def busy(ms):
    """Work for the current stream, about that long."""
    x = torch.ones(1 << 28, device="cuda")  # 2 GB read and written a pass: 0.3 ms
    for _ in range(int(ms / 0.3) + 1):
        x.mul_(1.0)


@pytest.mark.parametrize("name", NAMES)
def test_buffers_are_allocated_on_the_calls_stream(b, name, monkeypatch):
    f = calls(b)[name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    at = []
    empty, empty_like = torch.empty, torch.empty_like

    def record(make):
        def call(*a, **kw):
            at.append(torch.cuda.current_stream().cuda_stream)
            return make(*a, **kw)
        return call
    monkeypatch.setattr(torch, "empty", record(empty))
    monkeypatch.setattr(torch, "empty_like", record(empty_like))
    f(stream=s)
    torch.cuda.synchronize()
    assert at and all(x == s.cuda_stream for x in at)
    at.clear()
    f(stream=torch.cuda.current_stream())
    f()
    torch.cuda.synchronize()
    assert at and all(x == torch.cuda.current_stream().cuda_stream for x in at)


@pytest.mark.parametrize("name", ["linear", "cache_evict", "decode_paged_weights", "decode_paged"])
def test_pending_work_on_freed_memory_does_not_reach_the_outputs(b, name):
    """The current stream still has to write memory that it has freed; the call on the other stream must not be
    given that memory."""
    f = calls(b)[name]
    want = [t.clone() for t in outputs(f())]
    sizes = [t.numel() * t.element_size() for t in want]
    s = torch.cuda.Stream()
    fill = lambda: [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(77) for n in sizes for _ in range(20)]  # noqa: E731
    f(stream=s)
    busy(1)
    fill()
    torch.cuda.synchronize()
    busy(30)
    fill()
    got = outputs(f(stream=s))
    torch.cuda.synchronize()
    assert same(got, want)


def test_an_output_dropped_while_the_current_stream_reads_it(b):
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w = (torch.randn(256, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    want, other = b.linear(x, w).clone(), b.linear(w, w)
    s = torch.cuda.Stream()
    busy(1)
    torch.cuda.synchronize()
    y = b.linear(x, w, stream=s)
    s.synchronize()
    busy(30)
    got = y.clone()  # waits behind the work above
    del y
    z = [b.linear(w, w, stream=s) for _ in range(4)]
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(t, other) for t in z)
