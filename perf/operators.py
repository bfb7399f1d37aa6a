"""Cases of the operators around the paged attention calls, to be timed and compared.

One layer's serving step over a paged KV cache runs: the projection of the new tokens
(`linear`: bias, activation and residual in the product's epilogue), per-head norms and the
rotation of queries and keys with the write into the pages (`append`), the attention that also
accumulates how much weight every cached token received (`decode` for single tokens, `chunk`
for a prompt's chunk), and the eviction of the tokens with the least weight (`evict`).

`run` computes each operator in plain torch operations in fp32 (`own` false) or through the
library's calls (`own` true); `exact` computes it in fp64, on its own.
"""
import math

import torch

own = False

DEV = "cuda"
PAGE = 16
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 sequences: fused QKV projection in, positions ahead of the cache
        # slots as they are after evictions
        dict(name="append_decode_64", op="append", batch=64, chunk=1, lo=1, hi=1024, hq=32, hkv=8, d=128, rot=128,
             axes=1, inter=False, norm=True, packed=True, ragged=False, dtype="bf16"),
        # a padded batch of image / video prompts: three position axes (time, height, width)
        dict(name="append_chunk_3axes", op="append", batch=4, chunk=2048, lo=0, hi=512, hq=32, hkv=8, d=128, rot=128,
             axes=3, inter=False, norm=True, packed=True, ragged=True, dtype="bf16"),
        # fp32, partial rotation of neighbouring pairs, no head norms, odd lengths
        dict(name="append_f32_odd", op="append", batch=3, chunk=37, lo=5, hi=300, hq=8, hkv=8, d=64, rot=32,
             axes=1, inter=True, norm=False, packed=False, ragged=True, dtype="f32"),
        # one sequence, one token, fp32: the smallest call, where latency counts
        dict(name="decode_f32_single", op="decode", batch=1, lo=256, hi=256, hq=8, hkv=8, d=64, dtype="f32"),
        # the batched decode with one query head per KV head, ragged lengths
        dict(name="decode_mha_batch", op="decode", batch=16, lo=512, hi=4096, hq=32, hkv=32, d=128, dtype="bf16"),
        # long contexts, four query heads per KV head
        dict(name="decode_gqa_long", op="decode", batch=4, lo=32768, hi=32768, hq=32, hkv=8, d=128, dtype="bf16"),
        # the last 32 queries of a prompt's chunk score the whole prompt (an observation window)
        dict(name="chunk_window32", op="chunk", batch=4, chunk=512, window=32, lo=2048, hi=8000, hq=32, hkv=8,
             d=128, dtype="bf16"),
        # every query of a chunk counts, causal inside the chunk
        dict(name="chunk_full", op="chunk", batch=2, chunk=2048, window=0, lo=1024, hi=2048, hq=32, hkv=8,
             d=128, dtype="bf16"),
        # a budget of 2048 tokens, overrun by a few hundred: what a serving loop evicts now and then
        dict(name="evict_2k", op="evict", batch=4, lo=2048, hi=2304, budget=2048, sink=4, recent=256, hkv=8, d=128,
             dtype="bf16"),
        # long prompts cut down to 4096 tokens right after their prefill
        dict(name="evict_32k", op="evict", batch=16, lo=16384, hi=32768, budget=4096, sink=4, recent=512, hkv=8, d=128,
             dtype="bf16"),
        # the output projection of a decode step: a few tokens, residual added in the epilogue
        dict(name="linear_o_proj_8", op="linear", m=8, n=4096, k=4096, act="none", bias=True, res=True),
        # a prompt's up projection with its activation
        dict(name="linear_up_4096", op="linear", m=4096, n=11008, k=4096, act="gelu_tanh", bias=True, res=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lens(rng, most):
    hi = _log(rng, 1, most)
    return max(1, int(hi * rng.uniform(0.1, 1.0))), hi


def draw(rng):
    op = rng.choice(["append", "decode", "chunk", "evict", "linear"])
    if op == "append":
        batch = _log(rng, 1, 64)
        chunk = _log(rng, 1, max(1, 8192 // batch)) if rng.random() < 0.6 else 1
        hq, hkv = rng.choice([(8, 8), (8, 2), (14, 2), (28, 4), (16, 16), (32, 8)])
        d = rng.choice([64, 128])
        rot = rng.choice([d, d, d // 2, d // 4])
        lo, hi = _lens(rng, 1024)
        return dict(op=op, batch=batch, chunk=chunk, lo=lo, hi=hi, hq=hq, hkv=hkv, d=d, rot=rot,
                    axes=rng.choice([1, 2, 3]), inter=rng.random() < 0.5, norm=rng.random() < 0.7,
                    packed=rng.random() < 0.5, ragged=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "decode":
        lo, hi = _lens(rng, 32768)
        hq, hkv = rng.choice([(8, 8), (16, 8), (32, 8), (32, 4), (16, 2), (32, 32)])
        d = rng.choice([64, 128, 128])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        size = hi * hkv * d * (4 if dtype == "f32" else 2)
        most = 4 * 32768 * 8 * 128 * 2 // size
        if most < 1:
            lo, hi, most = lo // 4 + 1, hi // 4 + 1, 1
        return dict(op=op, batch=_log(rng, 1, max(1, min(64, most))), lo=lo, hi=hi, hq=hq, hkv=hkv, d=d, dtype=dtype)
    if op == "chunk":
        chunk = _log(rng, 1, 2048)
        lo, hi = _lens(rng, 8192)
        hq, hkv = rng.choice([(8, 8), (16, 8), (32, 8), (32, 4), (16, 2)])
        window = 0 if rng.random() < 0.4 else _log(rng, 1, chunk)
        most = 2 * 2048 * 4096 * 32 // ((window or chunk) * (hi + chunk) * hq)
        if most < 1:
            chunk, hi, lo, window, most = chunk // 4 + 1, hi // 4 + 1, lo // 4 + 1, window // 4, 1
        return dict(op=op, batch=_log(rng, 1, max(1, min(16, most))), chunk=chunk, window=window, lo=lo, hi=hi, hq=hq,
                    hkv=hkv, d=128, dtype="bf16")
    if op == "evict":
        lo, hi = _lens(rng, 32768)
        hkv = rng.choice([1, 2, 4, 8, 8])
        budget = max(1, int(hi * rng.uniform(0.1, 1.0)))
        sink = min(budget, rng.choice([0, 1, 4]))
        d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "f32"])
        most = 16 * 4096 * 8 * 256 // (budget * hkv * d * (4 if dtype == "f32" else 2))
        if most < 1:
            budget, most, sink = budget // 8 + 1, 1, 0
        return dict(op=op, batch=_log(rng, 1, max(1, min(16, most))), lo=lo, hi=hi, budget=budget, sink=sink,
                    recent=int((budget - sink) * rng.uniform(0.0, 0.5)), hkv=hkv, d=d, dtype=dtype)
    m = _log(rng, 1, 4096)
    sizes = [256, 1000, 1024, 1536, 2048, 4096, 4097, 6144, 11008]
    n, k = rng.choice(sizes), rng.choice([72, 256, 1024, 1536, 2048, 4096])
    return dict(op="linear", m=m, n=n, k=k, act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                bias=rng.random() < 0.6, res=rng.random() < 0.5)


# ------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _lengths(g, case):
    """Lengths spread evenly over lo .. hi, in an order of the seed's."""
    n = case["batch"]
    at = torch.linspace(case["lo"], case["hi"], n, device=DEV, dtype=torch.float64) if n > 1 else \
        torch.full((1,), float(case["hi"]), device=DEV, dtype=torch.float64)
    return at.round().to(torch.int32)[torch.randperm(n, generator=g, device=DEV)].contiguous()


def _total(case):
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    return sum(int(round(lo + (hi - lo) * i / (n - 1))) for i in range(n)) if n > 1 else hi


def _table(g, batch, blocks, extra=0):
    """A shuffled pool: the pages of `batch` sequences of `blocks` each, and `extra` more of each."""
    order = torch.randperm(batch * (blocks + extra), generator=g, device=DEV).to(torch.int32).view(batch, blocks + extra)
    return order[:, :blocks].contiguous(), order[:, blocks:].contiguous()


def _pool(g, pages, hkv, d, dtype):
    return torch.randn(pages, hkv, PAGE, d, generator=g, device=DEV, dtype=dtype)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16)
        s["w"] = (torch.randn(n, k, generator=g, device=DEV) / math.sqrt(k)).to(torch.bfloat16)
        s["bias"] = (0.3 * torch.randn(n, generator=g, device=DEV)).to(torch.bfloat16) if case["bias"] else None
        s["res"] = torch.randn(m, n, generator=g, device=DEV).to(torch.bfloat16) if case["res"] else None
        s["y"] = torch.empty(m, n, device=DEV, dtype=torch.bfloat16)
        return s
    t, d, hkv, batch = TYPES[case["dtype"]], case["d"], case["hkv"], case["batch"]
    s["lens"] = _lengths(g, case)
    s["scale"] = 1.0 / math.sqrt(d)
    blocks = (case["hi"] + case.get("chunk", 0) + PAGE - 1) // PAGE
    if case["op"] == "evict":
        new_blocks = (case["budget"] + PAGE - 1) // PAGE
        s["table"], s["new_table"] = _table(g, batch, blocks, new_blocks)
        pages = batch * (blocks + new_blocks)
        # attention weight piles up on a few tokens; tokens that got none tie
        w = torch.rand(batch, hkv, blocks * PAGE, generator=g, device=DEV)
        s["sums"] = torch.where(w < 0.2, torch.zeros_like(w), (w * w * 64).round() / 16 * w.lt(0.5) + w.pow(8) * 50)
        s["new_sums"] = torch.zeros(batch, hkv, new_blocks * PAGE, device=DEV)
        s["new_lens"] = torch.zeros(batch, dtype=torch.int32, device=DEV)
        s["kept"] = torch.zeros(batch, hkv, case["budget"], dtype=torch.int32, device=DEV)
        s["k"], s["v"] = _pool(g, pages, hkv, d, t), _pool(g, pages, hkv, d, t)
        return s
    s["table"], _ = _table(g, batch, blocks)
    hq = case["hq"]
    s["k"], s["v"] = _pool(g, batch * blocks, hkv, d, t), _pool(g, batch * blocks, hkv, d, t)
    if case["op"] == "append":
        c, rot, axes = case["chunk"], case["rot"], case["axes"]
        x = torch.randn(batch, c, hq + 2 * hkv, d, generator=g, device=DEV).to(t)
        parts = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
        s["x"] = parts if case["packed"] else tuple(p.contiguous() for p in parts)
        s["q_norm"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(t) if case["norm"] else None
        s["k_norm"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(t) if case["norm"] else None
        s["inv_freq"] = (1e6 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot)).float()
        s["pair_axis"] = (torch.arange(rot // 2, device=DEV) * axes // (rot // 2)).to(torch.int32) if axes > 1 else None
        if axes > 1:  # video: frames, rows and columns of patches after a text prefix
            i = torch.arange(c, device=DEV)
            grid = torch.stack([i // 256, i // 16 % 16, i % 16])[:axes]
            s["pos"] = (grid[:, None, :] + 7 * s["lens"][None, :, None]).to(torch.int32).contiguous()
        else:  # text: ahead of the cache by what was evicted
            ahead = torch.randint(0, 200000, (batch, 1), generator=g, device=DEV)
            s["pos"] = (s["lens"][:, None] + ahead + torch.arange(c, device=DEV))[None].to(torch.int32).contiguous()
        s["chunk_lens"] = torch.randint(0, c + 1, (batch,), generator=g, device=DEV).to(torch.int32) if case["ragged"] else None
        s["q_out"] = torch.zeros(batch, c, hq, d, device=DEV, dtype=t)
        return s
    s["sums"] = torch.rand(batch, hkv, blocks * PAGE, generator=g, device=DEV)
    s["new_sums"] = torch.zeros_like(s["sums"])
    s["decay"] = 0.98
    if case["op"] == "decode":
        s["q"] = (2 * torch.randn(batch, hq, d, generator=g, device=DEV)).to(t)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(batch, hq, device=DEV)
        return s
    s["q"] = (2 * torch.randn(batch, case["chunk"], hq, d, generator=g, device=DEV)).to(t)
    # the log-sum-exps that the chunk's prefill returned
    logits, mask = _chunk_logits(s, case["chunk"])
    lse = logits.masked_fill_(~mask, -math.inf).logsumexp(-1)
    s["lse"] = torch.zeros(batch, hq, case["chunk"], device=DEV)
    s["lse"][:] = lse.view(batch, hq, -1)
    return s


# ------------------------------------------------------------------------------------ plain forms

def _rows(pool, table):
    """[B, Hkv, T, D] in fp32: the tokens of every table row, in order."""
    x = pool[table.long()].float()
    b, n, h, p, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, n * p, d)


def _chunk_logits(s, n):
    """The scaled logits of the chunk's last n queries, and which (query, key) pairs count."""
    q, k = s["q"][:, s["q"].shape[1] - n:].float(), _rows(s["k"], s["table"])
    b, _, hq, d = q.shape
    hkv, total = k.shape[1], k.shape[2]
    q = q.permute(0, 2, 1, 3).reshape(b, hkv, (hq // hkv) * n, d)
    logits = (q @ k.transpose(-1, -2)).view(b, hkv, hq // hkv, n, total) * s["scale"]
    last = s["lens"].long()[:, None] + torch.arange(s["q"].shape[1] - n, s["q"].shape[1], device=DEV)
    mask = torch.arange(total, device=DEV) <= last[:, :, None]
    return logits, mask[:, None, None]


def _angles(s):
    """cos and sin [B, C, rot / 2]: the angles in fp64 (positions run far), rounded after."""
    pairs = s["inv_freq"].numel()
    axis = s["pair_axis"].long() if s["pair_axis"] is not None else torch.zeros(pairs, dtype=torch.long, device=DEV)
    a = s["pos"].double()[axis].permute(1, 2, 0) * s["inv_freq"].double()
    return a.cos().float()[:, :, None], a.sin().float()[:, :, None]


def _turn(x, w, cos, sin, inter):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    n = cos.shape[-1]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if inter else (x[..., :n], x[..., n:2 * n])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _plain_append(s):
    case = s["case"]
    q, k, v = s["x"]
    cos, sin = _angles(s)
    b, c = q.shape[:2]
    i = torch.arange(c, device=DEV)
    live = (i < s["chunk_lens"][:, None]) if s["chunk_lens"] is not None else torch.ones(b, c, dtype=torch.bool, device=DEV)
    qn = _turn(q, s["q_norm"], cos, sin, case["inter"]).to(q.dtype)
    s["q_out"].copy_(torch.where(live[:, :, None, None], qn, s["q_out"]))
    at = (s["lens"].long()[:, None] + i)
    page = s["table"].long().gather(1, at // PAGE)[live]
    slot = (at % PAGE)[live]
    s["k"][page, :, slot] = _turn(k, s["k_norm"], cos, sin, case["inter"]).to(k.dtype)[live]
    s["v"][page, :, slot] = v[live]
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _accumulate(s, w, n):
    t = torch.arange(w.shape[-1], device=DEV) < n[:, None, None]
    s["new_sums"].copy_(torch.where(t, s["decay"] * s["sums"] + w, s["new_sums"]))
    return s["new_sums"]


def _plain_decode(s):
    q, k, v = s["q"].float(), _rows(s["k"], s["table"]), _rows(s["v"], s["table"])
    b, hq, d = q.shape
    hkv = k.shape[1]
    logits = (q.view(b, hkv, hq // hkv, d) @ k.transpose(-1, -2)) * s["scale"]
    live = torch.arange(k.shape[2], device=DEV) < s["lens"][:, None]
    logits = logits.masked_fill(~live[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = (logits - top).exp()
    total = p.sum(-1, keepdim=True)
    p = p / total
    out = (p @ v).view(b, hq, d).to(s["q"].dtype)
    lse = (top + total.log()).view(b, hq)
    return {"out": out, "lse": lse, "sums": _accumulate(s, p.sum(2), s["lens"])}


def _plain_chunk(s):
    case = s["case"]
    n = case["window"] or case["chunk"]
    logits, mask = _chunk_logits(s, n)
    lse = s["lse"][:, :, case["chunk"] - n:].reshape(logits.shape[:-1])
    p = (logits - lse[..., None]).exp() * mask
    return _accumulate(s, p.sum((2, 3)), s["lens"] + case["chunk"])


def _plain_evict(s):
    case = s["case"]
    budget, sums, lens = case["budget"], s["sums"], s["lens"].long()[:, None, None]
    t = torch.arange(sums.shape[-1], device=DEV)
    forced = (t < case["sink"]) | (t >= lens - case["recent"])
    rank = torch.where(t >= lens, -math.inf, torch.where(forced, math.inf, sums))
    take = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    none = sums.shape[-1]
    take = torch.where(take < lens, take, none).sort(-1).values
    short = budget - take.shape[-1]
    if short > 0:
        take = torch.cat([take, take.new_full(take.shape[:-1] + (short,), none)], -1)
    live = take < none
    s["kept"].copy_(torch.where(live, take, -1))
    s["new_lens"].copy_(lens[:, 0, 0].clamp(max=budget))
    src = take.clamp(max=none - 1)
    s["new_sums"].zero_()
    s["new_sums"][..., :budget] = torch.where(live, sums.gather(-1, src), 0.0)
    b, h, _ = src.shape
    page = s["table"].long().gather(1, (src // PAGE).view(b, -1)).view(src.shape)[live]
    heads = torch.arange(h, device=DEV)[None, :, None].expand(src.shape)[live]
    j = torch.arange(budget, device=DEV).expand(src.shape)
    to = s["new_table"].long()[:, None, :].expand(b, h, -1).gather(2, j // PAGE)[live]
    j, src = (j % PAGE)[live], (src % PAGE)[live]
    s["k"][to, heads, j] = s["k"][page, heads, src]
    s["v"][to, heads, j] = s["v"][page, heads, src]
    return {"kept": s["kept"], "lens": s["new_lens"], "sums": s["new_sums"], "k": s["k"], "v": s["v"]}


def _act(y, act):
    if act == "relu":
        return y.clamp(min=0)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if act == "silu":
        return y / (1 + torch.exp(-y))
    return y


def _plain_linear(s):
    y = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(y, s["case"]["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------------------------ the calls

def _own(s):
    from paged_kv_attention_28_gb300 import binding as B
    case = s["case"]
    op = case["op"]
    if op == "append":
        q, k, v = s["x"]
        B.qk_norm_rope_append(q, k, v, s["k"], s["v"], s["table"], s["lens"], chunk_lens=s["chunk_lens"],
                              positions=s["pos"], inv_freq=s["inv_freq"], pair_axis=s["pair_axis"], q_norm=s["q_norm"],
                              k_norm=s["k_norm"], eps=1e-6, interleaved=case["inter"], out=s["q_out"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if op == "decode":
        if "ws" not in s:
            b, hq, d = s["q"].shape
            nb = B.decode_weights_workspace_size(b, s["table"].shape[1], hq, case["hkv"], d, PAGE,
                                                 dtype=B.PKV_F32 if case["dtype"] == "f32" else B.PKV_BF16)
            s["ws"] = B.alloc_workspace(nb, DEV)
        out, lse, sums = B.decode_paged_weights(s["q"], s["k"], s["v"], s["table"], s["lens"], s["sums"], s["scale"],
                                                sums_out=s["new_sums"], decay=s["decay"], out=s["out"], lse=s["lse"],
                                                workspace=s["ws"])
        return {"out": out, "lse": lse, "sums": sums}
    if op == "chunk":
        return B.chunk_weights(s["q"], s["k"], s["table"], s["lens"], s["lse"], s["sums"], s["scale"],
                               sums_out=s["new_sums"], decay=s["decay"], window=case["window"])
    if op == "evict":
        B.cache_evict(s["k"], s["v"], s["table"], s["lens"], s["sums"], s["new_table"], case["budget"],
                      n_sink=case["sink"], n_recent=case["recent"], kept=s["kept"], new_lens=s["new_lens"],
                      new_sums=s["new_sums"])
        return {"kept": s["kept"], "lens": s["new_lens"], "sums": s["new_sums"], "k": s["k"], "v": s["v"]}
    return B.linear(s["x"], s["w"], bias=s["bias"], activation=case["act"], residual=s["res"], out=s["y"])


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "decode": _plain_decode, "chunk": _plain_chunk, "evict": _plain_evict,
            "linear": _plain_linear}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------ fp64

def _tokens(pool, row, n, h):
    """Tokens 0 .. n-1 of one sequence and KV head, fp64."""
    at = torch.arange(n, device=DEV)
    return pool[row.long()[at // PAGE], h, at % PAGE].double()


def _exact_append(s, case):
    rot, d = case["rot"], case["d"]
    k_pool, v_pool = s["k"].double(), s["v"].double()
    q_out = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=DEV)
    q, k, v = (x.double() for x in s["x"])
    turned = []
    for x, w in ((q, s["q_norm"]), (k, s["k_norm"])):
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * w.double()
        y = x.clone()
        for i in range(rot // 2):
            axis = int(s["pair_axis"][i]) if s["pair_axis"] is not None else 0
            ang = (s["pos"][axis].double() * s["inv_freq"][i].double())[:, :, None]
            lo, hi = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)
            y[..., lo] = x[..., lo] * torch.cos(ang) - x[..., hi] * torch.sin(ang)
            y[..., hi] = x[..., lo] * torch.sin(ang) + x[..., hi] * torch.cos(ang)
        turned.append(y)
    for b in range(case["batch"]):
        n = int(s["chunk_lens"][b]) if s["chunk_lens"] is not None else case["chunk"]
        at = int(s["lens"][b]) + torch.arange(n, device=DEV)
        page = s["table"][b].long()[at // PAGE]
        q_out[b, :n] = turned[0][b, :n]
        k_pool[page, :, at % PAGE] = turned[1][b, :n]
        v_pool[page, :, at % PAGE] = v[b, :n]
    return {"q": q_out, "k": k_pool, "v": v_pool}


def _exact_decode(s, case):
    b, hq, d = s["q"].shape
    g = hq // case["hkv"]
    out = torch.zeros(b, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device=DEV)
    sums = torch.zeros(s["sums"].shape, dtype=torch.float64, device=DEV)
    for i in range(b):
        n = int(s["lens"][i])
        for h in range(case["hkv"]):
            z = _tokens(s["k"], s["table"][i], n, h) @ s["q"][i, h * g:(h + 1) * g].double().t() / math.sqrt(d)
            lse[i, h * g:(h + 1) * g] = torch.logsumexp(z, 0)
            p = torch.softmax(z, 0)
            out[i, h * g:(h + 1) * g] = p.t() @ _tokens(s["v"], s["table"][i], n, h)
            sums[i, h, :n] = s["decay"] * s["sums"][i, h, :n].double() + p.sum(1)
    return {"out": out, "lse": lse, "sums": sums}


def _exact_chunk(s, case):
    g, c, d = case["hq"] // case["hkv"], case["chunk"], case["d"]
    first = c - (case["window"] or c)
    sums = torch.zeros(s["sums"].shape, dtype=torch.float64, device=DEV)
    for i in range(case["batch"]):
        n = int(s["lens"][i]) + c
        at = torch.arange(n, device=DEV)
        after = at[:, None] > int(s["lens"][i]) + torch.arange(first, c, device=DEV)
        for h in range(case["hkv"]):
            keys = _tokens(s["k"], s["table"][i], n, h)
            total = s["decay"] * s["sums"][i, h, :n].double()
            for j in range(h * g, (h + 1) * g):
                z = keys @ s["q"][i, first:, j].double().t() / math.sqrt(d) - s["lse"][i, j, first:].double()
                total = total + z.masked_fill(after, -math.inf).exp().sum(1)
            sums[i, h, :n] = total
    return sums


def _exact_evict(s, case):
    kept, new_sums = torch.full_like(s["kept"], -1), torch.zeros_like(s["new_sums"]).double()
    lens = []
    for i in range(case["batch"]):
        n = int(s["lens"][i])
        lens.append(min(n, case["budget"]))
        for h in range(case["hkv"]):
            if n <= case["budget"]:
                take = list(range(n))
            else:
                w = s["sums"][i, h, :n].tolist()
                hold = set(range(min(n, case["sink"]))) | set(range(n - case["recent"], n))
                rest = sorted((t for t in range(n) if t not in hold), key=lambda t: (-w[t], t))
                take = sorted(hold | set(rest[:case["budget"] - len(hold)]))
            at = torch.tensor(take, device=DEV, dtype=torch.long)
            kept[i, h, :len(take)] = at.to(torch.int32)
            new_sums[i, h, :len(take)] = s["sums"][i, h, at].double()
    return {"kept": kept, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "sums": new_sums, "k": None, "v": None}


def _exact_linear(s, case):
    y = torch.nn.functional.linear(s["x"].double(), s["w"].double(), None if s["bias"] is None else s["bias"].double())
    f = torch.nn.functional
    y = {"none": lambda z: z, "relu": f.relu, "gelu": f.gelu, "gelu_tanh": lambda z: f.gelu(z, approximate="tanh"),
         "silu": f.silu}[case["act"]](y)
    return y if s["res"] is None else y + s["res"].double()


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "chunk": _exact_chunk, "evict": _exact_evict,
            "linear": _exact_linear}[case["op"]](s, case)


# ------------------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * (m * k + n * k + m * n * (2 if case["res"] else 1) + (n if case["bias"] else 0)),
                "flops": 2 * m * n * k}
    size = 4 if case["dtype"] == "f32" else 2
    d, hkv, batch = case["d"], case["hkv"], case["batch"]
    total = _total(case)
    if op == "append":
        tokens = batch * case["chunk"] * (0.5 if case["ragged"] else 1)
        return {"bytes": tokens * (2 * size * (case["hq"] + 2 * hkv) * d + 4 * case["axes"]) + 4 * tokens,
                "flops": tokens * (case["hq"] + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if op == "decode":
        return {"bytes": total * hkv * (2 * d * size + 8) + 4 * total // PAGE + 2 * batch * case["hq"] * d * size,
                "flops": 4 * total * case["hq"] * d}
    if op == "chunk":
        n = case["window"] or case["chunk"]
        c = case["chunk"]
        pairs = n * total + batch * (n * c - n * (n - 1) // 2)
        return {"bytes": (total + batch * c) * hkv * (d * size + 8) + batch * n * case["hq"] * (d * size + 4),
                "flops": 2 * pairs * case["hq"] * d}
    kept = sum(min(case["budget"], x) for x in ([case["hi"]] if batch == 1 else
               [int(round(case["lo"] + (case["hi"] - case["lo"]) * i / (batch - 1))) for i in range(batch)]))
    return {"bytes": total * hkv * 4 + kept * hkv * (4 * d * size + 8), "flops": 0}
