"""Measured cases of the operators on both sides of the paged cache's attention: appending new keys
and values with the rotation of their positions (bf16, FP8 and block-scaled int8 caches), attention
over an int8 cache with one scale per page and head, and the adjustment of logits before sampling
(penalties for repeated tokens, biases, grammar masks).

Every operator has a plain form in elementary torch operations (``own`` false) and the
framework's call (``own`` true) on the same state. ``exact`` evaluates the definitions again
in 64 bits.
"""
import math

import numpy as np
import torch

own = False

# (query heads, KV heads, head dim): the framework's 8B, 14B and 70B shapes, its small test
# shapes of head dim 64 and of one KV head
HEADS = {"8b": (32, 8, 128), "14b": (40, 8, 128), "70b": (64, 8, 128), "tiny": (4, 2, 64), "one_kv": (5, 1, 128)}
THETA = 500000.0
PAGE = 16


def listed():
    return [
        # one layer's new keys, values and queries of a few short conversations: launch latency
        dict(name="append_tokens_small", op="append", heads="tiny", kind="bf16", seqs=4, ctx_lo=1, ctx_hi=64, new_lo=1,
             new_hi=1, caches=1, q=True, offset=0),
        # the same of a decode step of 24 requests into a block-scaled cache, whose last pages' scales grow
        dict(name="append_tokens_14b_int8", op="append", heads="14b", kind="int8", seqs=24, ctx_lo=0, ctx_hi=60,
             new_lo=1, new_hi=1, caches=1, q=True, offset=0),
        # one layer's rows of a serving step's prompt chunks, after an eviction that moved their positions
        dict(name="append_chunks_8b", op="append", heads="8b", kind="bf16", seqs=4, ctx_lo=0, ctx_hi=6048, new_lo=1900,
             new_hi=2016, caches=1, q=True, offset=40000),
        # keys and values of the skipped layers' caches from one wide projection, for the 16 prompts
        # of the prefill benchmark (16 x 500..1000 tokens)
        dict(name="append_wide_8b", op="append", heads="8b", kind="bf16", seqs=16, ctx_lo=0, ctx_hi=0, new_lo=500,
             new_hi=1000, caches=8, q=False, offset=0),
        # one layer's keys and values of the same prompts into an int8 cache, read back as bf16 values
        dict(name="append_prompts_int8", op="append", heads="8b", kind="int8", seqs=16, ctx_lo=0, ctx_hi=40, new_lo=500,
             new_hi=1000, caches=1, q=False, offset=0),
        # a decode step's attention: 24 requests of about 1100 cached tokens
        dict(name="attend_tokens_14b_int8", op="attend", heads="14b", seqs=24, ctx_lo=1000, ctx_hi=1250, new_lo=1,
             new_hi=1, window=0, sinks=0),
        # a decode step over long contexts
        dict(name="attend_tokens_long_int8", op="attend", heads="8b", seqs=16, ctx_lo=12000, ctx_hi=16384, new_lo=1,
             new_hi=1, window=0, sinks=0),
        # prompt chunks of a serving step after cached prefixes of up to three chunks
        dict(name="attend_chunks_8b_int8", op="attend", heads="8b", seqs=4, ctx_lo=0, ctx_hi=6048, new_lo=1900,
             new_hi=2016, window=0, sinks=0),
        # logits of one request with a history of a few hundred tokens
        dict(name="adjust_one", op="adjust", rows=1, vocab=128256, hist_lo=600, hist_hi=600, penalties=True, bias=0,
             mask=False, mixed=False),
        # a decode batch in which requests have penalties, biases and grammars of their own
        dict(name="adjust_mixed_14b", op="adjust", rows=24, vocab=152064, hist_lo=1000, hist_hi=2250, penalties=True,
             bias=32, mask=True, mixed=True),
        # a large batch of long conversations
        dict(name="adjust_batch", op="adjust", rows=256, vocab=128256, hist_lo=4000, hist_hi=8064, penalties=True,
             bias=0, mask=True, mixed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "adjust"])
    if op == "append":
        heads, kind = rng.choice(sorted(HEADS)), rng.choice(["bf16", "fp8", "int8"])
        _, n_kv, d_h = HEADS[heads]
        q, caches = rng.random() < 0.6, rng.choice([1, 1, 1, 2, 5, 8])
        if rng.random() < 0.5:
            seqs, new = _log(rng, 1, 48), rng.choice([1, 1, 1, rng.randint(2, 9)])
        else:
            seqs, new = rng.randint(1, 8), _log(rng, 10, 2016)
        while caches > 1 and seqs * new * caches * n_kv * d_h > 12000 * 8 * 8 * 128:
            caches -= 1
        ctx = rng.choice([0, _log(rng, 1, 200)])
        return dict(op=op, heads=heads, kind=kind, seqs=seqs, ctx_lo=ctx // 2, ctx_hi=ctx, new_lo=max(1, new - new // 8),
                    new_hi=new, caches=caches, q=q, offset=rng.choice([0, 0, _log(rng, 1, 1 << 20)]))
    if op == "attend":
        heads = rng.choice(sorted(HEADS))
        n_q, _, d_h = HEADS[heads]
        limit = 4 * 2016 * 5000 * 32 * 128  # no more query-key products than the largest listed chunks
        if rng.random() < 0.5:
            seqs, new = _log(rng, 1, 48), rng.choice([1, 1, 1, rng.randint(2, 9)])
            ctx = _log(rng, 1, 12000)
        else:
            seqs, new = rng.randint(1, 6), _log(rng, 5, 2016)
            ctx = rng.choice([0, _log(rng, 1, 6048)])
        while seqs > 1 and seqs * new * (ctx + new) * n_q * d_h > limit:
            seqs -= 1
        window = rng.choice([0, 0, _log(rng, 16, 4096)])
        return dict(op=op, heads=heads, seqs=seqs, ctx_lo=ctx // 2, ctx_hi=ctx, new_lo=max(1, new - new // 8),
                    new_hi=new, window=window, sinks=rng.choice([0, 1, 4, 17]) if window else 0)
    hist = _log(rng, 1, 8064)
    penalties, bias, mask = rng.random() < 0.8, rng.choice([0, 0, 1, 32, 300]), rng.random() < 0.5
    vocab = rng.choice([1024, 5120, 128256, 152064, _log(rng, 2, 130000)])
    return dict(op="adjust", rows=min(_log(rng, 1, 256), 256 * 128256 // vocab), vocab=vocab,
                hist_lo=hist // 2, hist_hi=hist, penalties=penalties, bias=bias, mask=mask, mixed=rng.random() < 0.5)


# ---------------------------------------------------------------- states

_models = {}


def _model(heads, caches=1):
    """The handle of a model of these heads, as a program holds the handle of its model."""
    from swiftkv_prefill_skipping_gb300 import api
    if (heads, caches) not in _models:
        n_q, n_kv, d_h = HEADS[heads]
        shape = api.Shape(L=caches, d=128, n_q=n_q, n_kv=n_kv, d_h=d_h, ffn=64, vocab=128, rope_theta=THETA)
        _models[heads, caches] = api.Model(shape, l=caches)
    return _models[heads, caches]


def _lengths(lo, hi, seqs):
    """Ragged lengths over [lo, hi], the same for every seed: seeds change values, not shapes."""
    at = (torch.arange(seqs, dtype=torch.float64) * 0.6180339887498949 + 0.37) % 1.0
    return (lo + (at * (hi - lo + 1)).floor().long()).tolist()


def _pages(gen, lens):
    """Block table of sequences of these lengths over a shuffled pool, -1 past each one's pages."""
    need = (torch.tensor(lens) + PAGE - 1) // PAGE
    total = int(need.sum())
    perm = torch.randperm(total + 3, generator=gen)[:total].to(torch.int32)
    table = torch.full((len(lens), max(1, int(need.max()))), -1, dtype=torch.int32)
    table[torch.arange(table.shape[1])[None] < need[:, None]] = perm
    return table, total + 3


def _adjust_state(case, cpu, dev):
    R, V = case["rows"], case["vocab"]
    st = dict(case=case, logits=torch.randn(R, V, device="cuda", generator=dev) * 3.0)
    st["out"] = torch.empty_like(st["logits"])
    lens = torch.tensor(_lengths(case["hist_lo"], case["hist_hi"], R), dtype=torch.int32)
    N = int(lens.max())
    # histories come back to a part of the vocabulary; the first half of each is its prompt
    st["tokens"] = (torch.rand(R, max(1, N), device="cuda", generator=dev) ** 3 * V).to(torch.int32).clamp_(max=V - 1)
    st["lens"], st["prompt_lens"] = lens.cuda(), (lens // 2).cuda()
    f = torch.rand(3, R, generator=cpu)
    one = torch.ones(R)
    rep, pres, freq = 1.2 * one, 0.4 * one, 0.1 * one
    if case["mixed"]:  # each request has its own settings, some of them off
        rep = torch.where(f[0] < 0.3, one, 0.8 + f[0])
        pres = torch.where(f[1] < 0.3, 0 * one, f[1] * 3 - 1.5)
        freq = torch.where(f[2] < 0.3, 0 * one, f[2] - 0.5)
    st["repetition"], st["presence"], st["frequency"] = rep.cuda(), pres.cuda(), freq.cuda()
    if case["bias"]:
        B = case["bias"]
        # ids that differ within a row, with unused entries behind some of them
        first = torch.randint(0, V, (R, 1), device="cuda", generator=dev)
        ids = (first + torch.arange(B, device="cuda") * max(1, V // B)) % V
        unused = (torch.arange(B, device="cuda") >= V) | (torch.rand(R, B, device="cuda", generator=dev) < 0.2)
        st["bias_ids"] = torch.where(unused, -1, ids).to(torch.int32)
        st["bias"] = torch.randn(R, B, device="cuda", generator=dev) * 4.0
    if case["mask"]:
        W = (V + 31) // 32
        # grammars allow a part of the ids; every third row of a mixed batch has none and allows all
        keep = torch.rand(R, W, 32, device="cuda", generator=dev) < 0.3
        if case["mixed"]:
            keep[::3] = True
        bit = torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
        word = (keep.long() * bit).sum(-1)
        st["mask"] = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
    return st


def _codes8(x):
    """int8 codes and scales of blocks x [..., PAGE, d]: one scale for each block."""
    scale = x.abs().amax((-1, -2)) / 127.0
    return torch.round(x / scale[..., None, None]).to(torch.int8), scale


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(int(seed) * 2 + 1)
    dev = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    if case["op"] == "adjust":
        return _adjust_state(case, cpu, dev)
    n_q, n_kv, d_h = HEADS[case["heads"]]
    P, C = case["seqs"], case.get("caches", 1)
    st = dict(case=case, heads=(n_q, n_kv, d_h))
    new = _lengths(case["new_lo"], case["new_hi"], P)
    ctx = _lengths(case["ctx_lo"], case["ctx_hi"], P)[::-1]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    table, pages = _pages(cpu, [a + b for a, b in zip(ctx, new)])
    T = cu[-1]
    st.update(cu=np.array(cu, np.int32), ctx=np.array(ctx, np.int32), table=table.cuda())
    shape = (C, pages, n_kv, PAGE, d_h)
    kind = case.get("kind", "int8")
    if own:
        from swiftkv_prefill_skipping_gb300 import api
        st["model"] = _model(case["heads"], C)
        st["kv"] = api.KVCache(st["model"], pages, table.numpy(), dtype=kind)
    names = ("k", "v") if kind == "bf16" else ("k", "v", "k_scale", "v_scale")
    if case["op"] == "attend":
        st["q"] = torch.randn(T, n_q, d_h, device="cuda", generator=dev).to(torch.bfloat16)
        for name in ("k", "v"):
            st[name], st[name + "_scale"] = _codes8(torch.randn(shape, device="cuda", generator=dev))
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(n_q, T, device="cuda")
    else:
        # one projection's rows: [Q heads |] then for each cache its K and V heads
        Q = n_q if case["q"] else 0
        rows = torch.randn(T, Q + 2 * C * n_kv, d_h, device="cuda", generator=dev).to(torch.bfloat16)
        st["q"] = rows[:, :Q] if Q else None
        kv = rows[:, Q:].view(T, C, 2, n_kv, d_h) if not Q else rows[:, Q:].unflatten(1, (C, 2, n_kv))
        st["new_k"], st["new_v"] = kv[:, :, 0], kv[:, :, 1]
        st["q_out"] = torch.empty(T, n_q, d_h, dtype=torch.bfloat16, device="cuda") if Q else None
        # an eviction took tokens away before: positions are ahead of the cache's rows
        st["offsets"] = np.array([case["offset"] + 7 * s for s in range(P)], np.int32) if case["offset"] else None
        for name in ("k", "v"):  # what earlier calls left in the pages
            if kind == "bf16":
                st[name] = torch.randn(shape, device="cuda", generator=dev).to(torch.bfloat16)
                continue
            old = torch.randn(shape, device="cuda", generator=dev)
            if kind == "int8":  # block maxima around those of the new rows: some scales grow
                size = 0.5 + torch.rand(shape[:3], device="cuda", generator=dev)
                st[name], st[name + "_scale"] = _codes8(old * size[..., None, None])
            else:
                st[name + "_scale"] = old.abs().amax(-1) / 448.0
                st[name] = (old / st[name + "_scale"][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            st[name + "_value"] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    if own:
        for name in names:
            getattr(st["kv"], name).copy_(st[name])
            st[name] = getattr(st["kv"], name)
    return st


# ---------------------------------------------------------------- plain forms

def _places(st):
    """Of every new token: its sequence, its row in the cache, and that row's page."""
    cu, ctx = torch.from_numpy(st["cu"]).cuda().long(), torch.from_numpy(st["ctx"]).cuda().long()
    t = torch.arange(int(st["cu"][-1]), device="cuda")
    s = torch.searchsorted(cu, t, right=True) - 1
    row = ctx[s] + t - cu[s]
    return s, row, st["table"].long()[s, row // PAGE]


def _rotated(x, pos):
    """x [T, ..., d_h] turned by its position: pairs (i, i + d_h / 2) by pos * THETA^(-2 i / d_h). Angles in 64 bits."""
    half = x.shape[-1] // 2
    freq = THETA ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = (pos.double()[:, None] * freq).view(pos.shape[0], *(1,) * (x.dim() - 2), half)
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * c - b * s, b * c + a * s], -1).to(torch.bfloat16)


def _append_blocks(st, name, x, s, row, page):
    """New rows x [T, caches, heads, d_h] into int8 pages of one scale each."""
    codes, scale = st[name], st[name + "_scale"]
    hit = torch.zeros(codes.shape[1], dtype=torch.bool, device="cuda")
    hit[page] = True
    pages = torch.nonzero(hit)[:, 0]
    at = torch.zeros(codes.shape[1], dtype=torch.long, device="cuda")
    at[pages] = torch.arange(len(pages), device="cuda")
    first = torch.full((len(pages),), PAGE, device="cuda").scatter_reduce_(0, at[page], row % PAGE, "amin")
    fresh = torch.zeros(codes.shape[0], len(pages), *codes.shape[2:], device="cuda")
    is_new = torch.zeros(len(pages), PAGE, dtype=torch.bool, device="cuda")
    fresh[:, at[page], :, row % PAGE] = x.float()
    is_new[at[page], row % PAGE] = True
    mine = fresh.abs().amax((-1, -2)) / 127.0
    old = torch.where((first > 0)[:, None], scale[:, pages], 0.0)
    both = torch.maximum(mine, old)
    ratio = torch.where(both > 0, old / both, 1.0)
    was = torch.round(codes[:, pages].float() * ratio[..., None, None])
    now = torch.round(fresh / torch.where(both > 0, both, 1.0)[..., None, None])
    slot = torch.arange(PAGE, device="cuda")
    before = (slot[None] < first[:, None])[:, None, :, None]
    value = torch.where(is_new[:, None, :, None], now, torch.where(before, was, codes[:, pages].float()))
    codes[:, pages] = value.to(torch.int8)
    scale[:, pages] = both


def _append_plain(st):
    s, row, page = _places(st)
    pos = row if st["offsets"] is None else row + torch.from_numpy(st["offsets"]).cuda().long()[s]
    k, v = _rotated(st["new_k"], pos), st["new_v"]
    if st["q"] is not None:
        st["q_out"].copy_(_rotated(st["q"], pos))
    kind = st["case"]["kind"]
    for name, x in (("k", k), ("v", v)):
        if kind == "int8":
            _append_blocks(st, name, x, s, row, page)
        elif kind == "bf16":
            st[name][:, page, :, row % PAGE] = x
        else:
            x = x.float()
            scale = x.abs().amax(-1) / 448.0
            code = (x / torch.where(scale > 0, scale, 1.0)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            st[name][:, page, :, row % PAGE] = code
            st[name + "_scale"][:, page, :, row % PAGE] = scale


def _appended(st):
    """The cache after an append, codes as the values they stand for."""
    kind = st["case"]["kind"]
    if kind == "bf16":
        return {"q": st["q_out"], "k": st["k"], "v": st["v"]}
    out = {"q": st["q_out"]}
    for name in ("k", "v"):
        if kind == "int8":
            out[name] = torch.mul(st[name], st[name + "_scale"][..., None, None], out=st[name + "_value"])
        else:
            code = st[name].view(torch.float8_e4m3fn).float()
            out[name] = torch.mul(code, st[name + "_scale"][..., None], out=st[name + "_value"])
    return out


def _padded(st):
    """Where each new token stands in a [seqs, longest] grid, the visible keys of each, and the
    pool rows of the cached keys: (row of the grid's token, real, page, slot, visible)."""
    c = st["case"]
    cu, ctx = torch.from_numpy(st["cu"]).cuda().long(), torch.from_numpy(st["ctx"]).cuda().long()
    new = cu[1:] - cu[:-1]
    N, K = int((st["cu"][1:] - st["cu"][:-1]).max()), int((st["ctx"] + st["cu"][1:] - st["cu"][:-1]).max())
    i, j = torch.arange(N, device="cuda"), torch.arange(K, device="cuda")
    real = i[None] < new[:, None]
    row = torch.where(real, cu[:-1, None] + i[None], 0)
    pos = ctx[:, None] + i[None]
    seen = (j[None, None] <= pos[..., None]) & real[..., None]
    if c["window"]:
        seen &= (j[None, None] > pos[..., None] - c["window"]) | (j < c["sinks"])[None, None]
    page = st["table"].long()[:, j // PAGE].clamp(min=0)
    return row, real, page, j % PAGE, seen


def _keys(st, name, page, slot):
    """Cached vectors in float32: [seqs, KV heads, keys, head dim]."""
    x = st[name][0][page, :, slot[None]].transpose(1, 2).float()
    return x * st[name + "_scale"][0][page].transpose(1, 2)[..., None]


def _attend_plain(st):
    n_q, n_kv, d_h = st["heads"]
    row, real, page, slot, seen = _padded(st)
    P, N = row.shape
    q = st["q"][row].float().view(P, N, n_kv, n_q // n_kv, d_h).permute(0, 2, 3, 1, 4).reshape(P, n_kv, -1, d_h)
    s = torch.matmul(q, _keys(st, "k", page, slot).transpose(2, 3)).view(P, n_kv, n_q // n_kv, N, -1)
    s = (s * (1.0 / math.sqrt(d_h))).masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s.sub_(m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(P, n_kv, -1, p.shape[-1]), _keys(st, "v", page, slot)).view(P, n_kv, -1, N, d_h) / total
    out = torch.empty_like(st["q"])
    lse = torch.empty(n_q, st["q"].shape[0], device="cuda")
    out[row[real]] = o.permute(0, 3, 1, 2, 4).reshape(P, N, n_q, d_h)[real].to(torch.bfloat16)
    lse[:, row[real]] = (m + torch.log(total)).reshape(P, n_q, N).permute(1, 0, 2)[:, real]
    return {"out": out, "lse": lse}


def _adjust_plain(st):
    c, x = st["case"], st["logits"].clone()
    R, V = x.shape
    if c["penalties"]:
        at = torch.arange(st["tokens"].shape[1], device="cuda")[None]
        written = at < st["lens"][:, None]
        ids = st["tokens"].long()
        seen = torch.zeros(R, V, dtype=torch.int32, device="cuda").scatter_add_(1, ids, written.to(torch.int32))
        count = torch.zeros(R, V, device="cuda").scatter_add_(1, ids, (written & (at >= st["prompt_lens"][:, None])).float())
        rep = st["repetition"][:, None]
        x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
        x = x - st["frequency"][:, None] * count - st["presence"][:, None] * (count > 0)
    if c["bias"]:
        used = st["bias_ids"] >= 0
        x.scatter_add_(1, st["bias_ids"].long().clamp(min=0), torch.where(used, st["bias"], 0.0))
    if c["mask"]:
        i = torch.arange(V, device="cuda")
        x = x.masked_fill(((st["mask"][:, i // 32] >> (i % 32).int()) & 1) == 0, -math.inf)
    return x


# ---------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    if own:
        from swiftkv_prefill_skipping_gb300 import api
        if c["op"] == "append":
            api.append(st["model"], st["new_k"], st["new_v"], st["cu"], st["ctx"], st["kv"], q=st["q"], q_out=st["q_out"],
                       pos_offsets=st["offsets"])
            return _appended(st)
        if c["op"] == "attend":
            api.attend(st["model"], st["q"], st["cu"], st["ctx"], st["kv"], window=c["window"], sinks=c["sinks"],
                       out=st["out"], lse=st["lse"])
            return {"out": st["out"], "lse": st["lse"]}
        more = {}
        if c["penalties"]:
            more.update(tokens=st["tokens"], lens=st["lens"], prompt_lens=st["prompt_lens"], repetition=st["repetition"],
                        presence=st["presence"], frequency=st["frequency"])
        if c["bias"]:
            more.update(bias_ids=st["bias_ids"], bias=st["bias"])
        if c["mask"]:
            more.update(mask=st["mask"])
        return api.adjust_logits(st["logits"], out=st["out"], **more)
    if c["op"] == "append":
        _append_plain(st)
        return _appended(st)
    if c["op"] == "attend":
        return _attend_plain(st)
    return _adjust_plain(st)


# ---------------------------------------------------------------- what a pass cannot do without

def _visible(n, ctx, window, sinks):
    """(query-key pairs, keys some row sees) of a chunk of n tokens after ctx cached ones."""
    pos = np.arange(ctx, ctx + n, dtype=np.int64)
    if not window:
        return int((pos + 1).sum()), ctx + n
    near = np.minimum(pos + 1, window)
    far = np.minimum(np.maximum(pos + 1 - window, 0), sinks)
    first = max(0, ctx - window + 1)
    return int((near + far).sum()), ctx + n - first + min(first, sinks)


def work(case):
    if case["op"] == "adjust":
        R, V = case["rows"], case["vocab"]
        hist = (case["hist_lo"] + case["hist_hi"]) / 2 if case["penalties"] else 0
        return {"bytes": R * (V * 8 + hist * 4 + case["bias"] * 8 + (V / 8 if case["mask"] else 0)), "flops": 4 * R * V}
    n_q, n_kv, d_h = HEADS[case["heads"]]
    P = case["seqs"]
    if case["op"] == "append":
        T = sum(_lengths(case["new_lo"], case["new_hi"], P))
        vec = n_kv * {"bf16": 2 * d_h, "fp8": d_h + 4, "int8": d_h + 0.25}[case["kind"]]
        q = 4 * n_q * d_h if case["q"] else 0
        return {"bytes": T * (case["caches"] * 2 * (2 * n_kv * d_h + vec) + q),
                "flops": T * 6 * d_h * (case["caches"] * n_kv + (n_q if case["q"] else 0))}
    bytes_, flops = 0, 0.0
    for n, ctx in zip(_lengths(case["new_lo"], case["new_hi"], P), _lengths(case["ctx_lo"], case["ctx_hi"], P)[::-1]):
        pairs, keys = _visible(n, ctx, case["window"], case["sinks"])
        bytes_ += keys * 2 * n_kv * (d_h + 0.25) + n * n_q * (4 * d_h + 4)
        flops += 4.0 * pairs * n_q * d_h
    return {"bytes": bytes_, "flops": flops}


# ---------------------------------------------------------------- the definitions in 64 bits

def _turned(x, pos):
    """The rotation as a product of complex numbers."""
    d = x.shape[-1]
    w = torch.pow(THETA, -2.0 * torch.arange(d // 2, dtype=torch.float64, device="cuda") / d)
    z = torch.complex(x[..., :d // 2].double(), x[..., d // 2:].double())
    turn = torch.polar(torch.ones_like(w)[None], torch.outer(pos.double(), w))
    z = z * turn.view(len(pos), *(1,) * (x.dim() - 2), d // 2)
    return torch.cat([z.real, z.imag], -1)


def _exact_append(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    out = {"q": None}
    cache = {}
    for name in ("k", "v"):
        if kind == "bf16":
            cache[name] = st[name].double()
        elif kind == "int8":
            cache[name] = (st[name].double(), st[name + "_scale"].double())
        else:
            cache[name] = st[name].view(torch.float8_e4m3fn).double() * st[name + "_scale"].double()[..., None]
    if st["q"] is not None:
        out["q"] = torch.empty(st["q_out"].shape, dtype=torch.float64, device="cuda")
    for s in range(case["seqs"]):
        r0, r1, c0 = int(st["cu"][s]), int(st["cu"][s + 1]), int(st["ctx"][s])
        at = torch.arange(c0, c0 + r1 - r0, device="cuda")
        pos = at + (int(st["offsets"][s]) if st["offsets"] is not None else 0)
        if st["q"] is not None:
            out["q"][r0:r1] = _turned(st["q"][r0:r1], pos)
        for name, x in (("k", _turned(st["new_k"][r0:r1], pos)), ("v", st["new_v"][r0:r1].double())):
            pages = st["table"][s].long()[at // PAGE]
            if kind == "bf16":
                cache[name][:, pages, :, at % PAGE] = x
                continue
            x = x.to(torch.bfloat16).double()  # what the cache quantizes are the values a bf16 cache would hold
            if kind == "fp8":
                scale = (x.abs().amax(-1, keepdim=True) / 448).float().double()
                code = (x / scale.clamp(min=1e-300)).float().to(torch.float8_e4m3fn).double()
                cache[name][:, pages, :, at % PAGE] = code * scale
                continue
            codes, scales = cache[name]
            for lo in range(c0 // PAGE * PAGE, c0 + r1 - r0, PAGE):  # page by page, all caches and heads at once
                a, b = max(lo, c0), min(lo + PAGE, c0 + r1 - r0)
                page = int(st["table"][s, lo // PAGE])
                rows = x[a - c0:b - c0].permute(1, 2, 0, 3)  # caches, heads, rows, dims
                top = (rows.abs().amax((2, 3)) / 127).float().double()
                if a > lo:
                    top = torch.maximum(top, scales[:, page])
                    codes[:, page, :, :a - lo] = torch.round(codes[:, page, :, :a - lo] * (scales[:, page] / top)[..., None, None])
                codes[:, page, :, a - lo:b - lo] = torch.round(rows / top[..., None, None])
                scales[:, page] = top
    for name in ("k", "v"):
        out[name] = cache[name][0] * cache[name][1][..., None, None] if kind == "int8" else cache[name]
    return out


def _exact_attend(case, seed):
    if work(case)["flops"] > 3e12:
        return None
    st = prepare(case, seed)
    n_q, n_kv, d_h = st["heads"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(n_q, st["q"].shape[0], dtype=torch.float64, device="cuda")
    for s in range(case["seqs"]):
        r0, r1, c0 = int(st["cu"][s]), int(st["cu"][s + 1]), int(st["ctx"][s])
        keys = torch.arange(c0 + r1 - r0, device="cuda")
        if case["window"]:  # the keys that any of the rows can see
            keys = keys[(keys < case["sinks"]) | (keys > c0 - case["window"])]
        pages = st["table"][s].long()[keys // PAGE]
        K, V = (st[n][0][pages, :, keys % PAGE].double() * st[n + "_scale"][0][pages].double()[..., None] for n in ("k", "v"))
        behind = torch.arange(c0, c0 + r1 - r0, device="cuda")[:, None] - keys[None]
        hidden = behind < 0
        if case["window"]:
            hidden |= (behind >= case["window"]) & (keys >= case["sinks"])[None]
        for h in range(n_q):
            g = h // (n_q // n_kv)
            z = (st["q"][r0:r1, h].double() @ K[:, g].T) * d_h ** -0.5
            z = z.masked_fill(hidden, -math.inf)
            norm = torch.logsumexp(z, 1)
            out[r0:r1, h] = torch.exp(z - norm[:, None]) @ V[:, g]
            lse[h, r0:r1] = norm
    return {"out": out, "lse": lse}


def _exact_adjust(case, seed):
    st = prepare(case, seed)
    out = st["logits"].double().cpu().numpy()
    tokens, lens, prompts = (st[n].cpu().numpy() for n in ("tokens", "lens", "prompt_lens"))
    rep, pres, freq = (st[n].cpu().numpy().astype(np.float64) for n in ("repetition", "presence", "frequency"))
    for r, x in enumerate(out):
        if case["penalties"]:
            history = tokens[r, :lens[r]]
            ids = np.unique(history)
            x[ids] *= np.where(x[ids] > 0, 1.0 / rep[r], rep[r])
            ids, times = np.unique(history[prompts[r]:], return_counts=True)
            x[ids] -= freq[r] * times + pres[r]
        if case["bias"]:
            ids = st["bias_ids"][r].cpu().numpy()
            x[ids[ids >= 0]] += st["bias"][r].cpu().numpy()[ids >= 0]
        if case["mask"]:
            words = st["mask"][r].cpu().numpy().view(np.uint8)
            x[np.unpackbits(words, bitorder="little")[:len(x)] == 0] = -np.inf
    return out


def exact(case, seed):
    return {"append": _exact_append, "attend": _exact_attend, "adjust": _exact_adjust}[case["op"]](case, seed)
