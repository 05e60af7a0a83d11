"""Measured cases of the serving operators over the paged KV cache: attention of new tokens
(prompt chunks and single tokens, with an optional sliding window and sink tokens), the
attention weight each cached key received, eviction of the keys that received least, and
sampling of the next token.

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
PAGE = 16


def listed():
    return [
        # a few short conversations on the small head-dim-64 shape: launch latency
        dict(name="attend_tokens_small", op="attend", heads="tiny", seqs=4, ctx_lo=1, ctx_hi=64, new_lo=1, new_hi=1,
             window=0, sinks=0, fp8=False),
        # a decode step's attention: 24 requests of about 1100 cached tokens
        dict(name="attend_tokens_14b", op="attend", heads="14b", seqs=24, ctx_lo=1000, ctx_hi=1250, new_lo=1, new_hi=1,
             window=0, sinks=0, fp8=False),
        # a decode step over long streams that keep 4 sinks and the last 4096 tokens, FP8 cache
        dict(name="attend_tokens_window_fp8", op="attend", heads="8b", seqs=16, ctx_lo=12000, ctx_hi=16384, new_lo=1,
             new_hi=1, window=4096, sinks=4, fp8=True),
        # prompt chunks of a serving step after cached prefixes of up to three chunks
        dict(name="attend_chunks_8b", op="attend", heads="8b", seqs=4, ctx_lo=0, ctx_hi=6048, new_lo=1900, new_hi=2016,
             window=0, sinks=0, fp8=False),
        # the same chunks through a window of 1024 tokens and 4 sinks
        dict(name="attend_chunks_window", op="attend", heads="8b", seqs=4, ctx_lo=4032, ctx_hi=6048, new_lo=1900,
             new_hi=2016, window=1024, sinks=4, fp8=False),
        # weight that a decode step's tokens gave to each of ~1100 cached keys
        dict(name="weights_tokens_14b", op="weights", heads="14b", seqs=24, ctx_lo=1000, ctx_hi=1250, new_lo=1,
             new_hi=1, window=0, sinks=0, fp8=False),
        # weight that a prompt's chunks gave to their keys
        dict(name="weights_chunks_8b", op="weights", heads="8b", seqs=4, ctx_lo=0, ctx_hi=4032, new_lo=1900,
             new_hi=2016, window=0, sinks=0, fp8=False),
        # a few requests shrunk to 512 keys in two caches
        dict(name="evict_small", op="evict", heads="14b", seqs=4, len_lo=900, len_hi=2100, keep=512, sinks=4,
             recent=64, caches=2),
        # a batch of long prompts shrunk to a quarter in four caches
        dict(name="evict_long", op="evict", heads="8b", seqs=16, len_lo=6000, len_hi=8064, keep=2048, sinks=4,
             recent=256, caches=4),
        # the next token of one request
        dict(name="sample_one", op="sample", rows=1, vocab=128256, temperature=0.8, top_k=50, top_p=0.95, min_p=0.0,
             mixed=False),
        # a decode batch in which every request has settings of its own
        dict(name="sample_mixed_14b", op="sample", rows=24, vocab=152064, temperature=1.0, top_k=0, top_p=0.9,
             min_p=0.05, mixed=True),
        # a large batch with a nucleus only
        dict(name="sample_batch", op="sample", rows=256, vocab=128256, temperature=1.0, top_k=0, top_p=0.95,
             min_p=0.0, mixed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "weights", "evict", "sample"])
    if op in ("attend", "weights"):
        heads = rng.choice(sorted(HEADS))
        n_q, _, d_h = HEADS[heads]
        limit = 4 * 2016 * 5000 * 32 * 128  # no more query-key products than the largest listed chunks
        if rng.random() < 0.5:
            seqs, new = _log(rng, 1, 48), rng.choice([1, 1, 1, rng.randint(2, 9)])
            ctx = _log(rng, 1, 16000)
        else:
            seqs, new = rng.randint(1, 6), _log(rng, 5, 2016)
            ctx = rng.choice([0, _log(rng, 1, 6048)])
        while seqs > 1 and seqs * new * (ctx + new) * n_q * d_h > limit:
            seqs -= 1
        window = rng.choice([0, 0, _log(rng, 16, 4096)])
        return dict(op=op, heads=heads, seqs=seqs, ctx_lo=ctx // 2, ctx_hi=ctx, new_lo=max(1, new - new // 8),
                    new_hi=new, window=window, sinks=rng.choice([0, 1, 4, 17]) if window else 0,
                    fp8=rng.random() < 0.4)
    if op == "evict":
        seqs, longest = rng.randint(1, 16), _log(rng, 40, 8064)
        keep = max(8, int(longest * rng.uniform(0.1, 0.9)))
        sinks = rng.choice([0, 1, 4])
        return dict(op="evict", heads=rng.choice(sorted(HEADS)), seqs=seqs, len_lo=max(1, longest // 3),
                    len_hi=longest, keep=keep, sinks=sinks, recent=rng.randint(0, (keep - sinks) // 2),
                    caches=rng.randint(1, 4))
    return dict(op="sample", rows=_log(rng, 1, 256), vocab=rng.choice([1024, 5120, 128256, 152064, _log(rng, 2, 130000)]),
                temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.3]), top_k=rng.choice([0, 1, 7, 50, 1000]),
                top_p=rng.choice([1.0, 0.99, 0.9, 0.5]), min_p=rng.choice([0.0, 0.02, 0.1]), mixed=rng.random() < 0.5)


# ---------------------------------------------------------------- states

_models = {}


def _model(heads, caches=1):
    """The handle of a model of these heads, as a program holds the handle of its model."""
    from swiftkv_prefill_skipping_gb300 import api
    if (heads, caches) not in _models:
        n_q, n_kv, d_h = HEADS[heads]
        shape = api.Shape(L=caches, d=128, n_q=n_q, n_kv=n_kv, d_h=d_h, ffn=64, vocab=128, rope_theta=10000.0)
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


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(int(seed) * 2 + 1)
    dev = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    st = dict(case=case)
    if case["op"] == "sample":
        R, V = case["rows"], case["vocab"]
        # a broad body of tokens and a few that stand out, as a language model's logits have
        x = torch.randn(R, V, device="cuda", generator=dev) * 2.0
        at = torch.randint(0, V, (R, 24), device="cuda", generator=dev)
        x.scatter_add_(1, at, torch.rand(R, 24, device="cuda", generator=dev) * 12.0)
        st["logits"] = x
        st["u"] = torch.rand(R, device="cuda", generator=dev)
        f = torch.rand(4, R, generator=cpu)
        one = torch.ones(R)
        t, k, p, m = (one * case["temperature"], one * case["top_k"], one * case["top_p"], one * case["min_p"])
        if case["mixed"]:  # each request has its own settings, some of them off
            t = torch.where(f[0] < 0.2, 0 * t, 0.5 + f[0])
            k = torch.where(f[1] < 0.5, 0 * k, (f[1] * 400).floor())
            p = torch.where(f[2] < 0.3, one, f[2])
            m = torch.where(f[3] < 0.5, 0 * m, 0.2 * f[3])
        st["temperature"], st["top_p"], st["min_p"] = t.cuda(), p.cuda(), m.cuda()
        st["top_k"] = k.to(torch.int32).cuda()
        return st
    n_q, n_kv, d_h = HEADS[case["heads"]]
    P = case["seqs"]
    st["heads"] = (n_q, n_kv, d_h)
    if case["op"] == "evict":
        C = case["caches"]
        lens = _lengths(case["len_lo"], case["len_hi"], P)
        # each sequence's pages, then pages of its own that receive the kept keys
        room = [n + PAGE * ((case["keep"] + PAGE - 1) // PAGE + 1) for n in lens]
        table, pages = _pages(cpu, room)
        own_pages = [(n + PAGE - 1) // PAGE for n in lens]
        width = (case["keep"] + PAGE - 1) // PAGE
        dst = torch.stack([table[s, own_pages[s]:own_pages[s] + width] for s in range(P)])
        st.update(lens=lens, table=table.cuda(), dst=dst.contiguous().cuda())
        shape = (C, pages, n_kv, PAGE, d_h)
        if own:
            from swiftkv_prefill_skipping_gb300 import api
            st["model"] = _model(case["heads"], C)
            st["kv"] = api.KVCache(st["model"], pages, table.numpy())
            st["k"], st["v"] = st["kv"].k, st["kv"].v
        else:
            st["k"] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
            st["v"] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        st["k"].normal_(generator=dev)
        st["v"].normal_(generator=dev)
        # accumulated weights are positive with a long tail
        st["scores"] = torch.empty(shape[:-1], device="cuda").normal_(generator=dev).mul_(1.5).exp_()
        return st
    new = _lengths(case["new_lo"], case["new_hi"], P)
    ctx = _lengths(case["ctx_lo"], case["ctx_hi"], P)[::-1]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    table, pages = _pages(cpu, [a + b for a, b in zip(ctx, new)])
    T = cu[-1]
    st.update(cu=np.array(cu, np.int32), ctx=np.array(ctx, np.int32), table=table.cuda())
    shape = (1, pages, n_kv, PAGE, d_h)
    if own:
        from swiftkv_prefill_skipping_gb300 import api
        st["model"] = _model(case["heads"])
        st["kv"] = api.KVCache(st["model"], pages, table.numpy(), dtype="fp8" if case["fp8"] else "bf16")
    # keys share a direction with the queries, so that a row's weights have a head and a tail
    q = torch.randn(T, n_q, d_h, device="cuda", generator=dev)
    k = torch.randn(shape, device="cuda", generator=dev)
    v = torch.randn(shape, device="cuda", generator=dev)
    st["q"] = q.to(torch.bfloat16)
    if case["fp8"]:
        ks, vs = k.abs().amax(-1) / 448.0, v.abs().amax(-1) / 448.0
        kc = (k / ks[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        vc = (v / vs[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        st.update(k=kc, v=vc, k_scale=ks, v_scale=vs)
    else:
        st.update(k=k.to(torch.bfloat16), v=v.to(torch.bfloat16))
    if own:
        for name in ("k", "v") + (("k_scale", "v_scale") if case["fp8"] else ()):
            getattr(st["kv"], name).copy_(st[name])
            st[name] = getattr(st["kv"], name)
    if case["op"] == "weights":
        st["lse"] = _attend_plain(st)["lse"]  # from the attention that came before
        st["scores"] = torch.zeros(pages, n_kv, PAGE, device="cuda")
    else:
        st["out"] = torch.empty(T, n_q, d_h, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(n_q, T, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms

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
    pool = st[name][0]
    x = pool[page, :, slot[None]].transpose(1, 2)
    if st["case"]["fp8"]:
        x = x.contiguous().view(torch.float8_e4m3fn).float()
        return x * st[name + "_scale"][0][page, :, slot[None]].transpose(1, 2)[..., None]
    return x.float()


def _scores(st):
    n_q, n_kv, d_h = st["heads"]
    row, real, page, slot, seen = _padded(st)
    P, N = row.shape
    q = st["q"][row].float().view(P, N, n_kv, n_q // n_kv, d_h).permute(0, 2, 3, 1, 4).reshape(P, n_kv, -1, d_h)
    s = torch.matmul(q, _keys(st, "k", page, slot).transpose(2, 3)).view(P, n_kv, n_q // n_kv, N, -1)
    s = (s * (1.0 / math.sqrt(d_h))).masked_fill_(~seen[:, None, None], -math.inf)
    return s, row, real, page, slot, seen


def _attend_plain(st):
    n_q, n_kv, d_h = st["heads"]
    s, row, real, page, slot, _ = _scores(st)
    P, N = row.shape
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s.sub_(m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(P, n_kv, -1, p.shape[-1]), _keys(st, "v", page, slot)).view(P, n_kv, -1, N, d_h) / total
    out = torch.empty_like(st["q"])
    lse = torch.empty(n_q, st["q"].shape[0], device="cuda")
    out[row[real]] = o.permute(0, 3, 1, 2, 4).reshape(P, N, n_q, d_h)[real].to(torch.bfloat16)
    lse[:, row[real]] = (m + torch.log(total)).reshape(P, n_q, N).permute(1, 0, 2)[:, real]
    return {"out": out, "lse": lse}


def _weights_plain(st):
    n_q, n_kv, _ = st["heads"]
    s, row, real, page, slot, seen = _scores(st)
    P, N = row.shape
    lse = st["lse"][:, row].view(n_kv, n_q // n_kv, P, N).permute(2, 0, 1, 3)
    w = torch.exp(s.sub_(lse[..., None])).sum(dim=(2, 3))
    touched = seen.any(1)
    st["scores"][page[touched], :, slot[None].expand(P, -1)[touched]] = w.transpose(1, 2)[touched]
    return st["scores"]


def _evict_plain(st):
    c = st["case"]
    C, P, keep = c["caches"], c["seqs"], c["keep"]
    n = torch.tensor(st["lens"], device="cuda")
    K = max(keep, max(st["lens"]))
    j = torch.arange(K, device="cuda")
    live = j[None] < n[:, None]
    page = torch.where(live, st["table"].long()[:, (j // PAGE).clamp(max=st["table"].shape[1] - 1)], 0)
    slot = j % PAGE
    sc = st["scores"][:, page, :, slot[None].expand(P, -1)].permute(2, 0, 3, 1).contiguous()  # [C, P, heads, K]
    held = live & ((j < c["sinks"])[None] | (j[None] >= (n - c["recent"])[:, None]))
    sc = sc.masked_fill(held[None, :, None], math.inf).masked_fill(~live[None, :, None], -math.inf)
    best = torch.sort(sc, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.sort(torch.where(torch.gather(live[None, :, None].expand_as(sc), 3, best), best, K), dim=-1).values
    some = kept < K
    ci, si, hi, ki = torch.nonzero(some, as_tuple=True)
    src = kept[some]
    p0, p1 = page[si, src], st["dst"].long()[si, ki // PAGE]
    for_all = (ci, p1, hi, ki % PAGE), (ci, p0, hi, src % PAGE)
    st["k"][for_all[0]] = st["k"][for_all[1]]
    st["v"][for_all[0]] = st["v"][for_all[1]]
    st["scores"][for_all[0]] = st["scores"][for_all[1]]
    return {"kept": torch.where(some, kept, -1).to(torch.int32), "k": st["k"], "v": st["v"], "scores": st["scores"]}


def _sample_plain(st):
    x = st["logits"].double()
    V = x.shape[1]
    t = st["temperature"].double()[:, None]
    m = x.amax(1, keepdim=True)
    w = torch.exp((x - m) / torch.where(t > 0, t, 1.0))
    greedy = (x == m).to(torch.int8).argmax(1)
    order = torch.sort(st["logits"], dim=1, descending=True, stable=True).indices
    k = st["top_k"].long()[:, None]
    k = torch.where((k > 0) & (k < V), k, V)
    ws = torch.gather(w, 1, order)
    ws = torch.where(torch.arange(V, device="cuda")[None] < k, ws, 0.0)
    run = torch.cumsum(ws, 1)
    p = st["top_p"].double()[:, None]
    ok = (torch.arange(V, device="cuda")[None] < k) & (((run - ws) < p * run[:, -1:]) | (p >= 1))
    ok[:, 0] = True
    ok &= ws >= st["min_p"].double()[:, None]
    keep = torch.zeros_like(ok).scatter_(1, order, ok)
    run = torch.cumsum(torch.where(keep, w, 0.0), 1)
    token = (run > st["u"].double()[:, None] * run[:, -1:]).to(torch.int8).argmax(1)
    return torch.where(t[:, 0] > 0, token, greedy).to(torch.int32)


# ---------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    if own:
        from swiftkv_prefill_skipping_gb300 import api
        if c["op"] == "attend":
            api.attend(st["model"], st["q"], st["cu"], st["ctx"], st["kv"], window=c["window"], sinks=c["sinks"],
                       out=st["out"], lse=st["lse"])
            return {"out": st["out"], "lse": st["lse"]}
        if c["op"] == "weights":
            return api.attention_weights(st["model"], st["q"], st["lse"], st["cu"], st["ctx"], st["kv"], st["scores"],
                                         window=c["window"], sinks=c["sinks"], decay=0.0)
        if c["op"] == "evict":
            kept = api.evict(st["model"], st["kv"], st["scores"], st["lens"], c["keep"], sinks=c["sinks"],
                             recent=c["recent"], dst_block_table=st["dst"])
            return {"kept": kept, "k": st["k"], "v": st["v"], "scores": st["scores"]}
        return api.sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                          min_p=st["min_p"])
    if c["op"] == "attend":
        return _attend_plain(st)
    if c["op"] == "weights":
        return _weights_plain(st)
    if c["op"] == "evict":
        return _evict_plain(st)
    return _sample_plain(st)


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
    if case["op"] == "sample":
        R, V = case["rows"], case["vocab"]
        return {"bytes": R * V * 4 + R * 24, "flops": 3 * R * V}
    n_q, n_kv, d_h = HEADS[case["heads"]]
    P = case["seqs"]
    if case["op"] == "evict":
        n = (case["len_lo"] + case["len_hi"]) / 2
        kept = min(n, case["keep"])
        lists = case["caches"] * P * n_kv
        return {"bytes": lists * (n * 4 + kept * (4 + 8 + 2 * 2 * 2 * d_h)), "flops": lists * n}
    n, ctx = (case["new_lo"] + case["new_hi"]) // 2, (case["ctx_lo"] + case["ctx_hi"]) // 2
    pairs, keys = _visible(n, ctx, case["window"], case["sinks"])
    vec = n_kv * (d_h + 4 if case["fp8"] else 2 * d_h)
    if case["op"] == "weights":
        return {"bytes": P * (keys * (vec + n_kv * 4) + n * n_q * (2 * d_h + 4)), "flops": P * 2.0 * pairs * n_q * d_h}
    return {"bytes": P * (keys * 2 * vec + n * n_q * (4 * d_h + 4)), "flops": P * 4.0 * pairs * n_q * d_h}


# ---------------------------------------------------------------- the definitions in 64 bits

def _cached(st, name, s, keys):
    """float64 vectors [keys, KV heads, head dim] of sequence s at these positions."""
    pages, slots = st["table"][s].long()[keys // PAGE], keys % PAGE
    if st["case"]["fp8"]:
        codes = st[name][0][pages, :, slots].view(torch.float8_e4m3fn)
        return codes.double() * st[name + "_scale"][0][pages, :, slots].double()[..., None]
    return st[name][0][pages, :, slots].double()


def exact(case, seed):
    if case["op"] in ("attend", "weights"):
        if work(case)["flops"] > 3e12:
            return None
        st = prepare(case, seed)
        n_q, n_kv, d_h = st["heads"]
        G = n_q // n_kv

        def each_head():
            """For each sequence and head: (sequence, head, its tokens' rows, keys, logits in 64 bits)."""
            for s in range(case["seqs"]):
                r0, r1, c0 = int(st["cu"][s]), int(st["cu"][s + 1]), int(st["ctx"][s])
                n = r1 - r0
                keys = torch.arange(c0 + n, device="cuda")
                if case["window"]:  # the keys that any of the rows can see
                    keys = keys[(keys < case["sinks"]) | (keys > c0 - case["window"])]
                K = _cached(st, "k", s, keys)
                for h in range(n_q):
                    z = (st["q"][r0:r1, h].double() @ K[:, h // (n_q // n_kv)].T) * d_h ** -0.5
                    at = torch.arange(c0, c0 + n, device="cuda")[:, None] - keys[None]  # how far behind the token
                    hidden = at < 0
                    if case["window"]:
                        hidden |= (at >= case["window"]) & (keys >= case["sinks"])[None]
                    yield s, h, slice(r0, r1), keys, z.masked_fill(hidden, -math.inf)

        if case["op"] == "attend":
            out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
            lse = torch.empty(n_q, st["q"].shape[0], dtype=torch.float64, device="cuda")
            held = (-1, None)
            for s, h, rows, keys, z in each_head():
                if held[0] != s:
                    held = (s, _cached(st, "v", s, keys))
                norm = torch.logsumexp(z, 1)
                out[rows, h] = torch.exp(z - norm[:, None]) @ held[1][:, h // G]
                lse[h, rows] = norm
            return {"out": out, "lse": lse}
        total = st["scores"].double()
        for s, h, rows, keys, z in each_head():
            given = torch.exp(z - st["lse"][h, rows].double()[:, None]).sum(0)
            total[st["table"][s].long()[keys // PAGE], h // G, keys % PAGE] += given
        return total
    st = prepare(case, seed)
    if case["op"] == "evict":
        _, n_kv, _ = st["heads"]
        table, scores = st["table"].cpu().numpy(), st["scores"].cpu().numpy().astype(np.float64)
        kept = np.full((case["caches"], case["seqs"], n_kv, case["keep"]), -1, np.int32)
        for s, n in enumerate(st["lens"]):
            j = np.arange(n)
            sure = (j < case["sinks"]) | (j >= n - case["recent"])
            room = min(n, case["keep"]) - int(sure.sum()) if n > case["keep"] else n
            for c in range(case["caches"]):
                for h in range(n_kv):
                    if n <= case["keep"]:
                        kept[c, s, h, :n] = j
                        continue
                    others = j[~sure]
                    value = scores[c, table[s, others // PAGE], h, others % PAGE]
                    chosen = others[np.lexsort((others, -value))[:room]]
                    kept[c, s, h] = np.sort(np.concatenate([j[sure], chosen]))
        return {"kept": kept, "k": None, "v": None, "scores": None}
    rows = []
    x = st["logits"].cpu().numpy().astype(np.float64)
    t, k, p, m, u = (st[a].cpu().numpy().astype(np.float64) for a in ("temperature", "top_k", "top_p", "min_p", "u"))
    for r in range(x.shape[0]):
        if t[r] <= 0:
            rows.append(int(np.argmax(x[r])))
            continue
        w = np.exp((x[r] - x[r].max()) / t[r])
        by = np.lexsort((np.arange(x.shape[1]), -x[r]))
        if 0 < k[r] < x.shape[1]:
            by = by[:int(k[r])]
        if p[r] < 1:
            before = np.concatenate([[0.0], np.cumsum(w[by])])
            by = by[:max(1, int(np.searchsorted(before[:-1], p[r] * before[-1], side="left")))]
        by = np.sort(by[w[by] >= m[r]])
        run_ = np.cumsum(w[by])
        rows.append(int(by[np.searchsorted(run_, u[r] * run_[-1], side="right")]))
    return np.array(rows, np.int32)
