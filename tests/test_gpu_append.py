"""swiftkv_append against the rotation in 64 bits and the caches' quantization rules, value for value.

Tolerances. Rotated values: the float32 cosine and sine are off by 2^-24 of their value each (past the
table by 2^-21 radians more), a product and the sum by 2^-24 of theirs, together below
2^-22 (|a| + |b|), past the table 2^-20; the rounding to bf16 adds 2^-8 of the value. Values that are not rotated,
and everything outside the new rows, have to be equal. FP8 and int8 codes and scales are decisions in float32
over the bf16 values that a bf16 cache holds: they have to be equal to the same decisions made here."""
import ctypes as C

import numpy as np
import pytest

from oracle import model as OM
from swiftkv_prefill_skipping_gb300 import binding as B

HEADS = {"gqa4": (8, 2, 128), "gqa5": (5, 1, 128), "mha": (2, 2, 128), "14b": (40, 8, 128), "d64": (4, 2, 64),
         "d64_mha": (6, 6, 64)}
THETA = 1e4
BATCHES = [([1], [0]), ([1, 1, 1, 1], [15, 16, 17, 2000]), ([16], [0]), ([17, 0, 3], [15, 9, 31]),
           ([0, 130, 1, 0, 20], [3, 7, 14, 0, 5]), ([300, 33], [0, 1])]


def model_of(heads, caches):
    from swiftkv_prefill_skipping_gb300 import api
    n_q, n_kv, d = HEADS[heads]
    return api.Model(api.Shape(L=caches, d=128, n_q=n_q, n_kv=n_kv, d_h=d, ffn=64, vocab=128, rope_theta=THETA), l=caches)


def turned(x, pos):
    """float64 rotation of x [T, heads, d]."""
    import torch
    half = x.shape[-1] // 2
    w = THETA ** (-torch.arange(half, dtype=torch.float64) / half)
    a = torch.outer(torch.as_tensor(pos, dtype=torch.float64), w)[:, None]
    c, s = torch.cos(a), torch.sin(a)
    lo, hi = x[..., :half].double(), x[..., half:].double()
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


class Case:
    """New rows of a ragged batch over pools that hold something everywhere; block-table entries of pages
    that get no new row are outside the pool."""

    def __init__(self, heads, new, ctx, kind="bf16", caches=1, total_caches=None, first=0, seed=0, scale=1.0):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        self.n_q, self.n_kv, self.d = HEADS[heads]
        self.kind, self.caches, self.first, self.new, self.ctx = kind, caches, first, new, ctx
        self.model = model_of(heads, total_caches or first + caches)
        g = torch.Generator().manual_seed(seed)
        P = len(new)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T, self.P = int(self.cu[-1]), P
        pages = [sorted({p // 16 for p in range(c, c + n)}) for c, n in zip(ctx, new)]
        self.num_pages = sum(map(len, pages)) + 3
        perm = torch.randperm(self.num_pages, generator=g)
        self.table = torch.full((P, max([p[-1] + 1 for p in pages if p], default=1) + 1), -1, dtype=torch.int32)
        self.table[:, ::2] = 10 ** 6
        at = 0
        for s in range(P):
            for p in pages[s]:
                self.table[s, p] = perm[at]
                at += 1
        self.kv = api.KVCache(self.model, self.num_pages, self.table.numpy(), dtype=kind)
        shape = tuple(self.kv.k.shape)
        for pool, sc in ((self.kv.k, self.kv.k_scale), (self.kv.v, self.kv.v_scale)):
            if kind == "bf16":
                pool.copy_(torch.randn(shape, generator=g).bfloat16())
            elif kind == "fp8":
                pool.copy_(torch.randint(0, 127, shape, generator=g).to(torch.uint8))
                sc.copy_(torch.rand(shape[:-1], generator=g))
            else:
                pool.copy_(torch.randint(-127, 128, shape, generator=g).to(torch.int8))
                sc.copy_(torch.rand(shape[:-2], generator=g) * 0.06 * scale)
        self.before = {n: getattr(self.kv, n).cpu().clone() for n in self.names()}
        self.k = (torch.randn(self.T, caches, self.n_kv, self.d, generator=g) * scale).bfloat16()
        self.v = (torch.randn(self.T, caches, self.n_kv, self.d, generator=g) * scale).bfloat16()
        self.q = torch.randn(self.T, self.n_q, self.d, generator=g).bfloat16()
        row = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, new)] + [np.zeros(0, int)]).astype(int)
        seq = np.repeat(np.arange(P), new)
        self.row, self.seq = row, seq
        self.page = self.table[torch.from_numpy(seq), torch.from_numpy(row // 16)].long()
        self.slot = torch.from_numpy(row % 16)

    def names(self):
        return ("k", "v") if self.kind == "bf16" else ("k", "v", "k_scale", "v_scale")

    def args(self):
        k, v = self.k.cuda(), self.v.cuda()
        return (k, v) if self.caches > 1 else (k[:, 0], v[:, 0])

    def run(self, q=True, status=0, **kw):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        k, v = self.args()
        out = api.append(self.model, k, v, self.cu, self.ctx, self.kv, cache=self.first, q=self.q.cuda() if q else None, **kw)
        torch.cuda.synchronize()
        assert self.model.status() == status
        return out

    def bf16_keys(self, off, rotate):
        """K as a bf16 cache of the same model holds it, whose values test_bf16 checks."""
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        kv = api.KVCache(self.model, self.num_pages, self.table.numpy())
        k, v = self.args()
        api.append(self.model, k, v, self.cu, self.ctx, kv, cache=self.first, pos_offsets=off, rotate=rotate)
        got = kv.k.cpu()
        return torch.stack([got[self.first + c][self.page, :, self.slot] for c in range(self.caches)], 1)

    def check(self, q_out, off=None, rotate=True):
        """Everything in the pools against the rules."""
        import torch
        pos = self.row + (np.asarray(off)[self.seq] if off is not None else 0)
        tol = 2.0 ** -20 if (pos >= 32768).any() else 2.0 ** -22

        def near(got, x):
            if not rotate:
                assert torch.equal(got, x)
                return
            flat = x.reshape(x.shape[0], -1, self.d)
            ref, y = turned(flat, pos).view(x.shape), x.double().abs()
            swap = torch.cat([y[..., self.d // 2:], y[..., :self.d // 2]], -1)
            err = (got.double() - ref).abs() - 2.0 ** -8 * ref.abs() - tol * (y + swap)
            assert bool((err <= 0).all()), float(err.max())

        if q_out is not None:
            near(q_out.cpu(), self.q)
        want = {n: t.clone() for n, t in self.before.items()}
        if self.T:
            keys = self.bf16_keys(off, rotate)
            near(keys, self.k)
            for name, x in (("k", keys), ("v", self.v)):
                for c in range(self.caches):
                    to = want[name][self.first + c]
                    if self.kind == "bf16":
                        to[self.page, :, self.slot] = x[:, c]
                        continue
                    sc = want[name + "_scale"][self.first + c]
                    if self.kind == "fp8":
                        f = x[:, c].float()
                        scale = f.abs().amax(-1) / 448
                        code = torch.where(scale[..., None] > 0, f / scale.clamp(min=1e-45)[..., None], 0.0)
                        to[self.page, :, self.slot] = code.to(torch.float8_e4m3fn).view(torch.uint8)
                        sc[self.page, :, self.slot] = scale
                        continue
                    for s in range(self.P):
                        for p in sorted(set(self.row[self.seq == s] // 16)):
                            rows = np.flatnonzero((self.seq == s) & (self.row // 16 == p))
                            lo, pg = self.row[rows[0]] % 16, int(self.table[s, p])
                            old = None
                            if lo:
                                old = np.zeros((lo, self.n_kv, self.d)).view(OM.Int8Rows)
                                old.codes = to[pg, :, :lo].permute(1, 0, 2).double().numpy()
                                old.scales = sc[pg].numpy()[None].copy()
                            r = OM.int8_append(old, x[rows, c].float().numpy())
                            to[pg, :, :lo + len(rows)] = torch.from_numpy(r.codes).permute(1, 0, 2).to(torch.int8)
                            sc[pg] = torch.from_numpy(r.scales[0])
        for n in self.names():
            got, ref = getattr(self.kv, n).cpu(), want[n]
            if n in ("k", "v") and self.kind == "bf16":
                got, ref = got.view(torch.int16), ref.view(torch.int16)
            assert torch.equal(got, ref), (n, int((got != ref).sum()))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("heads", list(HEADS))
def test_ragged_batches(heads, kind):
    for i, (new, ctx) in enumerate(BATCHES):
        c = Case(heads, new, ctx, kind, seed=i)
        c.check(c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("heads", ["gqa4", "gqa5", "d64"])
def test_several_caches_of_one_call(heads, kind):
    for new, ctx in (([1, 1], [15, 30]), ([40, 2], [3, 0])):
        c = Case(heads, new, ctx, kind, caches=3, total_caches=5, first=1, seed=7)
        c.check(c.run(q=False))
        c = Case(heads, new, ctx, kind, caches=2, seed=8)
        c.check(c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
def test_position_offsets_and_no_rotation(kind):
    new, ctx = [3, 1, 20], [10, 0, 5]
    for off in ([0, 0, 0], [5, 0, 32760], [32748, 40000, 1 << 20], [(1 << 30) - 13, 0, 123456789]):
        c = Case("gqa4", new, ctx, kind, seed=11)
        c.check(c.run(pos_offsets=off), off)
    c = Case("d64", new, ctx, kind, seed=12)
    c.check(c.run(rotate=False), rotate=False)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_strided_rows_q_in_place_and_another_stream(kind):
    """K, V and q as parts of one projection's rows; q is turned where it stands."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case("gqa4", [5, 1, 17], [14, 15, 0], kind, seed=13)
    rows = torch.full((c.T, c.n_q + 2 * c.n_kv + 1, c.d), 9.0, dtype=torch.bfloat16, device="cuda")
    q, k, v = rows[:, :c.n_q], rows[:, c.n_q:c.n_q + c.n_kv], rows[:, c.n_q + c.n_kv:-1]
    for part, x in ((q, c.q), (k, c.k[:, 0]), (v, c.v[:, 0])):
        part.copy_(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = api.append(c.model, k, v, c.cu, c.ctx, c.kv, q=q, q_out=q, stream=st)
    st.synchronize()
    assert out is q and c.model.status() == 0
    c.check(out)
    assert torch.equal(k.cpu(), c.k[:, 0]) and torch.equal(v.cpu(), c.v[:, 0]) and bool((rows[:, -1] == 9).all())
    # rows of a batch of one token may have any stride
    one = Case("gqa4", [1], [3], kind, seed=14)
    one.check(one.run())


@pytest.mark.gpu
def test_q_out_beside_q_in_wider_rows():
    """The turned q in the same rows as q itself, before or behind it."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case("gqa5", [5, 1, 17], [14, 15, 0], "bf16", seed=17)
    for first, second in ((0, c.n_q), (c.n_q + 1, 1)):
        rows = torch.full((c.T, 2 * c.n_q + 1, c.d), 9.0, dtype=torch.bfloat16, device="cuda")
        q, out = rows[:, first:first + c.n_q], rows[:, second:second + c.n_q]
        q.copy_(c.q)
        k, v = c.args()
        assert api.append(c.model, k, v, c.cu, c.ctx, c.kv, q=q, q_out=out) is out
        torch.cuda.synchronize()
        c.check(out)
        assert torch.equal(q.cpu(), c.q)
        with pytest.raises(B.SwiftKVError, match="overlaps q"):
            api.append(c.model, k, v, c.cu, c.ctx, c.kv, q=q, q_out=rows[:, 1:1 + c.n_q] if first == 0 else rows[:, 2:2 + c.n_q])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_more_sequences_than_the_parameters_hold(kind):
    new = [(7 * i) % 4 for i in range(700)]
    ctx = [(11 * i) % 37 for i in range(700)]
    c = Case("d64", new, ctx, kind, seed=15)
    c.check(c.run(pos_offsets=[i % 5 for i in range(700)]), [i % 5 for i in range(700)])


@pytest.mark.gpu
def test_int8_scales_grow_token_by_token():
    """A page filled by single tokens of growing and shrinking size, zeros and tiny values among them, holds what
    the rule gives token by token; a whole page at once has no error but its codes'."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    sizes = [0.0, 0.0, 1e-38, 1e-3, 1.0, 0.5, 2.0, 2.0, 60.0, 0.1, 61.0, 1e4, 3e38, 1.0, 0.0, 5.0, 7.0, 0.0, 2.0]
    m = model_of("gqa4", 1)
    kv = api.KVCache(m, 3, np.array([[2, 0]], np.int32), dtype="int8")
    g = torch.Generator().manual_seed(1)
    old = {"k": None, "v": None}
    for t, size in enumerate(sizes):
        x = {n: (torch.randn(1, 2, 128, generator=g).clamp(-1, 1) * size).bfloat16() for n in ("k", "v")}
        api.append(m, x["k"].cuda(), x["v"].cuda(), [0, 1], [t], kv, rotate=False)
        for n in ("k", "v"):
            old[n] = OM.int8_append(old[n], x[n].float().numpy())
            assert np.array_equal(kv.codes(0, 0, t + 1, n).cpu().numpy(), old[n].codes), (t, n)
            got = kv.scales(0, 0, t + 1, n).cpu().numpy()[::16]
            assert np.array_equal(got, old[n].scales), (t, n)
    assert m.status() == 0


@pytest.mark.gpu
def test_int8_values_that_are_not_finite():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m = model_of("gqa4", 1)
    kv = api.KVCache(m, 2, np.array([[1]], np.int32), dtype="int8")
    x = torch.randn(3, 2, 128, generator=torch.Generator().manual_seed(2)).bfloat16()
    x[0, 0, 5], x[1, 0, 7], x[2, 0, 0], x[1, 1, 3] = float("nan"), float("inf"), -float("inf"), float("nan")
    api.append(m, x.cuda(), x.cuda(), [0, 3], [0], kv, rotate=False)
    codes, scales = kv.codes(0, 0, 3).cpu(), kv.scales(0, 0, 3).cpu()
    top = torch.finfo(torch.bfloat16).max
    assert float(scales[0, 0]) == np.float32(top) / np.float32(127)
    assert codes[0, 0, 5] == 0 and codes[1, 0, 7] == 127 and codes[2, 0, 0] == -127 and codes[1, 1, 3] == 0
    rest = x[:, 1].float()
    rest[1, 3] = 0
    assert float(scales[0, 1]) == float(rest.abs().max() / 127)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
def test_pages_outside_the_pool_are_skipped(kind):
    import torch
    c = Case("gqa4", [20, 3], [10, 0], kind, seed=20)
    lost = c.table[0, 1].clone()
    c.table[0, 1] = c.num_pages
    c.kv.block_table.copy_(c.table.cuda())
    q = c.run(status=B.STATUS_BAD_PAGE)
    for n in c.names():
        assert torch.equal(getattr(c.kv, n).cpu()[:, lost].float(), c.before[n][:, lost].float())
    for n in ("k", "v"):  # (the page's int8 scale may have been large enough)
        assert not torch.equal(getattr(c.kv, n).cpu()[:, c.table[0, 0]].float(), c.before[n][:, c.table[0, 0]].float())
    c2 = Case("gqa4", [20, 3], [10, 0], kind, seed=20)
    assert torch.equal(q, c2.run())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
def test_captured_and_replayed(kind):
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case("14b", [1, 1, 6], [15, 40, 3], kind, seed=21)
    k, v = c.args()
    q, out = c.q.cuda(), torch.empty_like(c.q, device="cuda")
    graph = torch.cuda.CUDAGraph()
    kb, vb, qb = torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(q)
    with torch.cuda.graph(graph):
        api.append(c.model, kb, vb, c.cu, c.ctx, c.kv, q=qb, q_out=out)
    for name in c.names():
        getattr(c.kv, name).copy_(c.before[name].cuda())
    kb.copy_(k), vb.copy_(v), qb.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    c.check(out)


@pytest.mark.gpu
def test_two_graphs_that_share_the_workspace():
    """Batches whose lists do not fit the parameters are uploaded: two captured ones, replayed in turn, and a larger call
    between them, which makes the workspace grow."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    cases = [Case("d64", [(s * i) % 3 + 1 for i in range(400)], [(5 * s * i) % 40 for i in range(400)], "int8", seed=s)
             for s in (1, 2)]
    m = cases[0].model
    big = Case("d64", [1] * 9000, [0] * 9000, "bf16", seed=3)
    graphs, outs = [], []
    for c in cases:
        c.model = m
        c.run()                    # the workspace holds it
        k, v = (x.contiguous() for x in c.args())
        q, out = c.q.cuda(), torch.empty_like(c.q, device="cuda")
        c.keep = (k, v, q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.append(m, k, v, c.cu, c.ctx, c.kv, q=q, q_out=out)
        graphs.append(g)
        outs.append(out)
    big.model = m
    big.check(big.run())
    for _ in range(2):
        for c, g, out in zip(cases, graphs, outs):
            for name in c.names():
                getattr(c.kv, name).copy_(c.before[name].cuda())
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for c, out in zip(cases, outs):
            c.check(out)
    assert m.status() == 0


@pytest.mark.gpu
def test_calls_on_two_streams():
    """Appends to two models' caches at once."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    cases = [Case("gqa4", [300, 1, 7], [5, 15, 0], kind, seed=30 + i) for i, kind in enumerate(("bf16", "int8", "fp8"))]
    streams = [torch.cuda.Stream() for _ in cases]
    data = [(c.args(), c.q.cuda()) for c in cases]
    torch.cuda.synchronize()
    outs = [api.append(c.model, *kv, c.cu, c.ctx, c.kv, q=q, stream=st) for c, (kv, q), st in zip(cases, data, streams)]
    torch.cuda.synchronize()
    for c, out in zip(cases, outs):
        assert c.model.status() == 0
        c.check(out)


@pytest.mark.gpu
def test_refusals():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case("gqa4", [3], [0], caches=1, total_caches=2)
    k, v = c.args()
    q = c.q.cuda()

    def refused(what, *a, **kw):
        with pytest.raises((ValueError, B.SwiftKVError), match=what):
            api.append(c.model, *a, **kw)

    refused("bfloat16", k.float(), v, c.cu, c.ctx, c.kv)
    refused("bfloat16", k[:2], v, c.cu, c.ctx, c.kv)
    refused("contiguous", k.transpose(0, 1).contiguous().transpose(0, 1), v, c.cu, c.ctx, c.kv)
    refused("cache 2", k, v, c.cu, c.ctx, c.kv, cache=2)
    both = torch.stack([k, k], 1)
    refused("caches", both, both, c.cu, c.ctx, c.kv, cache=1)
    refused("v: bfloat16", both, torch.stack([v] * 3, 1), c.cu, c.ctx, c.kv)
    refused("q_out without q", k, v, c.cu, c.ctx, c.kv, q_out=q)
    buf = torch.cat([q, q])
    refused("overlaps", k, v, c.cu, c.ctx, c.kv, q=buf[:3], q_out=buf[1:4])
    refused("pos_offsets", k, v, c.cu, c.ctx, c.kv, pos_offsets=[0, 0])
    refused("positions", k, v, c.cu, c.ctx, c.kv, pos_offsets=[-1])
    refused("positions", k, v, c.cu, c.ctx, c.kv, pos_offsets=[(1 << 30) - 2])
    refused("pages", k, v, c.cu, [1000], c.kv)
    refused("32 bits", k, v, c.cu, c.ctx, c.kv, pos_offsets=np.array([1 << 32]))
    odd = torch.zeros(c.T * 256 + 8, dtype=torch.bfloat16, device="cuda")
    refused("16-byte", odd[1:1 + c.T * 256].view(c.T, 2, 128), v, c.cu, c.ctx, c.kv)
    refused("stride", torch.zeros(c.T, 260, dtype=torch.bfloat16, device="cuda")[:, :256].unflatten(1, (2, 128)), v, c.cu,
            c.ctx, c.kv)
    torch.cuda.synchronize()
    assert c.model.status() == 0
    assert all(torch.equal(getattr(c.kv, n).cpu(), c.before[n]) for n in c.names())
    # nothing to do
    assert api.append(c.model, k[:0], v[:0], [0], [], c.kv) is None
    assert api.append(c.model, k[:0], v[:0], [0, 0], [0], c.kv, q=q[:0]).shape[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3])
def test_q_out_over_k_or_v_is_refused(T):
    """Rows of q_out are written while other warps read K and V: a view that reaches into theirs, by one head at
    either end or in another token's row, is refused; parts beside them are not."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case("gqa4", [T], [0], "int8", caches=2)
    Q, K = c.n_q, c.n_kv
    W = 2 * Q + 4 * K
    # a row: room for q, K of both caches, V of both, room for q again
    wide = torch.zeros(T + 2, W, c.d, dtype=torch.bfloat16, device="cuda")
    rows = wide[1:-1]
    k, v = rows[:, Q:Q + 2 * K].unflatten(1, (2, K)), rows[:, Q + 2 * K:Q + 4 * K].unflatten(1, (2, K))
    k.copy_(c.k)
    v.copy_(c.v)
    q = c.q.cuda()
    flat, row = wide.flatten(), wide.stride(0)

    def at(head):  # q_out that starts `head` heads into the rows
        return flat.as_strided((T, Q, c.d), (row, c.d, 1), row + head * c.d)

    apart, over = [0, Q + 4 * K], [1, Q, Q + K + 1, Q + 4 * K - 1]
    (over if T > 1 else apart).extend((W + 1, 1 - W))  # over the neighbouring tokens' rows
    for head in over:
        with pytest.raises(B.SwiftKVError, match="q_out overlaps k or v"):
            api.append(c.model, k, v, c.cu, c.ctx, c.kv, q=q, q_out=at(head))
    torch.cuda.synchronize()
    assert all(torch.equal(getattr(c.kv, n).cpu(), c.before[n]) for n in c.names())
    for head in apart:
        out = api.append(c.model, k, v, c.cu, c.ctx, c.kv, q=q, q_out=at(head))
        c.check(out)
        assert torch.equal(k.cpu(), c.k) and torch.equal(v.cpu(), c.v)


@pytest.mark.gpu
def test_int8_caches_elsewhere_are_refused():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case("gqa4", [3], [0], "int8")
    lse, sc = torch.zeros(8, 3, device="cuda"), torch.zeros(1, c.num_pages, 2, 16, device="cuda")
    for call in (lambda: api.attention_weights(c.model, c.q.cuda(), lse, c.cu, c.ctx, c.kv, sc[0]),
                 lambda: api.evict(c.model, c.kv, sc, [3], 2)):
        with pytest.raises(B.SwiftKVError, match="EUNSUPPORTED"):
            call()


@pytest.mark.gpu
def test_strides_past_32_bits_are_refused():
    """A step between caches whose multiple wraps around to a row's width, and row strides whose low 32 bits would pass."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case("gqa4", [3], [0], caches=5, total_caches=5)
    (k, v), q = c.args(), c.q.cuda()
    r = B.NewRows()
    r.k, r.v, r.ldk, r.ldv, r.k_step, r.v_step = k.data_ptr(), v.data_ptr(), 1280, 1280, 1 << 62, 256
    for r.k_step, r.v_step in ((1 << 62, 256), (256, 1 << 62)):
        assert B.lib().swiftkv_append(c.model.handle, 0, 5, r, B.host(c.cu), None, None, 1, c.kv.pages_ref, 1, None) == -1
        assert b"k_step" in B.lib().swiftkv_last_error()
    wide = torch.empty(2 * ((1 << 32) + 1280) + 4096, dtype=torch.bfloat16, device="cuda")

    def rows(t):
        return wide.as_strided(t.shape, ((1 << 32) + 1280, *t.stride()[1:]))

    for kk, vv, qq in ((rows(k), v, q), (k, rows(v), q), (k, v, rows(q))):
        with pytest.raises(ValueError, match="32 bits"):
            api.append(c.model, kk, vv, c.cu, c.ctx, c.kv, q=qq)
    torch.cuda.synchronize()
    assert all(torch.equal(getattr(c.kv, n).cpu(), c.before[n]) for n in c.names())


def test_arguments_without_gpu():
    lib = B.lib()
    r = B.NewRows()
    assert lib.swiftkv_append(None, 0, 1, C.byref(r), None, None, None, 1, None, 1, None) == -1
    assert b"null model" in lib.swiftkv_last_error()
