"""Attention over an int8 cache with one scale for each page and head, and the model's own calls on such caches.

Tolerances of swiftkv_attend, for each element with its own mass M = sum_j p_ij |v_je|, as over the other
caches: scores are off by at most ds = d 2^-23 max_ij sum |q_i k_j| / sqrt(d), a weight by 2 ds and 2^-12 of it for
its exponential and the sums, P's rounding to bf16 by 2^-8 of it in chunks of more than 16 rows (two bf16 parts,
2^-16, in shorter ones), and the output's rounding to bf16 by 2^-8 of its value. Codes enter exactly. Nothing scales
with the largest value of the cache: pages may differ in size by any factor."""
import math

import numpy as np
import pytest

import oracle
import synth
from gpu_helpers import LOGIT_ABS_TOL, SMALL128, SMALL_BIAS, GQA8
from oracle import model as OM
from swiftkv_prefill_skipping_gb300 import binding as B
from test_gpu_serving import BATCHES, HEADS, WINDOWS, model_of, seen_mask

pytestmark = pytest.mark.gpu


class Case:
    """A ragged batch over an int8 cache. Rows that nobody sees hold large codes, pages without a visible row
    scales of NaN and table entries outside the pool. vmul, kmul: a factor for each page (cycled)."""

    def __init__(self, heads, new, ctx, window=0, sinks=0, seed=0, vmul=(1.0,), kmul=(1.0,), qmul=1.0, low=(), zero=()):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        self.n_q, self.n_kv, self.d = HEADS[heads]
        self.new, self.ctx, self.window, self.sinks = new, ctx, window, sinks
        self.model = model_of(heads)
        g = torch.Generator().manual_seed(seed)
        P = len(new)
        self.P, self.cu = P, np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.cu[-1])
        need = [(c + n + 15) // 16 for c, n in zip(ctx, new)]
        total = sum(need) + 5
        perm = torch.randperm(total, generator=g)
        table = torch.full((P, max(need, default=0) + 2), 10 ** 6, dtype=torch.int32)
        table[:, ::2] = -1
        pools = {n: torch.where(torch.rand(total, self.n_kv, 16, self.d, generator=g) < 0.5, -127, 127).to(torch.int8) for n in "kv"}
        scales = {n: torch.full((total, self.n_kv), float("nan")) for n in "kv"}
        self.masks, self.ref, at = [], [], 0
        for s in range(P):
            n, c0 = new[s], ctx[s]
            mask = seen_mask(n, c0, window, sinks)
            some = mask.any(0) if n else np.zeros(c0 + n, bool)
            self.masks.append(torch.from_numpy(mask))
            ref = {x: torch.zeros(c0 + n, self.n_kv, self.d, dtype=torch.float64) for x in "kv"}
            for p in range(need[s]):
                rows = np.flatnonzero(some[16 * p:16 * p + 16])
                if not len(rows):
                    continue
                table[s, p] = page = int(perm[at + p])
                for x, mul in (("k", kmul[p % len(kmul)]), ("v", vmul[p % len(vmul)])):
                    code = (torch.randn(len(rows), self.n_kv, self.d, generator=g) * 32).round().clamp(-127, 127)
                    if x == "k" and p in low:
                        code = code * 0 - 60
                    if x == "v" and p in zero:
                        code = code * 0
                    scale = torch.full((self.n_kv,), mul / 32, dtype=torch.float32) * (1 + torch.arange(self.n_kv) / 8)
                    if x == "v" and p in zero:
                        scale = scale * 0
                    pools[x][page][:, rows] = code.to(torch.int8).transpose(0, 1)
                    scales[x][page] = scale
                    ref[x][16 * p + rows] = code.double() * scale.double()[None, :, None]
            at += need[s]
            self.ref.append(ref)
        self.kv = api.KVCache(self.model, total, table.numpy(), dtype="int8")
        for x in "kv":
            getattr(self.kv, x)[1].copy_(pools[x])
            getattr(self.kv, x + "_scale")[1].copy_(scales[x])
        self.q = ((torch.randn(self.T, self.n_q, self.d, generator=g) + (0.5 if low else 0.0)) * qmul).bfloat16()

    def attend(self, **kw):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        lse = torch.full((self.n_q, self.T), float("nan"), device="cuda")
        out = api.attend(self.model, self.q.cuda(), self.cu, self.ctx, self.kv, cache=1, window=self.window,
                         sinks=self.sinks, lse=lse, **kw)
        torch.cuda.synchronize()
        assert self.model.status() == 0
        return out.cpu(), lse.cpu()

    def check(self):
        import torch
        out, lse = self.attend()
        G = self.n_q // self.n_kv
        for s in range(self.P):
            if not self.new[s]:
                continue
            rows = slice(int(self.cu[s]), int(self.cu[s + 1]))
            for h in range(self.n_q):
                q, k, v = self.q[rows, h].double(), self.ref[s]["k"][:, h // G], self.ref[s]["v"][:, h // G]
                z = (q @ k.T / math.sqrt(self.d)).masked_fill(~self.masks[s], -math.inf)
                ds = self.d * 2.0 ** -23 * float((q.abs() @ k.abs().T)[self.masks[s]].max()) / math.sqrt(self.d)
                ref_lse = torch.logsumexp(z, 1)
                p = torch.exp(z - ref_lse[:, None])
                ref = p @ v
                rel = 2 * ds + 2.0 ** -12 + (2.0 ** -8 if self.new[s] > 16 else 2.0 ** -16)
                tol = 2.0 ** -8 * ref.abs() + rel * (p @ v.abs()) + 2.0 ** -133
                err = (out[rows, h].double() - ref).abs()
                assert bool((err <= tol).all()), (s, h, float((err - tol).max()))
                el = (lse[h, rows].double() - ref_lse).abs()
                assert bool((el <= ds + 2.0 ** -12 + 2.0 ** -21 * ref_lse.abs()).all()), (s, h, float(el.max()))


@pytest.mark.parametrize("heads", list(HEADS))
def test_ragged_batches(heads):
    for i, (new, ctx) in enumerate(BATCHES):
        Case(heads, new, ctx, seed=i).check()


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("heads", ["gqa4", "gqa5", "d64"])
def test_window_and_sinks(heads, window, sinks):
    for i, (new, ctx) in enumerate([([1, 1, 3], [0, 250, 90]), ([260, 5], [33, 400]), ([70, 300], [0, 500])]):
        Case(heads, new, ctx, window, sinks, seed=10 + i).check()


@pytest.mark.parametrize("heads", ["gqa4", "d64"])
@pytest.mark.parametrize("new,ctx", [([1, 3], [300, 64]), ([200, 5], [100, 400])])
def test_pages_of_any_size(heads, new, ctx):
    """Value and key scales that differ by many powers of two from page to page, and pages that are zero."""
    Case(heads, new, ctx, seed=30, vmul=(1.0, 2.0 ** 40, 2.0 ** -40, 1e-3)).check()
    Case(heads, new, ctx, seed=31, vmul=(1e-30, 1e-38)).check()
    Case(heads, new, ctx, seed=32, vmul=(1.0, 2.0 ** 90), low=(1, 3, 5, 7)).check()
    Case(heads, new, ctx, seed=33, kmul=(1.0, 0.01, 8.0, 1e-20)).check()
    Case(heads, new, ctx, seed=34, zero=(0, 2, 6)).check()
    Case(heads, new, ctx, seed=35, zero=range(100)).check()
    Case(heads, new, ctx, seed=36, kmul=(0.0,)).check()


@pytest.mark.parametrize("mul", [2.0 ** -60, 2.0 ** -100, 2.0 ** -126, 2.0 ** -135])
@pytest.mark.parametrize("heads", ["gqa4", "gqa5", "d64"])
@pytest.mark.parametrize("new", [[16], [17], [130]])
def test_weights_of_pages_with_tiny_values_count(heads, new, mul):
    """Thousands of keys whose weights are small and whose values are next to nothing, behind a page of ordinary ones: their
    share of the sum is not lost, whatever their scale."""
    n = 600
    Case(heads, new, [16 * n], seed=38, vmul=(1.0,) + (mul,) * (n + 20), low=range(1, n + 20)).check()


@pytest.mark.parametrize("heads", ["gqa4", "gqa5", "d64"])
@pytest.mark.parametrize("new", [[16], [17], [300, 3]])
def test_pages_cleared_by_a_scale_of_zero(heads, new):
    """Codes under a scale of 0 stand for zeros, in chunks of either kind and beside values of any size."""
    for vmul in (1.0, 1e-30):
        c = Case(heads, new, [70 + 10 * i for i in range(len(new))], seed=37, vmul=(vmul,))
        for s in range(c.P):
            for p in (1, 3):
                page = int(c.kv.block_table[s, p])
                c.kv.v_scale[1, page, 0] = 0
                c.ref[s]["v"][16 * p:16 * p + 16, 0] = 0
                c.kv.k_scale[1, page, -1] = 0
                c.ref[s]["k"][16 * p:16 * p + 16, -1] = 0
        c.check()


@pytest.mark.parametrize("heads", list(HEADS))
def test_chunks_around_the_border_between_rows_and_tiles(heads):
    for window, sinks in ((0, 0), (37, 5)):
        Case(heads, [4, 5, 7, 8], [0, 700, 33, 16], window, sinks, seed=70).check()
        Case(heads, [15, 16, 17, 9, 18], [300, 1, 40, 0, 500], window, sinks, seed=71).check()


@pytest.mark.parametrize("heads", list(HEADS))
@pytest.mark.parametrize("window,sinks", [(0, 0), (900, 30), (2500, 0), (300, 1500)])
def test_tiles_cut_along_their_keys(heads, window, sinks):
    """Few tiles after long prefixes run in parts: rows that see nothing of a part, tiles that end before one, second tiles
    that are absent."""
    Case(heads, [40], [3000], window, sinks, seed=80).check()
    Case(heads, [300], [2500], window, sinks, seed=81, kmul=(1.0, 4.0, 0.1)).check()
    Case(heads, [17, 2, 500], [4000, 100, 1000], window, sinks, seed=82, vmul=(1.0, 2.0 ** 30, 1e-6)).check()


def test_cut_tiles_repeat_their_bits_and_replay():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case("gqa4", [100, 3], [5000, 40], seed=83)
    out, lse = c.attend()
    assert all(torch.equal(x, y) for x, y in zip((out, lse), c.attend()))
    q, got, l = c.q.cuda(), torch.zeros_like(c.q, device="cuda"), torch.zeros_like(lse, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.attend(c.model, q, c.cu, c.ctx, c.kv, cache=1, out=got, lse=l)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), out) and torch.equal(l.cpu(), lse)
    # rows of a wider buffer, and no log-sum-exp
    wide = torch.full((c.T, c.n_q + 1, c.d), 5.0, dtype=torch.bfloat16, device="cuda")
    api.attend(c.model, q, c.cu, c.ctx, c.kv, cache=1, out=wide[:, 1:])
    assert torch.equal(wide[:, 1:].cpu(), out) and bool((wide[:, 0] == 5).all())


@pytest.mark.parametrize("heads", ["gqa5", "gqa4", "d64"])
def test_more_items_than_ctas(heads):
    """CTAs walk several items, of which the second tile takes part in some only (odd groups)."""
    n = {"gqa5": 44, "gqa4": 24, "d64": 48}[heads]
    Case(heads, [100, 300, 5, 260] * (n // 4), [(37 * i) % 500 for i in range(n)], seed=50).check()
    Case(heads, [100, 300, 5, 260] * (n // 4), [(37 * i) % 500 for i in range(n)], 90, 20, seed=51).check()


@pytest.mark.parametrize("heads", ["gqa4", "d64"])
def test_queries_of_any_size(heads):
    for new, ctx in (([1, 2], [300, 64]), ([70], [100])):
        for qmul, kmul in ((1e20, 1e-20), (1e-20, 1e20), (20.0, 1.0), (1e-30, 1.0)):
            Case(heads, new, ctx, seed=40, qmul=qmul, kmul=(kmul,)).check()


def test_codes_of_minus_128_and_repeated_bits():
    import torch
    c = Case("gqa4", [3, 40], [70, 30], seed=41)
    a = c.attend()
    assert all(torch.equal(x, y) for x, y in zip(a, c.attend()))
    # -128 is not written by append, and stands for -128 all the same
    page = int(c.kv.block_table[0, 0])
    c.kv.v[1, page, :, :, 0] = -128
    c.ref[0]["v"][:16, :, 0] = -128 * c.kv.v_scale[1, page].cpu().double()[None]
    c.check()


def test_captured_and_on_another_stream():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    for new, ctx in (([1, 2], [500, 64]), ([70, 3], [100, 40])):
        c = Case("gqa4", new, ctx, seed=42)
        ref, _ = c.attend()
        q, out = c.q.cuda(), torch.zeros_like(c.q, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            api.attend(c.model, q, c.cu, c.ctx, c.kv, cache=1, out=out)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), ref)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        got = api.attend(c.model, q, c.cu, c.ctx, c.kv, cache=1, stream=st)
        st.synchronize()
        assert torch.equal(got.cpu(), ref)


def test_two_graphs_that_share_the_workspace():
    """Expansions and lists of two captured calls in one workspace, which a larger call outgrows between them."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    cases = [Case("gqa4", [70, 3, 200], [100, 40, 0], seed=60), Case("gqa4", [5, 33], [900, 20], 64, 3, seed=61)]
    big = Case("gqa4", [900, 900], [3000, 2000], seed=62)
    m = cases[0].model
    graphs = []
    for c in cases:
        c.model = m
        c.want = c.attend()
        q, out = c.q.cuda(), torch.zeros_like(c.q, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.attend(m, q, c.cu, c.ctx, c.kv, cache=1, window=c.window, sinks=c.sinks, out=out)
        graphs.append((g, q, out))
    big.model = m
    big.check()
    for _ in range(2):
        for c, (g, q, out) in zip(cases, graphs):
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for c, (g, q, out) in zip(cases, graphs):
            assert torch.equal(out.cpu(), c.want[0])
    assert m.status() == 0


def test_sequences_that_share_pages():
    """A common prefix in two sequences' tables, and one sequence named twice."""
    import torch
    c = Case("gqa5", [40, 2, 40], [80, 80, 80], seed=63)
    table = c.kv.block_table.clone()
    for s in (1, 2):
        c.kv.block_table[s, :5] = table[0, :5]       # 80 rows
        for x in "kv":
            c.ref[s][x][:80] = c.ref[0][x][:80]
    c.check()
    rows = c.kv.view([0, 0])
    from swiftkv_prefill_skipping_gb300 import api
    q = torch.cat([c.q[:40], c.q[:40]]).cuda()
    out = api.attend(c.model, q, [0, 40, 80], [80, 80], rows, cache=1)
    assert torch.equal(out[:40], out[40:])


def test_bad_pages_are_flagged():
    c = Case("gqa4", [2, 60], [40, 50], seed=43)
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    for s, p in ((0, 1), (1, 0)):
        kept = int(c.kv.block_table[s, p])
        c.kv.block_table[s, p] = 10 ** 6
        api.attend(c.model, c.q.cuda(), c.cu, c.ctx, c.kv, cache=1)
        torch.cuda.synchronize()
        assert c.model.status() == B.STATUS_BAD_PAGE
        c.kv.block_table[s, p] = kept
    c.check()


# ---------------------------------------------------------------- the model's own calls

SHAPES = {"tiny": (synth.TINY, 2, 1), "d128": (SMALL128, 2, 2), "bias": (SMALL_BIAS, 4, 1), "gqa8": (GQA8, 2, 2)}


def setup(name, lens, extra=40):
    from swiftkv_prefill_skipping_gb300 import api
    shape, l, g = SHAPES[name]
    batch = synth.prompt_batch(shape.vocab, len(lens), 0, 0, lens=lens, reserve_tokens=extra)
    m = api.load_synthetic(shape, l, g)
    kv = api.KVCache(m, batch.num_pages, batch.block_table, dtype="int8")
    prompts = [batch.tokens[batch.cu_seqlens[s]:batch.cu_seqlens[s + 1]] for s in range(len(lens))]
    return m, kv, batch, prompts, oracle.config_of(shape), oracle.synth_weights(shape), l, g


def check_caches(m, kv, s, caches):
    """The first cache, whose inputs are the same on both sides: where a bf16 value rounds the other way a code may
    move by one, or, where it was the block's largest, the block's scale by 2^-7 of itself. The others inherit
    differences of float32 and float64 accumulation, one step of 1/127 of the block's largest value here and there."""
    n = caches[0][0].shape[0]
    for which, t in (("k", 0), ("v", 1)):
        got, ref = kv.codes(0, s, n, which).cpu().numpy(), caches[0][t]
        assert (got == ref.codes).mean() >= 0.98 and np.abs(got - ref.codes).max() <= 2, which
        sc = kv.scales(0, s, n, which).cpu().numpy()[::16]
        assert np.abs(sc - ref.scales).max() <= 2.0 ** -7 * ref.scales.max()
        for c in range(m.num_caches):
            a, b = kv.gather(c, s, n, which).cpu().numpy().astype(np.float64), np.asarray(caches[c][t])
            assert np.linalg.norm(a - b) <= 2e-2 * np.linalg.norm(b), (c, which)


@pytest.mark.parametrize("name", list(SHAPES))
def test_prefill_forward_and_decode(name):
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, prompts, cfg, w, l, g = setup(name, [150, 3, 70])
    logits = api.prefill(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, kv)
    state = []
    with OM.kv_cache_int8():
        for s, p in enumerate(prompts):
            caches, ref = OM.swiftkv_prefill_one(cfg, w, p, l, g)
            assert np.abs(logits[s].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL
            check_caches(m, kv, s, caches)
            state.append((caches, OM.greedy(ref)))
        chunk = synth.uniform_int(5, 1, 9, 0, cfg.vocab - 1)
        toks = np.concatenate([chunk, [state[1][1]]])
        lg = api.forward(m, torch.as_tensor(toks, device="cuda"), [0, 9, 10], [150, 3], kv.view([0, 1]))
        for i, t in ((0, chunk), (1, [state[1][1]])):
            caches, ref = OM.swiftkv_forward_one(cfg, w, state[i][0], t, l, g)
            assert np.abs(lg[i].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL
            state[i] = (caches, OM.greedy(ref))
        lens = [159, 4, 70]
        for _ in range(3):
            lg, _ = api.decode_step(m, torch.tensor([t for _, t in state], device="cuda"), lens, kv)
            for s in range(3):
                caches, ref = OM.swiftkv_decode_step(cfg, w, state[s][0], state[s][1], l, g)
                assert np.abs(lg[s].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL
                state[s] = (caches, OM.greedy(ref))
            lens = [n + 1 for n in lens]
        for s in range(3):
            check_caches(m, kv, s, state[s][0])
    assert m.status() == 0
    m.free()


@pytest.mark.parametrize("impl", [0, 1])
def test_window_and_chained_rows(impl):
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, prompts, cfg, w, l, g = setup("d128", [140, 2])
    B.check(B.lib().swiftkv_set_rows_impl(m.handle, impl))
    m.set_attention_window(48, 3)
    logits = api.prefill(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, kv)
    with OM.attention_window(48, 3), OM.kv_cache_int8():
        refs = [OM.swiftkv_forward_one(cfg, w, None, p, l, g) for p in prompts]
        for s in range(2):
            assert np.abs(logits[s].cpu().numpy() - refs[s][1]).max() <= LOGIT_ABS_TOL
        toks = [OM.greedy(r[1]) for r in refs]
        lg, _ = api.decode_step(m, torch.tensor(toks, device="cuda"), [140, 2], kv)
        for s in range(2):
            _, ref = OM.swiftkv_decode_step(cfg, w, refs[s][0], toks[s], l, g)
            assert np.abs(lg[s].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL
    assert m.status() == 0
    m.free()


@pytest.mark.parametrize("gemm,fused", [(1, 0), (2, 0), (0, 1)])
def test_other_gemm_families(gemm, fused):
    """Every family hands its rows to the same pages; the fused norm rounds elsewhere (one more bf16 step)."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, prompts, cfg, w, l, g = setup("d128", [150, 30])
    B.check(B.lib().swiftkv_set_gemm_impl(m.handle, gemm))
    B.check(B.lib().swiftkv_set_norm_fusion(m.handle, fused))
    logits = api.prefill(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, kv)
    with OM.kv_cache_int8():
        for s, p in enumerate(prompts):
            caches, ref = OM.swiftkv_prefill_one(cfg, w, p, l, g)
            assert np.abs(logits[s].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL
            got = kv.gather(0, s, len(p), "v").cpu().numpy()
            assert np.linalg.norm(got - caches[0][1]) <= 2e-2 * np.linalg.norm(caches[0][1])
    assert m.status() == 0
    m.free()


def test_rows_nobody_wrote_stay():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, prompts, *_ = setup("d128", [33, 70])
    kv.k.fill_(77)
    kv.k_scale.fill_(-5.0)
    api.prefill(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, kv)
    torch.cuda.synchronize()
    used = torch.zeros(kv.num_pages, 16, dtype=torch.bool)
    for s, n in enumerate([33, 70]):
        for p in range(n):
            used[int(batch.block_table[s][p // 16]), p % 16] = True
    rows = kv.k.cpu().permute(1, 3, 0, 2, 4)
    assert bool((rows[~used] == 77).all())
    sc = kv.k_scale.cpu()
    assert bool((sc[:, ~used.any(1)] == -5).all()) and bool((sc[:, used.any(1)] > 0).all())


def test_score_pools_are_refused():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, *_ = setup("tiny", [20])
    m.set_score_pools(torch.zeros(m.num_caches, batch.num_pages, m.shape.n_kv, 16, device="cuda"))
    tok = torch.as_tensor(batch.tokens, device="cuda")
    with pytest.raises(B.SwiftKVError, match="EUNSUPPORTED"):
        api.prefill(m, tok, batch.cu_seqlens, kv)
    m.set_score_pools(None)
    api.prefill(m, tok, batch.cu_seqlens, kv)
    assert m.status() == 0


def test_a_layer_of_ones_own():
    """append, attend, adjust_logits and sample as a program with layers of its own calls them: a prompt, then single
    tokens, against one pass over the whole text."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m = model_of("gqa4", 1)
    g = torch.Generator(device="cuda").manual_seed(5)
    n, more = 100, 6
    rows = torch.randn(n + more, 12, 128, device="cuda", generator=g).bfloat16()
    head = torch.randn(8 * 128, 500, device="cuda", generator=g) / 32
    table = torch.randperm(8)[None].int().numpy()

    def part(a, b, kv):
        q = api.append(m, rows[a:b, 8:10], rows[a:b, 10:], [0, b - a], [a], kv, q=rows[a:b, :8])
        return api.attend(m, q, [0, b - a], [a], kv)

    for dtype in ("bf16", "fp8", "int8"):
        whole, step = (api.KVCache(m, 8, table, dtype=dtype) for _ in range(2))
        ref = part(0, n + more, whole)
        got = [part(0, n, step)] + [part(i, i + 1, step) for i in range(n, n + more)]
        got = torch.cat(got)
        # an int8 page filled in steps may differ by a step of 1/127 of its largest value (5 here) in each vector
        tol = 2.0 ** -6 if dtype != "int8" else 0.08
        assert float((got.float() - ref.float()).abs().max()) <= tol * max(1.0, float(ref.float().abs().max()))
        text = torch.zeros(1, more, dtype=torch.int32, device="cuda")
        lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        for i in range(more):  # a presence penalty beyond any logit: no token comes twice
            logits = got[n + i:n + i + 1].flatten(1).float() @ head
            logits = api.adjust_logits(logits, tokens=text, lens=lens, presence=1e6)
            text[:, i] = api.sample(logits, torch.rand(1, device="cuda", generator=g), temperature=2.0)
            lens += 1
        assert len(set(text[0].tolist())) == more
    assert m.status() == 0
