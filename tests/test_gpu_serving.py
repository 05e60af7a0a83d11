"""swiftkv_attend, swiftkv_attention_weights and swiftkv_evict against their definitions in 64 bits.

Every row of the pools that no token may see holds NaN, and every block-table entry that is not
needed points outside the pool, so a read too many shows.

Tolerances. The scores are fp32 tensor-core sums of d products: off by at most
ds = d 2^-23 max_ij sum|q_i k_j| / sqrt(d) (the bound of a d-term sum with a rounding of 2^-23,
twice fp32's half step, per addition). A softmax weight is then off by a factor within
exp(+-2 ds), its exponential (2^-22) and the fp32 sums of up to 2^12 positive terms (2^-12 2^-1 for
a running fp32 sum) add to that. P's rounding adds 2^-8 (bf16) for chunks of more than 4 rows; for
shorter ones 2^-17 (two bf16 parts), or with an FP8 cache 2^-11 (fp16) and 2^-25 of the largest value
per key for weights below fp16's normal range. The output's rounding to bf16 adds 2^-8 of its value."""
import ctypes as C
import math

import numpy as np
import pytest

from swiftkv_prefill_skipping_gb300 import binding as B

HEADS = {"gqa4": (8, 2, 128), "gqa5": (5, 1, 128), "gqa8": (16, 2, 128), "mha": (2, 2, 128), "d64": (4, 2, 64),
         "d64_mha": (6, 6, 64)}


def model_of(heads, caches=2):
    from swiftkv_prefill_skipping_gb300 import api
    n_q, n_kv, d = HEADS[heads]
    d_model = 128
    return api.Model(api.Shape(L=caches, d=d_model, n_q=n_q, n_kv=n_kv, d_h=d, ffn=64, vocab=128, rope_theta=1e4),
                     l=caches)


def seen_mask(n, c0, window, sinks):
    """[n, c0 + n]: which keys each row sees."""
    p = c0 + np.arange(n)[:, None]
    j = np.arange(c0 + n)[None]
    m = j <= p
    if window:
        m &= (j > p - window) | (j < sinks)
    return m


class Case:
    """A ragged batch over poisoned pools; K and V of visible keys are finite, all else is NaN."""

    def __init__(self, heads, new, ctx, window=0, sinks=0, fp8=False, seed=0, caches=2, cache=1, scale=1.0, ramp=None):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        self.n_q, self.n_kv, self.d = HEADS[heads]
        self.new, self.ctx, self.window, self.sinks, self.fp8, self.cache = new, ctx, window, sinks, fp8, cache
        self.model = model_of(heads, caches)
        g = torch.Generator().manual_seed(seed)
        P = len(new)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(self.cu[-1])
        need = [(c + n + 15) // 16 for c, n in zip(ctx, new)]
        width = max(max(need, default=0), 1) + 2
        total = sum(need) + 5
        perm = torch.randperm(total, generator=g)
        table = torch.full((P, width), 10 ** 6, dtype=torch.int32)
        table[:, ::2] = -1
        self.masks, first = [], 0
        self.k, self.v = [], []          # float64 [keys, n_kv, d] of each sequence, 0 where unseen
        nan = float("nan")
        pool = torch.full((total, self.n_kv, 16, self.d), nan)
        vpool = pool.clone()
        ks = torch.full((total, self.n_kv, 16), nan)
        vs = ks.clone()
        self.seen = []
        for s in range(P):
            n, c0 = new[s], ctx[s]
            mask = seen_mask(n, c0, window, sinks)
            some = mask.any(0) if n else np.zeros(c0 + n, bool)
            self.masks.append(mask)
            self.seen.append(some)
            kk = torch.randn(c0 + n, self.n_kv, self.d, generator=g) * scale
            vv = torch.randn(c0 + n, self.n_kv, self.d, generator=g)
            if ramp:  # scores near ramp[0] at the first key, ramp[1] at the last
                at = torch.linspace(ramp[0], ramp[1], c0 + n)[:, None, None]
                kk = kk + at / math.sqrt(self.d)
            for p in range(need[s]):
                if some[16 * p:16 * p + 16].any():
                    table[s, p] = perm[first + p]
            idx = np.flatnonzero(some)
            pg, sl = perm[first + torch.from_numpy(idx // 16)], torch.from_numpy(idx % 16)
            first += need[s]
            i = torch.from_numpy(idx)
            if fp8:
                for x, po, sc in ((kk, pool, ks), (vv, vpool, vs)):
                    sx = x.abs().amax(-1) / 448
                    code = (x / sx[..., None]).to(torch.float8_e4m3fn).float()
                    po[pg, :, sl] = code[i]
                    sc[pg, :, sl] = sx[i]
                    x.copy_(code * sx[..., None])  # what the cache stands for, up to one fp32 rounding
                    if po is pool:
                        kk = code.double() * sx.double()[..., None]
                    else:
                        vv = code.double() * sx.double()[..., None]
            else:
                kk, vv = kk.bfloat16().double(), vv.bfloat16().double()
                pool[pg, :, sl] = kk[i].float()
                vpool[pg, :, sl] = vv[i].float()
            self.k.append(kk)
            self.v.append(vv)
        self.table = table
        self.kv = api.KVCache(self.model, total, table.numpy(), dtype="fp8" if fp8 else "bf16")
        if fp8:
            self.kv.k.view(torch.float8_e4m3fn)[cache] = pool.to(torch.float8_e4m3fn).cuda()
            self.kv.v.view(torch.float8_e4m3fn)[cache] = vpool.to(torch.float8_e4m3fn).cuda()
            self.kv.k_scale[cache] = ks.cuda()
            self.kv.v_scale[cache] = vs.cuda()
        else:
            self.kv.k[cache] = pool.bfloat16().cuda()
            self.kv.v[cache] = vpool.bfloat16().cuda()
        self.q = (torch.randn(T, self.n_q, self.d, generator=g) * scale + (1.0 if ramp else 0.0)).bfloat16()
        self.T, self.P, self.total = T, P, total

    def logits(self, s, h):
        """float64 scores of sequence s, head h, -inf where hidden, and ds."""
        import torch
        q = self.q[self.cu[s]:self.cu[s + 1], h].double()
        k = self.k[s][:, h // (self.n_q // self.n_kv)]
        z = (q @ k.T) / math.sqrt(self.d)
        ds = self.d * 2.0 ** -23 * float((q.abs() @ k.abs().T).max()) / math.sqrt(self.d)
        return z.masked_fill(~torch.from_numpy(self.masks[s]), -math.inf), ds

    def attend(self, **kw):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        lse = torch.full((self.n_q, self.T), float("nan"), device="cuda")
        out = api.attend(self.model, self.q.cuda(), self.cu, self.ctx, self.kv, cache=self.cache, window=self.window,
                         sinks=self.sinks, lse=lse, **kw)
        torch.cuda.synchronize()
        assert self.model.status() == 0
        return out.cpu().double(), lse.cpu().double()

    def check_attend(self, out, lse):
        import torch
        for s in range(self.P):
            if not self.new[s]:
                continue
            rows = slice(int(self.cu[s]), int(self.cu[s + 1]))
            rows_kernel = self.new[s] <= 4
            vmax = float(self.v[s].abs().max())
            for h in range(self.n_q):
                z, ds = self.logits(s, h)
                ref_lse = torch.logsumexp(z, 1)
                p = torch.exp(z - ref_lse[:, None])
                v = self.v[s][:, h // (self.n_q // self.n_kv)]
                ref, mass = p @ v, p @ v.abs()
                rel = 2 * ds + 2.0 ** -12
                if not rows_kernel:
                    rel += 2.0 ** -8
                elif self.fp8:
                    rel += 2.0 ** -11
                tol = 2.0 ** -8 * ref.abs() + rel * mass + (p.shape[1] * 2.0 ** -25 * vmax if self.fp8 else 0)
                err = (out[rows, h] - ref).abs()
                assert bool((err <= tol).all()), (s, h, float((err - tol).max()))
                el = (lse[h, rows] - ref_lse).abs()
                assert bool((el <= ds + 2.0 ** -12 + 2.0 ** -21 * ref_lse.abs()).all()), (s, h, float(el.max()))

    def check_weights(self, decay=1.0, lse=None, **kw):
        """Runs attention_weights on the exact lse (rounded to fp32) and compares every entry."""
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        ref_lse = torch.zeros(self.n_q, self.T, dtype=torch.float64)
        for s in range(self.P):
            for h in range(self.n_q):
                if self.new[s]:
                    ref_lse[h, self.cu[s]:self.cu[s + 1]] = torch.logsumexp(self.logits(s, h)[0], 1)
        lse = ref_lse.float()
        g = torch.Generator().manual_seed(9)
        old = torch.randn(self.total, self.n_kv, 16, generator=g)
        scores = old.clone().cuda()
        api.attention_weights(self.model, self.q.cuda(), lse.cuda(), self.cu, self.ctx, self.kv, scores, cache=self.cache,
                              window=self.window, sinks=self.sinks, decay=decay, **kw)
        torch.cuda.synchronize()
        assert self.model.status() == 0
        got = scores.cpu()
        ref, tol = old.double(), torch.zeros(old.shape, dtype=torch.float64)
        G = self.n_q // self.n_kv
        for s in range(self.P):
            if not self.new[s]:
                continue
            idx = np.flatnonzero(self.seen[s])
            pg, sl = self.table[s][torch.from_numpy(idx // 16)].long(), torch.from_numpy(idx % 16)
            i = torch.from_numpy(idx)
            for kh in range(self.n_kv):
                w, t = torch.zeros(len(idx), dtype=torch.float64), torch.zeros(len(idx), dtype=torch.float64)
                for h in range(kh * G, kh * G + G):
                    z, ds = self.logits(s, h)
                    l = lse[h, self.cu[s]:self.cu[s + 1]].double()[:, None]
                    p = torch.exp(z - l)[:, i]
                    # a score's error, the exponent's roundings (|z|, |lse| times 2^-22), and the sums
                    rel = ds + 2.0 ** -22 * (z.masked_fill(z == -math.inf, 0).abs() + l.abs())[:, i] + 2.0 ** -12
                    w += p.sum(0)
                    t += (p * rel).sum(0)
                ref[pg, kh, sl] = decay * old[pg, kh, sl].double() + w
                tol[pg, kh, sl] = t + 2.0 ** -22 * (abs(decay) * old[pg, kh, sl].double().abs() + w)
        err = (got.double() - ref).abs()
        assert bool((err <= tol).all()), float((err - tol).max())


BATCHES = [
    ([1], [0]), ([1], [37]), ([1, 1, 1], [15, 16, 17]), ([4, 2, 3], [100, 0, 31]), ([5], [0]), ([5, 1, 130], [3, 200, 0]),
    ([128], [0]), ([129], [16]), ([257, 0, 64, 1], [40, 12, 0, 700]), ([300], [333]), ([1, 600], [1500, 0]),
]
WINDOWS = [(0, 0), (1, 0), (1, 3), (7, 1), (16, 4), (64, 0), (100, 20), (129, 70), (2000, 4), (30, 10 ** 9)]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("heads", list(HEADS))
def test_attend_ragged_batches(heads, fp8):
    for i, (new, ctx) in enumerate(BATCHES):
        c = Case(heads, new, ctx, fp8=fp8, seed=i)
        c.check_attend(*c.attend())


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("heads,fp8", [("gqa4", False), ("gqa5", False), ("d64", False), ("gqa4", True), ("mha", True),
                                       ("d64", True)])
def test_attend_window_and_sinks(heads, fp8, window, sinks):
    for i, (new, ctx) in enumerate([([1, 1, 3], [0, 250, 90]), ([260, 5], [33, 400]), ([70, 300], [0, 500])]):
        c = Case(heads, new, ctx, window, sinks, fp8, seed=10 + i)
        c.check_attend(*c.attend())


@pytest.mark.gpu
def test_attend_large_scores():
    """Sharp softmaxes: scores of +-100 and a running maximum that moves often."""
    for new, ctx in (([1, 3], [300, 64]), ([200], [100])):
        for fp8 in (False, True):
            c = Case("gqa4", new, ctx, 150, 2, fp8, seed=3, scale=3.0)
            c.check_attend(*c.attend())


@pytest.mark.gpu
@pytest.mark.parametrize("heads", ["gqa4", "d64"])
@pytest.mark.parametrize("ramp", [(-500, -500), (-500, 0), (0, 500), (500, -500), (-900, 900), (300, 300)])
def test_attend_scores_far_from_zero(ramp, heads):
    """Weights that would underflow or overflow against any maximum but the row's own, and maxima that
    rise by more than a block's range from one block to the next or fall after the first."""
    for new, ctx in (([1, 3], [300, 64]), ([200, 5], [100, 400])):
        for fp8, window in ((False, 0), (False, 150), (True, 0), (True, 90)):
            c = Case(heads, new, ctx, window, 2, fp8, seed=4, ramp=ramp)
            out, lse = c.attend()
            c.check_attend(out, lse)


@pytest.mark.gpu
def test_attend_does_not_follow_the_models_attention_family():
    import torch
    c = Case("gqa4", [130, 1, 70], [50, 90, 0], 60, 5, seed=4)
    ref = c.attend()
    for impl in (1, 2):
        B.check(B.lib().swiftkv_set_attention_impl(c.model.handle, impl))
        assert all(torch.equal(a, b) for a, b in zip(ref, c.attend()))


@pytest.mark.gpu
def test_attend_strided_rows_and_other_stream():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case("gqa4", [140, 1], [20, 70], 64, 4, seed=5)
    ref, _ = c.attend()
    wide = torch.zeros(c.T, c.n_q + 3, c.d, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:1 + c.n_q] = c.q.cuda()
    out = torch.full((c.T, c.n_q + 2, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    api.attend(c.model, wide[:, 1:1 + c.n_q], c.cu, c.ctx, c.kv, cache=1, window=64, sinks=4, out=out[:, 2:], stream=st)
    st.synchronize()
    assert bool((out[:, 2:].cpu().double() == ref).all()) and bool((out[:, :2] == 7).all())
    flat = api.attend(c.model, c.q.cuda().view(c.T, -1), c.cu, c.ctx, c.kv, cache=1, window=64, sinks=4)
    assert bool((flat.cpu().double() == ref).all())


@pytest.mark.gpu
def test_attend_tiles_do_not_depend_on_the_batch():
    """A chunk of more than 4 rows gives the same bits alone and next to others (shorter ones are cut
    by the call's total work)."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    for heads in ("gqa4", "gqa5", "d64"):
        a = Case(heads, [130, 1, 9], [64, 333, 10], 100, 4, seed=6)
        out, lse = a.attend()
        for s in (0, 2):
            sl = slice(int(a.cu[s]), int(a.cu[s + 1]))
            one = api.attend(a.model, a.q[sl].cuda(), [0, a.new[s]], [a.ctx[s]], a.kv.view([s]), cache=1, window=100,
                             sinks=4)
            assert bool((one.cpu().double() == out[sl]).all())


@pytest.mark.gpu
def test_attend_repeats_its_bits():
    c = Case("gqa4", [1, 3, 200], [900, 50, 300], 128, 4, seed=16)
    a = c.attend()
    for _ in range(3):
        b = c.attend()
        assert bool((a[0] == b[0]).all()) and bool((a[1] == b[1]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("heads", list(HEADS))
def test_weights_ragged_batches(heads, fp8):
    for i, (new, ctx) in enumerate(BATCHES):
        Case(heads, new, ctx, fp8=fp8, seed=20 + i).check_weights(decay=(1.0, 0.0, 0.5)[i % 3])


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("heads,fp8", [("gqa4", False), ("gqa5", True), ("d64", False)])
def test_weights_window_and_sinks(heads, fp8, window, sinks):
    for i, (new, ctx) in enumerate([([1, 2, 3], [0, 250, 90]), ([260, 5], [33, 400]), ([70, 300], [0, 500])]):
        Case(heads, new, ctx, window, sinks, fp8, seed=30 + i).check_weights(decay=(0.0, 1.0, -0.25)[i])


@pytest.mark.gpu
def test_weights_sum_to_the_number_of_rows():
    """Each row and head hands out a weight of one."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    for new, ctx in (([200, 1], [77, 40]), ([1, 1], [500, 3])):
        c = Case("gqa4", new, ctx, seed=7)
        lse = torch.empty(c.n_q, c.T, device="cuda")
        api.attend(c.model, c.q.cuda(), c.cu, c.ctx, c.kv, cache=1, lse=lse)
        sc = api.attention_weights(c.model, c.q.cuda(), lse, c.cu, c.ctx, c.kv,
                                   torch.zeros(c.total, c.n_kv, 16, device="cuda"), cache=1)
        assert abs(float(sc.double().sum()) - c.T * c.n_q) <= 1e-4 * c.T * c.n_q


@pytest.mark.gpu
def test_status_of_bad_pages():
    """A needed entry outside the pool sets the status and faults nothing; one that is not needed is
    not looked at (every Case has those)."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    for heads in ("gqa4", "d64"):
        for new in (200, 1):
            for fp8 in (False, True):
                c = Case(heads, [new], [100], fp8=fp8, seed=8)
                c.kv.block_table[0, 2] = 10 ** 6
                lse = torch.zeros(c.n_q, c.T, device="cuda")
                api.attend(c.model, c.q.cuda(), c.cu, c.ctx, c.kv, cache=1, lse=lse)
                torch.cuda.synchronize()
                assert c.model.status() == B.STATUS_BAD_PAGE
                sc = torch.zeros(c.total, c.n_kv, 16, device="cuda")
                api.attention_weights(c.model, c.q.cuda(), torch.zeros_like(lse), c.cu, c.ctx, c.kv, sc, cache=1)
                torch.cuda.synchronize()
                assert c.model.status() == B.STATUS_BAD_PAGE


@pytest.mark.gpu
def test_capture_replays_on_new_values():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case("gqa4", [1, 1, 40], [90, 300, 10], 64, 4, seed=11)
    q = c.q.cuda()
    lse = torch.empty(c.n_q, c.T, device="cuda")
    out = torch.empty_like(q)
    sc = torch.zeros(c.total, c.n_kv, 16, device="cuda")

    def step():
        api.attend(c.model, q, c.cu, c.ctx, c.kv, cache=1, window=64, sinks=4, out=out, lse=lse)
        api.attention_weights(c.model, q, lse, c.cu, c.ctx, c.kv, sc, cache=1, window=64, sinks=4, decay=0.0)

    fresh = model_of("gqa4")
    g = torch.cuda.CUDAGraph()
    with pytest.raises(B.SwiftKVError) as e:  # its workspace would have to grow inside the capture
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            api.attend(fresh, q, c.cu, c.ctx, c.kv, cache=1, out=out)
    assert e.value.code == -10
    step()
    with torch.cuda.graph(g):
        step()
    # a larger call grows the workspace; the graph still replays on its own
    big = Case("gqa4", [700], [900], seed=12)
    api.attend(c.model, big.q.cuda(), big.cu, big.ctx, big.kv, cache=1)
    for seed in (1, 2):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(seed)).bfloat16())
        g.replay()
        torch.cuda.synchronize()
        got = (out.clone(), lse.clone(), sc.clone())
        step()
        torch.cuda.synchronize()
        assert all(bool((a == b).all()) for a, b in zip(got, (out, lse, sc)))


@pytest.mark.gpu
def test_two_graphs_share_a_workspace():
    """Graphs of different batches, captured on one model, replayed in turn on one stream."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    cases = [Case("gqa4", [1, 200], [90, 10], 64, 4, seed=21), Case("gqa4", [150, 3, 6], [700, 30, 1], seed=22)]
    model, calls = cases[0].model, []
    for c in cases:
        q = c.q.cuda()
        lse, sc = torch.empty(c.n_q, c.T, device="cuda"), torch.zeros(c.total, c.n_kv, 16, device="cuda")
        out = torch.empty_like(q)

        def call(c=c, q=q, lse=lse, sc=sc, out=out):
            api.attend(model, q, c.cu, c.ctx, c.kv, cache=1, window=c.window, sinks=c.sinks, out=out, lse=lse)
            api.attention_weights(model, q, lse, c.cu, c.ctx, c.kv, sc, cache=1, window=c.window, sinks=c.sinks, decay=0.0)

        call()
        torch.cuda.synchronize()
        calls.append((call, (out, lse, sc), [t.clone() for t in (out, lse, sc)]))
    graphs = []
    for call, _, _ in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for _, got, _ in calls:
        for t in got:
            t.zero_()
    for i in (0, 1, 0, 1, 1, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        _, got, ref = calls[i]
        assert all(bool((a == b).all()) for a, b in zip(got, ref))
        got[0].zero_()
    assert model.status() == 0


@pytest.mark.gpu
def test_pages_far_into_the_pool():
    """Elements past 2^32 of a pool: the same bits as in a pool of a few pages."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    model = model_of("gqa8", 1)
    n_q, n_kv, d = HEADS["gqa8"]
    new, ctx, keep = [1, 3, 140], [90, 400, 33], 30
    cu, lens = np.concatenate([[0], np.cumsum(new)]), [a + b for a, b in zip(new, ctx)]
    pages = [(n + 15) // 16 for n in lens]
    table = np.zeros((3, max(pages)), np.int32)
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = at + np.arange(n)
        at += n
    dst = at + np.arange(3 * 2, dtype=np.int32).reshape(3, 2)
    base = (1 << 32) // (n_kv * 16 * d)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(at + 6, n_kv, 16, d, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(int(cu[-1]), n_q, d, generator=g).bfloat16().cuda()
    results = []
    for first in (0, base):
        kv = api.KVCache(model, first + at + 6, table + first)
        kv.k[0, first:], kv.v[0, first:] = k.cuda(), v.cuda()
        lse, sc = torch.empty(n_q, int(cu[-1]), device="cuda"), kv.new_scores()
        out = api.attend(model, q, cu, ctx, kv, window=100, sinks=4, lse=lse)
        api.attention_weights(model, q, lse, cu, ctx, kv, sc[0], window=100, sinks=4)
        to = torch.as_tensor(dst + first, device="cuda", dtype=torch.int32)
        kept = api.evict(model, kv, sc, lens, keep, sinks=2, recent=5, dst_block_table=to)
        moved = [t[0, first:].clone() for t in (kv.k, kv.v, sc)]
        api.evict(model, kv, sc, lens, keep, sinks=2, recent=5)
        results.append([out, lse, kept] + moved + [t[0, first:].clone() for t in (kv.k, kv.v, sc)])
        assert model.status() == 0
        del kv, sc
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_captured_eviction_replays_on_new_scores():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = EvictCase("gqa4", [200, 40], 32, 2, 8, seed=4)
    sc, dst = torch.rand_like(c.kv.new_scores()), c.dst.cuda()
    kept = torch.empty(2, 2, c.n_kv, 32, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.evict(c.model, c.kv, sc, [200, 40], 32, sinks=2, recent=8, dst_block_table=dst, kept=kept)
    for seed in (1, 2):
        sc.copy_(torch.rand(sc.shape, generator=torch.Generator().manual_seed(seed)))
        before = sc.clone()
        g.replay()
        torch.cuda.synchronize()
        got = kept.clone()
        sc.copy_(before)
        ref = api.evict(c.model, c.kv, sc, [200, 40], 32, sinks=2, recent=8, dst_block_table=dst)
        assert torch.equal(got, ref)


# ---------------------------------------------------------------- eviction

def kept_ref(score, n, keep, sinks, recent):
    if n <= keep:
        return np.concatenate([np.arange(n), np.full(keep - n, -1)])
    j = np.arange(n)
    held = (j < sinks) | (j >= n - recent)
    s = np.where(np.isnan(score), -np.inf, score.astype(np.float64))
    nan_last = np.where(np.isnan(score), 1, 0)
    others = j[~held]
    order = others[np.lexsort((others, -s[others], nan_last[others]))]
    return np.sort(np.concatenate([j[held], order[:keep - held.sum()]]))


class EvictCase:
    def __init__(self, heads, lens, keep, sinks, recent, fp8=False, caches=2, seed=0, ties=False, extra=True):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        self.n_q, self.n_kv, self.d = HEADS[heads]
        self.lens, self.keep, self.sinks, self.recent, self.fp8 = lens, keep, sinks, recent, fp8
        self.model = model_of(heads, caches)
        g = torch.Generator().manual_seed(seed)
        need = [(n + 15) // 16 for n in lens]
        dw = (keep + 15) // 16
        total = sum(need) + len(lens) * dw + 3
        perm = torch.randperm(total, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), max(max(need), 1) + 1), -1, dtype=torch.int32)
        first = 0
        for s, m in enumerate(need):
            self.table[s, :m] = perm[first:first + m]
            first += m
        self.dst = perm[first:first + len(lens) * dw].view(len(lens), dw).clone()
        self.kv = api.KVCache(self.model, total, self.table.numpy(), dtype="fp8" if fp8 else "bf16")
        dev = torch.Generator(device="cuda").manual_seed(seed)
        pools = [self.kv.k, self.kv.v] + ([self.kv.k_scale, self.kv.v_scale] if fp8 else [])
        for p in pools:
            if p.dtype == torch.uint8:
                p.copy_(torch.randint(0, 256, p.shape, device="cuda", generator=dev, dtype=torch.uint8))
            else:
                p.normal_(generator=dev)
        self.scores = torch.empty(caches, total, self.n_kv, 16, device="cuda").normal_(generator=dev)
        if ties:
            self.scores = (self.scores * 1.5).round()
            self.scores[0, :, :, 3] = float("nan")
            self.scores[-1, :, 0, 5] = float("inf")
            self.scores[-1, :, 0, 7] = -float("inf")
            self.scores[0, :, :, 9] = -0.0
        self.pools = pools + [self.scores]
        self.caches = caches

    def expected(self, before, inplace, only):
        """Pools and kept after the call."""
        import torch
        after = [p.clone() for p in before]
        kept = np.full((1 if only is not None else self.caches, len(self.lens), self.n_kv, self.keep), -1, np.int32)
        sc = before[-1].cpu().numpy()
        table, dst = self.table.numpy(), (self.table if inplace else self.dst).numpy()
        for ci, c in enumerate(range(self.caches) if only is None else [only]):
            for s, n in enumerate(self.lens):
                j = np.arange(n)
                for h in range(self.n_kv):
                    row = sc[c, table[s, j // 16], h, j % 16] if n else np.zeros(0, np.float32)
                    ids = kept_ref(row, n, self.keep, self.sinks, self.recent)
                    kept[ci, s, h] = ids
                    ids = ids[ids >= 0]
                    i = np.arange(len(ids))
                    src = (c, torch.as_tensor(table[s, ids // 16]).long(), h, torch.as_tensor(ids % 16))
                    to = (c, torch.as_tensor(dst[s, i // 16]).long(), h, torch.as_tensor(i % 16))
                    for p, q in zip(after, before):
                        p[to] = q[src]
        return after, kept

    def run(self, inplace, only=None):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        before = [p.clone() for p in self.pools]
        after, kept = self.expected([b.cpu() for b in before], inplace, only)
        scores = self.scores if only is None else self.scores[only]
        got = api.evict(self.model, self.kv, scores, self.lens, self.keep, self.sinks, self.recent, cache=only,
                        dst_block_table=None if inplace else self.dst.cuda())
        torch.cuda.synchronize()
        assert self.model.status() == 0
        assert np.array_equal(got.cpu().numpy(), kept)
        for p, q in zip(self.pools, after):
            assert torch.equal(torch.nan_to_num(p.float(), 123.0).cpu(), torch.nan_to_num(q.float(), 123.0))


@pytest.mark.gpu
@pytest.mark.parametrize("inplace", [True, False], ids=["inplace", "moved"])
@pytest.mark.parametrize("heads,fp8", [("gqa4", False), ("d64", False), ("gqa5", True), ("d64_mha", True)])
@pytest.mark.parametrize("lens,keep,sinks,recent", [
    ([1], 1, 0, 0), ([0, 5, 17], 4, 1, 1), ([100, 33, 16, 7], 16, 4, 12), ([700, 1500, 2], 333, 4, 64),
    ([513, 512, 511], 512, 0, 0), ([2000], 1999, 0, 1), ([3000, 64], 1, 0, 0), ([900], 128, 0, 128), ([40], 64, 30, 30)])
def test_evict(heads, fp8, lens, keep, sinks, recent, inplace):
    EvictCase(heads, lens, keep, sinks, recent, fp8, seed=keep).run(inplace)


@pytest.mark.gpu
@pytest.mark.parametrize("inplace", [True, False], ids=["inplace", "moved"])
def test_evict_ties_and_non_finite_scores(inplace):
    for keep in (1, 40, 500, 1100):
        EvictCase("gqa4", [1200, 300, 90], keep, 0, 0, ties=True, caches=3, seed=keep).run(inplace)
        EvictCase("gqa4", [1200, 300, 90], keep, min(keep, 3) // 2, min(keep, 20) // 2, ties=True, seed=keep).run(inplace)


@pytest.mark.gpu
def test_evict_one_cache_and_long_lists():
    EvictCase("gqa4", [900, 500], 100, 4, 16, caches=3, seed=1).run(True, only=1)
    EvictCase("gqa4", [900, 500], 100, 4, 16, caches=3, seed=2).run(False, only=2)
    # longer than the list that fits shared memory
    EvictCase("d64", [50001, 49153, 60], 7000, 4, 100, caches=1, seed=3).run(True)
    EvictCase("d64", [50001], 49990, 4, 100, caches=1, seed=4, ties=True).run(False)


@pytest.mark.gpu
def test_evict_bad_pages_leave_the_sequence_alone():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    for inplace in (True, False):
        c = EvictCase("gqa4", [100, 200], 32, 0, 0, seed=5)
        c.kv.block_table[0, 3] = -1
        before = [p.clone() for p in c.pools]
        kept = api.evict(c.model, c.kv, c.scores, c.lens, 32, dst_block_table=None if inplace else c.dst.cuda())
        torch.cuda.synchronize()
        assert c.model.status() == B.STATUS_BAD_PAGE
        assert bool((kept[:, 0] == -1).all()) and bool((kept[:, 1] >= 0).all())
        mine = torch.cat([c.table[0, :7], c.dst[0]]).long()
        mine = mine[mine >= 0]
        for p, q in zip(c.pools, before):
            assert torch.equal(p[:, mine], q[:, mine])


@pytest.mark.gpu
def test_refusals_on_the_gpu():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case("gqa4", [3, 40], [10, 20], seed=1)
    q = c.q.cuda()
    bad = [dict(window=-1), dict(sinks=-1), dict(cache=2), dict(cache=-1), dict(out=q)]
    for kw in bad:
        with pytest.raises(B.SwiftKVError):
            api.attend(c.model, q, c.cu, c.ctx, c.kv, **kw)
    with pytest.raises(B.SwiftKVError):
        api.attend(c.model, q, [1, 3, 43], c.ctx, c.kv)
    with pytest.raises(B.SwiftKVError):
        api.attend(c.model, q, [0, 50, 43], c.ctx, c.kv)
    with pytest.raises(B.SwiftKVError):
        api.attend(c.model, q, c.cu, [10, 10 ** 6], c.kv)
    for bad_q in (q.float(), q.cpu(), q[:5], q[:, :3], q.transpose(0, 1)):
        with pytest.raises(ValueError):
            api.attend(c.model, bad_q, c.cu, c.ctx, c.kv)
    with pytest.raises(ValueError):
        api.attend(c.model, q, c.cu, c.ctx, c.kv, lse=torch.empty(3, 3, device="cuda"))
    with pytest.raises(ValueError):
        api.attend(c.model, q, [0] * 4 + [43], None, c.kv)  # more chunks than block-table rows
    with pytest.raises(B.SwiftKVError):  # rows that start off 16 bytes
        buf = torch.zeros(c.T * c.n_q * c.d + 8, dtype=torch.bfloat16, device="cuda")
        api.attend(c.model, buf[1:1 + c.T * c.n_q * c.d].view(c.T, c.n_q, c.d), c.cu, c.ctx, c.kv)
    lse, sc = torch.zeros(c.n_q, c.T, device="cuda"), torch.zeros(c.total, c.n_kv, 16, device="cuda")
    for d in (float("nan"), float("inf")):
        with pytest.raises(B.SwiftKVError):
            api.attention_weights(c.model, q, lse, c.cu, c.ctx, c.kv, sc, decay=d)
    with pytest.raises(ValueError):
        api.attention_weights(c.model, q, lse, c.cu, c.ctx, c.kv, sc[:-1])
    all_sc = torch.zeros(2, c.total, c.n_kv, 16, device="cuda")
    for kw in (dict(keep=0), dict(keep=4, sinks=3, recent=2), dict(keep=4, sinks=-1), dict(keep=4, recent=-1)):
        with pytest.raises((B.SwiftKVError, ValueError)):
            api.evict(c.model, c.kv, all_sc, [13, 60], **kw)
    with pytest.raises(B.SwiftKVError):
        api.evict(c.model, c.kv, all_sc, [13, 10 ** 6], 8)
    with pytest.raises(B.SwiftKVError):
        api.evict(c.model, c.kv, all_sc, [-1, 5], 8)
    with pytest.raises(B.SwiftKVError):  # a destination too narrow
        api.evict(c.model, c.kv, all_sc, [13, 60], 40, dst_block_table=torch.zeros(2, 2, dtype=torch.int32, device="cuda"))
    other = model_of("d64")  # a cache of other heads
    for call in (lambda: api.attend(other, q, c.cu, c.ctx, c.kv),
                 lambda: api.attention_weights(other, q, lse, c.cu, c.ctx, c.kv, sc),
                 lambda: api.evict(other, c.kv, all_sc, [13, 60], 8)):
        with pytest.raises(ValueError, match="a cache of"):
            call()
    torch.cuda.synchronize()
    assert c.model.status() == 0
    assert api.attend(c.model, q[:0], [0], None, c.kv).shape == (0, c.n_q, c.d)
    assert api.attend(c.model, q[:0], [0, 0, 0], [5, 7], c.kv).shape == (0, c.n_q, c.d)


def test_refusals_without_a_gpu():
    lib = B.lib()
    fake = C.c_void_p(256)  # never dereferenced: a null model is refused first
    kv = B.KVPages()
    assert lib.swiftkv_attend(None, 0, fake, 128, fake, None, 1, C.byref(kv), 0, 0, fake, 128, None, None) == -1
    assert lib.swiftkv_attention_weights(None, 0, fake, 128, fake, fake, None, 1, C.byref(kv), 0, 0, 1.0, fake, None) == -1
    assert lib.swiftkv_evict(None, 0, C.byref(kv), None, fake, 1, 4, 0, 0, None, 0, fake, None) == -1
    assert b"null model" in lib.swiftkv_last_error()
