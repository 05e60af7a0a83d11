"""swiftkv_adjust_logits against its definition in 64 bits, and swiftkv_sample behind it.

Tolerance: the logit times or over the repetition penalty, the product of frequency and count, and three sums, each
rounded to float32: 4 half steps (2^-24) of the sum of the terms' sizes. Ids that nothing concerns keep their bits."""
import ctypes as C

import numpy as np
import pytest

from swiftkv_prefill_skipping_gb300 import binding as B


class Case:
    def __init__(self, rows, vocab, hist=0, bias=0, mask=None, seed=0, settings=None, pad=0, offset=0):
        """pad: further columns of the buffer the logits are a part of, offset: of its first ones not theirs."""
        import torch
        g = torch.Generator().manual_seed(seed)
        self.R, self.V = rows, vocab
        self.wide = torch.randn(rows, vocab + pad, generator=g) * 4
        self.offset = offset
        self.logits = self.wide[:, offset:offset + vocab]
        self.kw = {}
        if hist:
            t = torch.randint(0, max(1, min(vocab, 3 * hist // 2)), (rows, hist), generator=g)
            t[:, 1::7] = torch.randint(0, vocab, t[:, 1::7].shape, generator=g)
            t[torch.rand(t.shape, generator=g) < 0.05] = -1
            t[torch.rand(t.shape, generator=g) < 0.05] = vocab
            t[torch.rand(t.shape, generator=g) < 0.02] = 2 ** 31 - 1
            lens = torch.randint(0, hist + 1, (rows,), generator=g)
            lens[0] = hist
            self.kw.update(tokens=t.int(), lens=lens.int(), prompt_lens=(lens // 3).int())
            f = torch.rand(3, rows, generator=g)
            s = settings or dict(repetition=0.7 + f[0], presence=f[1] - 0.3, frequency=f[2] - 0.5)
            self.kw.update(s)
        if bias:
            ids = torch.randint(0, vocab, (rows, bias), generator=g)
            ids[torch.rand(ids.shape, generator=g) < 0.2] = -1
            ids[torch.rand(ids.shape, generator=g) < 0.05] = vocab
            self.kw.update(bias_ids=ids.int(), bias=torch.randn(rows, bias, generator=g) * 5)
        if mask is not None:
            keep = torch.rand(rows, (vocab + 31) // 32 * 32, generator=g) < mask
            keep[0] = False  # a row without any
            w = np.packbits(keep.numpy(), axis=1, bitorder="little").view(np.int32)
            self.kw["mask"] = torch.from_numpy(w.copy())

    def run(self, **kw):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        self.buf = self.wide.cuda()
        x = self.buf[:, self.offset:self.offset + self.V]
        args = {k: v.cuda() if hasattr(v, "cuda") else v for k, v in self.kw.items()}
        args.update(kw)
        if args.get("out") == "in place":
            args["out"] = x
        out = api.adjust_logits(x, **args)
        torch.cuda.synchronize()
        return out.cpu().numpy()

    def check(self, got):
        import torch
        x = self.logits.double().numpy()
        tol = np.zeros_like(x)
        per = {}
        for name, off in (("repetition", 1.0), ("presence", 0.0), ("frequency", 0.0)):
            v = self.kw.get(name, off)
            v = v.numpy() if hasattr(v, "numpy") else np.full(self.R, v, np.float32)
            per[name] = v.astype(np.float64)
        for r in range(self.R):
            size = np.zeros(self.V)
            if "tokens" in self.kw:
                n = int(self.kw["lens"][r]) if "lens" in self.kw else self.kw["tokens"].shape[1]
                n = min(max(n, 0), self.kw["tokens"].shape[1])
                t = self.kw["tokens"][r, :n].numpy()
                a = int(self.kw["prompt_lens"][r]) if "prompt_lens" in self.kw else 0
                ok = (t >= 0) & (t < self.V)
                seen = np.unique(t[ok])
                rep = per["repetition"][r] if per["repetition"][r] > 0 else 1.0
                with np.errstate(all="ignore"):
                    x[r, seen] = np.where(x[r, seen] > 0, x[r, seen] / rep, x[r, seen] * rep)
                size[seen] += np.abs(x[r, seen])
                ids, c = np.unique(t[(np.arange(n) >= a) & ok], return_counts=True)
                x[r, ids] -= per["frequency"][r] * c + per["presence"][r]
                size[ids] += np.abs(per["frequency"][r]) * c + np.abs(per["presence"][r])
            if "bias" in self.kw:
                last = {int(i): float(b) for i, b in zip(self.kw["bias_ids"][r], self.kw["bias"][r]) if 0 <= i < self.V}
                for i, b in last.items():
                    size[i] += abs(x[r, i]) + abs(b)
                    x[r, i] += b
            tol[r] = 4 * 2.0 ** -24 * size
            if "mask" in self.kw:
                bits = np.unpackbits(self.kw["mask"][r].numpy().view(np.uint8), bitorder="little")[:self.V]
                x[r, bits == 0] = -np.inf
        same = np.isnan(x) | np.isinf(x)
        assert np.array_equal(got[same], x[same], equal_nan=True)
        err = np.abs(got.astype(np.float64) - np.where(same, got, x))[~same]
        assert (err <= tol[~same]).all(), float((err - tol[~same]).max())


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 1000, 2048, 4097, 32000, 128256, 151669])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_everything_at_once(rows, vocab):
    for seed, (hist, bias, mask) in enumerate([(50, 7, 0.5), (700, 0, None), (0, 40, 0.9), (0, 0, 0.3), (3, 1, None)]):
        c = Case(rows, vocab, hist, bias, mask, seed=seed)
        c.check(c.run())
        c.check(c.run(out="in place"))


@pytest.mark.gpu
@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (4, 4), (7, 2), (8, 4)])
def test_rows_of_a_wider_buffer(pad, offset):
    """Alignments of rows and of the output; what lies beside the rows stays."""
    import torch
    for rows, vocab in ((3, 4099), (130, 70001)):
        c = Case(rows, vocab, 60, 5, 0.7, seed=1, pad=pad, offset=offset)
        c.check(c.run())
        c.check(c.run(out="in place"))
        beside = torch.ones(vocab + pad, dtype=torch.bool)
        beside[offset:offset + vocab] = False
        assert torch.equal(c.buf.cpu()[:, beside], c.wide[:, beside])
        out = torch.full((rows, vocab + 5), 7.0, device="cuda")
        c.check(c.run(out=out[:, 1:1 + vocab]))
        assert bool((out[:, 0] == 7).all()) and bool((out[:, 1 + vocab:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("vocab,gap", [(4099, 0), (4100, 0), (70001, 3)])
def test_out_beside_the_logits_in_wider_rows(vocab, gap):
    """Logits and results as parts of the same rows: apart from each other, though their ranges are not."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case(5, vocab, 60, 5, 0.7, seed=3)
    args = {k: v.cuda() for k, v in c.kw.items()}
    for x_at, out_at in ((0, vocab + gap), (vocab + gap, 0)):
        wide = torch.full((5, 2 * vocab + gap), 7.0, device="cuda")
        x, out = wide[:, x_at:x_at + vocab], wide[:, out_at:out_at + vocab]
        x.copy_(c.logits)
        c.check(api.adjust_logits(x, out=out, **args).cpu().numpy())
        assert torch.equal(x.cpu(), c.logits) and bool((wide[:, vocab:vocab + gap] == 7).all())
        with pytest.raises(B.SwiftKVError, match="overlaps"):
            api.adjust_logits(x, out=wide[:, gap + 1:gap + 1 + vocab], **args)


@pytest.mark.gpu
@pytest.mark.parametrize("first,more", [(0, 1), (1, 3), (4, 4), (3, 1)])
def test_lists_that_are_parts_of_wider_ones(first, more):
    """Histories and masks whose rows start anywhere and have other words before and behind them."""
    import torch
    for rows, vocab, hist in ((3, 5000, 70), (50, 40000, 2100)):
        c = Case(rows, vocab, hist, 0, 0.6, seed=9)
        kw = {}
        for name, fill in (("tokens", 17), ("mask", -1)):
            t = c.kw[name]
            wide = torch.full((rows, t.shape[1] + first + more), fill, dtype=torch.int32)
            wide[:, first:first + t.shape[1]] = t
            kw[name] = wide.cuda()[:, first:first + t.shape[1]]
        c.check(c.run(**kw))
        c.check(c.run(out="in place", **kw))


@pytest.mark.gpu
def test_many_rows_and_long_histories():
    for rows, vocab, hist, bias in ((300, 32000, 90, 3), (70, 151669, 5000, 2046), (2, 128256, 200000, 0), (1, 700000, 100, 9)):
        c = Case(rows, vocab, hist, bias, 0.6, seed=2)
        c.check(c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("hist", [32766, 32767, 32768, 70000])
def test_one_id_throughout_a_history(hist):
    """The largest counts, beside neighbours in the prompt alone, in both, and in none, on even and odd ids."""
    import torch
    for rows, vocab in ((2, 301), (80, 40000)):
        c = Case(rows, vocab, hist, mask=0.9, seed=8)
        t = c.kw["tokens"]
        for r in range(rows):
            t[r, :] = 4 + r % 2
            c.kw["prompt_lens"][r] = 0
        t[1, :3], c.kw["prompt_lens"][1] = torch.tensor([4, 6, 5]), 3
        c.kw["lens"][:] = hist
        c.check(c.run())
        c.check(c.run(out="in place"))


@pytest.mark.gpu
def test_settings_that_are_off_and_lengths_out_of_range():
    import torch
    nan = float("nan")
    for s in (dict(repetition=1.0, presence=0.0, frequency=0.0), dict(repetition=0.0, presence=0.5, frequency=0.0),
              dict(repetition=-2.0), dict(repetition=nan, frequency=0.25), dict(presence=-1.5),
              dict(repetition=torch.tensor([nan, 0.0, -1.0, 1.5]))):
        c = Case(4, 5000, 80, seed=3, settings=s)
        c.check(c.run())
    c = Case(4, 5000, 80, seed=4)
    c.kw["lens"] = torch.tensor([-5, 1000, 80, 0], dtype=torch.int32)
    c.kw["prompt_lens"] = torch.tensor([0, 1000, -3, 7], dtype=torch.int32)
    c.check(c.run())
    del c.kw["lens"], c.kw["prompt_lens"]
    c.check(c.run())


@pytest.mark.gpu
def test_logits_that_are_not_finite():
    import torch
    c = Case(5, 4000, 300, 20, 0.8, seed=5)
    c.logits[:, ::5] = float("-inf")
    c.logits[:, 1::50] = float("inf")
    c.logits[:, 2::50] = float("nan")
    c.check(c.run())
    c.check(c.run(out="in place"))


@pytest.mark.gpu
def test_nothing_to_change_keeps_the_bits():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    x = torch.randn(9, 5003, device="cuda")
    assert torch.equal(api.adjust_logits(x), x)
    t = torch.zeros(9, 0, dtype=torch.int32, device="cuda")
    assert torch.equal(api.adjust_logits(x, tokens=t, repetition=2.0), x)
    e = torch.zeros(9, 0, device="cuda")
    assert torch.equal(api.adjust_logits(x, bias_ids=e.int(), bias=e), x)
    assert api.adjust_logits(x[:0]).shape == (0, 5003)


@pytest.mark.gpu
def test_captured_replays_read_the_lengths_anew():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case(6, 50000, 400, 10, 0.5, seed=6)
    x = c.logits.contiguous().cuda()
    kw = {k: v.cuda() for k, v in c.kw.items()}
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.adjust_logits(x, out=out, **kw)
    for lens in ([400] * 6, [0, 1, 2, 3, 4, 5], [399, 100, 7, 0, 250, 1]):
        c.kw["lens"] = torch.tensor(lens, dtype=torch.int32)
        kw["lens"].copy_(c.kw["lens"])
        graph.replay()
        torch.cuda.synchronize()
        c.check(out.cpu().numpy())


@pytest.mark.gpu
def test_on_two_streams_and_sampled():
    """Masked rows sample an allowed id; a row that allows nothing gives id 0."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    cases = [Case(8, 30000, 100, 4, 0.01, seed=s) for s in (7, 8)]
    streams = [torch.cuda.Stream() for _ in cases]
    data = [(c.logits.contiguous().cuda(), {k: v.cuda() for k, v in c.kw.items()}) for c in cases]
    u = torch.rand(8, device="cuda")
    torch.cuda.synchronize()
    got = []
    for (x, kw), st in zip(data, streams):
        y = api.adjust_logits(x, stream=st, **kw)
        got.append((y, api.sample(y, u, top_p=0.9, stream=st)))
    torch.cuda.synchronize()
    for c, (y, token) in zip(cases, got):
        c.check(y.cpu().numpy())
        token = token.cpu()
        assert int(token[0]) == 0
        for r in range(1, 8):
            i = int(token[r])
            assert int(c.kw["mask"][r, i // 32]) >> (i % 32) & 1


@pytest.mark.gpu
def test_refusals():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    x = torch.zeros(4, 100, device="cuda")
    i, f = torch.zeros(4, 7, dtype=torch.int32, device="cuda"), torch.zeros(4, 7, device="cuda")

    def refused(what, *a, **kw):
        with pytest.raises((ValueError, B.SwiftKVError), match=what):
            api.adjust_logits(*a, **kw)

    refused("logits", x.half())
    refused("logits", x.t())
    refused("tokens", x, tokens=i.long())
    refused("tokens", x, tokens=i[:3])
    refused("lens", x, tokens=i, lens=i[:, 0])
    refused("belong to tokens", x, lens=i[0, :4].contiguous())
    refused("repetition", x, tokens=i, repetition=f[:, :4])
    refused("go together", x, bias=f)
    refused("bias_ids", x, bias=f, bias_ids=i[:, :6].contiguous())
    refused("mask", x, mask=i[:, :3])
    refused("mask", x, mask=i[:, :4].float())
    refused("out", x, out=x[:, :99])
    refused("overlaps", x[:, :90], out=x[:, 10:])
    refused("EUNSUPPORTED", x, tokens=torch.zeros(4, 1 << 20, dtype=torch.int32, device="cuda"))
    refused("EUNSUPPORTED", x, bias=torch.zeros(4, 2047, device="cuda"),
            bias_ids=torch.zeros(4, 2047, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("which", ["logits", "out", "tokens", "lens", "prompt_lens", "repetition", "presence", "frequency",
                                   "bias_ids", "bias", "mask"])
def test_misaligned_arrays_are_refused_without_gpu(which):
    a, at = B.Adjustments(), dict(logits=256, out=1 << 40)  # addresses that are never used: refused first
    for name in ("tokens", "lens", "prompt_lens", "repetition", "presence", "frequency", "bias_ids", "bias", "mask"):
        setattr(a, name, 256)
    a.max_tokens = a.ld_tokens = a.num_bias = a.ld_mask = 2000
    a.num_bias = 1 << 20  # refused later on, so that no kernel runs where the check is missing
    if which in at:
        at[which] += 2
    else:
        setattr(a, which, 258)
    lib = B.lib()
    assert lib.swiftkv_adjust_logits(at["logits"], 1, 100, 100, C.byref(a), at["out"], 100, None) == -1
    assert b"misaligned" in lib.swiftkv_last_error()


def test_arguments_without_gpu():
    lib, a = B.lib(), B.Adjustments()
    call = lambda rows=1, V=100, ld=100, out=1 << 40, ldo=100: lib.swiftkv_adjust_logits(256, rows, V, ld, C.byref(a), out, ldo, None)  # noqa: E731
    assert call(rows=0) == 0
    assert call(rows=-1) == -1 and call(V=0) == -1 and call(ld=99) == -1 and call(ldo=99) == -1 and call(out=None) == -1
    assert call(V=(1 << 30) + 1, ld=1 << 31, ldo=1 << 31) == -9 and call(rows=(1 << 27) + 1) == -9
    assert call(out=260) == -1 and b"overlaps" in lib.swiftkv_last_error()
    a.max_tokens = -1
    assert call() == -1
    a.max_tokens = 5
    assert call() == -1 and b"null tokens" in lib.swiftkv_last_error()
    a.tokens, a.ld_tokens, a.max_tokens = 256, 4, 5
    assert call(rows=2) == -1
    a.ld_tokens, a.num_bias = 5, 3
    assert call() == -1 and b"null bias" in lib.swiftkv_last_error()


@pytest.mark.gpu
def test_sizes_past_32_bits_are_refused():
    """Sizes whose low 32 bits would pass."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    big, x = torch.empty(1, (1 << 32) + 4, device="cuda"), torch.zeros(1, 100, device="cuda")
    ids = big.view(torch.int32)
    for a, kw in ((big, {}), (big.view(-1, 1), {}), (x, dict(tokens=ids)), (x, dict(bias_ids=ids, bias=big))):
        with pytest.raises(ValueError, match="32 bits"):
            api.adjust_logits(a, out=x, **kw)
