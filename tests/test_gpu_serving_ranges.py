"""Operators over an FP8 cache where vectors differ widely in size: each key and value vector has a
scale of its own, so two of them may be any factor apart, and no output may depend on that beyond
the roundings of its own terms.

Tolerances, for each element (row i, head h, dimension e) with its own mass M = sum_j p_ij |v_je|:
the scores' errors as in test_gpu_serving (2 ds + 2^-12 of M, ds the bound of a d-term fp32 sum), P's
rounding (2^-8 of M in chunks of more than 4 rows; two bf16 parts, 2^-8 of 2^-8, in shorter ones) and
the output's own rounding to bf16, 2^-8 of its value. Nothing scales with the largest value of the
cache. Weights: as in test_gpu_serving."""
import math

import numpy as np
import pytest

from test_gpu_serving import HEADS, model_of, seen_mask

pytestmark = pytest.mark.gpu


class Fp8Batch:
    """One sequence of n new rows after c0 keys over an FP8 cache. vmul, kmul: a factor for each key's
    vectors; low: keys (indices) that every row scores near -40; zero: (key, dims) of V set to 0.
    peak: a factor for each value vector's first dimension."""

    def __init__(self, heads, n, c0, window=0, sinks=0, vmul=None, kmul=1.0, qmul=1.0, low=(), zero=None, peak=None,
                 seed=0):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        self.n_q, self.n_kv, self.d = HEADS[heads]
        self.n, self.c0, self.window, self.sinks = n, c0, window, sinks
        self.model = model_of(heads, 1)
        g = torch.Generator().manual_seed(seed)
        keys = c0 + n
        pages = (keys + 15) // 16
        perm = torch.randperm(pages + 2, generator=g)[:pages]
        self.kv = api.KVCache(self.model, pages + 2, perm[None].to(torch.int32).numpy(), dtype="fp8")
        k = torch.randn(keys, self.n_kv, self.d, generator=g)
        v = torch.randn(keys, self.n_kv, self.d, generator=g)
        q = torch.randn(n, self.n_q, self.d, generator=g) + 1.0
        if len(low):
            k[list(low)] -= 40.0 / math.sqrt(self.d)  # times q's mean of 1: -40 in the score
        if zero is not None:
            v[zero[0], :, zero[1]] = 0.0
        if peak is not None:
            v[..., 0] *= peak
        if vmul is not None:
            v = v * torch.as_tensor(vmul, dtype=torch.float32)[:, None, None]
        k = k * kmul
        j = torch.arange(keys)
        pg, sl = perm[j // 16], j % 16
        self.ref = {}
        for name, x in (("k", k), ("v", v)):
            sx = x.abs().amax(-1) / 448
            code = (x / sx[..., None]).to(torch.float8_e4m3fn)
            self.ref[name] = code.double() * sx.double()[..., None]
            getattr(self.kv, name).view(torch.float8_e4m3fn)[0, pg.cuda(), :, sl.cuda()] = code.cuda()
            getattr(self.kv, name + "_scale")[0, pg.cuda(), :, sl.cuda()] = sx.cuda()
        self.pg, self.sl, self.pages = pg, sl, pages + 2
        self.q = (q * qmul).bfloat16()
        self.mask = torch.from_numpy(seen_mask(n, c0, window, sinks))

    def logits(self, h):
        k = self.ref["k"][:, h // (self.n_q // self.n_kv)]
        q = self.q[:, h].double()
        z = q @ k.T / math.sqrt(self.d)
        # sum |q_i k_i| where somebody sees the key
        ds = self.d * 2.0 ** -23 * float((q.abs() @ k.abs().T)[self.mask].max()) / math.sqrt(self.d)
        return z.masked_fill(~self.mask, -math.inf), ds

    def check_attend(self):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        lse = torch.full((self.n_q, self.n), float("nan"), device="cuda")
        out = api.attend(self.model, self.q.cuda(), [0, self.n], [self.c0], self.kv, window=self.window,
                         sinks=self.sinks, lse=lse).cpu().double()
        assert self.model.status() == 0
        lse = lse.cpu().double()
        for h in range(self.n_q):
            z, ds = self.logits(h)
            ref_lse = torch.logsumexp(z, 1)
            p = torch.exp(z - ref_lse[:, None])
            v = self.ref["v"][:, h // (self.n_q // self.n_kv)]
            ref, mass = p @ v, p @ v.abs()
            tol = 2.0 ** -8 * ref.abs() + (2 * ds + 2.0 ** -12 + (2.0 ** -16 if self.n <= 4 else 2.0 ** -8)) * mass
            err = (out[:, h] - ref).abs()
            assert bool((err <= tol).all()), (h, float((err / tol).max()))
            assert bool(((lse[h] - ref_lse).abs() <= ds + 2.0 ** -12 + 2.0 ** -21 * ref_lse.abs()).all()), h

    def check_weights(self):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        zs = [self.logits(h) for h in range(self.n_q)]
        lse = torch.stack([torch.logsumexp(z, 1) for z, _ in zs]).float()
        sc = api.attention_weights(self.model, self.q.cuda(), lse.cuda(), [0, self.n], [self.c0], self.kv,
                                   torch.zeros(self.pages, self.n_kv, 16, device="cuda"), window=self.window,
                                   sinks=self.sinks, decay=0.0)
        assert self.model.status() == 0
        got = sc.cpu().double()[self.pg, :, self.sl]
        G = self.n_q // self.n_kv
        for kh in range(self.n_kv):
            ref, tol = 0, 0
            for h in range(kh * G, kh * G + G):
                z, ds = zs[h]
                l = lse[h].double()[:, None]
                p = torch.exp(z - l)
                rel = ds + 2.0 ** -22 * (z.masked_fill(z == -math.inf, 0).abs() + l.abs()) + 2.0 ** -12
                ref, tol = ref + p.sum(0), tol + (p * rel).sum(0)
            err = (got[:, kh] - ref).abs()
            assert bool((err <= tol + 2.0 ** -22 * ref).all()), (kh, float(err.max()))


ROWS = [("gqa4", 1), ("gqa4", 3), ("gqa8", 4), ("d64", 2), ("gqa4", 40), ("d64", 70)]


@pytest.mark.parametrize("heads,n", ROWS)
@pytest.mark.parametrize("span", [3, 6, 30])
def test_value_vectors_of_growing_and_falling_size(heads, n, span):
    for c0 in (200, 3000):
        at = np.arange(c0 + n) / (c0 + n)
        for mul in (10.0 ** (span * at), 10.0 ** (-span * at), 10.0 ** (span * (np.floor(at * 400) % 7 - 3) / 3)):
            Fp8Batch(heads, n, c0, vmul=mul, seed=span).check_attend()


@pytest.mark.parametrize("heads,n", ROWS)
@pytest.mark.parametrize("size", [1e3, 1e5, 1e6, 1e9])
def test_a_large_value_vector_of_negligible_weight(heads, n, size):
    for c0, where in ((300, 0), (300, 150), (300, 299), (4000, 2000), (4000, 4)):
        mul = np.ones(c0 + n)
        mul[where] = size
        Fp8Batch(heads, n, c0, vmul=mul, low=[where], seed=1).check_attend()


@pytest.mark.parametrize("heads,n", ROWS)
def test_a_large_value_vector_with_empty_dimensions(heads, n):
    """Where its dimensions are zero the other keys' values are the whole output."""
    for size in (1e4, 1e8):
        for where in (0, 100):
            mul = np.ones(250 + n)
            mul[where] = size
            Fp8Batch(heads, n, 250, vmul=mul, zero=(where, slice(0, HEADS[heads][2] // 2)), seed=2).check_attend()


@pytest.mark.parametrize("heads,n", [("gqa4", 3), ("gqa8", 4), ("d64", 4), ("gqa4", 60)])
def test_a_large_value_vector_outside_the_window_of_later_rows(heads, n):
    c0, window = 400, 50
    mul = np.ones(c0 + n)
    mul[c0 - window + 1] = 1e7  # the first row's last visible key, hidden from the rows after it
    Fp8Batch(heads, n, c0, window=window, sinks=2, vmul=mul, low=[c0 - window + 1], seed=3).check_attend()


@pytest.mark.parametrize("heads,n", ROWS)
def test_values_far_below_their_vectors_largest(heads, n):
    """One dimension 2^15 times the others: their codes are e4m3's subnormals."""
    for c0 in (30, 1000):
        Fp8Batch(heads, n, c0, peak=2.0 ** 15, seed=7).check_attend()


@pytest.mark.parametrize("heads,n", ROWS)
def test_value_vectors_near_the_ends_of_the_range(heads, n):
    for size in (1e-36, 1e-30, 1e30):
        Fp8Batch(heads, n, 100, vmul=np.full(100 + n, size), seed=4).check_attend()


@pytest.mark.parametrize("heads,n", ROWS)
@pytest.mark.parametrize("power", [20, 60, -30, -60])
def test_queries_of_any_size(heads, n, power):
    """q 2^power times as large and K as much smaller: the same scores."""
    for c0 in (100, 2000):
        Fp8Batch(heads, n, c0, qmul=2.0 ** power, kmul=2.0 ** -power, seed=5).check_attend()


@pytest.mark.parametrize("heads,n", ROWS + [("gqa4", 7)])
@pytest.mark.parametrize("power", [20, 60, -30, -60])
def test_weights_of_queries_of_any_size(heads, n, power):
    for c0 in (100, 2000):
        Fp8Batch(heads, n, c0, qmul=2.0 ** power, kmul=2.0 ** -power, seed=6).check_weights()
