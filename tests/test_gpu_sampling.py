"""swiftkv_sample against the definition in 64 bits: temperature, top-k, top-p and min-p, ties,
masked and non-finite logits, strides and alignments, settings per row and for all rows. The
tokens are whole numbers and have to be equal: the kernel's sums are exact and its weights within
2^-40, so a draw of random inputs comes within that of a border with a probability below 1e-6."""
import ctypes as C

import numpy as np
import pytest

from swiftkv_prefill_skipping_gb300 import binding as B


def ref_token(x, t, k, p, m, u):
    """The definition, one row in float64."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    V, best = len(x), x.max()
    if best == -np.inf:
        return 0
    if not t > 0:
        return int(np.argmax(x))
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == best, 1.0, np.where(x == -np.inf, 0.0, np.exp((x - best) / float(np.float32(t)))))
    order = np.lexsort((np.arange(V), -x))
    if 0 < k < V:
        order = order[:k]
    if p < 1:
        c = np.cumsum(w[order])
        before = c - w[order]
        keep = before < float(np.float32(p)) * c[-1]
        keep[0] = True
        order = order[keep]
    if m > 0:
        order = order[w[order] >= min(float(np.float32(m)), 1.0)]
    ids = np.sort(order)
    c = np.cumsum(w[ids])
    u = float(np.float32(u))
    u = min(max(u, 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    return int(ids[np.searchsorted(c, u * c[-1], side="right")])


def logits_of(rng, R, V, sigma=2.0, spikes=8):
    x = rng.standard_normal((R, V)).astype(np.float32) * np.float32(sigma)
    for r in range(R):
        x[r, rng.integers(0, V, spikes)] += rng.random(spikes).astype(np.float32) * 10
    return x


def run(x, u, t, k, p, m, ld=None, offset=0, scalars=False):
    """api.sample on rows of stride ld that start `offset` floats into an allocation."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    R, V = x.shape
    ld = ld or V
    buf = torch.full((offset + R * ld + 8,), 1e30, device="cuda")  # larger than any logit: must not be read as one
    view = torch.as_strided(buf, (R, V), (ld, 1), offset)
    view.copy_(torch.from_numpy(x))
    f = lambda a, d: torch.from_numpy(np.ascontiguousarray(a)).to(d).cuda()  # noqa: E731
    uu = f(u, torch.float32)
    if scalars:
        return api.sample(view, uu, float(t[0]), int(k[0]), float(p[0]), float(m[0])).cpu().numpy()
    return api.sample(view, uu, f(t, torch.float32), f(k, torch.int32), f(p, torch.float32),
                      f(m, torch.float32)).cpu().numpy()


def check(x, u, t, k, p, m, **kw):
    got = run(x, u, t, k, p, m, **kw)
    ref = [ref_token(x[r], t[r], int(k[r]), p[r], m[r], u[r]) for r in range(len(x))]
    assert got.tolist() == ref


SIZES = [1, 2, 3, 31, 33, 1000, 1024, 4099, 8192, 8193, 16385, 32769, 50257, 128256, 152064]


@pytest.mark.gpu
@pytest.mark.parametrize("V", SIZES)
def test_settings_per_row(V):
    rng = np.random.default_rng(V)
    R = 12 if V > 20000 else 40
    x = logits_of(rng, R, V)
    t = rng.choice([0.0, 0.3, 0.8, 1.0, 1.7], R)
    k = rng.choice([0, 1, 2, 40, 1000, V, V + 5, -3], R)
    p = rng.choice([1.0, 0.999, 0.9, 0.5, 0.01, 0.0, 2.0], R)
    m = rng.choice([0.0, 0.01, 0.2, 1.0, 3.0, -1.0], R)
    check(x, rng.random(R), t, k, p, m)


@pytest.mark.gpu
@pytest.mark.parametrize("t,k,p,m", [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.0, 0, 0.95, 0.0), (1.3, 0, 1.0, 0.05),
                                     (0.9, 64, 0.9, 0.02), (0.0, 0, 1.0, 0.0), (1e-3, 0, 0.9, 0.0), (1e30, 0, 0.5, 0.0),
                                     (float("inf"), 7, 1.0, 0.5), (1e-42, 3, 0.5, 0.1)])
@pytest.mark.parametrize("V", [777, 128256])
def test_one_setting_for_all_rows(V, t, k, p, m):
    rng = np.random.default_rng(5)
    R = 16
    x = logits_of(rng, R, V)
    one = np.ones(R)
    check(x, rng.random(R), one * t, (one * k).astype(int), one * p, one * m, scalars=True)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [64, 5000, 130000])
def test_ties_go_to_the_lowest_id(V):
    """Few distinct values: every threshold falls among ties."""
    rng = np.random.default_rng(V + 1)
    R = 24
    x = rng.integers(-2, 3, (R, V)).astype(np.float32)
    x[0] = 0.0
    x[1] = np.where(rng.random(V) < 0.5, 0.0, -0.0)  # +0 and -0 are equal logits
    k = rng.choice([0, 1, 3, V // 3 + 1, V // 2], R)
    # top_p values whose product with a whole number of equal weights is exact in 64 bits
    p = rng.choice([1.0, 0.5, 0.25, 0.75], R)
    t = np.full(R, np.inf)  # every weight 1: borders fall exactly between ids
    check(x, rng.choice([0.0, 0.25, 0.5, 0.9999], R), t, k, p, np.zeros(R))
    check(x, rng.random(R), np.ones(R), k, rng.choice([1.0, 0.3], R), rng.choice([0.0, 0.1], R))


@pytest.mark.gpu
@pytest.mark.parametrize("V", [100, 40000])
def test_masked_and_non_finite_logits(V):
    rng = np.random.default_rng(3)
    R = 12
    x = logits_of(rng, R, V)
    x[:, rng.random(V) < 0.3] = -np.inf
    x[0] = -np.inf                      # nothing left: id 0
    x[1] = np.nan                       # NaN counts as -inf
    x[2, 5:9] = np.nan
    x[3] = np.finfo(np.float32).min     # all at the type's lowest value
    x[4] = -np.inf
    x[4, V - 1] = -3.0                  # one id left
    x[5, [7, 11]] = np.inf              # two ids share the mass
    x[6, 3] = np.finfo(np.float32).max
    x[7] = np.finfo(np.float32).min
    x[7, 2] = np.finfo(np.float32).max
    x[8, 4] = -np.finfo(np.float32).tiny
    for k, p, m in ((0, 1.0, 0.0), (5, 0.9, 0.0), (V, 0.5, 0.1), (V - 1, 1.0, 0.0)):
        one = np.ones(R)
        check(x, rng.random(R), one, (one * k).astype(int), one * p, one * m)
    one = np.ones(R)
    check(x, rng.random(R), 0 * one, (0 * one).astype(int), one, 0 * one)


@pytest.mark.gpu
def test_uniform_numbers_at_and_past_the_ends():
    rng = np.random.default_rng(9)
    x = logits_of(rng, 8, 3000)
    u = np.array([0.0, -0.0, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, np.nan, 1e-40])
    one = np.ones(8)
    for p in (1.0, 0.8):
        check(x, u, one, (0 * one).astype(int), one * p, 0 * one)


@pytest.mark.gpu
@pytest.mark.parametrize("ld,offset", [(5003, 0), (5004, 1), (5008, 4), (6001, 3)])
def test_strides_and_alignments(ld, offset):
    rng = np.random.default_rng(ld)
    R, V = 9, 5003
    x = logits_of(rng, R, V)
    one = np.ones(R)
    check(x, rng.random(R), one, (one * 100).astype(int), one * 0.9, one * 0.01, ld=ld, offset=offset)


@pytest.mark.gpu
def test_a_row_does_not_depend_on_the_batch():
    rng = np.random.default_rng(12)
    x = logits_of(rng, 64, 33000)
    one = np.ones(64)
    u = rng.random(64)
    args = (one, (0 * one).astype(int), 0.97 * one, 0 * one)
    whole = run(x, u, *args)
    for r in (0, 13, 63):
        assert run(x[r:r + 1], u[r:r + 1], *[a[r:r + 1] for a in args])[0] == whole[r]


@pytest.mark.gpu
def test_frequencies_follow_the_weights():
    """4096 evenly spread uniform numbers: each id is drawn as often as its share says, to one."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    rng = np.random.default_rng(1)
    V, n = 37, 4096
    x = rng.standard_normal(V).astype(np.float32)
    u = (torch.arange(n, device="cuda") + 0.5) / n
    got = api.sample(torch.from_numpy(x).cuda().repeat(n, 1), u, temperature=0.8)
    w = np.exp((x.astype(np.float64) - x.max()) / np.float64(np.float32(0.8)))
    count = np.bincount(got.cpu().numpy(), minlength=V)
    assert np.abs(count - n * w / w.sum()).max() <= 1.0


@pytest.mark.gpu
def test_streams_and_graph_replay():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    rng = np.random.default_rng(4)
    R, V = 6, 20000
    xs = [logits_of(rng, R, V) for _ in range(3)]
    us = [rng.random(R).astype(np.float32) for _ in range(3)]
    ref = [[ref_token(x[r], 1.0, 0, 0.9, 0.0, u[r]) for r in range(R)] for x, u in zip(xs, us)]
    dev = [(torch.from_numpy(x).cuda(), torch.from_numpy(u).cuda()) for x, u in zip(xs, us)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [api.sample(x, u, top_p=0.9, stream=s) for (x, u), s in zip(dev, streams)]
    torch.cuda.synchronize()
    assert [o.tolist() for o in outs] == ref
    x, u = dev[0][0].clone(), dev[0][1].clone()
    out = torch.empty(R, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.sample(x, u, top_p=0.9, out=out)
    for i in (1, 2, 0):
        x.copy_(dev[i][0])
        u.copy_(dev[i][1])
        g.replay()
        torch.cuda.synchronize()
        assert out.tolist() == ref[i]


@pytest.mark.gpu
def test_empty_batch_and_refusals_on_the_gpu():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    assert api.sample(torch.empty(0, 10, device="cuda"), torch.empty(0, device="cuda")).shape == (0,)
    x, u = torch.zeros(2, 10, device="cuda"), torch.zeros(2, device="cuda")
    with pytest.raises(ValueError):
        api.sample(x.half(), u)
    with pytest.raises(ValueError):
        api.sample(x.t(), u)
    with pytest.raises(ValueError):
        api.sample(x, u[:1])
    with pytest.raises(ValueError):
        api.sample(x, u, temperature=torch.ones(3, device="cuda"))
    with pytest.raises(ValueError):
        api.sample(x, u, top_k=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        api.sample(x.expand(2, 10)[:1].expand(2, 10), u)  # rows that overlap
    with pytest.raises(B.SwiftKVError):
        api.sample(torch.zeros(1, 360449, device="cuda"), u[:1])


def test_refusals_without_a_gpu():
    lib = B.lib()
    fake, s = C.c_void_p(256), B.Sampling()  # never dereferenced: refused first
    call = lib.swiftkv_sample
    assert call(fake, -1, 10, 10, C.byref(s), fake, fake, None) == -1
    assert call(fake, 1, 0, 10, C.byref(s), fake, fake, None) == -1
    assert call(fake, 1, 10, 9, C.byref(s), fake, fake, None) == -1
    assert call(None, 1, 10, 10, C.byref(s), fake, fake, None) == -1
    assert call(fake, 1, 10, 10, None, fake, fake, None) == -1
    assert call(fake, 1, 10, 10, C.byref(s), None, fake, None) == -1
    assert call(fake, 1, 10, 10, C.byref(s), fake, None, None) == -1
    assert call(C.c_void_p(258), 1, 10, 10, C.byref(s), fake, fake, None) == -1
    assert call(fake, 1, 360449, 360449, C.byref(s), fake, fake, None) == -9
    assert call(None, 0, 10, 10, None, None, None, None) == 0
