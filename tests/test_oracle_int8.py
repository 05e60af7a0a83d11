"""The oracle's int8 cache: one scale for each page of 16 rows and head, which may grow as rows are appended."""
import numpy as np
import pytest

import oracle
import synth
from oracle import model as OM


def rows(n, h=2, d=8, seed=0, size=1.0):
    return OM.bf16(np.random.default_rng(seed).standard_normal((n, h, d)) * size)


def test_one_call_by_hand():
    x = np.zeros((3, 1, 2))
    x[0, 0], x[1, 0], x[2, 0] = (1.0, -127.0), (63.5, 0.25), (0.5, 1.5)
    c = OM.int8_append(None, x)
    assert c.scales.shape == (1, 1) and c.scales[0, 0] == 1.0
    assert np.array_equal(c.codes[:, 0], [[1, -127], [64, 0], [0, 2]])      # ties to even
    assert np.array_equal(np.asarray(c), c.codes)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 40])
def test_whole_blocks_are_off_by_half_a_step(n):
    x = rows(n)
    c = OM.int8_append(None, x)
    step = c.scales.astype(np.float64)[np.arange(n) // 16][..., None]
    assert np.abs(np.asarray(c) - x).max() <= step.max() / 2 * (1 + 1e-6)
    assert (np.abs(np.asarray(c) - x) <= step / 2 * (1 + 1e-6)).all() and np.abs(c.codes).max() == 127
    for p in range(c.scales.shape[0]):
        for h in range(2):
            top = np.float32(np.abs(x[16 * p:16 * p + 16, h]).max())
            assert c.scales[p, h] == top / np.float32(127)


def test_appended_rows_against_loops():
    """Any split into calls: scales are those of the page's largest value, earlier codes are rounded again at each growth."""
    x = rows(50, size=np.linspace(0.1, 3.0, 50)[:, None, None])
    whole = OM.int8_append(None, x)
    for cuts in ([1] * 50, [7, 20, 1, 22], [16, 16, 18]):
        c, at = None, 0
        codes, scales = np.zeros((50, 2, 8)), np.zeros((4, 2), np.float32)
        for n in cuts:
            c = OM.int8_append(c, x[at:at + n])
            for h in range(2):
                for p in range(at // 16, (at + n + 15) // 16):
                    lo, hi = max(at, 16 * p), min(at + n, 16 * p + 16)
                    need = np.float32(np.abs(x[lo:hi, h]).max()) / np.float32(127)
                    if need > scales[p, h]:
                        for r in range(16 * p, lo):
                            codes[r, h] = np.rint(codes[r, h].astype(np.float32) * (scales[p, h] / need))
                        scales[p, h] = need
                    for r in range(lo, hi):
                        codes[r, h] = np.rint(x[r, h].astype(np.float32) / scales[p, h])
            at += n
            assert np.array_equal(c.codes, codes[:at]) and np.array_equal(c.scales, scales[:(at + 15) // 16])
        assert np.array_equal(c.scales, whole.scales)
    # a page's values are off by half a step of its last scale for each growth behind them, and half for their own code
    assert np.abs(np.asarray(c) - x).max() <= whole.scales.max() * 2


def test_zero_rows_and_growth_from_zero():
    c = OM.int8_append(None, np.zeros((3, 1, 4)))
    assert not c.scales.any() and not c.codes.any()
    c = OM.int8_append(c, np.ones((1, 1, 4)))
    assert np.array_equal(c.codes[:, 0, 0], [0, 0, 0, 127])


def test_in_the_model():
    """Caches hold code * scale, logits move by a small nonzero amount, a prompt in chunks is the whole prompt where no page
    is cut, and a decode step is a chunk of one."""
    shape, l, g = synth.TINY, 2, 1
    cfg, w = oracle.config_of(shape), oracle.synth_weights(shape)
    toks = synth.uniform_int(3, 1, 40, 0, cfg.vocab - 1)
    exact, ref = OM.swiftkv_prefill_one(cfg, w, toks, l, g)
    with OM.kv_cache_int8():
        caches, got = OM.swiftkv_prefill_one(cfg, w, toks, l, g)
        one, _ = OM.swiftkv_forward_one(cfg, w, None, toks[:32], l, g)
        two, lg = OM.swiftkv_forward_one(cfg, w, one, toks[32:], l, g)
        a, la = OM.swiftkv_decode_step(cfg, w, caches, 5, l, g)
        b, lb = OM.swiftkv_forward_one(cfg, w, caches, [5], l, g)
    assert 0 < np.abs(got - ref).max() <= 5e-2
    assert np.abs(lg - got).max() <= 1e-9 and np.array_equal(la, lb)
    for c in range(len(caches)):
        for t in (0, 1):
            assert isinstance(caches[c][t], OM.Int8Rows)
            assert np.array_equal(np.asarray(caches[c][t]), caches[c][t].codes * caches[c][t].scales.astype(float)[np.arange(40) // 16][..., None])
            assert np.array_equal(two[c][t].codes, caches[c][t].codes) and np.array_equal(a[c][t].codes, b[c][t].codes)
    assert not isinstance(exact[0][0], OM.Int8Rows)
