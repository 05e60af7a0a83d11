"""Operators over the paged cache at the shapes between the others: groups of 3, 6 and 7 query heads, more
sequences than a call's lists hold in its parameters, and windows at the ends of the type's range."""
import numpy as np
import pytest

import test_gpu_serving as S

pytestmark = pytest.mark.gpu
GROUPS = {"g3": (6, 2, 128), "g6": (6, 1, 64), "g6_128": (12, 2, 128), "g7": (14, 2, 128)}
S.HEADS.update(GROUPS)  # Case looks its heads up there


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("heads", list(GROUPS))
def test_groups(heads, fp8):
    for i, (new, ctx, window, sinks) in enumerate([([1, 4, 2], [100, 33, 0], 0, 0), ([3, 1], [700, 5], 90, 7),
                                                   ([130, 5, 300], [20, 400, 0], 0, 0), ([200, 4], [90, 333], 64, 3)]):
        c = S.Case(heads, new, ctx, window, sinks, fp8, seed=50 + i)
        c.check_attend(*c.attend())
        c.check_weights(decay=(1.0, 0.0, 0.5, 1.0)[i])


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_many_sequences(fp8):
    """Lists past the kernels' parameters, and more items than the GPU has warps."""
    for i, (P, lo, hi, window) in enumerate([(300, 0, 60, 0), (700, 1, 30, 9), (260, 900, 1000, 0)]):
        rng = np.random.default_rng(i)
        new = rng.integers(0, 3, P).tolist()
        c = S.Case("gqa4" if i else "d64", new, rng.integers(lo, hi, P).tolist(), window, 2 if window else 0, fp8, seed=60 + i)
        c.check_attend(*c.attend())
        c.check_weights(decay=0.5)


@pytest.mark.parametrize("inplace", [True, False], ids=["inplace", "moved"])
def test_evict_many_sequences(inplace):
    rng = np.random.default_rng(5)
    S.EvictCase("d64", rng.integers(0, 90, 1100).tolist(), 20, 2, 5, caches=1, seed=8).run(inplace)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_windows_at_the_ends_of_the_range(fp8):
    """A window or sinks of 2^31 - 1 hide nothing: the bits of a call without a window."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    top = 2 ** 31 - 1
    for new, ctx in (([1, 3], [300, 64]), ([200, 5], [100, 400])):
        c = S.Case("gqa4", new, ctx, fp8=fp8, seed=9)
        lse = torch.empty(c.n_q, c.T, device="cuda")
        q, outs, scores = c.q.cuda(), [], []
        for window, sinks in ((0, 0), (0, top), (top, 0), (top, top), (1, top), (5, 1 << 30)):
            outs.append(api.attend(c.model, q, c.cu, c.ctx, c.kv, cache=1, window=window, sinks=sinks, lse=lse))
            sc = torch.zeros(c.total, c.n_kv, 16, device="cuda")
            scores.append(api.attention_weights(c.model, q, lse, c.cu, c.ctx, c.kv, sc, cache=1, window=window, sinks=sinks))
        for i in (1, 2, 3):
            assert torch.equal(outs[0], outs[i]) and torch.equal(scores[0], scores[i])
        for i in (4, 5):  # sinks that hide nothing: other cuts of the same keys
            c.check_attend(outs[i].cpu().double(), lse.cpu().double())
            assert bool(((scores[0] - scores[i]).abs() <= 2.0 ** -12 * scores[0].abs() + 1e-6).all())
        assert c.model.status() == 0
