"""The bf16 copy of an 8-bit cache that attend's tiles read: pages that no row sees have a place in a block of it, but
nothing is written there. Whatever the workspace held before, NaN above all, must not reach an output. Tolerances
are those of the two caches' own tests."""
import pytest

import test_gpu_int8_cache as I8
import test_gpu_serving as F8

pytestmark = pytest.mark.gpu

BATCHES = [([24], [0]), ([24, 5, 40, 17, 100], [0, 82, 700, 3, 130]), ([33, 0, 2, 260], [50, 9, 4, 300])]


def fill_with_nan(model, heads):
    """A call of the same model whose K, V and scales are all NaN, over more pages than the next one's."""
    from swiftkv_prefill_skipping_gb300 import api
    c = F8.Case(heads, [300] * 3, [900] * 3, fp8=True, seed=1)
    for pool, scale in ((c.kv.k, c.kv.k_scale), (c.kv.v, c.kv.v_scale)):
        pool.fill_(0x7f)
        scale.fill_(float("nan"))
    out = api.attend(model, c.q.cuda(), c.cu, c.ctx, c.kv, cache=1)
    assert bool(out.isnan().all()) and model.status() == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (37, 5), (64, 20), (200, 90)])
@pytest.mark.parametrize("heads", ["gqa4", "gqa5", "d64"])
def test_pages_without_rows_hold_anything(heads, window, sinks):
    for i, (new, ctx) in enumerate(BATCHES):
        c = F8.Case(heads, new, ctx, window, sinks, fp8=True, seed=20 + i)
        fill_with_nan(c.model, heads)
        c.check_attend(*c.attend())
        c = I8.Case(heads, new, ctx, window, sinks, seed=30 + i)
        fill_with_nan(c.model, heads)
        c.check()
