"""swiftkv_append with 8 query heads for each KV head and with more heads than a warp takes in a step; rules and tolerances of
test_gpu_append."""
import pytest

import test_gpu_append as A

pytestmark = pytest.mark.gpu

SHAPES = {"gqa8": (16, 2, 128), "70b": (64, 8, 128), "gqa8_d64": (24, 3, 64)}


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("heads", list(SHAPES))
def test_eight_query_heads_for_each_kv_head(monkeypatch, heads, kind):
    monkeypatch.setitem(A.HEADS, heads, SHAPES[heads])
    for i, (new, ctx) in enumerate(A.BATCHES):
        c = A.Case(heads, new, ctx, kind, seed=40 + i)
        c.check(c.run())
    off = [100 * s for s in range(3)]
    c = A.Case(heads, [17, 3, 40], [33000, 5, 31], kind, caches=3, total_caches=4, first=1, seed=50)
    c.check(c.run(pos_offsets=off), off)
