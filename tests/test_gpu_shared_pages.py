"""Sequences that share pages of a common prefix, which attend allows always and evict to other pages:
the same bits as with a copy of the prefix for each. And the model's window when it is turned off again."""
import numpy as np
import pytest

from gpu_helpers import LOGIT_ABS_TOL
from oracle import model as OM
from test_gpu_bounded_cache import setup
from test_gpu_serving import HEADS, model_of

pytestmark = pytest.mark.gpu


class Shared:
    """Sequences of `lens` keys whose first `prefix` pages hold the same: `kv` with a copy for each, `one`
    with one copy that all name. Random pools, so every other row differs."""

    def __init__(self, heads, lens, prefix, dtype, caches=1, room=0, seed=0):
        import torch
        from swiftkv_prefill_skipping_gb300 import api
        self.n_q, self.n_kv, self.d = HEADS[heads]
        self.model = model_of(heads, caches)
        g = torch.Generator().manual_seed(seed)
        need = [(n + 15) // 16 for n in lens]
        total = sum(need) + room
        perm = torch.randperm(total, generator=g).to(torch.int32).numpy()
        table = np.full((len(lens), max(need)), -1, np.int32)
        at = 0
        for s, m in enumerate(need):
            table[s, :m] = perm[at:at + m]
            at += m
        self.free = perm[at:]
        self.kv = api.KVCache(self.model, total, table, dtype=dtype)
        self.pools = [self.kv.k, self.kv.v] + ([self.kv.k_scale, self.kv.v_scale] if dtype == "fp8" else [])
        for p in self.pools:
            if p.dtype == torch.uint8:  # codes of normal values
                p.copy_((torch.randn(p.shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            elif p.dim() == 4:
                p.copy_(torch.rand(p.shape, generator=g) / 50 + 1e-3)
            else:
                p.copy_(torch.randn(p.shape, generator=g))
        self.scores = torch.rand(self.kv.k.shape[:-1], generator=g).cuda()
        self.pools.append(self.scores)
        for s in range(1, len(lens)):
            for p in self.pools:
                p[:, table[s, :prefix].tolist()] = p[:, table[0, :prefix].tolist()]
        shared = table.copy()
        shared[:, :prefix] = table[0, :prefix]
        self.one = self.kv.view(range(len(lens)))
        self.one.block_table.copy_(torch.from_numpy(shared))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (100, 20), (7, 0)])
@pytest.mark.parametrize("heads", ["gqa4", "gqa5", "d64"])
def test_attend_over_a_shared_prefix(heads, window, sinks, dtype):
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    for new, ctx in (([1, 1, 3], [90, 200, 80]), ([140, 9, 1], [80, 100, 300]), ([20, 150], [85, 81])):
        c = Shared(heads, [a + b for a, b in zip(new, ctx)], 5, dtype, seed=len(new))
        T = sum(new)
        cu = np.concatenate([[0], np.cumsum(new)])
        q = torch.randn(T, c.n_q, c.d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
        got = []
        for kv in (c.kv, c.one):
            lse = torch.empty(c.n_q, T, device="cuda")
            got.append((api.attend(c.model, q, cu, ctx, kv, window=window, sinks=sinks, lse=lse), lse))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert not got[0][0].isnan().any() and c.model.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attend_names_a_sequence_twice(dtype):
    """Two chunks of one sequence, as in trying continuations: the bits of each on its own, tiles and rows."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Shared("gqa4", [300], 0, dtype, seed=3)
    q = torch.randn(60, c.n_q, c.d, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    out = api.attend(c.model, q, [0, 30, 60], [270, 200], c.kv.view([0, 0]), window=64, sinks=2)
    for s, ctx in ((0, 270), (1, 200)):
        one = api.attend(c.model, q[30 * s:30 * s + 30], [0, 30], [ctx], c.kv, window=64, sinks=2)
        assert torch.equal(out[30 * s:30 * s + 30], one)
    assert c.model.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_evict_from_a_shared_prefix_to_other_pages(dtype):
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    lens, keep = [200, 330, 81, 40], 48
    got = []
    for shared in (False, True):
        c = Shared("gqa4", lens, 2, dtype, caches=2, room=12, seed=4)
        dst = torch.from_numpy(c.free.reshape(4, 3)).cuda()
        before = [p.clone() for p in c.pools]
        kept = api.evict(c.model, c.one if shared else c.kv, c.scores, lens, keep, sinks=2, recent=8, dst_block_table=dst)
        source = c.kv.block_table[c.kv.block_table >= 0].long()
        for p, b in zip(c.pools, before):  # the source was only read
            assert torch.equal(p[:, source], b[:, source])
        got.append([kept] + [p[:, dst.long().flatten()] for p in c.pools])
        assert c.model.status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_a_window_that_is_turned_off_is_off():
    """A decode step after set_attention_window(0) over a cache that a windowed prefill filled sees every
    key again: the oracle's logits without a window, which are not those with it."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, prompts, cfg, w, l, g = setup("d128", [200])
    m.set_attention_window(32, 5)
    api.prefill(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, kv)
    with OM.attention_window(32, 5):
        caches, _ = OM.swiftkv_forward_one(cfg, w, None, prompts[0], l, g)
        _, windowed = OM.swiftkv_forward_one(cfg, w, caches, [7], l, g)
    _, whole = OM.swiftkv_forward_one(cfg, w, caches, [7], l, g)
    assert np.abs(windowed - whole).max() > 4 * LOGIT_ABS_TOL  # the test can tell them apart
    tok = torch.tensor([7], device="cuda")
    a, _ = api.decode_step(m, tok, [200], kv)
    assert np.abs(a[0].cpu().numpy() - windowed).max() <= LOGIT_ABS_TOL
    m.set_attention_window(0)
    b, _ = api.decode_step(m, tok, [200], kv)
    assert np.abs(b[0].cpu().numpy() - whole).max() <= LOGIT_ABS_TOL
    assert m.status() == 0
    m.free()
