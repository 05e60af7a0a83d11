"""Scores that the model's calls collect belong to the keys: a row that a call writes starts from nothing,
whatever its entry held - a page's former owner's scores, or those of keys that an eviction moved or
dropped. The same bits as with entries that were cleared by hand."""
import pytest

from test_gpu_bounded_cache import setup

pytestmark = pytest.mark.gpu


def entries(scores, kv, s, n):
    """[num_caches, n, n_kv]: the scores of sequence s's first n rows."""
    import torch
    j = torch.arange(n, device="cuda")
    return scores[:, kv.block_table[s][j // 16].long(), :, j % 16].permute(1, 0, 2)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("name", ["tiny", "d128", "bias"])
@pytest.mark.parametrize("decay", [1.0, 0.5])
def test_rows_that_are_written_start_from_nothing(name, dtype, decay):
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    lens = [130, 6]
    got = []
    for old in (0.0, 1000.0):
        m, kv, batch, prompts, cfg, *_ = setup(name, lens, dtype=dtype)
        scores = kv.new_scores() + old
        m.set_score_pools(scores, decay)
        api.prefill(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, kv)
        tok = torch.arange(12, device="cuda", dtype=torch.int32)
        api.forward(m, tok, [0, 9, 10], lens, kv)               # a chunk and a token
        api.forward(m, tok, [0, 1, 3], [139, 7], kv, pos_offsets=[5, 0])
        api.decode_step(m, tok[:2], [140, 9], kv)
        torch.cuda.synchronize()
        assert m.status() == 0
        got.append([entries(scores, kv, s, n).clone() for s, n in ((0, 141), (1, 10))])
        assert bool((got[-1][0] > 0).all()) and bool((got[-1][1] > 0).all())
        touched = torch.zeros_like(scores, dtype=torch.bool)
        for s, n in ((0, 141), (1, 10)):
            j = torch.arange(n, device="cuda")
            touched[:, kv.block_table[s][j // 16].long(), :, j % 16] = True
        assert bool((scores[~touched] == old).all())            # all else stays as it was
        m.free()
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("name", ["tiny", "d128"])
def test_rows_behind_an_eviction_start_from_nothing(name, dtype):
    """Prompt, eviction in place, tokens behind the kept keys and a second eviction: no choice hangs on
    scores of keys that are gone."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    lens, keep = [150, 20, 70], 48
    got = []
    for clear in (True, False):
        m, kv, batch, *_ = setup(name, lens, dtype=dtype)
        scores = kv.new_scores()
        m.set_score_pools(scores)
        api.prefill(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, kv)
        api.evict(m, kv, scores, lens, keep, sinks=2, recent=8)
        left = [min(n, keep) for n in lens]
        gone = [n - k for n, k in zip(lens, left)]
        if clear:
            for s, k in enumerate(left):
                j = torch.arange(k, kv.block_table.shape[1] * 16, device="cuda")
                page = kv.block_table[s][j // 16].long()
                scores[:, page[page >= 0], :, (j % 16)[page >= 0]] = 0
        tok = torch.arange(90, device="cuda", dtype=torch.int32)
        api.forward(m, tok, [0, 30, 40, 42], left, kv, pos_offsets=gone)
        left = [left[0] + 30, left[1] + 10, left[2] + 2]
        got.append([entries(scores, kv, s, n).clone() for s, n in enumerate(left)])
        got[-1].append(api.evict(m, kv, scores, left, 40, sinks=2, recent=4))
        assert m.status() == 0
        m.free()
    for a, b in zip(*got):
        assert torch.equal(a, b)
