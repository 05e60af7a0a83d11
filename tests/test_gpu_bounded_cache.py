"""The model's own calls over a bounded cache: sliding window with sinks, attention weights collected
per cache, eviction by them, position offsets after it and sampled tokens, against the oracle.

The tolerances are those of the model parity tests. Collected weights: a cached vector and a query are
within KV_REL_TOL of the oracle's each, so a score z is off by at most 2 KV_REL_TOL |z| + the same
again for the norm of the vectors it is a product of, and a softmax weight by twice that."""
import numpy as np
import pytest

import oracle
import synth
from gpu_helpers import KV_REL_TOL, LOGIT_ABS_TOL, SMALL128, SMALL_BIAS, rel_l2
from oracle import model as OM
from swiftkv_prefill_skipping_gb300 import binding as B

pytestmark = pytest.mark.gpu
SHAPES = {"tiny": (synth.TINY, 2, 1), "d128": (SMALL128, 2, 2), "bias": (SMALL_BIAS, 4, 1)}


def setup(name, lens, extra=40, dtype="bf16"):
    """Model, cache with room for `extra` more tokens per sequence, prompts, oracle config and weights."""
    from swiftkv_prefill_skipping_gb300 import api
    shape, l, g = SHAPES[name]
    batch = synth.prompt_batch(shape.vocab, len(lens), 0, 0, lens=lens, reserve_tokens=extra)
    m = api.load_synthetic(shape, l, g)
    kv = api.KVCache(m, batch.num_pages, batch.block_table, dtype=dtype)
    prompts = [batch.tokens[batch.cu_seqlens[s]:batch.cu_seqlens[s + 1]] for s in range(len(lens))]
    return m, kv, batch, prompts, oracle.config_of(shape), oracle.synth_weights(shape), l, g


def check_caches(kv, m, s, caches):
    for c in range(m.num_caches):
        n = caches[c][0].shape[0]
        for which, t in (("k", 0), ("v", 1)):
            assert rel_l2(kv.gather(c, s, n, which).float().cpu().numpy(), caches[c][t]) <= KV_REL_TOL, (c, which)


@pytest.mark.parametrize("window,sinks", [(1, 0), (24, 4), (64, 0), (200, 17), (4096, 0)])
@pytest.mark.parametrize("name", list(SHAPES))
def test_window_in_prefill_forward_and_decode(name, window, sinks):
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, prompts, cfg, w, l, g = setup(name, [150, 3, 70])
    m.set_attention_window(window, sinks)
    logits = api.prefill(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, kv)
    state = []
    with OM.attention_window(window, sinks):
        for s, p in enumerate(prompts):
            caches, ref = OM.swiftkv_forward_one(cfg, w, None, p, l, g)
            assert np.abs(logits[s].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL
            check_caches(kv, m, s, caches)
            state.append((caches, OM.greedy(ref)))
        # a chunk after the prefix for sequence 0, a single token for sequence 1
        chunk = synth.uniform_int(5, 1, 9, 0, cfg.vocab - 1)
        toks = np.concatenate([chunk, [state[1][1]]])
        lg = api.forward(m, torch.as_tensor(toks, device="cuda"), [0, 9, 10], [150, 3], kv.view([0, 1]))
        caches, ref = OM.swiftkv_forward_one(cfg, w, state[0][0], chunk, l, g)
        assert np.abs(lg[0].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL
        check_caches(kv, m, 0, caches)
        state[0] = (caches, OM.greedy(ref))
        caches, ref = OM.swiftkv_forward_one(cfg, w, state[1][0], [state[1][1]], l, g)
        assert np.abs(lg[1].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL
        state[1] = (caches, OM.greedy(ref))
        lens = [159, 4, 70]
        for _ in range(2):
            lg, _ = api.decode_step(m, torch.tensor([t for _, t in state], device="cuda"), lens, kv)
            for s in range(3):
                caches, ref = OM.swiftkv_decode_step(cfg, w, state[s][0], state[s][1], l, g)
                caches = caches if caches is not None else state[s][0]
                assert np.abs(lg[s].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL
                state[s] = (caches, OM.greedy(ref))
            lens = [n + 1 for n in lens]
    assert m.status() == 0
    m.free()


@pytest.mark.parametrize("name", ["tiny", "d128"])
def test_window_over_an_fp8_cache(name):
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, prompts, cfg, w, l, g = setup(name, [140, 2], dtype="fp8")
    m.set_attention_window(48, 3)
    logits = api.prefill(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, kv)
    with OM.attention_window(48, 3), OM.kv_cache_fp8():
        refs = [OM.swiftkv_forward_one(cfg, w, None, p, l, g) for p in prompts]
        for s in range(2):
            assert np.abs(logits[s].cpu().numpy() - refs[s][1]).max() <= LOGIT_ABS_TOL
        toks = [OM.greedy(r[1]) for r in refs]
        lg, _ = api.decode_step(m, torch.tensor(toks, device="cuda"), [140, 2], kv)
        for s in range(2):
            _, ref = OM.swiftkv_decode_step(cfg, w, refs[s][0], toks[s], l, g)
            assert np.abs(lg[s].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL
    assert m.status() == 0
    m.free()


def test_pages_behind_the_window_may_be_given_back():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, prompts, cfg, w, l, g = setup("d128", [200])
    m.set_attention_window(32, 5)
    api.prefill(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, kv)
    tok = torch.tensor([7], device="cuda")
    a, _ = api.decode_step(m, tok, [200], kv)
    gone = kv.block_table[0, 1:10].long()          # rows 16 .. 159: behind the window, past the sinks
    for pool in (kv.k, kv.v):
        pool[:, gone] = float("nan")               # another sequence's data by now
    kv.block_table[0, 1:10] = -1
    b, _ = api.decode_step(m, tok, [200], kv)
    torch.cuda.synchronize()
    assert m.status() == 0 and torch.equal(a, b)
    m.set_attention_window(0)
    api.decode_step(m, tok, [200], kv)             # now they are needed
    m.free()


def test_window_off_is_the_ordinary_path_bit_for_bit():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, prompts, *_ = setup("d128", [100, 30])
    tok = torch.as_tensor(batch.tokens, device="cuda")
    a = api.prefill(m, tok, batch.cu_seqlens, kv)
    m.set_attention_window(20, 2)
    m.set_score_pools(kv.new_scores())
    api.prefill(m, tok, batch.cu_seqlens, kv)
    m.set_attention_window(0)
    m.set_score_pools(None)
    assert torch.equal(a, api.prefill(m, tok, batch.cu_seqlens, kv))
    m.free()


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("name", list(SHAPES))
def test_collected_weights(name, window):
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, prompts, cfg, w, l, g = setup(name, [130, 6])
    m.set_attention_window(window, 2 if window else 0)
    scores = kv.new_scores()
    m.set_score_pools(scores)
    logits = api.prefill(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, kv)
    nxt = [OM.greedy(logits[s].cpu().numpy()) for s in range(2)]
    api.decode_step(m, torch.tensor(nxt, device="cuda"), [130, 6], kv)
    m.set_score_pools(None)
    torch.cuda.synchronize()
    G = cfg.n_q // cfg.n_kv
    for s, p in enumerate(prompts):
        n = len(p) + 1
        ref = np.zeros((m.num_caches, n, cfg.n_kv))
        calls = []
        with OM.attention_window(window, 2 if window else 0), OM.observe_attention(calls.append):
            caches, _ = OM.swiftkv_forward_one(cfg, w, None, p, l, g)
            OM.swiftkv_forward_one(cfg, w, caches, [nxt[s]], l, g)
        assert len(calls) == 2 * cfg.L
        for i, pr in enumerate(calls):
            given = pr.sum(1).reshape(cfg.n_kv, G, -1).sum(1).T          # [keys, n_kv]
            ref[OM.cache_of_layer(i % cfg.L, l, g), :given.shape[0]] += given
        bt = kv.block_table[s]
        j = torch.arange(n, device="cuda")
        got = scores[:, bt[j // 16].long(), :, j % 16].permute(1, 0, 2).cpu().numpy()
        assert rel_l2(got, ref) <= 4 * KV_REL_TOL
        rows = sum((len(p) if j < l else 1) + 1 for j in range(cfg.L))    # each row and head hands out one
        assert abs(got.astype(np.float64).sum() - rows * cfg.n_q) <= 1e-3 * rows * cfg.n_q
    m.free()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("name", ["tiny", "d128"])
def test_collect_evict_go_on_and_sample(name, dtype):
    """Prompts, their keys' weights, eviction in every cache, then tokens drawn by swiftkv_sample and
    fed back at their true positions, as a server with a bounded cache does it."""
    import contextlib
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    lens, keep = [150, 20, 70], 48
    m, kv, batch, prompts, cfg, w, l, g = setup(name, lens, dtype=dtype)
    scores = kv.new_scores()
    m.set_score_pools(scores)
    logits = api.prefill(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, kv)
    kept = api.evict(m, kv, scores, lens, keep, sinks=2, recent=16).cpu().numpy()
    left = [min(n, keep) for n in lens]
    gone = [n - k for n, k in zip(lens, left)]
    with OM.kv_cache_fp8() if dtype == "fp8" else contextlib.nullcontext():
        state = []
        for s, p in enumerate(prompts):
            caches, _ = OM.swiftkv_forward_one(cfg, w, None, p, l, g)
            shrunk = []
            for c in range(m.num_caches):
                idx = kept[c, s][:, :left[s]]                              # [n_kv, left]
                assert (np.diff(idx, axis=1) > 0).all() and (idx[:, :2] == [0, 1]).all()
                shrunk.append(tuple(np.stack([t[idx[h], h] for h in range(cfg.n_kv)], axis=1) for t in caches[c]))
            state.append(shrunk)
        u = torch.rand(4, 3, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
        lg = logits
        for step in range(4):
            toks = api.sample(lg, u[step], temperature=0.9, top_k=40, top_p=0.95)
            lg = api.forward(m, toks, [0, 1, 2, 3], [k + step for k in left], kv, pos_offsets=gone)
            for s, t in enumerate(toks.tolist()):
                state[s], ref = OM.swiftkv_forward_one(cfg, w, state[s], [t], l, g, pos_offset=gone[s])
                assert np.abs(lg[s].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL, (step, s)
    assert m.status() == 0
    # the collected pools moved with the keys and go on collecting for the new ones
    bt = kv.block_table[0]
    j = torch.arange(left[0], left[0] + 4, device="cuda")
    assert bool((scores[:, bt[j // 16].long(), :, j % 16] > 0).all())
    m.free()


def test_refusals():
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, prompts, *_ = setup("tiny", [20])
    with pytest.raises(B.SwiftKVError):
        m.set_attention_window(-1)
    with pytest.raises(B.SwiftKVError):
        m.set_attention_window(4, -1)
    sc = kv.new_scores()
    with pytest.raises(B.SwiftKVError):
        m.set_score_pools(sc, decay=float("nan"))
    with pytest.raises(ValueError):
        m.set_score_pools(sc[:-1])
    with pytest.raises(ValueError):
        m.set_score_pools(sc.double())
    tok = torch.as_tensor(batch.tokens, device="cuda")
    with pytest.raises(B.SwiftKVError):
        api.forward(m, tok, [0, 20], None, kv, pos_offsets=[-1])
    with pytest.raises(B.SwiftKVError):
        api.forward(m, tok, [0, 20], None, kv, pos_offsets=[1 << 30])
    with pytest.raises(ValueError):
        api.forward(m, tok, [0, 20], None, kv, pos_offsets=[0, 0])
    # pools of fewer pages than the cache, in each of the model's calls
    small = torch.zeros_like(sc[:, :-1].contiguous())
    m.set_score_pools(small)
    for call in (lambda: api.prefill(m, tok, [0, 20], kv), lambda: api.forward(m, tok, [0, 20], [0], kv),
                 lambda: api.forward(m, tok, [0, 20], [0], kv, pos_offsets=[3]),
                 lambda: api.decode_step(m, tok[:1], [20], kv)):
        with pytest.raises(B.SwiftKVError, match="score pools"):
            call()
    torch.cuda.synchronize()
    assert not small.any() and m.status() == 0
    m.set_score_pools(None)
    before = m.memory()[1]
    api.attend(m, torch.zeros(300, m.shape.n_q, m.shape.d_h, dtype=torch.bfloat16, device="cuda")[:20], [0, 20], None, kv)
    assert m.memory()[1] > before  # the operators' workspace counts
    m.free()
