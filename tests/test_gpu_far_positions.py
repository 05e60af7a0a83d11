"""Positions far beyond the table of rotations (swiftkv_forward_at allows them up to 2^30): rotated keys
and logits against the oracle, whose angles are computed in 64 bits, at the model parity tolerances. The
angle of dimension 1 at position 2^30 is some 10^9 radians, so a float32 product of position and
frequency holds nothing of it."""
import numpy as np
import pytest

import oracle
import synth
from gpu_helpers import KV_REL_TOL, LOGIT_ABS_TOL, SMALL128, SMALL_BIAS, rel_l2
from oracle import model as OM

pytestmark = pytest.mark.gpu
SHAPES = {"tiny": (synth.TINY, 2, 1), "d128": (SMALL128, 2, 2), "bias": (SMALL_BIAS, 4, 1)}


@pytest.mark.parametrize("gemm", [0, 1])
@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("offset", [32768 - 30, 100_000, (1 << 20) + 3, (1 << 24) + 1, (1 << 30) - 200])
def test_chunks_and_tokens_at_far_positions(name, offset, gemm):
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    from swiftkv_prefill_skipping_gb300 import binding as B
    shape, l, g = SHAPES[name]
    lens = [90, 3, 1]
    batch = synth.prompt_batch(shape.vocab, 3, 0, 0, lens=lens, reserve_tokens=4)
    m = api.load_synthetic(shape, l, g)
    B.check(B.lib().swiftkv_set_gemm_impl(m.handle, gemm))
    kv = api.KVCache(m, batch.num_pages, batch.block_table)
    cfg, w = oracle.config_of(shape), oracle.synth_weights(shape)
    lg = api.forward(m, torch.as_tensor(batch.tokens, device="cuda"), batch.cu_seqlens, None, kv, pos_offsets=[offset] * 3)
    state = []
    for s in range(3):
        p = batch.tokens[batch.cu_seqlens[s]:batch.cu_seqlens[s + 1]]
        caches, ref = OM.swiftkv_forward_one(cfg, w, None, p, l, g, pos_offset=offset)
        assert np.abs(lg[s].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL
        for c in range(m.num_caches):
            assert rel_l2(kv.gather(c, s, lens[s], "k").float().cpu().numpy(), caches[c][0]) <= KV_REL_TOL, c
        state.append((caches, OM.greedy(ref)))
    lg = api.forward(m, torch.tensor([t for _, t in state], device="cuda"), [0, 1, 2, 3], lens, kv, pos_offsets=[offset] * 3)
    for s in range(3):
        _, ref = OM.swiftkv_forward_one(cfg, w, state[s][0], [state[s][1]], l, g, pos_offset=offset)
        assert np.abs(lg[s].cpu().numpy() - ref).max() <= LOGIT_ABS_TOL
    assert m.status() == 0
    m.free()
