"""Checks of the operators' arguments that need no GPU: nothing here reaches a kernel."""
import ctypes as C

import numpy as np
import pytest
import torch

from swiftkv_prefill_skipping_gb300 import api
from swiftkv_prefill_skipping_gb300 import binding as B


def model_on(device="cuda:0", n_kv=2, d_h=64, caches=2):
    """A Model without its handle: every call that gets past the checks fails on it."""
    m = object.__new__(api.Model)
    m.shape = api.Shape(L=caches, d=128, n_q=4, n_kv=n_kv, d_h=d_h, ffn=64, vocab=128, rope_theta=1e4)
    m.l, m.g, m.num_caches, m.handle = caches, 1, caches, C.c_void_p()
    m.device = torch.device(device)
    return m


@pytest.mark.parametrize("device", ["cuda:0", "cuda:1"])
def test_score_pools_have_to_be_on_the_models_device(device):
    m = model_on(device)
    with pytest.raises(ValueError, match=f"on {device}"):
        m.set_score_pools(torch.zeros(2, 5, 2, 16))
    assert getattr(m, "_scores", None) is None


def test_operators_refuse_a_cache_on_another_device():
    m = model_on()
    kv = api.KVCache(m, 4, np.zeros((1, 2), np.int32), device=torch.device("cpu"))
    q, lse = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 1)
    for call in (lambda: api.attend(m, q, [0, 1], None, kv),
                 lambda: api.attention_weights(m, q, lse, [0, 1], None, kv, kv.new_scores()[0]),
                 lambda: api.evict(m, kv, kv.new_scores(), [5], 2)):
        with pytest.raises(ValueError, match="model on cuda:0"):
            call()


@pytest.mark.parametrize("which", ["tokens", "u", "temperature", "top_k", "top_p", "min_p"])
def test_sample_refuses_misaligned_arrays(which):
    s, at = B.Sampling(), dict(tokens=256, u=256)  # addresses that are never used: refused first
    if which in at:
        at[which] += 2
    else:
        setattr(s, which, 258)
    vocab = 360449  # refused later on, so that no kernel runs where the check is missing
    assert B.lib().swiftkv_sample(256, 1, vocab, vocab, C.byref(s), at["u"], at["tokens"], None) == -1
    assert b"misaligned" in B.lib().swiftkv_last_error()


@pytest.mark.parametrize("big", [1 << 31, (1 << 32) + 5, -(1 << 31) - 1])
def test_numbers_past_32_bits_are_refused(big):
    """They would wrap on their way into the call: 2^32 + 5 would be a window of 5."""
    m = model_on("cpu")
    kv = api.KVCache(m, 4, np.zeros((1, 2), np.int32), device=torch.device("cpu"))
    q, lse, sc = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 1), kv.new_scores()
    wide = np.array([big], np.int64)
    calls = [lambda: m.set_attention_window(big), lambda: m.set_attention_window(4, big),
             lambda: api.attend(m, q, [0, 1], None, kv, window=big), lambda: api.attend(m, q, [0, 1], None, kv, window=2, sinks=big),
             lambda: api.attend(m, q, [0, 1], None, kv, cache=big),
             lambda: api.attend(m, q, [0, 1], wide, kv), lambda: api.attend(m, q, [0, 1], torch.tensor(wide), kv),
             lambda: api.attend(m, q, np.array([0, big]), None, kv),
             lambda: api.attention_weights(m, q, lse, [0, 1], None, kv, sc[0], window=big),
             lambda: api.attention_weights(m, q, lse, [0, 1], wide, kv, sc[0]),
             lambda: api.evict(m, kv, sc, wide, 2), lambda: api.evict(m, kv, sc, [5], 2, sinks=big),
             lambda: api.evict(m, kv, sc, [5], 2, recent=big), lambda: api.evict(m, kv, sc, [5], big),
             lambda: api.forward(m, torch.zeros(1, dtype=torch.int32), [0, 1], [0], kv, pos_offsets=wide)]
    for call in calls:
        with pytest.raises((ValueError, OverflowError), match="32 bits"):
            call()


@pytest.mark.parametrize("T", [1, 3])
def test_append_refuses_values_of_one_cache_for_keys_of_several(T):
    """v of one cache beside k of two: its rows end, or another part of the projection begins, where the second's would be."""
    m = model_on("cpu")
    kv = api.KVCache(m, 4, np.zeros((1, 2), np.int32), device=torch.device("cpu"))
    wide = torch.zeros(T, 2, 2, 2, 64, dtype=torch.bfloat16)  # K and V of the first cache, then of the second
    k, v = wide[:, :, 0], wide[:, :, 1]
    for one in (v[:, 0], v[:, 0].contiguous(), wide.flatten(1, 3)[:, 2:4]):
        with pytest.raises(ValueError, match="v: bfloat16"):
            api.append(m, k, one, [0, T], None, kv)
        with pytest.raises(ValueError, match="v: bfloat16"):
            api.append(m, k.contiguous(), one, [0, T], None, kv)
        with pytest.raises(ValueError, match="v: bfloat16"):
            api.append(m, one, v, [0, T], None, kv)
