"""Limits and ownership of the operators over the paged cache: what is refused before a launch, what
memory they hold, which stream their outputs belong to."""
import ctypes as C

import numpy as np
import pytest

from swiftkv_prefill_skipping_gb300 import binding as B
from test_gpu_bounded_cache import setup
from test_gpu_serving import HEADS, Case, EvictCase, model_of

pytestmark = pytest.mark.gpu


def test_evict_refuses_lists_past_what_its_kernels_count():
    """Refused on the host: nothing is launched, so the pointers are never used."""
    c = EvictCase("d64", [40], 8, 0, 0)
    lib, fake = B.lib(), 1 << 20
    scores = (C.c_void_p * 2)(c.scores[0].data_ptr(), c.scores[1].data_ptr())
    lens = np.array([40], np.int32)
    for keep in ((1 << 30) + 1, 2 ** 31 - 1):
        assert lib.swiftkv_evict(c.model.handle, -1, c.kv.pages_ref, scores, B.host(lens), 1, keep, 0, 0, None, 0, fake, None) == -9
    wide = B.KVPages.from_buffer_copy(c.kv.pages)
    wide.max_pages_per_seq = 1 << 27
    lens = np.array([(1 << 30) + 1], np.int32)
    assert lib.swiftkv_evict(c.model.handle, -1, C.byref(wide), scores, B.host(lens), 1, 8, 0, 0, None, 0, fake, None) == -9
    assert b"2^30" in lib.swiftkv_last_error()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("mode", ["plain", "window", "scores"])
def test_the_models_calls_refuse_pools_off_16_bytes(mode, dtype):
    """Refused on the host, as by the operators: the kernels would read such a pool 16 bytes at a time."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    m, kv, batch, *_ = setup("tiny", [20], dtype=dtype)
    if mode == "window":
        m.set_attention_window(8, 1)
    if mode == "scores":
        m.set_score_pools(kv.new_scores())
    tok = torch.as_tensor(batch.tokens, device="cuda")
    for name, step in (("_kp", 2), ("_vp", 8)) + ((("_ks", 4), ("_vs", 8)) if dtype == "fp8" else ()):
        pools = getattr(kv, name)
        for c in range(m.num_caches):
            was, pools[c] = pools[c], pools[c] + step
            for call in (lambda: api.prefill(m, tok, [0, 20], kv), lambda: api.forward(m, tok, [0, 20], [0], kv),
                         lambda: api.forward(m, tok, [0, 20], [0], kv, pos_offsets=[3]),
                         lambda: api.decode_step(m, tok[:1], [20], kv)):
                with pytest.raises(B.SwiftKVError, match="16-byte"):
                    call()
            pools[c] = was
    assert m.status() == 0
    m.free()


def test_evict_refuses_misaligned_lists():
    """Refused on the host: nothing is launched."""
    c = EvictCase("d64", [40], 8, 0, 0)
    scores = (C.c_void_p * 2)(c.scores[0].data_ptr(), c.scores[1].data_ptr())
    lens = np.array([40], np.int32)
    for kept, dst in ((4098, None), (4096, 4097), (4096, 4098)):
        assert B.lib().swiftkv_evict(c.model.handle, -1, c.kv.pages_ref, scores, B.host(lens), 1, 8, 0, 0, dst,
                                     1 if dst else 0, kept, None) == -1
        assert b"misaligned" in B.lib().swiftkv_last_error()


def test_outputs_belong_to_the_stream_they_are_written_on():
    """A call on another stream takes no memory that the current stream's work still writes: a block that
    was freed while a fill was waiting on the current stream is not handed out as the output."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    c = Case("gqa4", [140, 1], [20, 70], seed=5)
    e = EvictCase("gqa4", [200, 40], 32, 2, 8, seed=4)
    q, dst, x, u = c.q.cuda(), e.dst.cuda(), torch.randn(300, 1000, device="cuda"), torch.rand(300, device="cuda")
    scores = e.scores.clone()
    side = torch.cuda.Stream()

    def attend(**kw):
        return api.attend(c.model, q, c.cu, c.ctx, c.kv, cache=1, **kw)

    def evict(**kw):  # to other pages: the source and its scores stay
        return api.evict(e.model, e.kv, scores, e.lens, 32, sinks=2, recent=8, dst_block_table=dst, **kw)

    def sample(**kw):
        return api.sample(x, u, top_p=0.9, **kw)

    for call in (attend, evict, sample):
        ref = call()
        torch.cuda.synchronize()
        block = torch.empty_like(ref)
        was = block.data_ptr()
        torch.cuda._sleep(100_000_000)
        block.fill_(7)
        del block
        got = call(stream=side)
        assert got.data_ptr() != was
        torch.cuda.synchronize()
        assert torch.equal(got, ref)


@pytest.mark.parametrize("captured", [False, True])
def test_workspace_that_was_outgrown(captured):
    """Over an FP8 cache a chunk's workspace holds a bf16 copy of its keys. After growing step by step
    swiftkv_memory gives what the device has lost, and without a graph that is the last block alone."""
    import gc
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    n_q, n_kv, d = HEADS["gqa8"]
    steps, new = (2000, 16000, 32000, 64000), 8
    pages = steps[-1] // 16 + 1

    def make():
        m = model_of("gqa8", 1)
        return m, api.KVCache(m, pages, np.arange(pages, dtype=np.int32)[None], dtype="fp8")

    q = torch.randn(new, n_q, d, device="cuda").bfloat16()
    out = torch.empty_like(q)

    def call(m, kv, keys):
        api.attend(m, q, [0, new], [keys - new], kv, out=out)

    other = make()
    call(*other, steps[-1])
    m, kv = make()
    call(m, kv, 500)

    def free_bytes():  # less what other tests left behind, which a capture would give back in between
        torch.cuda.synchronize()
        gc.collect()
        torch.cuda.empty_cache()
        return torch.cuda.mem_get_info()[0]

    held, free = m.memory()[1], free_bytes()
    graphs = []
    for keys in steps:
        call(m, kv, keys)
        if captured:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                call(m, kv, keys)
        lost = free - free_bytes()
        assert abs(m.memory()[1] - held - lost) <= (8 << 20), (keys, m.memory()[1] - held, lost)
    if captured:
        ref = []
        for keys in steps:
            call(m, kv, keys)
            ref.append(out.clone())
        for g, r in zip(graphs, ref):
            out.zero_()
            g.replay()
            assert torch.equal(out, r)
    else:
        assert m.memory() == other[0].memory()
    assert m.status() == 0


def test_sample_takes_any_number_as_top_k():
    """From vocab on it is off, 2^32 + 5 as well, and so is anything below 1."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    x, u = torch.randn(200, 3000, device="cuda"), torch.rand(200, device="cuda")
    ref = api.sample(x, u)
    assert not torch.equal(ref, api.sample(x, u, top_k=5))
    for k in (3000, (1 << 31) - 1, 1 << 31, (1 << 32) + 5, (1 << 63) + 5, -1, -(1 << 31), 5 - (1 << 32)):
        assert torch.equal(ref, api.sample(x, u, top_k=k))


def test_two_models_on_two_streams_at_once():
    """Calls on different models need no order: tiles, rows and weights of both, side by side, with the bits
    that each gives alone."""
    import torch
    from swiftkv_prefill_skipping_gb300 import api
    cases = [Case("gqa4", [700, 1, 300], [900, 500, 0], 200, 4, seed=31), Case("d64", [650, 2], [1200, 900], fp8=True, seed=32)]
    streams, calls = [torch.cuda.Stream() for _ in cases], []
    for c in cases:
        q, lse = c.q.cuda(), torch.empty(c.n_q, c.T, device="cuda")
        out, sc = torch.empty_like(q), torch.zeros(c.total, c.n_kv, 16, device="cuda")

        def call(stream, c=c, q=q, lse=lse, out=out, sc=sc):
            api.attend(c.model, q, c.cu, c.ctx, c.kv, cache=1, window=c.window, sinks=c.sinks, out=out, lse=lse, stream=stream)
            api.attention_weights(c.model, q, lse, c.cu, c.ctx, c.kv, sc, cache=1, window=c.window, sinks=c.sinks, decay=0.0,
                                  stream=stream)

        call(None)
        torch.cuda.synchronize()
        calls.append((call, (out, lse, sc), [t.clone() for t in (out, lse, sc)]))
    for _, got, _ in calls:
        for t in got:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(8):
        for (call, _, _), st in zip(calls, streams):
            call(st)
    torch.cuda.synchronize()
    for _, got, ref in calls:
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert all(c.model.status() == 0 for c in cases)
