"""Torch-facing layer over the C ABI: weights in, paged caches, prefill, decode.

PyTorch provides device memory and streams only; all computation happens in
libswiftkv.so. Every call checks the library's return code and raises
``SwiftKVError`` on failure.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np
import torch

from . import binding as B


def _stream(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


# the current stream's handle without a Stream object around it, where PyTorch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(dev: torch.device, stream) -> int:
    # dev.index is set: the devices here are those of CUDA tensors
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev.index)
    return (stream if stream is not None else torch.cuda.current_stream(dev)).cuda_stream


def _empty(shape, dtype, dev: torch.device, stream) -> torch.Tensor:
    """An output that work on `stream` (None: the current one) will write. Its memory is that stream's:
    a block of the current stream may still be in use by what was enqueued there before."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


_I32 = np.dtype(np.int32)


def _int32(*values: int) -> None:
    """ctypes takes a number's low 32 bits without a word."""
    for x in values:
        if not -0x80000000 <= x <= 0x7fffffff:
            raise ValueError(f"{x} does not fit 32 bits")


def _ints(a) -> np.ndarray:
    """A call's host list as int32. (NumPy refuses Python numbers past 32 bits by itself, but wraps an
    array's.)"""
    if type(a) is np.ndarray and a.dtype is _I32:
        return a
    if type(a) not in (list, tuple):
        a = np.asarray(a)
        if not np.array_equal(a.astype(np.int32), a):
            raise ValueError("a list with numbers that do not fit 32 bits")
    return np.ascontiguousarray(a, dtype=np.int32)


def _ptr(a) -> Optional[int]:
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        assert a.flags["C_CONTIGUOUS"]
        return a.ctypes.data
    assert a.is_contiguous()
    return a.data_ptr()


@dataclass
class Shape:
    L: int
    d: int
    n_q: int
    n_kv: int
    d_h: int
    ffn: int
    vocab: int
    rope_theta: float
    rms_eps: float = 1e-5
    qkv_bias: bool = False

    @classmethod
    def of(cls, s):
        return cls(L=s.L, d=s.d, n_q=s.n_q, n_kv=s.n_kv, d_h=s.d_h, ffn=s.ffn, vocab=s.vocab,
                   rope_theta=s.rope_theta, rms_eps=s.rms_eps, qkv_bias=s.qkv_bias)

    def config(self) -> B.ModelConfig:
        return B.ModelConfig(self.L, self.d, self.n_q, self.n_kv, self.d_h, self.ffn, self.vocab,
                             int(self.qkv_bias), self.rope_theta, self.rms_eps)


class Model:
    """A SwiftKV model on the current CUDA device, packed for (l, g)."""

    def __init__(self, shape, l: int, g: int = 1):
        self.shape = Shape.of(shape)
        self.l, self.g = l, g
        self.num_caches = B.cache_count(self.shape.L, l, g)
        self._cfg = self.shape.config()
        h = C.c_void_p()
        B.check(B.lib().swiftkv_model_create(C.byref(self._cfg), l, g, C.byref(h)))
        self.handle = h
        self.device = torch.device("cuda", torch.cuda.current_device())

    def load_layer(self, j: int, w: dict, stream=None) -> None:
        lw = B.LayerWeights(*[_ptr(w.get(k)) for k in (
            "gamma_attn", "wq", "wk", "wv", "bq", "bk", "bv", "wo", "gamma_mlp", "wg", "wu", "wd")])
        B.check(B.lib().swiftkv_load_layer(self.handle, j, C.byref(lw), _stream(stream)))

    def load_globals(self, w: dict, stream=None) -> None:
        B.check(B.lib().swiftkv_load_globals(self.handle, _ptr(w["embed"]), _ptr(w["gamma_final"]),
                                             _ptr(w["lm_head"]), _stream(stream)))

    def free(self) -> None:
        if getattr(self, "handle", None) is not None and self.handle.value:
            B.lib().swiftkv_free(self.handle)
            self.handle = C.c_void_p()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass

    def status(self, clear: bool = True) -> int:
        return B.check(B.lib().swiftkv_status(self.handle, int(clear)))

    def set_attention_window(self, window: int, sinks: int = 0) -> None:
        """Later calls see the last `window` tokens and the first `sinks` (0: all of them)."""
        _int32(window, sinks)
        B.check(B.lib().swiftkv_set_attention_window(self.handle, window, sinks))

    def set_score_pools(self, scores: Optional[torch.Tensor], decay: float = 1.0) -> None:
        """Later calls add every layer's attention weights to scores (float32 [num_caches, num_pages,
        n_kv, 16] on the model's device, e.g. KVCache.new_scores(); kept alive here); None turns that
        off. Rows that a call writes start from 0. Sequences of a call must not share pages while it
        is on."""
        if scores is None:
            B.check(B.lib().swiftkv_set_score_pools(self.handle, None, 0, decay))
        else:
            s = self.shape
            if scores.dim() != 4 or scores.shape[0] != self.num_caches or tuple(scores.shape[2:]) != (s.n_kv, 16):
                raise ValueError(f"scores: float32 [{self.num_caches}, pages, {s.n_kv}, 16]")
            base = _flat(scores, torch.float32, tuple(scores.shape), self.device, "scores")
            step = scores.stride(0) * 4
            ptrs = (C.c_void_p * self.num_caches)(*[base + c * step for c in range(self.num_caches)])
            B.check(B.lib().swiftkv_set_score_pools(self.handle, ptrs, scores.shape[1], decay))
        self._scores = scores

    def memory(self):
        wb, sb = C.c_size_t(), C.c_size_t()
        B.check(B.lib().swiftkv_memory(self.handle, C.byref(wb), C.byref(sb)))
        return wb.value, sb.value


def load_synthetic(shape, l: int, g: int = 1, seed: int = 0, gain_std: float = 0.0) -> Model:
    """Model with the seeded synthetic weights of the shared generator (inputs only)."""
    import synth
    m = Model(shape, l, g)
    for j in range(shape.L):
        rep = j < l or (j - l) % g == 0
        kinds = None if rep else ("wq", "wo", "wg", "wu", "wd", "gamma_attn", "gamma_mlp", "bq")
        m.load_layer(j, synth.layer_weights(shape, j, seed=seed, gain_std=gain_std, kinds=kinds))
    m.load_globals(synth.global_weights(shape, seed=seed, gain_std=gain_std))
    return m


_KV_DTYPES = {"bf16": torch.bfloat16, "fp8": torch.uint8, "int8": torch.int8}  # in the order of kv_dtype


class KVCache:
    """Caller-owned paged KV cache: num_caches x (K, V) pools of [num_pages][n_kv][16][d_h]
    elements plus a device block table. dtype "bf16": bfloat16 elements; dtype "fp8":
    uint8 float8-e4m3 codes with float32 scales [num_pages][n_kv][16] per pool (per-token
    FP8); dtype "int8": int8 codes with float32 scales [num_pages][n_kv], one for each page and
    head."""

    def __init__(self, model: Model, num_pages: int, block_table: np.ndarray, device=None, dtype: str = "bf16"):
        if dtype not in _KV_DTYPES:
            raise ValueError(f"KV cache dtype {dtype!r}")
        s = model.shape
        dev = device or torch.device("cuda", torch.cuda.current_device())
        self.num_pages, self.dtype = num_pages, dtype
        self.heads = (s.n_kv, s.d_h)
        shape = (model.num_caches, num_pages, s.n_kv, 16, s.d_h)
        elem = _KV_DTYPES[dtype]
        self.k = torch.zeros(shape, dtype=elem, device=dev)
        self.v = torch.zeros(shape, dtype=elem, device=dev)
        self.device = self.k.device
        self.k_scale = self.v_scale = None
        if dtype != "bf16":
            per = shape[:-1] if dtype == "fp8" else shape[:-2]
            self.k_scale = torch.zeros(per, dtype=torch.float32, device=dev)
            self.v_scale = torch.zeros(per, dtype=torch.float32, device=dev)
        self.block_table = torch.as_tensor(np.ascontiguousarray(block_table, dtype=np.int32), device=dev)
        n = model.num_caches
        self._kp = (C.c_void_p * n)(*[self.k[c].data_ptr() for c in range(n)])
        self._vp = (C.c_void_p * n)(*[self.v[c].data_ptr() for c in range(n)])
        self._ks = self._vs = None
        if dtype != "bf16":
            self._ks = (C.c_void_p * n)(*[self.k_scale[c].data_ptr() for c in range(n)])
            self._vs = (C.c_void_p * n)(*[self.v_scale[c].data_ptr() for c in range(n)])
        self.num_caches = n
        self._set_pages(self._pages(self.block_table))

    def _pages(self, block_table: torch.Tensor) -> B.KVPages:
        ptr = lambda a: C.cast(a, C.POINTER(C.c_void_p)) if a is not None else None  # noqa: E731
        return B.KVPages(ptr(self._kp), ptr(self._vp), self.num_caches, self.num_pages, 16, block_table.data_ptr(),
                         block_table.shape[1], list(_KV_DTYPES).index(self.dtype), ptr(self._ks), ptr(self._vs))

    def _set_pages(self, pages: B.KVPages) -> None:
        self.pages, self.pages_ref = pages, C.byref(pages)
        self.num_rows = self.block_table.shape[0]

    def new_scores(self) -> torch.Tensor:
        """Zeroed accumulated attention weights, one per cached key: [num_caches, num_pages, n_kv, 16]."""
        return torch.zeros((self.num_caches, self.num_pages, self.k.shape[2], 16), dtype=torch.float32,
                           device=self.k.device)

    def view(self, rows: Sequence[int]) -> "KVCache":
        """The same pools with block table rows `rows` (in that order): a batch that holds
        only some of the sequences, or holds them in another order."""
        out = object.__new__(KVCache)
        out.__dict__.update(self.__dict__)
        out.block_table = self.block_table[torch.as_tensor(list(rows), dtype=torch.long,
                                                           device=self.block_table.device)].contiguous()
        out._set_pages(out._pages(out.block_table))
        return out

    def _rows(self, pool: torch.Tensor, s: int, n: int) -> torch.Tensor:
        bt = self.block_table[s]
        pos = torch.arange(n, device=pool.device)
        return pool[bt[pos // 16].long(), :, pos % 16]

    def gather(self, c: int, s: int, n: int, which: str = "k") -> torch.Tensor:
        """Cache c's first n rows of sequence s, [n, n_kv, d_h] (test/inspection helper);
        for an fp8 or int8 cache the values code * scale in float32."""
        pool = self.k[c] if which == "k" else self.v[c]
        if self.dtype == "bf16":
            return self._rows(pool, s, n)
        return self.codes(c, s, n, which) * self.scales(c, s, n, which)[..., None]

    def codes(self, c: int, s: int, n: int, which: str = "k") -> torch.Tensor:
        """fp8 or int8 cache: the codes of cache c's first n rows of sequence s, as float32."""
        pool = self.k[c] if which == "k" else self.v[c]
        rows = self._rows(pool, s, n)
        return (rows.view(torch.float8_e4m3fn) if self.dtype == "fp8" else rows).float()

    def scales(self, c: int, s: int, n: int, which: str = "k") -> torch.Tensor:
        """fp8 or int8 cache: the float32 scales [n, n_kv] of cache c's first n rows of sequence s."""
        pool = self.k_scale[c] if which == "k" else self.v_scale[c]
        if self.dtype == "int8":
            return pool[self.block_table[s][torch.arange(n, device=pool.device) // 16].long()]
        return self._rows(pool, s, n)


def prefill(model: Model, tokens: torch.Tensor, cu_seqlens: Sequence[int], kv: KVCache,
            logits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """SwiftKV prefill: fills every cache of kv, returns [P, V] last-token logits."""
    cu = np.ascontiguousarray(cu_seqlens, dtype=np.int32)
    P = len(cu) - 1
    if logits is None:
        logits = torch.empty((P, model.shape.vocab), dtype=torch.float32, device=kv.k.device)
    tokens = tokens.to(torch.int32).contiguous()
    B.check(B.lib().swiftkv_prefill(model.handle, tokens.data_ptr(), cu.ctypes.data, P, model.l, model.g,
                                    C.byref(kv.pages), logits.data_ptr(), _stream(stream)))
    return logits


def prefill_host(model: Model, tokens: np.ndarray, cu_seqlens: Sequence[int], kv: KVCache,
                 logits: Optional[np.ndarray] = None, stream=None) -> np.ndarray:
    """prefill with host token ids and host logits (copies inside the call; synchronous)."""
    cu = np.ascontiguousarray(cu_seqlens, dtype=np.int32)
    P = len(cu) - 1
    if logits is None:
        logits = np.empty((P, model.shape.vocab), dtype=np.float32)
    B.check(B.lib().swiftkv_prefill_host(model.handle, _ptr(tokens), cu.ctypes.data, P, model.l, model.g,
                                         C.byref(kv.pages), _ptr(logits), _stream(stream)))
    return logits


def forward(model: Model, tokens: torch.Tensor, cu_seqlens: Sequence[int], ctx_lens: Optional[Sequence[int]],
            kv: KVCache, logits: Optional[torch.Tensor] = None, stream=None,
            pos_offsets: Optional[Sequence[int]] = None) -> torch.Tensor:
    """Serving forward over prompt chunks and decode tokens: chunk s follows ctx_lens[s]
    tokens already in kv (None: none); returns [P, V] logits of each chunk's last token. After an
    eviction ctx_lens[s] counts the keys that are left and pos_offsets[s] those that are gone."""
    cu = np.ascontiguousarray(cu_seqlens, dtype=np.int32)
    P = len(cu) - 1
    ctx = None if ctx_lens is None else np.ascontiguousarray(ctx_lens, dtype=np.int32)
    if ctx is not None and len(ctx) != P:
        raise ValueError(f"ctx_lens has {len(ctx)} entries for {P} chunks")
    if logits is None:
        logits = torch.empty((P, model.shape.vocab), dtype=torch.float32, device=kv.k.device)
    tokens = tokens.to(torch.int32).contiguous()
    if pos_offsets is not None:
        off = np.ascontiguousarray(_ints(pos_offsets))
        if len(off) != P:
            raise ValueError(f"pos_offsets has {len(off)} entries for {P} chunks")
        B.check(B.lib().swiftkv_forward_at(model.handle, tokens.data_ptr(), cu.ctypes.data,
                                           None if ctx is None else ctx.ctypes.data, off.ctypes.data, P, model.l,
                                           model.g, C.byref(kv.pages), logits.data_ptr(), _stream(stream)))
        return logits
    B.check(B.lib().swiftkv_forward(model.handle, tokens.data_ptr(), cu.ctypes.data,
                                    None if ctx is None else ctx.ctypes.data, P, model.l, model.g,
                                    C.byref(kv.pages), logits.data_ptr(), _stream(stream)))
    return logits


def decode_step(model: Model, tokens: torch.Tensor, seq_lens: Sequence[int], kv: KVCache, stream=None):
    """One decode token per sequence; returns (logits [B, V], next token ids [B])."""
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    Bsz = len(sl)
    dev = kv.device
    logits = torch.empty((Bsz, model.shape.vocab), dtype=torch.float32, device=dev)
    nxt = torch.empty((Bsz,), dtype=torch.int32, device=dev)
    tokens = tokens.to(torch.int32).contiguous()
    B.check(B.lib().swiftkv_decode_step(model.handle, tokens.data_ptr(), sl.ctypes.data, Bsz, C.byref(kv.pages),
                                        logits.data_ptr(), nxt.data_ptr(), _stream(stream)))
    return logits, nxt


def _fits(model: Model, kv: KVCache) -> None:
    if kv.heads != (model.shape.n_kv, model.shape.d_h):
        raise ValueError(f"a cache of (n_kv, d_h) {kv.heads} for a model of {(model.shape.n_kv, model.shape.d_h)}")
    if kv.device != model.device:
        raise ValueError(f"a cache on {kv.device} for a model on {model.device}")


def _chunks(cu_seqlens, ctx_lens, kv: KVCache, model: Model):
    """Host int32 arrays of a ragged batch, checked against the block table: (cu, ctx, P, T)."""
    _fits(model, kv)
    cu = _ints(cu_seqlens)
    ctx = None if ctx_lens is None else _ints(ctx_lens)
    P = cu.shape[0] - 1 if cu.ndim == 1 else -1
    if P < 0 or (ctx is not None and ctx.shape != (P,)):
        raise ValueError("cu_seqlens: [P + 1], ctx_lens: [P]")
    if P > kv.num_rows:
        raise ValueError(f"{P} chunks, but the block table has {kv.num_rows} rows")
    return cu, ctx, P, int(cu[P])


def _rows_of(t: torch.Tensor, T: int, model: Model, dev, name: str) -> int:
    """Row stride of bf16 rows [T, n_q, d_h] (or [T, n_q * d_h]) whose heads are contiguous."""
    s, shape, stride = model.shape, t.shape, t.stride()
    if t.dtype is not torch.bfloat16 or t.device != dev or shape[0] != T or not (
            len(shape) == 3 and shape[1] == s.n_q and shape[2] == s.d_h and stride[2] == 1 and
            (s.n_q == 1 or stride[1] == s.d_h) or
            len(shape) == 2 and shape[1] == s.n_q * s.d_h and stride[1] == 1):
        raise ValueError(f"{name}: bfloat16 [{T}, {s.n_q}, {s.d_h}] on {dev}, the heads of a row contiguous")
    ld = stride[0] if T > 1 else s.n_q * s.d_h
    if ld > 0x7fffffff:
        _int32(ld)
    return ld


def _flat(t: torch.Tensor, dtype, shape: tuple, dev, name: str) -> int:
    """Address of a contiguous tensor of this type and shape on dev."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous {dtype} {list(shape)} on {dev}")
    return t.data_ptr()


def _new_rows(t: torch.Tensor, T: int, heads: int, caches: int, d_h: int, dev, name: str):
    """Row stride and the stride between caches of bf16 rows [T, heads, d_h], or [T, caches, heads, d_h]."""
    shape, stride = t.shape, t.stride()
    many = len(shape) == 4 or caches > 1
    if t.dtype is not torch.bfloat16 or t.device != dev or shape != ((T, caches, heads, d_h) if many else (T, heads, d_h)):
        raise ValueError(f"{name}: bfloat16 [{T}, {heads}, {d_h}] or, for several caches, [{T}, {caches}, {heads}, {d_h}] on {dev}")
    if T and (stride[-1] != 1 or heads > 1 and stride[-2] != d_h):
        raise ValueError(f"{name}: the heads of a row have to be contiguous")
    step = stride[1] if many and caches > 1 else heads * d_h
    ld = stride[0] if T > 1 else max(0, (caches - 1) * step) + heads * d_h
    if ld > 0x7fffffff:
        _int32(ld)
    return ld, step


def append(model: Model, k: torch.Tensor, v: torch.Tensor, cu_seqlens: Sequence[int], ctx_lens: Optional[Sequence[int]],
           kv: KVCache, cache: int = 0, q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
           pos_offsets: Optional[Sequence[int]] = None, rotate: bool = True, stream=None) -> Optional[torch.Tensor]:
    """Writes the keys and values of chunks of new tokens, k and v [T, n_kv, d_h] bf16 (rows may be strided:
    parts of one projection), into cache `cache` of kv, ahead of attend. Chunk s follows ctx_lens[s] cached
    tokens (None: none). Keys, and q [T, n_q, d_h] if given, are rotated to their positions, pos_offsets[s]
    ahead of the cache's rows (after an eviction: the tokens that are gone); with rotate=False nothing is.
    k and v of shape [T, n, n_kv, d_h] fill the n caches from `cache` on. Returns the rotated q: q_out, which may
    be q itself, or a new tensor; None without q."""
    cu, ctx, P, T = _chunks(cu_seqlens, ctx_lens, kv, model)
    if cache:
        _int32(cache)
    dev, s = kv.device, model.shape
    off = None if pos_offsets is None else _ints(pos_offsets)
    if off is not None and off.shape != (P,):
        raise ValueError("pos_offsets: [P]")
    shape = k.shape
    n = shape[1] if len(shape) == 4 else 1
    r = B.NewRows()
    r.ldk, r.k_step = ld = _new_rows(k, T, s.n_kv, n, s.d_h, dev, "k")
    if v.shape != shape or v.dtype is not torch.bfloat16 or v.device != dev or v.stride() != k.stride():
        ld = _new_rows(v, T, s.n_kv, n, s.d_h, dev, "v")
    r.ldv, r.v_step = ld
    r.k, r.v = k.data_ptr(), v.data_ptr()
    if q is not None:
        r.ldq = _rows_of(q, T, model, dev, "q")
        if q_out is None:
            q_out = _empty((T, s.n_q, s.d_h), torch.bfloat16, dev, stream)
        r.ldq_out = _rows_of(q_out, T, model, dev, "q_out")
        r.q, r.q_out = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    B.check(B.lib().swiftkv_append(model.handle, cache, n, r, B.host(cu), B.host(ctx), B.host(off), P, kv.pages_ref,
                                   int(rotate), _stream_of(dev, stream)))
    return q_out


def attend(model: Model, q: torch.Tensor, cu_seqlens: Sequence[int], ctx_lens: Optional[Sequence[int]], kv: KVCache,
           cache: int = 0, window: int = 0, sinks: int = 0, out: Optional[torch.Tensor] = None,
           lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of chunks of new tokens, q [T, n_q, d_h] bf16, over one cache of kv that already
    holds their keys and values. Chunk s follows ctx_lens[s] cached tokens (None: none). A token at
    position p sees positions <= p; with window > 0 only those above p - window, and the first
    `sinks`. Returns out [T, n_q, d_h] bf16; lse (float32 [n_q, T]), if given, receives each row's
    log-sum-exp, which attention_weights takes."""
    cu, ctx, P, T = _chunks(cu_seqlens, ctx_lens, kv, model)
    if cache or window or sinks:
        _int32(cache, window, sinks)
    dev = kv.device
    ldq = _rows_of(q, T, model, dev, "q")
    if out is None:
        out = _empty((T, model.shape.n_q, model.shape.d_h), torch.bfloat16, dev, stream)
    ldo = _rows_of(out, T, model, dev, "out")
    lp = None if lse is None else _flat(lse, torch.float32, (model.shape.n_q, T), dev, "lse")
    B.check(B.lib().swiftkv_attend(model.handle, cache, q.data_ptr(), ldq, B.host(cu), B.host(ctx), P, kv.pages_ref,
                                   window, sinks, out.data_ptr(), ldo, lp, _stream_of(dev, stream)))
    return out


def attention_weights(model: Model, q: torch.Tensor, lse: torch.Tensor, cu_seqlens: Sequence[int],
                      ctx_lens: Optional[Sequence[int]], kv: KVCache, scores: torch.Tensor, cache: int = 0,
                      window: int = 0, sinks: int = 0, decay: float = 1.0, stream=None) -> torch.Tensor:
    """Adds the attention weight that each cached key received from these tokens, summed over them
    and the query heads of its KV head, to scores (float32 [num_pages, n_kv, 16], one per key of the
    cache): scores = decay * scores + weight for every key some token sees, the others unchanged. The
    entry of a key that is new to the cache has to be 0.
    q and lse are those of the attend call before. Returns scores."""
    cu, ctx, P, T = _chunks(cu_seqlens, ctx_lens, kv, model)
    if cache or window or sinks:
        _int32(cache, window, sinks)
    dev, s = kv.device, model.shape
    ldq = _rows_of(q, T, model, dev, "q")
    lp = _flat(lse, torch.float32, (s.n_q, T), dev, "lse")
    sp = _flat(scores, torch.float32, (kv.num_pages, s.n_kv, 16), dev, "scores")
    B.check(B.lib().swiftkv_attention_weights(model.handle, cache, q.data_ptr(), ldq, lp, B.host(cu), B.host(ctx), P,
                                              kv.pages_ref, window, sinks, decay, sp, _stream_of(dev, stream)))
    return scores


def evict(model: Model, kv: KVCache, scores: torch.Tensor, seq_lens: Sequence[int], keep: int, sinks: int = 0,
          recent: int = 0, cache: Optional[int] = None, dst_block_table: Optional[torch.Tensor] = None,
          kept: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Shrinks each sequence to at most `keep` keys, per cache and KV head: the first `sinks`, the
    last `recent`, and of the others those with the largest scores (float32 [num_caches, num_pages,
    n_kv, 16]; with `cache`, that cache's [num_pages, n_kv, 16]), ties to the earlier key. Kept rows
    move in order to rows 0.. of the sequence's own pages, or of dst_block_table's (int32 [P, n],
    pages no sequence uses now; the source is then only read). Returns kept, the former indices
    [caches, P, n_kv, keep] int32, -1 behind a shorter list; sequence s then holds
    min(seq_lens[s], keep) keys."""
    _fits(model, kv)
    sl = _ints(seq_lens)
    _int32(keep, sinks, recent)
    P, dev, s = sl.shape[0], kv.device, model.shape
    if P > kv.num_rows:
        raise ValueError(f"{P} sequences, but the block table has {kv.num_rows} rows")
    if keep < 1 or (cache is not None and not 0 <= cache < kv.num_caches):
        raise ValueError(f"keep {keep}, cache {cache} of {kv.num_caches}")
    pool = (kv.num_pages, s.n_kv, 16)
    n = kv.num_caches if cache is None else 1
    base = _flat(scores, torch.float32, pool if cache is not None else (n,) + pool, dev, "scores")
    dst, width = None, 0
    if dst_block_table is not None:
        rows, width = dst_block_table.shape if dst_block_table.dim() == 2 else (-1, 0)
        if rows < P:
            raise ValueError(f"dst_block_table: int32 [{P}, pages]")
        dst = _flat(dst_block_table, torch.int32, (rows, width), dev, "dst_block_table")
    shape = (n, P, s.n_kv, keep)
    if kept is None:
        kept = _empty(shape, torch.int32, dev, stream)
        kp = kept.data_ptr()
    else:
        kp = _flat(kept, torch.int32, shape, dev, "kept")
    step, first = 4 * kv.num_pages * s.n_kv * 16, cache or 0
    ptrs = (C.c_void_p * kv.num_caches)(*[base + (c - first) * step if 0 <= c - first < n else None
                                          for c in range(kv.num_caches)])
    B.check(B.lib().swiftkv_evict(model.handle, -1 if cache is None else cache, kv.pages_ref, ptrs, B.host(sl), P, keep,
                                  sinks, recent, dst, width, kp, _stream_of(dev, stream)))
    return kept


def _matrix(t: torch.Tensor, dtype, rows: int, cols: Optional[int], dev, name: str):
    """Address, row stride and columns of a matrix [rows, cols] whose rows are contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or t.dtype is not dtype or t.device != dev or shape[0] != rows or (
            cols is not None and shape[1] != cols) or (shape[1] > 1 and stride[1] != 1):
        raise ValueError(f"{name}: {dtype} [{rows}, {'n' if cols is None else cols}] on {dev}, contiguous within a row")
    return t.data_ptr(), stride[0] if rows > 1 else shape[1], shape[1]


def adjust_logits(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, lens: Optional[torch.Tensor] = None,
                  prompt_lens: Optional[torch.Tensor] = None, repetition=1.0, presence=0.0, frequency=0.0,
                  bias_ids: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Penalties, biases and grammar masks on float32 logits [P, V] (rows may be strided), ahead of sample.
    tokens int32 [P, N] are the rows' histories, the first lens[r] of row r (None: all N), of which the first
    prompt_lens[r] are its prompt (None: none). Ids in the history have their logit divided by `repetition` where
    it is positive and multiplied by it elsewhere; `frequency` for each time behind the prompt and `presence`
    once are subtracted; all three are numbers or float32 [P]. bias [P, B] float32 is added to the ids bias_ids
    [P, B] int32 (-1: unused; the last entry of an id counts). mask int32 [P, (V + 31) // 32] allows id i of row r
    by bit i % 32 of mask[r, i // 32]; the others become -inf. Returns out, which may be logits itself, or a
    new tensor. Enqueued without synchronising."""
    if logits.dim() != 2 or logits.dtype is not torch.float32 or not logits.is_cuda:
        raise ValueError("logits: float32 CUDA [P, V]")
    (P, V), (ld, step), dev = logits.shape, logits.stride(), logits.device
    if P <= 1:
        ld = V
    if V < 1 or (V > 1 and step != 1) or ld < V:
        raise ValueError("logits: at least one column, contiguous within a row, rows that do not overlap")
    i32, f32, vec, a = torch.int32, torch.float32, (P,), B.Adjustments()
    if P > 0x7fffffff or V > 0x7fffffff:
        _int32(P, V)
    if tokens is not None:
        a.tokens, a.ld_tokens, n = _matrix(tokens, i32, P, None, dev, "tokens")
        if n > 0x7fffffff:
            _int32(n)
        a.max_tokens = n
        if lens is not None:
            a.lens = _flat(lens, i32, vec, dev, "lens")
        if prompt_lens is not None:
            a.prompt_lens = _flat(prompt_lens, i32, vec, dev, "prompt_lens")
        if isinstance(repetition, torch.Tensor):
            a.repetition = _flat(repetition, f32, vec, dev, "repetition")
        else:
            a.repetition_all = repetition
        if isinstance(presence, torch.Tensor):
            a.presence = _flat(presence, f32, vec, dev, "presence")
        else:
            a.presence_all = presence
        if isinstance(frequency, torch.Tensor):
            a.frequency = _flat(frequency, f32, vec, dev, "frequency")
        else:
            a.frequency_all = frequency
    elif lens is not None or prompt_lens is not None:
        raise ValueError("lens and prompt_lens belong to tokens")
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias go together")
    if bias is not None:
        n = bias.shape[1] if bias.dim() == 2 else -1
        if n > 0x7fffffff:
            _int32(n)
        a.bias_ids, a.bias, a.num_bias = (_flat(bias_ids, i32, (P, n), dev, "bias_ids"),
                                          _flat(bias, f32, (P, n), dev, "bias"), n)
    if mask is not None:
        a.mask, a.ld_mask, _ = _matrix(mask, i32, P, (V + 31) // 32, dev, "mask")
    if out is None:
        out = _empty((P, V), f32, dev, stream)
    op, ldo, _ = _matrix(out, f32, P, V, dev, "out")
    args = (logits.data_ptr(), P, V, ld, a, op, ldo, _stream_of(dev, stream))
    if torch.cuda.current_device() == dev.index:
        B.check(B.lib().swiftkv_adjust_logits(*args))
    else:
        with torch.cuda.device(dev):
            B.check(B.lib().swiftkv_adjust_logits(*args))
    return out


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
           out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token id (int32) per row of float32 logits [P, V] (rows may be strided), drawn with the
    uniform numbers u [P] in [0, 1). temperature, top_k, top_p and min_p are numbers, or one value
    per row as tensors on the same device (float32; top_k int32); temperature <= 0 takes the argmax,
    top_k <= 0, top_p >= 1 and min_p <= 0 are off. Enqueued without synchronising."""
    if logits.dim() != 2 or logits.dtype is not torch.float32 or not logits.is_cuda:
        raise ValueError("logits: float32 CUDA [P, V]")
    (P, V), (ld, step), dev = logits.shape, logits.stride(), logits.device
    if P <= 1:
        ld = V
    if V < 1 or (V > 1 and step != 1) or ld < V:
        raise ValueError("logits: at least one column, contiguous within a row, rows that do not overlap")
    vec, f32, s = (P,), torch.float32, B.Sampling()
    if isinstance(temperature, torch.Tensor):
        s.temperature = _flat(temperature, f32, vec, dev, "temperature")
    else:
        s.temperature_all = temperature
    if isinstance(top_k, torch.Tensor):
        s.top_k = _flat(top_k, torch.int32, vec, dev, "top_k")
    else:
        s.top_k_all = max(0, min(int(top_k), 0x7fffffff))
    if isinstance(top_p, torch.Tensor):
        s.top_p = _flat(top_p, f32, vec, dev, "top_p")
    else:
        s.top_p_all = top_p
    if isinstance(min_p, torch.Tensor):
        s.min_p = _flat(min_p, f32, vec, dev, "min_p")
    else:
        s.min_p_all = min_p
    if out is None:
        out = _empty(vec, torch.int32, dev, stream)
    args = (logits.data_ptr(), P, V, ld, s, _flat(u, f32, vec, dev, "u"), _flat(out, torch.int32, vec, dev, "out"),
            _stream_of(dev, stream))
    if torch.cuda.current_device() == dev.index:
        B.check(B.lib().swiftkv_sample(*args))
    else:
        with torch.cuda.device(dev):
            B.check(B.lib().swiftkv_sample(*args))
    return out
