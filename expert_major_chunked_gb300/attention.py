"""The attention operators beside the MoE layer, on torch tensors (include/moe_attention.h has their definitions).

    prefill(q, k, v, cu_q)                      causal attention over packed prompts, grouped heads
    assign_slots(ctx_lens, new_lens, ...)       block tables and slot maps of a step, from the requests' lengths
    append(k, v, slot_map, cache)               keys and values into the 8-bit paged cache
    decode(q, cache, block_table, kv_lens)      one query token a request over that cache

Every call enqueues kernels of libmoe_prefill.so on `stream` (default: the current stream) and returns at once. Results
and scratch are allocated for that stream; where it is not the current stream, the caller orders its inputs before it
(a wait on an event) and the results after it, and the tensors given are marked as used there.
The operators are for serving and have no backward pass. Where an input asks for gradients, results that the call allocates
raise an error when gradients are taken through them; buffers that are given for results, and the cache, have none.
"""

from __future__ import annotations

import importlib.util
import operator
import threading
from typing import NamedTuple, Optional

import torch

from . import binding as _b
from . import build as _build


class KvCache(NamedTuple):
    """The 8-bit paged cache: e4m3 codes [blocks][kv heads][block size][head dim] (torch.float8_e4m3fn or uint8) and
    one float32 scale for each (block, kv head); a stored value is code * scale."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @classmethod
    def empty(cls, num_blocks: int, n_kv_heads: int, block_size: int, head_dim: int, device="cuda") -> "KvCache":
        shape = (num_blocks, n_kv_heads, block_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
        return cls(k, v, *(torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in range(2)))


class Slots(NamedTuple):
    """What assign_slots computes for a step (all on the device)."""
    cu_new: torch.Tensor     # int32 [requests + 1]: the step's tokens are packed request after request
    kv_lens: torch.Tensor    # int32 [requests]: ctx + new
    slot_map: torch.Tensor   # int64 [max_tokens]: block * block_size + offset, -1 where there is none
    positions: torch.Tensor  # int32 [max_tokens]: position in the request, -1 past the last token
    used: torch.Tensor       # int32 [1]: blocks needed from the free list (more than it has: it was too small)


_DTYPES = (torch.bfloat16, torch.float16)
_CODES = (torch.float8_e4m3fn, torch.uint8)
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
_MAX = (1 << 31) - 1
_lock = threading.Lock()
_native = None


def _load():
    """The extension module attention_py (csrc/attention_py.cpp), which makes the calls: it tests the arguments, allocates
    results and calls the library. It returns None for arguments that it does not take (also tensors of another device
    than the current one); the functions below then say what is wrong with them."""
    global _native
    with _lock:
        if _native is None:
            _b.lib()  # builds and loads libmoe_prefill.so
            spec = importlib.util.spec_from_file_location("attention_py", _build.build_extension())
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            _native = module
    return _native


def _tensor(name, t):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, not {type(t).__name__}")
    if max(t.shape, default=0) > _MAX:
        raise ValueError(f"{name} has shape {tuple(t.shape)}: sizes must be below 2^31")


def _rows(name, t, dtype=None, shape=None):
    _tensor(name, t)
    if t.dim() != 3 or not t.is_cuda or t.dtype not in _DTYPES or t.stride(2) != 1:
        raise ValueError(f"{name} must be a [tokens][heads][head_dim] CUDA tensor, bf16 or f16, head_dim dense")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _ints(name, t, dtype=_I32, dim=1):
    _tensor(name, t)
    if t.dtype != dtype or t.dim() != dim or not t.is_cuda or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name} must be a {dim}-D {dtype} CUDA tensor with dense rows")


def _results(q, out, lse, lse_shape):
    if out is not None:
        _rows("out", out, q.dtype, q.shape)
    if lse is not None:
        _tensor("lse", lse)
    if lse is not None and (lse.dtype != _F32 or tuple(lse.shape) != lse_shape or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {lse_shape}")


def _scale(scale):
    try:
        float(1.0 if scale is None else scale)
    except (TypeError, ValueError, OverflowError, RuntimeError):
        raise ValueError(f"scale must be a number, not {scale!r}") from None


def _size(name, v):
    try:
        v = operator.index(v)
    except TypeError:
        raise ValueError(f"{name} must be a whole number, not {v!r}") from None
    if not 0 <= v <= _MAX:
        raise ValueError(f"{name} is {v}: it must be from 0 to 2^31 - 1")


def _cache(cache):
    if not isinstance(cache, tuple) or len(cache) != 4:
        raise ValueError("cache must be a KvCache, or a tuple of its four tensors")
    k, v, ks, vs = cache
    for name, t in zip(KvCache._fields, cache):
        _tensor(f"the cache's {name}", t)
    if k.dim() != 4 or k.dtype not in _CODES or v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("the cache's codes must be two [blocks][kv heads][block size][head dim] tensors, "
                         "float8_e4m3fn or uint8")
    if ks.shape != k.shape[:2] or vs.shape != ks.shape or ks.dtype != _F32 or vs.dtype != _F32:
        raise ValueError("the cache's scales must be float32 [blocks][kv heads]")
    if not all(t.is_cuda and t.is_contiguous() for t in cache):
        raise ValueError("the cache must be contiguous CUDA tensors")


def _same_device(**tensors):
    first = None
    for name, t in tensors.items():
        if t is None:
            continue
        if first is None:
            first = name, t.device
        elif t.device != first[1]:
            raise ValueError(f"{name} is on {t.device}, {first[0]} on {first[1]}")


def _done(result):
    """What the extension returned: results, or the status of a call that the library refused."""
    if type(result) is int:
        raise _b.MoeError(result, _b.moe_prefill_last_error())
    return result


def _elsewhere(call, device, stream, tensors, *args):
    """call(*args) with `device`, or `stream` where there is one, current; the tensors are marked as used there."""
    if stream is None:
        if torch.cuda.current_device() == device.index:
            raise ValueError("an argument is not of the kind that the call takes")
        with torch.cuda.device(device):
            return call(*args)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return call(*args)


class _NoBackward(torch.autograd.Function):
    """A result as it is, with the inputs behind it."""

    @staticmethod
    def forward(ctx, result, *inputs):
        return result.detach()

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the attention operators have no backward pass: they are for serving")


def _wants_grad(*inputs):
    return torch.is_grad_enabled() and any(t.requires_grad for t in inputs)


def _without_backward(call, inputs, out, lse, *args):
    """call(*args)'s (out, lse); those that were not given raise where gradients are taken through them."""
    with torch.no_grad():
        results = call(*args)
    return tuple(r if given is not None else _NoBackward.apply(r, *inputs) for r, given in zip(results, (out, lse)))


def prefill(q, k, v, cu_q, cu_k=None, scale: Optional[float] = None, out=None, lse=None, stream=None):
    """Causal attention over packed sequences; returns (out [tokens][heads][dim], lse float32 [heads][tokens]).

    q [total_q][heads][dim], k and v [total_k][kv heads][dim] (bf16 or f16, any strides with 16-byte aligned rows, such
    as views of one fused projection); sequence b owns rows cu_q[b]:cu_q[b+1] of q and cu_k[b]:cu_k[b+1] of k and v
    (int32 CUDA tensors; cu_k defaults to cu_q). Its queries are the last ones of its keys: query i sees keys up to
    i + k_len - q_len, so a chunk of a longer prompt passes its keys from the start of the prompt. A query that sees no
    key gets zeros and lse = -inf. scale defaults to 1 / sqrt(dim). Rows of out and lse past cu_q[-1] are not written.
    """
    if cu_k is None:
        cu_k = cu_q
    if stream is None:
        r = (_native or _load()).prefill(q, k, v, cu_q, cu_k, scale, out, lse)
        if r is not None:
            return _done(r)
    _rows("q", q)
    _rows("k", k, q.dtype)
    _rows("v", v, q.dtype, k.shape)
    if q.shape[2] != k.shape[2]:
        raise ValueError(f"k has head_dim {k.shape[2]}, q has {q.shape[2]}")
    _ints("cu_q", cu_q)
    _ints("cu_k", cu_k)
    if cu_q.shape[0] < 1 or cu_q.shape != cu_k.shape:
        raise ValueError("cu_q and cu_k must both have one entry more than there are sequences")
    _scale(scale)
    _results(q, out, lse, (q.shape[1], q.shape[0]))
    _same_device(q=q, k=k, v=v, cu_q=cu_q, cu_k=cu_k, out=out, lse=lse)
    if _wants_grad(q, k, v):
        return _without_backward(prefill, (q, k, v), out, lse, q, k, v, cu_q, cu_k, scale, out, lse, stream)
    return _elsewhere(prefill, q.device, stream, (q, k, v, cu_q, cu_k, out, lse), q, k, v, cu_q, cu_k, scale, out, lse)


def raise_on_device_error(stream=None) -> None:
    """Waits for the stream and raises MoeError when a wait inside a prefill kernel on its device has given up since the
    last check."""
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.device(s.device):
        _b._check(_b.lib().moe_attn_check(s.cuda_stream))


def assign_slots(ctx_lens, new_lens, free_blocks, block_table, block_size: int, max_tokens: int, stream=None) -> Slots:
    """Block tables and slot maps of a step. Request b holds ctx_lens[b] cached tokens in the blocks of its row of
    block_table and gets new_lens[b] tokens; the blocks it lacks are taken from free_blocks in order, request after
    request, and written into block_table (in place; entries past a request's last block become -1). max_tokens is the
    size of slot_map and positions: at least the step's tokens, more where the step's buffers are padded."""
    if stream is None:
        r = (_native or _load()).assign(ctx_lens, new_lens, free_blocks, block_table, block_size, max_tokens)
        if r is not None:
            return tuple.__new__(Slots, _done(r))
    _ints("ctx_lens", ctx_lens)
    _ints("new_lens", new_lens)
    _ints("free_blocks", free_blocks)
    _ints("block_table", block_table, dim=2)
    if not ctx_lens.shape[0] == new_lens.shape[0] == block_table.shape[0]:
        raise ValueError("ctx_lens, new_lens and block_table must have one row a request")
    _size("block_size", block_size)
    _size("max_tokens", max_tokens)
    _same_device(ctx_lens=ctx_lens, new_lens=new_lens, free_blocks=free_blocks, block_table=block_table)
    return _elsewhere(assign_slots, ctx_lens.device, stream, (ctx_lens, new_lens, free_blocks, block_table), ctx_lens,
                      new_lens, free_blocks, block_table, block_size, max_tokens)


def append(k, v, slot_map, cache: KvCache, stream=None) -> None:
    """Writes the tokens of k and v [tokens][kv heads][dim] into the cache at slot_map (int64 [tokens] or longer; a
    negative slot skips its token). Tokens of one block follow one another in ascending offsets, as assign_slots lays
    them out. The scale of a block is the smallest power of two that fits its largest magnitude; it grows, with the
    codes that are there rewritten, when a later token is larger."""
    if stream is None:
        r = (_native or _load()).append(k, v, slot_map, cache)
        if r is not None:
            _done(r)
            return
    _rows("k", k)
    _rows("v", v, k.dtype, k.shape)
    _ints("slot_map", slot_map, _I64)
    _cache(cache)
    kc, vc, ks, vs = cache
    if slot_map.shape[0] < k.shape[0]:
        raise ValueError(f"slot_map has {slot_map.shape[0]} entries for {k.shape[0]} tokens")
    if kc.shape[1] != k.shape[1] or kc.shape[3] != k.shape[2]:
        raise ValueError(f"the cache has {kc.shape[1]} kv heads of {kc.shape[3]}, k and v {k.shape[1]} of {k.shape[2]}")
    _same_device(k=k, v=v, slot_map=slot_map, cache_k=kc, cache_v=vc, k_scale=ks, v_scale=vs)
    return _elsewhere(append, k.device, stream, (k, v, slot_map, *cache), k, v, slot_map, cache)


def decode(q, cache: KvCache, block_table, kv_lens, scale: Optional[float] = None, out=None, lse=None, workspace=None,
           stream=None):
    """Attention of one query token a request over the cache; returns (out [requests][heads][dim], lse float32
    [requests][heads]). Request b attends to the first kv_lens[b] slots of the blocks in its row of block_table; a
    request without any gets zeros and lse = -inf. workspace: a uint8 CUDA tensor of decode_workspace() bytes to use
    again from call to call (by default one is kept for each stream)."""
    if stream is None:
        r = (_native or _load()).decode(q, cache, block_table, kv_lens, scale, out, lse, workspace)
        if r is not None:
            return _done(r)
    _rows("q", q)
    _ints("block_table", block_table, dim=2)
    _ints("kv_lens", kv_lens)
    _cache(cache)
    kc, vc, ks, vs = cache
    if kc.shape[3] != q.shape[2]:
        raise ValueError(f"the cache has head_dim {kc.shape[3]}, q has {q.shape[2]}")
    if not block_table.shape[0] == kv_lens.shape[0] == q.shape[0]:
        raise ValueError("block_table and kv_lens must have one row a request")
    _scale(scale)
    _results(q, out, lse, tuple(q.shape[:2]))
    if workspace is not None:
        _tensor("workspace", workspace)
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor")
    _same_device(q=q, block_table=block_table, kv_lens=kv_lens, cache_k=kc, cache_v=vc, k_scale=ks, v_scale=vs, out=out,
                 lse=lse, workspace=workspace)
    if _wants_grad(q):
        return _without_backward(decode, (q,), out, lse, q, cache, block_table, kv_lens, scale, out, lse, workspace, stream)
    return _elsewhere(decode, q.device, stream, (q, block_table, kv_lens, out, lse, workspace, *cache), q, cache,
                      block_table, kv_lens, scale, out, lse, workspace)


def decode_workspace(n_requests: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    """Bytes of scratch that decode() needs for a batch of this size."""
    need = _b.lib().moe_attn_decode_workspace(n_requests, n_heads, n_kv_heads, head_dim)
    if not need:
        raise _b.MoeError(-1, _b.moe_prefill_last_error())
    return need
