"""Torch-facing wrapper of the C ABI.  PyTorch supplies device memory and
streams; the verify step itself runs in the library's kernels.

    accepted_len, out_tokens = spec_verify(target, draft, draft_tokens,
                                           uniforms, temperature)

``target`` [B, K+1, V] and ``draft`` [B, K, V] are CUDA tensors of
torch.bfloat16 or torch.float32; ``draft_tokens`` [B, K] int32;
``uniforms`` [B, K+1] float32; ``temperature`` [B] float32 (0 = greedy).

``paged_plan``, ``paged_append`` and ``paged_attention`` are the target
model's pass over a paged key/value cache, with the request lengths on the
device: a step plans its pages and slots, and every layer appends the new
tokens' keys and values and attends.  ``paged_append_rotary`` appends with
the position rotation on the way; ``PagedCacheFp4`` is a cache of 4 bits, with
``paged_append_fp4``, ``paged_read_fp4`` and ``paged_attention_fp4``.
"""
from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional

import torch

from . import _native as N
from . import _native as _N

_DTYPES = {torch.bfloat16: N.SV_BF16, torch.float32: N.SV_F32}
_CACHE_DTYPES = {torch.bfloat16: N.SV_BF16, torch.float16: N.SV_F16}
_workspaces: dict = {}
_attention_workspaces: dict = {}   # (device, stream, D): workspace of calls outside captures
_captured_workspaces: dict = {}    # (device, stream, D): (capture, workspace of that capture)


class VerifyResult(NamedTuple):
    accepted_len: torch.Tensor           # [B] int32, -1 = error row
    out_tokens: torch.Tensor             # [B, K+1] int32, -1 padded
    logp: Optional[torch.Tensor] = None  # [B, K] float32 log p_t(x_t)
    logq: Optional[torch.Tensor] = None  # [B, K] float32 log q_t(x_t)


def _check(t: torch.Tensor, name: str, dtype=None, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_HERE = contextlib.nullcontext()


def _device(dev: torch.device):
    """Makes ``dev`` the current device, on which the library launches."""
    if dev.index == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(dev)


def _stream(stream: Optional[torch.cuda.Stream], dev: torch.device) -> torch.cuda.Stream:
    """``stream``, the device's current one if None."""
    if stream is None:
        return torch.cuda.current_stream(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, expected {dev}")
    return stream


def workspace_for(B: int, K: int, V: int, dtype: int, device: torch.device,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """A cached device workspace large enough for this shape, one per
    (device, stream): calls on one stream run in order and may share it,
    calls on different streams may overlap and must not."""
    need = N.spec_verify_workspace_bytes(B, K, V, dtype)
    if need == 0:
        raise ValueError(f"invalid shape B={B} K={K} V={V}")
    index = device.index if device.index is not None else torch.cuda.current_device()
    st = stream if stream is not None else torch.cuda.current_stream(index)
    key = (index, st.cuda_stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        with torch.cuda.stream(st):   # allocated for use on this stream
            ws = torch.empty(max(need, 1 << 20), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def spec_verify(target: torch.Tensor, draft: torch.Tensor, draft_tokens: torch.Tensor,
                uniforms: torch.Tensor, temperature: torch.Tensor, *,
                k_per_row: Optional[torch.Tensor] = None,
                want_logprobs: bool = False, out: Optional[VerifyResult] = None,
                workspace: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> VerifyResult:
    """Verify a batch on the current (or given) CUDA stream; no host sync.

    ``k_per_row`` ([B] int32, optional): row b verifies only its first
    k_per_row[b] drafted tokens (adaptive verification, spec_verify_ragged).
    """
    if target.dim() != 3:
        raise ValueError("target must be [B, K+1, V]")
    B, K1, V = target.shape
    K = K1 - 1
    dev = target.device
    if target.dtype not in _DTYPES:
        raise TypeError(f"target dtype {target.dtype} is not bfloat16 or float32")
    dt = _DTYPES[target.dtype]
    _check(target, "target", device=dev)
    _check(draft, "draft", dtype=target.dtype, shape=(B, K, V), device=dev)
    _check(draft_tokens, "draft_tokens", dtype=torch.int32, shape=(B, K), device=dev)
    _check(uniforms, "uniforms", dtype=torch.float32, shape=(B, K + 1), device=dev)
    _check(temperature, "temperature", dtype=torch.float32, shape=(B,), device=dev)
    st = _stream(stream, dev)
    if out is None:
        with torch.cuda.stream(st):   # outputs belong to the stream that writes them
            out = VerifyResult(
                torch.empty(B, dtype=torch.int32, device=dev),
                torch.empty(B, K + 1, dtype=torch.int32, device=dev),
                torch.empty(B, K, dtype=torch.float32, device=dev) if want_logprobs else None,
                torch.empty(B, K, dtype=torch.float32, device=dev) if want_logprobs else None)
    if workspace is None:
        workspace = workspace_for(B, K, V, dt, dev, st)
    lp = out.logp.data_ptr() if out.logp is not None else None
    lq = out.logq.data_ptr() if out.logq is not None else None
    ws_bytes = workspace.numel() * workspace.element_size()
    if k_per_row is None:
        with _device(dev):
            status = N.spec_verify_raw(
                target.data_ptr(), draft.data_ptr(), dt, draft_tokens.data_ptr(), uniforms.data_ptr(),
                temperature.data_ptr(), B, K, V, out.accepted_len.data_ptr(),
                out.out_tokens.data_ptr(), lp, lq, workspace.data_ptr(), ws_bytes, st.cuda_stream)
    else:
        _check(k_per_row, "k_per_row", dtype=torch.int32, shape=(B,), device=dev)
        with _device(dev):
            status = N.spec_verify_ragged_raw(
                target.data_ptr(), draft.data_ptr(), dt, draft_tokens.data_ptr(), uniforms.data_ptr(),
                temperature.data_ptr(), k_per_row.data_ptr(), B, K, V, out.accepted_len.data_ptr(),
                out.out_tokens.data_ptr(), lp, lq, workspace.data_ptr(), ws_bytes, st.cuda_stream)
    if status != N.SV_OK:
        raise N.SpecVerifyError(status)
    return out


def device_errors(workspace: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> int:
    """SV_DEV_* flags of the last call on ``workspace`` (synchronises the stream)."""
    st = stream if stream is not None else torch.cuda.current_stream(workspace.device)
    with _device(workspace.device):
        return N.spec_verify_device_errors(workspace.data_ptr(), st.cuda_stream)


def plug(result: VerifyResult, tokens: torch.Tensor, seq_len: torch.Tensor, *,
         last_token: Optional[torch.Tensor] = None, flags: Optional[torch.Tensor] = None,
         stream: Optional[torch.cuda.Stream] = None) -> None:
    """Append each row's emitted tokens to ``tokens`` [B, max_len] (int32) at
    ``seq_len`` [B] (int32, advanced in place) on the device; no host sync.
    ``last_token`` [B] int32 receives each row's last emitted token;
    ``flags`` (one int32) collects SV_DEV_PLUG_CLIPPED / SV_DEV_BAD_LENGTH."""
    B, K1 = result.out_tokens.shape
    dev = result.out_tokens.device
    if tokens.dim() != 2 or tokens.shape[0] != B:
        raise ValueError("tokens must be [B, max_len]")
    _check(tokens, "tokens", dtype=torch.int32, device=dev)
    _check(seq_len, "seq_len", dtype=torch.int32, shape=(B,), device=dev)
    if last_token is not None:
        _check(last_token, "last_token", dtype=torch.int32, shape=(B,), device=dev)
    if flags is not None:
        _check(flags, "flags", dtype=torch.int32, shape=(1,), device=dev)
    st = _stream(stream, dev)
    with _device(dev):
        status = N.spec_verify_plug_raw(
            result.accepted_len.data_ptr(), result.out_tokens.data_ptr(), B, K1 - 1,
            tokens.data_ptr(), seq_len.data_ptr(), tokens.shape[1],
            last_token.data_ptr() if last_token is not None else None,
            flags.data_ptr() if flags is not None else None, st.cuda_stream)
    if status != N.SV_OK:
        raise N.SpecVerifyError(status, "spec_verify_plug")


def spec_verify_and_plug(target: torch.Tensor, draft: torch.Tensor, draft_tokens: torch.Tensor,
                         uniforms: torch.Tensor, temperature: torch.Tensor, tokens: torch.Tensor,
                         seq_len: torch.Tensor, *, k_per_row: Optional[torch.Tensor] = None,
                         last_token: Optional[torch.Tensor] = None,
                         want_logprobs: bool = False, out: Optional[VerifyResult] = None,
                         workspace: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> VerifyResult:
    """spec_verify followed by plug, with the plug step fused into the
    verify call's second launch (same results as the two calls).  Plug flags
    go to the workspace word: read them with ``device_errors(workspace)``."""
    if target.dim() != 3:
        raise ValueError("target must be [B, K+1, V]")
    B, K1, V = target.shape
    K = K1 - 1
    dev = target.device
    if target.dtype not in _DTYPES:
        raise TypeError(f"target dtype {target.dtype} is not bfloat16 or float32")
    dt = _DTYPES[target.dtype]
    _check(target, "target", device=dev)
    _check(draft, "draft", dtype=target.dtype, shape=(B, K, V), device=dev)
    _check(draft_tokens, "draft_tokens", dtype=torch.int32, shape=(B, K), device=dev)
    _check(uniforms, "uniforms", dtype=torch.float32, shape=(B, K + 1), device=dev)
    _check(temperature, "temperature", dtype=torch.float32, shape=(B,), device=dev)
    if tokens.dim() != 2 or tokens.shape[0] != B:
        raise ValueError("tokens must be [B, max_len]")
    _check(tokens, "tokens", dtype=torch.int32, device=dev)
    _check(seq_len, "seq_len", dtype=torch.int32, shape=(B,), device=dev)
    if last_token is not None:
        _check(last_token, "last_token", dtype=torch.int32, shape=(B,), device=dev)
    if k_per_row is not None:
        _check(k_per_row, "k_per_row", dtype=torch.int32, shape=(B,), device=dev)
    st = _stream(stream, dev)
    if out is None:
        with torch.cuda.stream(st):   # outputs belong to the stream that writes them
            out = VerifyResult(
                torch.empty(B, dtype=torch.int32, device=dev),
                torch.empty(B, K + 1, dtype=torch.int32, device=dev),
                torch.empty(B, K, dtype=torch.float32, device=dev) if want_logprobs else None,
                torch.empty(B, K, dtype=torch.float32, device=dev) if want_logprobs else None)
    if workspace is None:
        workspace = workspace_for(B, K, V, dt, dev, st)
    with _device(dev):
        status = N.spec_verify_and_plug_raw(
            target.data_ptr(), draft.data_ptr(), dt, draft_tokens.data_ptr(), uniforms.data_ptr(),
            temperature.data_ptr(), k_per_row.data_ptr() if k_per_row is not None else None, B, K, V,
            out.accepted_len.data_ptr(), out.out_tokens.data_ptr(),
            out.logp.data_ptr() if out.logp is not None else None,
            out.logq.data_ptr() if out.logq is not None else None,
            tokens.data_ptr(), seq_len.data_ptr(), tokens.shape[1],
            last_token.data_ptr() if last_token is not None else None,
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), st.cuda_stream)
    if status != N.SV_OK:
        raise N.SpecVerifyError(status, "spec_verify_and_plug")
    return out


class TreeResult(NamedTuple):
    accepted_len: torch.Tensor                  # [B] int32: depth of the accepted path, -1 = error row
    out_tokens: torch.Tensor                    # [B, N+1] int32: path tokens, bonus, -1 padded
    accepted_nodes: Optional[torch.Tensor] = None   # [B, N] int32: path node indices, -1 padded


def verify_tree(target: torch.Tensor, node_tokens: torch.Tensor, parents: torch.Tensor, *,
                want_nodes: bool = False, workspace: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> TreeResult:
    """Greedy verification of one draft tree per row (spec_verify_tree):
    ``target`` [B, N+1, V] (slot 0 after the context, slot i+1 after node i),
    ``node_tokens`` and ``parents`` [B, N] int32 (parents[b, i] in [-1, i))."""
    if target.dim() != 3:
        raise ValueError("target must be [B, N+1, V]")
    B, N1, V = target.shape
    N = N1 - 1
    dev = target.device
    if target.dtype not in _DTYPES:
        raise TypeError(f"target dtype {target.dtype} is not bfloat16 or float32")
    dt = _DTYPES[target.dtype]
    _check(target, "target", device=dev)
    _check(node_tokens, "node_tokens", dtype=torch.int32, shape=(B, N), device=dev)
    _check(parents, "parents", dtype=torch.int32, shape=(B, N), device=dev)
    need = _N.spec_verify_tree_workspace_bytes(B, N, V, dt)
    if need == 0:
        raise ValueError(f"invalid tree shape B={B} N={N} V={V}")
    st = _stream(stream, dev)
    with torch.cuda.stream(st):   # blocks the allocator may reuse only after st's work
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        res = TreeResult(torch.empty(B, dtype=torch.int32, device=dev),
                         torch.empty(B, N + 1, dtype=torch.int32, device=dev),
                         torch.empty(B, N, dtype=torch.int32, device=dev) if want_nodes else None)
    with _device(dev):
        status = _N.spec_verify_tree_raw(
            target.data_ptr(), dt, node_tokens.data_ptr(), parents.data_ptr(), B, N, V,
            res.accepted_len.data_ptr(), res.out_tokens.data_ptr(),
            res.accepted_nodes.data_ptr() if res.accepted_nodes is not None else None,
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), st.cuda_stream)
    if status != _N.SV_OK:
        raise _N.SpecVerifyError(status, "spec_verify_tree")
    return res


class PagedPlan(NamedTuple):
    cu_new: torch.Tensor       # [B+1] int32: exclusive sums of the new tokens
    kv_len: torch.Tensor       # [B] int32: cached tokens once the new ones are, 0 = not served
    slot_map: torch.Tensor     # [max_tokens] int32: place of every new token, -1 = none
    positions: torch.Tensor    # [max_tokens] int32: position of every new token, -1 = none
    page_count: torch.Tensor   # [B] int32: pages held now
    free_count: torch.Tensor   # [1] int32: pages on the stack now


def _ints(t, name, shape, dev):
    """The address of a contiguous int32 tensor of this shape on ``dev``."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.shape == shape
            and t.device == dev and t.is_cuda and t.is_contiguous()):
        _check(t, name, dtype=torch.int32, shape=shape, device=dev)   # says what is wrong
    return t.data_ptr()


def _flags_ptr(flags, dev):
    return None if flags is None else _ints(flags, "flags", (1,), dev)


def _scratch(t, name, dev):
    """(address, bytes) of a contiguous tensor on ``dev``, of any type."""
    if not (isinstance(t, torch.Tensor) and t.device == dev and t.is_cuda and t.is_contiguous()):
        _check(t, name, device=dev)   # says what is wrong
    return t.data_ptr(), t.numel() * t.element_size()


def _stream_handle(stream, dev):
    """The raw handle of ``stream``, the device's current one if None (without
    the Stream object, whose making costs as much as a kernel's launch)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev.index)
    return _stream(stream, dev).cuda_stream


def _on(stream):
    """Makes what is allocated inside belong to ``stream`` (None: the current one)."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def paged_plan(seq_len: torch.Tensor, num_new: torch.Tensor, page_count: torch.Tensor,
               block_table: torch.Tensor, free_pages: torch.Tensor, free_count: torch.Tensor, *,
               page_size: int, max_tokens: int, out: Optional[PagedPlan] = None,
               flags: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> PagedPlan:
    """Pages, slots, positions and packed offsets of a step (spec_paged_plan).

    Row b has ``seq_len[b]`` cached tokens and brings ``num_new[b]``; it holds
    ``page_count[b]`` pages, the first entries of ``block_table`` [B,
    max_pages].  Pages it no longer needs go to the stack ``free_pages``
    (``free_count`` [1] entries), missing ones come from it; both arrays are
    updated in place.  The counts come back in the result, whose tensors may
    be ``page_count`` and ``free_count`` themselves (pass them in ``out``).
    All tensors are int32; ``flags`` (one int32) collects SV_DEV_* bits."""
    if seq_len.dim() != 1 or block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("seq_len must be [B], block_table [B, max_pages], free_pages [n_pages]")
    B, max_pages, n_pages, dev = seq_len.shape[0], block_table.shape[1], free_pages.shape[0], seq_len.device
    ins = (_ints(seq_len, "seq_len", (B,), dev), _ints(num_new, "num_new", (B,), dev),
           _ints(page_count, "page_count", (B,), dev),
           _ints(block_table, "block_table", (B, max_pages), dev),
           _ints(free_pages, "free_pages", (n_pages,), dev), _ints(free_count, "free_count", (1,), dev))
    sizes = (B + 1, B, max_tokens, max_tokens, B, 1)
    if out is None:
        if max_tokens < 0:
            raise ValueError("max_tokens must not be negative")
        with _on(stream):   # outputs belong to the stream that writes them
            out = PagedPlan(*[torch.empty(n, dtype=torch.int32, device=dev) for n in sizes])
        outs = [t.data_ptr() for t in out]
    else:
        outs = [_ints(t, "out." + name, (n,), dev)
                for t, name, n in zip(out, PagedPlan._fields, sizes)]
    with _device(dev):
        status = N.spec_paged_plan_raw(*ins, B, page_size, max_pages, n_pages, max_tokens, *outs,
                                       _flags_ptr(flags, dev), _stream_handle(stream, dev))
    if status != N.SV_OK:
        raise N.SpecVerifyError(status, "spec_paged_plan")
    return out


def _check_cache(k_cache, v_cache):
    """(dtype code, n_pages, Hk, page_size, D) of a paged cache."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [n_pages, Hk, page_size, D]")
    dt = _CACHE_DTYPES.get(k_cache.dtype)
    if dt is None:
        raise TypeError(f"k_cache dtype {k_cache.dtype} is not bfloat16 or float16")
    if not (k_cache.is_cuda and k_cache.is_contiguous() and v_cache.is_contiguous()
            and v_cache.dtype is k_cache.dtype and v_cache.shape == k_cache.shape
            and v_cache.device == k_cache.device):
        _check(k_cache, "k_cache")
        _check(v_cache, "v_cache", dtype=k_cache.dtype, shape=k_cache.shape, device=k_cache.device)
    return (dt, *k_cache.shape)


def _check_packed(t, name, dtype, shape, dev):
    """A packed [T, heads, D] tensor whose heads are dense; its token stride."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    T, heads, D = shape
    if T * heads == 0:
        return heads * D
    stride_t, stride_h, stride_d = t.stride()
    if stride_d != 1 or (stride_h != D and heads > 1):
        raise ValueError(f"{name} must have dense heads (strides [any, {D}, 1])")
    return stride_t if T > 1 else heads * D


def paged_append(k_new: torch.Tensor, v_new: torch.Tensor, slot_map: torch.Tensor,
                 k_cache: torch.Tensor, v_cache: torch.Tensor, *,
                 flags: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> None:
    """Write the new tokens' keys and values [T, Hk, D] (dense heads, any
    token stride) to the slots ``slot_map`` [T] of the paged cache [n_pages,
    Hk, page_size, D]; a negative slot skips its token (spec_paged_append)."""
    dt, n_pages, Hk, page_size, D = _check_cache(k_cache, v_cache)
    dev = k_cache.device
    if slot_map.dim() != 1:
        raise ValueError("slot_map must be [T]")
    T = slot_map.shape[0]
    slots = _ints(slot_map, "slot_map", (T,), dev)
    k_stride = _check_packed(k_new, "k_new", k_cache.dtype, (T, Hk, D), dev)
    v_stride = _check_packed(v_new, "v_new", k_cache.dtype, (T, Hk, D), dev)
    with _device(dev):
        status = N.spec_paged_append_raw(
            k_new.data_ptr(), k_stride, v_new.data_ptr(), v_stride, slots, dt, T, Hk, D, page_size,
            n_pages, k_cache.data_ptr(), v_cache.data_ptr(), _flags_ptr(flags, dev),
            _stream_handle(stream, dev))
    if status != N.SV_OK:
        raise N.SpecVerifyError(status, "spec_paged_append")


class AttentionResult(NamedTuple):
    out: torch.Tensor                      # [T, Hq, D]
    lse: Optional[torch.Tensor] = None     # [T, Hq] float32: log of the softmax's sum


def _capture_id(stream, handle):
    """0 outside captures, else a number for the capture that the stream is in."""
    if stream is None and not torch.cuda.is_current_stream_capturing():
        return 0
    return N.spec_stream_capture_id(handle)


def attention_workspace(D: int, device: torch.device,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The cached workspace of ``paged_attention`` on a (device, stream), its
    counters zeroed once; calls on different streams must not share one.

    A stream that is being captured has another one for each capture, whose
    counters the graph zeroes whenever it runs: graphs captured on one stream
    may be replayed in any order, on any streams, beside calls outside them.
    Of a stream's captures the last one's is kept here; those before it live
    in their graphs' memory pools, so graphs that share a pool must not be
    replayed at the same time."""
    need = N.spec_paged_attention_workspace_bytes(D)
    if need == 0:
        raise ValueError(f"invalid head dimension {D}")
    index = device.index if device.index is not None else torch.cuda.current_device()
    st = stream if stream is not None else torch.cuda.current_stream(index)
    key = (index, st.cuda_stream, D)
    with _device(st.device):
        capture = _capture_id(st, st.cuda_stream)
    if capture:
        owner, ws = _captured_workspaces.get(key, (0, None))
        if owner != capture:
            ws = None
    else:
        ws = _attention_workspaces.get(key)
    if ws is None:
        with torch.cuda.stream(st):   # allocated and zeroed on the stream that uses it
            ws = torch.empty(need, dtype=torch.uint8, device=device)
            ws[:N.SV_ATTENTION_COUNTER_BYTES].zero_()
        if capture:
            _captured_workspaces[key] = (capture, ws)
        else:
            _attention_workspaces[key] = ws
    return ws


def attention_errors(workspace: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> int:
    """SV_DEV_TIMEOUT if a ``paged_attention`` call with ``workspace`` has given
    up since this was last asked, else 0 (synchronises the stream).  Such a
    call leaves rows unwritten, and those after it give NaN until this clears
    the workspace.  The workspace of calls without one is
    ``attention_workspace(D, device, stream)``."""
    address, size = _scratch(workspace, "workspace", workspace.device)
    if size < N.SV_ATTENTION_COUNTER_BYTES:
        raise ValueError("workspace is smaller than its counters")
    st = _stream(stream, workspace.device)
    with _device(workspace.device):
        return N.spec_paged_attention_device_errors(address, st.cuda_stream)


def _attention_scratch(workspace, D, dev, stream, handle):
    """(address, bytes) of the caller's workspace, or of the cached one."""
    if workspace is not None:
        return _scratch(workspace, "workspace", dev)
    if not _capture_id(stream, handle):
        workspace = _attention_workspaces.get((dev.index, handle, D))
    if workspace is None:
        workspace = attention_workspace(D, dev, stream)
    return workspace.data_ptr(), workspace.numel()


def _attention_outputs(out, q, want_lse, stream):
    T, Hq, D = q.shape
    if out is None:
        with _on(stream):   # outputs belong to the stream that writes them
            return AttentionResult(
                torch.empty(T, Hq, D, dtype=q.dtype, device=q.device),
                torch.empty(T, Hq, dtype=torch.float32, device=q.device) if want_lse else None)
    _check(out.out, "out.out", dtype=q.dtype, shape=(T, Hq, D), device=q.device)
    if out.lse is not None:
        _check(out.lse, "out.lse", dtype=torch.float32, shape=(T, Hq), device=q.device)
    return out


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    block_table: torch.Tensor, cu_new: torch.Tensor, kv_len: torch.Tensor, *,
                    scale: Optional[float] = None, want_lse: bool = False,
                    out: Optional[AttentionResult] = None, flags: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> AttentionResult:
    """Causal attention of the packed new tokens ``q`` [T, Hq, D] (dense heads,
    any token stride) over the paged cache [n_pages, Hk, page_size, D]
    (spec_paged_attention).  Request b has tokens cu_new[b]..cu_new[b+1]-1,
    the last of its ``kv_len[b]`` cached ones; a token that sees no key gets
    zeros.  ``scale`` defaults to D ** -0.5.  A ``workspace`` of the caller's
    (spec_paged_attention_workspace_bytes) has its first
    SV_ATTENTION_COUNTER_BYTES zero before its first use, and is used by one
    call at a time.  ``flags`` (one int32) collects SV_DEV_* bits;
    SV_DEV_TIMEOUT stays in the workspace as well (``attention_errors``)."""
    dt, n_pages, Hk, page_size, D = _check_cache(k_cache, v_cache)
    dev = k_cache.device
    if q.dim() != 3:
        raise ValueError(f"q must be [T, Hq, {D}], got {tuple(q.shape)}")
    T, Hq, _ = q.shape
    q_stride = _check_packed(q, "q", k_cache.dtype, (T, Hq, D), dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = block_table.shape
    tables = (_ints(block_table, "block_table", (B, max_pages), dev),
              _ints(cu_new, "cu_new", (B + 1,), dev), _ints(kv_len, "kv_len", (B,), dev))
    out = _attention_outputs(out, q, want_lse, stream)
    with _device(dev):
        handle = _stream_handle(stream, dev)
        scratch = _attention_scratch(workspace, D, dev, stream, handle)
        status = N.spec_paged_attention_raw(
            q.data_ptr(), q_stride, k_cache.data_ptr(), v_cache.data_ptr(), dt, *tables, B, T, Hq, Hk,
            D, page_size, max_pages, n_pages, D ** -0.5 if scale is None else scale,
            out.out.data_ptr(), out.lse.data_ptr() if out.lse is not None else None,
            *scratch, _flags_ptr(flags, dev), handle)
    if status != N.SV_OK:
        raise N.SpecVerifyError(status, "spec_paged_attention")
    return out


# ------------------------------------------- rotation on the way, caches of 4 bits

def rotary_table(max_positions: int, rotary_dim: int, *, base: float = 10000.0,
                 inv_freq: Optional[torch.Tensor] = None, device=None) -> torch.Tensor:
    """Cosines and sines [max_positions, rotary_dim] float32 of the angles
    position * inv_freq, formed in float64.  ``inv_freq`` [rotary_dim / 2]
    defaults to base ** (-2 i / rotary_dim)."""
    if max_positions < 1 or rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("max_positions must be positive, rotary_dim positive and even")
    if inv_freq is None:
        inv_freq = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    elif inv_freq.shape != (rotary_dim // 2,):
        raise ValueError(f"inv_freq must have shape {(rotary_dim // 2,)}, got {tuple(inv_freq.shape)}")
    rates = inv_freq.to(device=device, dtype=torch.float64)
    angle = torch.arange(max_positions, dtype=torch.float64, device=rates.device)[:, None] * rates
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class PagedCacheFp4(NamedTuple):
    """A paged cache of 4-bit keys and values: two e2m1 codes a byte (the even
    column's in the low half) and an e4m3 scale for each group of 16 columns."""
    k: torch.Tensor         # [n_pages, Hk, page_size, D / 2] uint8
    k_scale: torch.Tensor   # [n_pages, Hk, page_size, D / 16] float8_e4m3fn
    v: torch.Tensor
    v_scale: torch.Tensor


def paged_cache_fp4(n_pages: int, Hk: int, page_size: int, D: int, device=None) -> PagedCacheFp4:
    """An empty cache (all zeros)."""
    if D not in (64, 128):
        raise ValueError(f"invalid head dimension {D}")
    shape = (n_pages, Hk, page_size)
    make = lambda n: torch.zeros(*shape, n, dtype=torch.uint8, device=device)
    return PagedCacheFp4(make(D // 2), make(D // 16).view(torch.float8_e4m3fn),
                         make(D // 2), make(D // 16).view(torch.float8_e4m3fn))


def _check_cache_fp4(cache):
    """The four addresses, and (n_pages, Hk, page_size, D), of a 4-bit cache."""
    k, k_scale, v, v_scale = cache
    if k.dim() != 4:
        raise ValueError("cache.k must be [n_pages, Hk, page_size, D / 2]")
    dev, (n_pages, Hk, page_size, half) = k.device, k.shape
    scales = (n_pages, Hk, page_size, half // 8)
    for t, name, dtype, shape in ((k, "k", torch.uint8, k.shape), (k_scale, "k_scale", torch.float8_e4m3fn, scales),
                                  (v, "v", torch.uint8, k.shape), (v_scale, "v_scale", torch.float8_e4m3fn, scales)):
        if not (t.is_cuda and t.is_contiguous() and t.dtype is dtype and t.shape == shape and t.device == dev):
            _check(t, "cache." + name, dtype=dtype, shape=shape, device=dev)
    return (k.data_ptr(), k_scale.data_ptr(), v.data_ptr(), v_scale.data_ptr()), (n_pages, Hk, page_size, 2 * half)


def _append_inputs(q, k_new, v_new, positions, cos_sin, slot_map, q_out, dtype, Hk, D, dev, stream):
    """What both rotated appends take, as their C arguments up to T and Hq, and q_out."""
    if slot_map.dim() != 1:
        raise ValueError("slot_map must be [T]")
    T = slot_map.shape[0]
    if (positions is None) != (cos_sin is None):
        raise ValueError("positions and cos_sin come together")
    if cos_sin is None:
        if q is not None:
            raise ValueError("q needs positions and cos_sin")
        table = (None, None, 0, 0)
    else:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [max_positions, rotary_dim]")
        if not (cos_sin.dtype is torch.float32 and cos_sin.device == dev and cos_sin.is_cuda and cos_sin.is_contiguous()):
            _check(cos_sin, "cos_sin", dtype=torch.float32, device=dev)   # says what is wrong
        table = (_ints(positions, "positions", (T,), dev), cos_sin.data_ptr(), *cos_sin.shape)
    ins = (k_new.data_ptr(), _check_packed(k_new, "k_new", dtype, (T, Hk, D), dev),
           v_new.data_ptr(), _check_packed(v_new, "v_new", dtype, (T, Hk, D), dev), *table)
    slots = _ints(slot_map, "slot_map", (T,), dev)
    if q is None:
        if q_out is not None:
            raise ValueError("q_out needs q")
        return (None, 0, *ins), slots, T, 0, (None, 0), None
    if q.dim() != 3:
        raise ValueError(f"q must be [T, Hq, {D}], got {tuple(q.shape)}")
    Hq = q.shape[1]
    shape = (T, Hq, D)
    stride = _check_packed(q, "q", dtype, shape, dev)
    if q_out is None:
        with _on(stream):   # outputs belong to the stream that writes them
            q_out = torch.empty(shape, dtype=dtype, device=dev)
        out_stride = Hq * D
    else:
        out_stride = _check_packed(q_out, "q_out", dtype, shape, dev)
    return (q.data_ptr(), stride, *ins), slots, T, Hq, (q_out.data_ptr(), out_stride), q_out


def paged_append_rotary(q: Optional[torch.Tensor], k_new: torch.Tensor, v_new: torch.Tensor,
                        positions: torch.Tensor, cos_sin: torch.Tensor, slot_map: torch.Tensor,
                        k_cache: torch.Tensor, v_cache: torch.Tensor, *, interleaved: bool = False,
                        q_out: Optional[torch.Tensor] = None, flags: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """``paged_append`` with the position rotation on the way
    (spec_paged_append_rotary); returns the rotated queries.

    ``q`` [T, Hq, D] (or None) and ``k_new`` are rotated by ``positions`` [T]
    int32 (a plan's; negative ones are padding, whose queries become zeros)
    with the table ``cos_sin`` [max_positions, rotary_dim] (``rotary_table``):
    pairs are columns i and i + rotary_dim / 2, or neighbours if
    ``interleaved``.  ``q_out`` may be ``q`` itself."""
    dt, n_pages, Hk, page_size, D = _check_cache(k_cache, v_cache)
    dev = k_cache.device
    if positions is None or cos_sin is None:
        raise ValueError("positions and cos_sin are needed")
    ins, slots, T, Hq, result, q_out = _append_inputs(q, k_new, v_new, positions, cos_sin, slot_map, q_out,
                                                      k_cache.dtype, Hk, D, dev, stream)
    with _device(dev):
        status = N.spec_paged_append_rotary_raw(
            *ins, int(interleaved), slots, dt, T, Hq, Hk, D, page_size, n_pages, *result, k_cache.data_ptr(),
            v_cache.data_ptr(), _flags_ptr(flags, dev), _stream_handle(stream, dev))
    if status != N.SV_OK:
        raise N.SpecVerifyError(status, "spec_paged_append_rotary")
    return q_out


def paged_append_fp4(q: Optional[torch.Tensor], k_new: torch.Tensor, v_new: torch.Tensor,
                     positions: Optional[torch.Tensor], cos_sin: Optional[torch.Tensor], slot_map: torch.Tensor,
                     cache: PagedCacheFp4, *, k_gain: float = 1.0, v_gain: float = 1.0,
                     interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                     flags: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """``paged_append_rotary`` into a 4-bit cache (spec_paged_append_fp4).  With
    ``positions`` and ``cos_sin`` None (and ``q`` too) nothing is rotated.  The
    gains are the cache's, the same in every call."""
    addresses, (n_pages, Hk, page_size, D) = _check_cache_fp4(cache)
    dev = cache.k.device
    dt = _CACHE_DTYPES.get(k_new.dtype)
    if dt is None:
        raise TypeError(f"k_new dtype {k_new.dtype} is not bfloat16 or float16")
    ins, slots, T, Hq, result, q_out = _append_inputs(q, k_new, v_new, positions, cos_sin, slot_map, q_out,
                                                      k_new.dtype, Hk, D, dev, stream)
    with _device(dev):
        status = N.spec_paged_append_fp4_raw(
            *ins, int(interleaved), slots, dt, T, Hq, Hk, D, page_size, n_pages, k_gain, v_gain, *result,
            *addresses, _flags_ptr(flags, dev), _stream_handle(stream, dev))
    if status != N.SV_OK:
        raise N.SpecVerifyError(status, "spec_paged_append_fp4")
    return q_out


def paged_read_fp4(cache: PagedCacheFp4, slot_map: torch.Tensor, dtype: torch.dtype = torch.bfloat16, *,
                   k_gain: float = 1.0, v_gain: float = 1.0, flags: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> tuple:
    """Keys and values [T, Hk, D] that a 4-bit cache holds at the slots
    ``slot_map`` [T], zeros for negative ones (spec_paged_read_fp4)."""
    addresses, (n_pages, Hk, page_size, D) = _check_cache_fp4(cache)
    dev = cache.k.device
    dt = _CACHE_DTYPES.get(dtype)
    if dt is None:
        raise TypeError(f"dtype {dtype} is not bfloat16 or float16")
    if slot_map.dim() != 1:
        raise ValueError("slot_map must be [T]")
    T = slot_map.shape[0]
    slots = _ints(slot_map, "slot_map", (T,), dev)
    with _on(stream):   # outputs belong to the stream that writes them
        k, v = (torch.empty(T, Hk, D, dtype=dtype, device=dev) for _ in range(2))
    with _device(dev):
        status = N.spec_paged_read_fp4_raw(
            *addresses, slots, dt, T, Hk, D, page_size, n_pages, k_gain, v_gain, k.data_ptr(), v.data_ptr(),
            _flags_ptr(flags, dev), _stream_handle(stream, dev))
    if status != N.SV_OK:
        raise N.SpecVerifyError(status, "spec_paged_read_fp4")
    return k, v


def paged_attention_fp4(q: torch.Tensor, cache: PagedCacheFp4, block_table: torch.Tensor,
                        cu_new: torch.Tensor, kv_len: torch.Tensor, *, scale: Optional[float] = None,
                        k_gain: float = 1.0, v_gain: float = 1.0, want_lse: bool = False,
                        out: Optional[AttentionResult] = None, flags: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> AttentionResult:
    """``paged_attention`` over a 4-bit cache (spec_paged_attention_fp4), with
    the same workspaces; ``q`` is bfloat16 or float16."""
    addresses, (n_pages, Hk, page_size, D) = _check_cache_fp4(cache)
    dev = cache.k.device
    dt = _CACHE_DTYPES.get(q.dtype)
    if dt is None:
        raise TypeError(f"q dtype {q.dtype} is not bfloat16 or float16")
    if q.dim() != 3:
        raise ValueError(f"q must be [T, Hq, {D}], got {tuple(q.shape)}")
    T, Hq, _ = q.shape
    q_stride = _check_packed(q, "q", q.dtype, (T, Hq, D), dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = block_table.shape
    tables = (_ints(block_table, "block_table", (B, max_pages), dev),
              _ints(cu_new, "cu_new", (B + 1,), dev), _ints(kv_len, "kv_len", (B,), dev))
    out = _attention_outputs(out, q, want_lse, stream)
    with _device(dev):
        handle = _stream_handle(stream, dev)
        scratch = _attention_scratch(workspace, D, dev, stream, handle)
        status = N.spec_paged_attention_fp4_raw(
            q.data_ptr(), q_stride, *addresses, dt, *tables, B, T, Hq, Hk, D, page_size, max_pages, n_pages,
            D ** -0.5 if scale is None else scale, k_gain, v_gain, out.out.data_ptr(),
            out.lse.data_ptr() if out.lse is not None else None, *scratch, _flags_ptr(flags, dev), handle)
    if status != N.SV_OK:
        raise N.SpecVerifyError(status, "spec_paged_attention_fp4")
    return out
