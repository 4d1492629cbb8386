"""Python binding of the operators beside the KDA forward: the rest of a
linear-attention layer, in the order it runs them.

    kda.rope(q, k, positions, inv_freq, ...)      rotary positions
    kda.qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, ...)
                                                  the same behind a norm of q and k
    kda.lin_attn_fwd(q, k, v, log_decay, ...)     linear attention over a paged pool
    kda.gated_delta_fwd(q, k, v, log_decay, beta, ...)
                                                  the gated delta rule over the pool
    kda.gated_norm(o, weight, gate=z, ...)        norm and gate of the output

Argument marshalling only; the kernels are in ``libkda.so`` (``include/kda.h``
describes each call).  Every call runs on the current GPU, where its tensors have to
be.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct
from typing import Optional

import torch

from . import (KDA_ERR_WORKSPACE, KDA_OK, STATE_DTYPES, _check, _host_bounds, _on_current_device, _per_sequence,
               _same_device, load_library)

_DTYPES = STATE_DTYPES  # kda_dtype has the same values as kda_state_dtype
_LAYOUTS = {"half": 0, "interleaved": 1}
_FLAGS = (torch.bool, torch.uint8)
_ACTIVATIONS = {"none": 0, "sigmoid": 1, "silu": 2}


class _RopeTensor(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("in_stride_t", ctypes.c_int64), ("in_stride_h", ctypes.c_int64),
                ("out_stride_t", ctypes.c_int64), ("out_stride_h", ctypes.c_int64),
                ("num_heads", ctypes.c_int32)]


class _NormRopeTensor(ctypes.Structure):
    _fields_ = [("x", _RopeTensor), ("weight", ctypes.c_void_p), ("weight_stride_h", ctypes.c_int64)]


# Two of them, as bytes: a third of the time that ctypes takes for their fields
_NORM_ROPE_TENSORS = struct.Struct("@" + "PPqqqqi4xPq" * 2)
assert _NORM_ROPE_TENSORS.size == 2 * ctypes.sizeof(_NormRopeTensor)
_NO_TENSOR = (0,) * 9


def _rows(x: torch.Tensor, name: str, dtype=None):
    """(T, H, D, token stride, head stride) of a [1, T, H, D] or [T, H, D] CUDA view,
    dense in its last dimension."""
    shape, stride = x.shape, x.stride()
    if len(shape) == 4 and shape[0] == 1:
        _, T, H, D = shape
        _, st, sh, s1 = stride
    elif len(shape) == 3:
        T, H, D = shape
        st, sh, s1 = stride
    elif len(shape) == 4:
        raise ValueError(f"{name}: packed input must have batch dim 1")
    else:
        raise ValueError(f"{name} must be [1, T, H, D] or [T, H, D], got {tuple(x.shape)}")
    if dtype is not None and x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if s1 != 1 and D > 1:
        raise ValueError(f"{name} must be dense in its last dimension")
    # the stride of a dimension of one entry says nothing
    return T, H, D, st if T > 1 else H * D, sh if H > 1 else D


# The current stream's handle by device index, without a Stream object around it.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device):
    if stream is not None:
        return stream.cuda_stream
    if _current_stream is not None and device.index is not None:
        return _current_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _empty(shape, dtype, device, stream):
    """New memory of the stream that the call runs on: another stream's could be given
    out again, once the caller has dropped it, while the call still uses it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _host_int32(cu_seqlens_cpu, N: int):
    """_host_bounds, without its conversions where nothing has to be converted."""
    h = cu_seqlens_cpu
    if (isinstance(h, torch.Tensor) and h.dtype is torch.int32 and h.numel() == N + 1
            and h.is_contiguous() and h.device.type == "cpu"):
        return h
    return _host_bounds(h, N)


@functools.lru_cache(maxsize=1024)
def lin_attn_workspace_size(total_tokens: int, num_seqs: int, num_heads: int) -> int:
    """Bytes of workspace a ``lin_attn_fwd`` call with these sizes needs."""
    return int(load_library().kda_lin_attn_workspace_size(total_tokens, num_seqs, num_heads))


def lin_attn_fwd(q, k, v, log_decay, cu_seqlens, *, state_cache, state_indices,
                 has_initial_state, out, scale: Optional[float] = None, cu_seqlens_cpu=None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Linear attention with a decay for each head (``kda_lin_attn_fwd``):

        S_t = exp(g_t) S_{t-1} + v_t k_t^T,    o_t = scale * S_t q_t

    q, k [1, T, Hqk, 128] and v [1, T, H, 128] are bf16 (views with strides of
    their own are taken as they are), H a multiple of Hqk; ``log_decay`` is fp32
    [H], or [1, T, H] for a decay of each token.  ``scale`` defaults to
    128 ** -0.5.  Prompts, ragged batches and single tokens go in one call; the
    pool arguments are those of ``chunk_fwd``.  ``workspace`` (uint8, at least
    ``lin_attn_workspace_size`` bytes; one for each stream) saves a call of more than
    8 tokens, or with ``stream``, its allocation, about 5 us of the 18 that it takes on the
    host.  Writes ``out`` and the selected pool slots in place and returns ``out``."""
    lib = load_library()
    dev = q.device
    T, Hk, H, N, q_st, q_sh, k_st, k_sh, v_st, v_sh, p_st, slots, per_token, at = _packed(
        q, k, v, log_decay, cu_seqlens, state_cache, state_indices, has_initial_state, out)
    _on_current_device(at)
    host = None if cu_seqlens_cpu is None else _host_int32(cu_seqlens_cpu, N)
    if workspace is None and T <= _LIN_STEP_MAX and stream is None:
        workspace, given = _header(dev, stream), _HEADER
    else:
        workspace, given = _packed_workspace(lin_attn_workspace_size(T, N, H), workspace, dev, stream)
    rc = lib.kda_lin_attn_fwd(
        q.data_ptr(), q_st, q_sh, k.data_ptr(), k_st, k_sh, v.data_ptr(), v_st, v_sh,
        log_decay.data_ptr(), per_token, cu_seqlens.data_ptr(),
        None if host is None else host.data_ptr(), N, T, H, Hk,
        state_cache.data_ptr(), p_st, slots,
        state_indices.data_ptr(), has_initial_state.data_ptr(), out.data_ptr(),
        0.08838834764831845 if scale is None else float(scale), STATE_DTYPES[state_cache.dtype],
        workspace.data_ptr(), given, _stream(stream, dev))
    if rc != KDA_OK:
        _check(rc, lib)
    return out


@functools.lru_cache(maxsize=1024)
def gated_delta_workspace_size(total_tokens: int, num_seqs: int, num_heads: int) -> int:
    """Bytes of workspace a ``gated_delta_fwd`` call with these sizes needs."""
    return int(load_library().kda_gated_delta_workspace_size(total_tokens, num_seqs, num_heads))


def gated_delta_fwd(q, k, v, log_decay, beta, cu_seqlens, *, state_cache, state_indices,
                    has_initial_state, out, scale: Optional[float] = None, cu_seqlens_cpu=None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gated delta rule with a decay for each head (``kda_gated_delta_fwd``):

        S_t = exp(g_t) S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,  o_t = scale * S_t q_t

    with q and k divided by their lengths.  Tensors, pool and options are those of
    ``lin_attn_fwd``; ``beta`` is contiguous fp32 [1, T, H] (or [T, H]), from 0 to 2,
    ``log_decay`` at most 0 (below -104 a token clears the state).  Prompts, ragged
    batches and single tokens go in one call.  The workspace holds what the chunks of
    long sequences need, 59 KB for 64 tokens and a head; where ``cu_seqlens_cpu`` says that
    none has more than 16 tokens, a call allocates none.  Writes ``out`` and the selected
    pool slots in place and returns ``out``."""
    lib = load_library()
    dev = q.device
    T, Hk, H, N, q_st, q_sh, k_st, k_sh, v_st, v_sh, p_st, slots, per_token, at = _packed(
        q, k, v, log_decay, cu_seqlens, state_cache, state_indices, has_initial_state, out)
    if beta.dtype is not torch.float32 or not beta.is_cuda:
        raise TypeError("beta must be a float32 CUDA tensor")
    if beta.get_device() != at:
        _same_device(dev, beta=beta)
    bs = beta.shape
    if not beta.is_contiguous() or not (bs == (1, T, H) or bs == (T, H)):
        raise ValueError(f"beta must be a contiguous [1, T, H] tensor; got shape {tuple(bs)}")
    _on_current_device(at)
    host = None if cu_seqlens_cpu is None else _host_int32(cu_seqlens_cpu, N)
    args = (q.data_ptr(), q_st, q_sh, k.data_ptr(), k_st, k_sh, v.data_ptr(), v_st, v_sh,
            log_decay.data_ptr(), per_token, beta.data_ptr(), cu_seqlens.data_ptr(),
            None if host is None else host.data_ptr(), N, T, H, Hk,
            state_cache.data_ptr(), p_st, slots,
            state_indices.data_ptr(), has_initial_state.data_ptr(), out.data_ptr(),
            0.08838834764831845 if scale is None else float(scale), STATE_DTYPES[state_cache.dtype])
    rc = KDA_ERR_WORKSPACE
    if workspace is None and (T <= _DELTA_STEP_MAX or host is not None and T <= N * _DELTA_STEP_MAX):
        # it has no chunks unless a sequence is longer than they are on average, which the library
        # sees before it does anything
        rc = lib.kda_gated_delta_fwd(*args, _header(dev, stream).data_ptr(), _HEADER, _stream(stream, dev))
    if rc == KDA_ERR_WORKSPACE:
        need = gated_delta_workspace_size(T, N, H)
        if workspace is not None and host is not None and T <= N * _DELTA_STEP_MAX:
            need = min(need, _HEADER)  # it may be enough: the library says
        workspace, given = _packed_workspace(need, workspace, dev, stream)
        rc = lib.kda_gated_delta_fwd(*args, workspace.data_ptr(), given, _stream(stream, dev))
    if rc != KDA_OK:
        _check(rc, lib)
    return out


def _packed(q, k, v, log_decay, cu_seqlens, state_cache, state_indices, hs, out):
    """(T, Hqk, H, N, strides of q, k and v, slot stride, slots, whether each token has its
    decay, GPU) of a call over packed sequences and the pool of their states, its arguments
    checked."""
    bf16 = torch.bfloat16
    at = q.get_device()  # -1 without a GPU
    qs, vs, ps, gs = q.shape, v.shape, state_cache.shape, log_decay.shape
    (_, q_st, q_sh, q_1), (_, k_st, k_sh, k_1), (_, v_st, v_sh, v_1), (p_st, *plane) = (
        x.stride() if x.dim() == 4 else (0, 0, 0, 0) for x in (q, k, v, state_cache))
    N = cu_seqlens.numel() - 1
    # One look at the usual forms; _packed_args looks at each argument, takes the others and
    # says what is wrong.
    if (at >= 0 and q_1 == k_1 == v_1 == 1 and plane == [16384, 128, 1]
            and qs[0] == vs[0] == 1 and qs[3] == vs[3] == 128
            and qs[1] == vs[1] and k.shape == qs and qs[2] > 0 and vs[2] % qs[2] == 0
            and q.dtype is k.dtype is v.dtype is out.dtype is bf16
            and k.get_device() == v.get_device() == out.get_device() == log_decay.get_device()
            == cu_seqlens.get_device() == state_indices.get_device() == hs.get_device()
            == state_cache.get_device() == at
            and out.shape == vs and out.is_contiguous()
            and log_decay.dtype is torch.float32 and log_decay.is_contiguous()
            and (gs == vs[2:3] or gs == vs[:3])
            and cu_seqlens.dtype is state_indices.dtype is torch.int32
            and cu_seqlens.dim() == 1 and N >= 0 and cu_seqlens.is_contiguous()
            and state_indices.numel() == N and state_indices.is_contiguous()
            and hs.dtype in _FLAGS and hs.numel() == N and hs.is_contiguous()
            and state_cache.dtype in STATE_DTYPES and ps[1] == vs[2] and ps[2] == ps[3] == 128):
        _, T, Hk, _ = qs
        H = vs[2]
        if T == 1:  # the stride of a dimension of one entry says nothing
            q_st = k_st = Hk * 128
            v_st = H * 128
        if Hk == 1:
            q_sh = k_sh = 128
        if H == 1:
            v_sh = 128
    else:
        T, Hk, H, N, (q_st, q_sh, k_st, k_sh, v_st, v_sh) = _packed_args(
            q, k, v, log_decay, cu_seqlens, state_cache, state_indices, hs, out)
    return T, Hk, H, N, q_st, q_sh, k_st, k_sh, v_st, v_sh, p_st, ps[0], len(gs) > 1, at


_HEADER = 256  # bytes of a workspace that holds a status word alone
# With so few tokens every sequence of linear attention's goes token by token: nothing of the
# workspace but the status word is used.  (Above, chunks may be dealt out by counters in it.)
_LIN_STEP_MAX = 8
_DELTA_STEP_MAX = 16  # of each of the gated delta rule's, which has no counters
_headers = {}  # of each GPU, by stream


def _header(dev, stream):
    """The workspace of a call that needs no other and whose caller cannot read its status:
    one for each GPU and current stream, which any number of calls may write.  (An allocation
    takes 5 us of such a call's 20 on the host.  Its memory may be what earlier work of the
    stream that makes it still uses: other streams have their own.)"""
    if stream is None:
        on = _stream(None, dev)
        ws = _headers.get(dev.index, {}).get(on)
        if ws is not None:
            return ws
    ws = _empty(_HEADER, torch.uint8, dev, stream)
    # (memory of a graph's own is the graph's)
    if stream is None and not torch.cuda.is_current_stream_capturing():
        _headers.setdefault(dev.index, {})[on] = ws
    return ws


def _packed_workspace(need, workspace, dev, stream):
    """(workspace, its bytes): a new one, or the caller's once it is checked."""
    if workspace is None:
        return _empty(max(need, 256), torch.uint8, dev, stream), need
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    given = workspace.numel() * workspace.element_size()
    if given < need:
        raise ValueError(f"workspace too small: {need} bytes needed")
    return workspace, given


def _packed_args(q, k, v, log_decay, cu_seqlens, state_cache, state_indices, hs, out):
    """(T, Hqk, H, N, strides of q, k and v), every argument checked for itself."""
    bf16 = torch.bfloat16
    T, Hk, D, q_st, q_sh = _rows(q, "q", bf16)
    Tk, Hk2, Dk, k_st, k_sh = _rows(k, "k", bf16)
    Tv, H, Dv, v_st, v_sh = _rows(v, "v", bf16)
    if D != 128 or (Tk, Hk2, Dk) != (T, Hk, D) or (Tv, Dv) != (T, D):
        raise ValueError("q and k must be [1, T, Hqk, 128] and v [1, T, H, 128]")
    if Hk < 1 or H % Hk:
        raise ValueError(f"{H} heads of v are not a multiple of {Hk} heads of q and k")
    if log_decay.dtype != torch.float32 or not log_decay.is_cuda:
        raise TypeError("log_decay must be a float32 CUDA tensor")
    if not log_decay.is_contiguous() or tuple(log_decay.shape) not in ((H,), (T, H), (1, T, H)):
        raise ValueError(f"log_decay must be a contiguous [H] or [1, T, H] tensor; got shape "
                         f"{tuple(log_decay.shape)}")
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
        raise TypeError("cu_seqlens must be an int32 CUDA tensor")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous 1-D tensor of N + 1 bounds")
    N = cu_seqlens.numel() - 1
    if out.dtype != bf16 or not out.is_cuda:
        raise TypeError("out must be a bfloat16 CUDA tensor")
    if tuple(out.shape) != tuple(v.shape) or not out.is_contiguous():
        raise ValueError("out must be contiguous and have the shape of v")
    if state_cache.dtype not in STATE_DTYPES or not state_cache.is_cuda:
        raise TypeError(f"state_cache dtype {state_cache.dtype} on {state_cache.device} not supported")
    if state_cache.dim() != 4 or tuple(state_cache.shape[1:]) != (H, 128, 128):
        raise ValueError("state_cache must be [slots, H, 128, 128]")
    if tuple(state_cache.stride()[1:]) != (128 * 128, 128, 1):
        raise ValueError("each slot plane of state_cache must be dense (only stride(0) may pad)")
    if state_indices.dtype != torch.int32 or not state_indices.is_cuda:
        raise TypeError("state_indices must be an int32 CUDA tensor")
    if hs.dtype not in _FLAGS or not hs.is_cuda:
        raise TypeError("has_initial_state must be a bool/uint8 CUDA tensor")
    _per_sequence(state_indices, "state_indices", N)
    _per_sequence(hs, "has_initial_state", N)
    _same_device(q.device, k=k, v=v, log_decay=log_decay, cu_seqlens=cu_seqlens, out=out,
                 state_cache=state_cache, state_indices=state_indices, has_initial_state=hs)
    return T, Hk, H, N, (q_st, q_sh, k_st, k_sh, v_st, v_sh)


def rope_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: Optional[str] = None,
                     factor: float = 1.0, original_positions: int = 0,
                     fast_turns: float = 32.0, slow_turns: float = 1.0,
                     device="cuda"):
    """(inv_freq fp64 [rot_dim / 2], factor on cos and sin) for ``rope``.

    Without ``scaling``, inv_freq[i] = base ** (-2 i / rot_dim).  For contexts
    ``factor`` times as long as those trained on:

    ``"linear"``  every frequency divided by ``factor`` (positions interpolated);
    ``"base"``    base * factor ** (r / (r - 2)): the slowest pair is divided by
                  ``factor``, the fastest kept;
    ``"ramp"``    pairs that turn more than ``fast_turns`` times within
                  ``original_positions`` kept, those that turn less than
                  ``slow_turns`` times divided by ``factor``, a linear ramp over
                  the pairs between, and cos and sin times 0.1 ln(factor) + 1.
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must be over 1 and factor at least 1")
    r = rot_dim
    amplitude = 1.0
    if scaling == "base":
        if r < 4:
            raise ValueError("scaling 'base' needs rot_dim of at least 4")
        base = base * factor ** (r / (r - 2.0))
    freq = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "ramp":
        if original_positions <= 0 or not fast_turns > slow_turns > 0:
            raise ValueError("scaling 'ramp' needs original_positions and fast_turns > slow_turns > 0")

        def pair_turning(turns):
            return r * math.log(original_positions / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo = max(math.floor(pair_turning(fast_turns)), 0)
        hi = min(math.ceil(pair_turning(slow_turns)), r - 1)
        for i in range(r // 2):
            slow = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            freq[i] *= (1.0 - slow) + slow / factor
        amplitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"scaling {scaling!r} is not one of 'linear', 'base', 'ramp'")
    return torch.tensor(freq, dtype=torch.float64, device=device), amplitude


def _rope_rows(q, k, positions, inv_freq, layout, q_out, k_out):
    """(the fields of q's and k's ``_RopeTensor``, D), every argument checked."""
    if layout not in _LAYOUTS:
        raise ValueError(f"layout {layout!r} is not one of {sorted(_LAYOUTS)}")
    if q.dtype not in _DTYPES:
        raise TypeError(f"q dtype {q.dtype} not supported")
    q_out = q if q_out is None else q_out
    if k is None and k_out is not None:
        raise ValueError("k_out is given without k")
    k_out = k if k_out is None else k_out
    rows = []
    for name, x, y in (("q", q, q_out), ("k", k, k_out)):
        if x is None:
            continue
        Tx, H, Dx, st, sh = _rows(x, name, q.dtype)
        if x is q:
            T, D = Tx, Dx
        To, Ho, Do, ost, osh = (Tx, H, Dx, st, sh) if y is x else _rows(y, name + "_out", q.dtype)
        if Tx != T or Dx != D or To != Tx or Ho != H or Do != Dx:
            raise ValueError(f"{name} and {name}_out must be [1, T, H, D] with q's T and D")
        rows.append((x.data_ptr(), y.data_ptr(), st, sh, ost, osh, H))
    if positions.dtype not in (torch.int32, torch.int64) or not positions.is_cuda:
        raise TypeError("positions must be an int32 or int64 CUDA tensor")
    if positions.numel() != T or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous tensor of {T} entries, one per token")
    if inv_freq.dtype != torch.float64 or not inv_freq.is_cuda:
        raise TypeError("inv_freq must be a float64 CUDA tensor")
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous() or 2 * inv_freq.numel() > D:
        raise ValueError("inv_freq must be a contiguous 1-D tensor of at most D / 2 frequencies")
    dev, at = q.device, q.get_device()
    if not (q_out.get_device() == positions.get_device() == inv_freq.get_device() == at
            and (k is None or k.get_device() == k_out.get_device() == at)):
        _same_device(dev, k=k, q_out=q_out, k_out=k_out, positions=positions, inv_freq=inv_freq)
    _on_current_device(at)
    return rows, D


def rope(q, k, positions, inv_freq, *, layout: str = "half", factor: float = 1.0,
         q_out=None, k_out=None, inverse: bool = False, stream=None):
    """Rotary positions on q [1, T, Hq, D] and, unless None, k [1, T, Hk, D]
    (``kda_rope``): the first 2 * len(inv_freq) dimensions of each head turn by
    position * inv_freq, the others are kept.  ``positions`` is int32 or int64
    [T], ``inv_freq`` fp64, as from ``rope_frequencies``.  Without ``q_out`` and
    ``k_out`` it works in place.  ``inverse`` turns back (times ``factor`` again):
    the gradient of the inputs from that of the outputs.  Returns (q_out, k_out)."""
    lib = load_library()
    rows, D = _rope_rows(q, k, positions, inv_freq, layout, q_out, k_out)
    q_out, k_out = q if q_out is None else q_out, k if k_out is None else k_out
    T, n = positions.numel(), len(rows)
    arr = (_RopeTensor * 2)(*rows)
    rc = lib.kda_rope(arr, n, positions.data_ptr(), positions.element_size(),
                      inv_freq.data_ptr(), T, D, 2 * inv_freq.numel(), _LAYOUTS[layout],
                      float(factor), 1 if inverse else 0, _DTYPES[q.dtype], _stream(stream, q.device))
    if rc != KDA_OK:
        _check(rc, lib)
    return q_out, k_out


def _head_weight(w, name, H, D):
    """(address, elements between heads) of a norm's weights."""
    if w is None:
        return 0, 0
    if w.dtype != torch.float32 or not w.is_cuda:
        raise TypeError(f"{name} must be a float32 CUDA tensor")
    if w.shape not in ((D,), (H, D)) or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{D}] or [{H}, {D}] tensor; got shape "
                         f"{tuple(w.shape)}")
    return w.data_ptr(), D if w.dim() == 2 else 0


def qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, *, layout: str = "half",
                 factor: float = 1.0, eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """Norms of queries and keys for each head and the rotary positions in one pass
    (``kda_qk_norm_rope``): each row of q [1, T, Hq, D] and, unless None, k [1, T, Hk, D]
    becomes x / sqrt(mean(x^2) + eps) * weight and is then turned as by ``rope``.
    ``q_weight`` and ``k_weight`` are fp32 [D], [H, D] for a weight of each head, or
    None.  The other arguments are those of ``rope``; without ``q_out`` and ``k_out``
    it works in place.  Returns (q_out, k_out)."""
    lib = load_library()
    q_out = q if q_out is None else q_out
    both = k is not None
    tensors = None
    if both:
        k_out = k if k_out is None else k_out
        tensors = _usual_turn(q, k, q_out, k_out, q_weight, k_weight, positions, inv_freq)
    if tensors is None or layout not in _LAYOUTS:
        tensors = _checked_turn(q, k, q_out, k_out, q_weight, k_weight, positions, inv_freq, layout)
    _on_current_device(q.get_device())
    freqs = inv_freq.numel()
    rc = lib.kda_qk_norm_rope(tensors, 2 if both else 1, float(eps), positions.data_ptr(), positions.element_size(),
                              inv_freq.data_ptr(), positions.numel(), q.shape[-1], 2 * freqs,
                              _LAYOUTS[layout], float(factor), _DTYPES[q.dtype], _stream(stream, q.device))
    if rc != KDA_OK:
        _check(rc, lib)
    return q_out, k_out


def _usual_turn(q, k, q_out, k_out, q_weight, k_weight, positions, inv_freq):
    """The tensors' fields of a ``qk_norm_rope`` call, packed, after one look at the usual
    forms; None for any other, which ``_checked_turn`` takes or says what is wrong with."""
    qs, ks = q.shape, k.shape
    if len(qs) != 4 or len(ks) != 4:
        return None
    one, T, H, D = qs
    one_k, Tk, Hk, Dk = ks
    (_, q_st, q_sh, q_1), (_, k_st, k_sh, k_1) = q.stride(), k.stride()
    at, dtype, f32 = q.get_device(), q.dtype, torch.float32
    if not (at >= 0 and one == one_k == 1 and T == Tk > 1 and D == Dk and H > 1 and Hk > 1 and q_1 == k_1 == 1
            and dtype in _DTYPES and k.dtype is dtype and k.get_device() == at
            and positions.dtype in (torch.int64, torch.int32) and positions.get_device() == at
            and positions.numel() == T and positions.is_contiguous()
            and inv_freq.dtype is torch.float64 and inv_freq.get_device() == at and inv_freq.dim() == 1
            and inv_freq.is_contiguous() and 2 * inv_freq.numel() <= D):
        return None
    out = (q_st, q_sh), (k_st, k_sh)
    if q_out is not q or k_out is not k:
        (_, qo_st, qo_sh, qo_1), (_, ko_st, ko_sh, ko_1) = (x.stride() if x.dim() == 4 else (0, 0, 0, 0) for x in (q_out, k_out))
        if not (q_out.shape == qs and k_out.shape == ks and qo_1 == ko_1 == 1 and q_out.dtype is k_out.dtype is dtype
                and q_out.get_device() == k_out.get_device() == at):
            return None
        out = (qo_st, qo_sh), (ko_st, ko_sh)
    weights = []
    for w, heads in ((q_weight, H), (k_weight, Hk)):
        if w is None:
            weights += 0, 0
            continue
        ws = w.shape
        if not (w.dtype is f32 and w.get_device() == at and w.is_contiguous() and (ws == (D,) or ws == (heads, D))):
            return None
        weights += w.data_ptr(), D if len(ws) == 2 else 0
    return _NORM_ROPE_TENSORS.pack(q.data_ptr(), q_out.data_ptr(), q_st, q_sh, *out[0], H, *weights[:2],
                                   k.data_ptr(), k_out.data_ptr(), k_st, k_sh, *out[1], Hk, *weights[2:])


def _checked_turn(q, k, q_out, k_out, q_weight, k_weight, positions, inv_freq, layout):
    """The same, every argument checked for itself."""
    rows, D = _rope_rows(q, k, positions, inv_freq, layout, q_out, k_out)
    if k is None and k_weight is not None:
        raise ValueError("k_weight is given without k")
    at = q.get_device()
    fields = _NO_TENSOR
    if k is not None:
        fields = (*rows[1], *_head_weight(k_weight, "k_weight", rows[1][6], D))
        if k_weight is not None and k_weight.get_device() != at:
            _same_device(q.device, k_weight=k_weight)
    tensors = _NORM_ROPE_TENSORS.pack(*rows[0], *_head_weight(q_weight, "q_weight", rows[0][6], D), *fields)
    if q_weight is not None and q_weight.get_device() != at:
        _same_device(q.device, q_weight=q_weight)
    return tensors


def gated_norm(x, weight=None, *, gate=None, activation: str = "sigmoid", eps: float = 1e-6,
               out=None, stream=None) -> torch.Tensor:
    """Root-mean-square norm of each row of x [1, T, H, D] with a weight and a
    gate (``kda_gated_norm``): x / sqrt(mean(x^2) + eps) * weight * act(gate).
    ``weight`` is fp32 [D] or None, ``gate`` like x or None, ``activation``
    "sigmoid", "silu" or "none"; ``out`` defaults to a new tensor and may be x.
    Returns ``out``."""
    lib = load_library()
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is not one of {sorted(_ACTIVATIONS)}")
    if x.dtype not in _DTYPES:
        raise TypeError(f"x dtype {x.dtype} not supported")
    T, H, D, x_st, x_sh = _rows(x, "x")
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    To, Ho, Do, o_st, o_sh = _rows(out, "out", x.dtype)
    if (To, Ho, Do) != (T, H, D):
        raise ValueError("out must have the shape of x")
    g_st = g_sh = 0
    if gate is not None:
        Tg, Hg, Dg, g_st, g_sh = _rows(gate, "gate", x.dtype)
        if (Tg, Hg, Dg) != (T, H, D):
            raise ValueError("gate must have the shape of x")
    if weight is not None:
        if weight.dtype != torch.float32 or not weight.is_cuda:
            raise TypeError("weight must be a float32 CUDA tensor")
        if weight.dim() != 1 or weight.numel() != D or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous 1-D tensor of {D} values")
    at = x.get_device()
    if not (out.get_device() == at and (gate is None or gate.get_device() == at)
            and (weight is None or weight.get_device() == at)):
        _same_device(x.device, gate=gate, weight=weight, out=out)
    _on_current_device(at)
    rc = lib.kda_gated_norm(
        x.data_ptr(), x_st, x_sh, None if gate is None else gate.data_ptr(), g_st, g_sh,
        None if weight is None else weight.data_ptr(), out.data_ptr(), o_st, o_sh, T, H, D,
        float(eps), _ACTIVATIONS[activation], _DTYPES[x.dtype], _stream(stream, x.device))
    if rc != KDA_OK:
        _check(rc, lib)
    return out
