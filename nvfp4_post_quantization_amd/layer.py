"""Binding of libnvfp4mi_layer.so (include/nvfp4mi_layer.h beside this file):
tokens sorted by expert and back, the expert layer for any number of tokens, and
low-rank adapters beside a W4A16 product.  Its functions are the package's, and like
those plain calls: autograd records none of them, and a gradient is the call that
makes it (moe_dispatch_grad, moe_combine_grad).
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import (_BF16, _U8, _c_void_p, _check, _dev, _flat, _i64, _row_major, _rows_out, _scalar, _scratch)
from . import load as _load_products

__all__ = [
    "moe_sort_workspace_bytes", "moe_sort", "moe_dispatch", "moe_dispatch_grad", "moe_combine", "moe_combine_grad",
    "moe_sorted_workspace_bytes", "moe_forward_sorted", "matmul_lora_workspace_bytes", "matmul_w4a16_lora",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4mi_layer.so")

_size_t, _int = ctypes.c_size_t, ctypes.c_int
_p = _c_void_p
_SIGS = {
    "nvfp4_moe_sort_workspace_bytes": (_size_t, [_i64, _i64, _i64]),
    "nvfp4_moe_sort": (_int, [_p, _i64, _i64, _i64, _p, _p, _p, _p, _size_t, _p]),
    "nvfp4_moe_dispatch": (_int, [_p, _i64, _i64, _i64, _p, _i64, _p, _i64, _p]),
    "nvfp4_moe_combine": (_int, [_p, _i64, _p, _p, _i64, _i64, _i64, _p, _i64, _p]),
    "nvfp4_moe_combine_grad": (_int, [_p, _i64, _p, _i64, _p, _p, _i64, _i64, _i64, _p, _i64, _p, _p]),
    "nvfp4_moe_forward_sorted_workspace_bytes": (_size_t, [_i64, _i64, _i64, _i64, _i64]),
    "nvfp4_moe_forward_sorted": (_int, [_p, _i64, _i64, _i64, _p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _p, _p, _p,
                                        _i64, _p, _size_t, _p]),
    "nvfp4_matmul_w4a16_lora_workspace_bytes": (_size_t, [_i64, _i64, _i64, _i64]),
    "nvfp4_matmul_w4a16_lora": (_int, [_p, _i64, _i64, _i64, _p, _p, _p, _i64, _p, _i64, _i64, _p, _p, _p, _p, _i64,
                                       _p, _size_t, _p]),
}

_lib = None
_I32, _F32 = torch.int32, torch.float32
_device_now, _stream_now = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def load() -> ctypes.CDLL:
    """Load libnvfp4mi_layer.so (built with libnvfp4mi.so, which it uses)."""
    global _lib
    if _lib is None:
        _load_products()
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m nvfp4_post_quantization_amd.build` (hipcc, gfx950)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _call(fn: str, device, *args) -> None:
    """fn(*args, the device's current stream), with the device made current."""
    index, lib = device.index, _lib or load()
    if _device_now() == index:
        status = getattr(lib, fn)(*args, _stream_now(index))
    else:
        with torch.cuda.device(device):
            status = getattr(lib, fn)(*args, _stream_now(index))
    if status:
        _check(fn, status)


# Small calls are the host's: each helper asks a good tensor as little as it can (a
# tenth of such a call) and leaves it to the package's own to say what is wrong.

def _choices(t: torch.Tensor, name: str) -> torch.Size:
    """(tokens, top_k) of a contiguous int32 [tokens, top_k] tensor."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _I32 and t.is_cuda and t.dim() == 2 and t.is_contiguous()):
        _dev(t, _I32, name, 2)
        raise ValueError(f"{name} must be contiguous")
    return t.shape


def _matrix(t: torch.Tensor, dtype, name: str, rows: int, cols: int | None, device) -> tuple[int, int]:
    """Columns and row stride of a [rows, cols] tensor with contiguous rows on `device`."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == 2 and t.device == device:
        have, wide = t.shape
        ld, one = t.stride()
        if have == rows and one == 1 and (cols is None or wide == cols):
            return wide, ld if rows > 1 else wide
    _dev(t, dtype, name, 2)
    if t.shape[0] != rows or (cols is not None and t.shape[1] != cols) or t.device != device:
        raise ValueError(f"{name} must be [{rows}, {'cols' if cols is None else cols}] on {device}")
    return t.shape[1], _row_major(t, name)


def _out(out: torch.Tensor | None, dtype, name: str, rows: int, cols: int, device) -> tuple[torch.Tensor, int]:
    """The [rows, cols] output, made here or checked, and its row stride."""
    if out is None:
        return torch.empty(rows, cols, dtype=dtype, device=device), cols
    return out, _matrix(out, dtype, name, rows, cols, device)[1]


def moe_sort_workspace_bytes(tokens: int, top_k: int, experts: int) -> int:
    return int(load().nvfp4_moe_sort_workspace_bytes(tokens, top_k, experts))


def moe_sort(ids: torch.Tensor, experts: int, out=None, workspace: torch.Tensor | None = None):
    """Choices (token * top_k + place) sorted by expert: (order i32
    [tokens * top_k], place i32 [tokens, top_k], offsets i32 [experts + 1]).

    order[row] = choice (-1 behind the last row), place[token, s] = row (-1 where
    ids[token, s] names no expert), rows of expert e: offsets[e] .. offsets[e+1].
    Choices of an expert stay in their order.  out=(order, place, offsets) reuses
    buffers; workspace: uint8, at least moe_sort_workspace_bytes(...) bytes."""
    tokens, top_k = _choices(ids, "ids")
    dev = ids.device
    if out is None:
        order = torch.empty(tokens * top_k, dtype=_I32, device=dev)
        place = torch.empty_like(ids)
        offsets = torch.empty(max(experts, 0) + 1, dtype=_I32, device=dev)
    else:
        order = _flat(out[0], _I32, (tokens * top_k,), "order", dev)
        place = _flat(out[1], _I32, (tokens, top_k), "place", dev)
        offsets = _flat(out[2], _I32, (experts + 1,), "offsets", dev)
    ws = _scratch(workspace, dev, moe_sort_workspace_bytes, tokens, top_k, experts)
    _call("nvfp4_moe_sort", dev, ids.data_ptr(), tokens, top_k, experts, order.data_ptr(), place.data_ptr(),
          offsets.data_ptr(), ws.data_ptr(), ws.numel())
    return order, place, offsets


def moe_dispatch(x: torch.Tensor, place: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """xs[place[t, s]] = x[t]: rows of any dtype (bf16 activations, packed nibbles,
    codes) to their sorted rows, [tokens * top_k, cols].  Rows to which no choice
    goes, those behind the last, are not written (without `out` they hold
    anything).  Rows contiguous, any row stride."""
    tokens, top_k = _choices(place, "place")
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev, size, dtype = place.device, x.element_size(), x.dtype
    cols, ldx = _matrix(x, dtype, "x", tokens, None, dev)
    out, ldo = _out(out, dtype, "out", tokens * top_k, cols, dev)
    _call("nvfp4_moe_dispatch", dev, x.data_ptr(), tokens, cols * size, ldx * size, place.data_ptr(), top_k,
          out.data_ptr(), ldo * size)
    return out


def moe_combine(ys: torch.Tensor, place: torch.Tensor, weights: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """y[t] = sum over s of weights[t, s] * ys[place[t, s]] (fp32 sums, one
    rounding), bf16 [tokens, cols] of bf16 ys [tokens * top_k, cols], cols a
    multiple of 8.  Places of -1 add nothing; weights (f32 [tokens, top_k]) None:
    all 1.  ys and out may have any row stride of 16-byte multiples."""
    tokens, top_k = _choices(place, "place")
    dev = place.device
    cols, ld = _matrix(ys, _BF16, "ys", tokens * top_k, None, dev)
    w = None if weights is None else _flat(weights, _F32, (tokens, top_k), "weights", dev).data_ptr()
    y, ldy = _out(out, _BF16, "out", tokens, cols, dev)
    _call("nvfp4_moe_combine", dev, ys.data_ptr(), ld, place.data_ptr(), w, tokens, top_k, cols, y.data_ptr(), ldy)
    return y


def moe_dispatch_grad(dxs: torch.Tensor, place: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of moe_dispatch: dx[t] = sum over s of dxs[place[t, s]]."""
    return moe_combine(dxs, place, None, out)


def moe_combine_grad(dy: torch.Tensor, ys: torch.Tensor, place: torch.Tensor, weights: torch.Tensor, out=None):
    """The gradient of moe_combine for dy = dL/dy: (dys bf16 [tokens * top_k, cols]
    with dys[place[t, s]] = weights[t, s] * dy[t], dweights f32 [tokens, top_k] =
    <dy[t], ys[place[t, s]]>, 0 where the place is -1).  Rows of dys to which no
    choice goes are not written.  out=(dys, dweights) reuses buffers."""
    tokens, top_k = _choices(place, "place")
    dev = place.device
    cols, lddy = _matrix(dy, _BF16, "dy", tokens, None, dev)
    rows = tokens * top_k
    _, ldys = _matrix(ys, _BF16, "ys", rows, cols, dev)
    _flat(weights, _F32, (tokens, top_k), "weights", dev)
    dys, lddys = _out(None if out is None else out[0], _BF16, "dys", rows, cols, dev)
    if out is None:
        dw = torch.empty_like(weights)
    else:
        dw = _flat(out[1], _F32, (tokens, top_k), "dweights", dev)
    _call("nvfp4_moe_combine_grad", dev, dy.data_ptr(), lddy, ys.data_ptr(), ldys, place.data_ptr(), weights.data_ptr(),
          tokens, top_k, cols, dys.data_ptr(), lddys, dw.data_ptr())
    return dys, dw


def moe_sorted_workspace_bytes(tokens: int, top_k: int, experts: int, hidden: int, inter: int) -> int:
    return int(load().nvfp4_moe_forward_sorted_workspace_bytes(tokens, top_k, experts, hidden, inter))


def moe_forward_sorted(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w13_packed: torch.Tensor,
                       w13_codes: torch.Tensor, w13_scale2: torch.Tensor, w2_packed: torch.Tensor,
                       w2_codes: torch.Tensor, w2_scale2: torch.Tensor, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None) -> torch.Tensor:
    """moe_forward for any number of tokens (the same arguments): beyond 64 the
    tokens are sorted by expert, and silu(W1 x) * (W3 x) and an expert's row are each
    rounded to fp16 with a power of two for every 32 columns; x and silu(..) * (..)
    enter the products as fp16 with a power of two a row (exact but for values 2^29
    and more below the row's largest).  out: any row stride of 16-byte multiples;
    workspace: uint8, at least moe_sorted_workspace_bytes(tokens, top_k, experts,
    hidden, inter) bytes."""
    _dev(x, _BF16, "x", 2)
    _dev(ids, _I32, "ids", 2)
    _dev(w13_packed, _U8, "w13_packed", 4)
    dev = x.device
    tokens, hidden = x.shape
    top_k = ids.shape[1]
    e, _, inter, _ = w13_packed.shape
    _flat(ids, _I32, (tokens, top_k), "ids", dev)
    _flat(weights, _F32, (tokens, top_k), "weights", dev)
    _flat(w13_packed, _U8, (e, 2, inter, hidden // 2), "w13_packed", dev)
    _flat(w13_codes, _U8, (e, 2, inter, hidden // 16), "w13_codes", dev)
    _flat(w13_scale2, _F32, (e,), "w13_scale2", dev)
    mid = (1,) if w2_packed.dim() == 4 else ()
    _flat(w2_packed, _U8, (e, *mid, hidden, inter // 2), "w2_packed", dev)
    _flat(w2_codes, _U8, (e, *mid, hidden, inter // 16), "w2_codes", dev)
    _flat(w2_scale2, _F32, (e,), "w2_scale2", dev)
    y, ldy = _rows_out(out, tokens, hidden, dev)
    ws = _scratch(workspace, dev, moe_sorted_workspace_bytes, tokens, top_k, e, hidden, inter)
    _call("nvfp4_moe_forward_sorted", dev, x.data_ptr(), tokens, hidden, _row_major(x, "x"), ids.data_ptr(),
          weights.data_ptr(), top_k, e, inter, w13_packed.data_ptr(), w13_codes.data_ptr(), w13_scale2.data_ptr(),
          w2_packed.data_ptr(), w2_codes.data_ptr(), w2_scale2.data_ptr(), y.data_ptr(), ldy, ws.data_ptr(), ws.numel())
    return y


def matmul_lora_workspace_bytes(tokens: int, out_features: int, k: int, rank: int) -> int:
    return int(load().nvfp4_matmul_w4a16_lora_workspace_bytes(tokens, out_features, k, rank))


def matmul_w4a16_lora(x: torch.Tensor, w_packed: torch.Tensor, w_codes: torch.Tensor, w_scale2: torch.Tensor,
                      adapter_ids: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor, lora_scale: torch.Tensor,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """matmul_w4a16 with each token's low-rank adapter: y[t] = x[t] w^T +
    lora_scale[a] * (x[t] A_a^T) B_a^T, a = adapter_ids[t], one rounding.

    adapter_ids i32 [tokens] (outside the adapters: none), lora_a bf16 [adapters,
    rank, k], lora_b bf16 [adapters, out_features, rank], lora_scale f32
    [adapters]; rank a multiple of 8, at most 256.  The others as matmul_w4a16;
    workspace: uint8, at least matmul_lora_workspace_bytes(tokens, out_features, k,
    rank) bytes."""
    _dev(x, _BF16, "x", 2)
    _dev(w_packed, _U8, "w_packed", 2)
    _dev(lora_a, _BF16, "lora_a", 3)
    dev = x.device
    tokens, k = x.shape
    o, (adapters, rank, _) = w_packed.shape[0], lora_a.shape
    _flat(w_packed, _U8, (o, k // 2), "w_packed", dev)
    _flat(w_codes, _U8, (o, k // 16), "w_codes", dev)
    _scalar(w_scale2, "w_scale2", dev)
    _flat(adapter_ids, _I32, (tokens,), "adapter_ids", dev)
    _flat(lora_a, _BF16, (adapters, rank, k), "lora_a", dev)
    _flat(lora_b, _BF16, (adapters, o, rank), "lora_b", dev)
    _flat(lora_scale, _F32, (adapters,), "lora_scale", dev)
    y, ldy = _rows_out(out, tokens, o, dev)
    ws = _scratch(workspace, dev, matmul_lora_workspace_bytes, tokens, o, k, rank)
    _call("nvfp4_matmul_w4a16_lora", dev, x.data_ptr(), tokens, k, _row_major(x, "x"), w_packed.data_ptr(),
          w_codes.data_ptr(), w_scale2.data_ptr(), o, adapter_ids.data_ptr(), adapters, rank, lora_a.data_ptr(),
          lora_b.data_ptr(), lora_scale.data_ptr(), y.data_ptr(), ldy, ws.data_ptr(), ws.numel())
    return y
