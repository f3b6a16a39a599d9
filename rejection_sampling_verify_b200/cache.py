"""The key-value cache around the verify step: Python binding.

Like the verify's binding, this module only marshals arguments: the raw
functions carry the ABI's names (``include/psi_verify.h``), and the tensor
helpers check shapes, allocate outputs and workspace with torch, and call
them on the current stream.  The order of a serving step is

    cache_resize   room for the drafted block in every sequence
    cache_append   per layer: norm, rotary positions, write of keys and values
    attend_block   per layer: attention of the block over the cache
    verify_*       of the block's logits
    cache_commit   the accepted path stays (tree verify); after a linear
                   verify the new length is lens + n_emitted
    cache_resize   pages behind the new length go back
    cache_fork     a sequence is continued more than once

With ``stream`` a call is made as under ``torch.cuda.stream(stream)``: outputs
and workspace are that stream's memory too.  The inputs' memory is the
caller's to keep, and its order with that stream the caller's to see to.
"""
from __future__ import annotations

import ctypes as C
import math
import os
from dataclasses import dataclass

from . import (PSI_OK, PsiError, _check_out, _check_workspace, _device_of, _dtype_code, _nbytes,
               _ptr, _torch, load_library)


class CacheLayout(C.Structure):
    """``psi_cache_layout``."""
    _fields_ = [("dtype", C.c_int), ("layers", C.c_int32), ("num_pages", C.c_int32),
                ("page_size", C.c_int32), ("kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("layer_stride", C.c_int64), ("page_stride", C.c_int64),
                ("slot_stride", C.c_int64), ("head_stride", C.c_int64)]


class PageStatePtrs(C.Structure):
    """``psi_page_state``: device pointers."""
    _fields_ = [("page_table", C.c_void_p), ("page_counts", C.c_void_p), ("refs", C.c_void_p),
                ("free_pages", C.c_void_p), ("n_free", C.c_void_p)]


def declare(lib):
    """Argument types of the cache's entry points."""
    vp, i32, i64, f32, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_size_t
    lay, st = C.POINTER(CacheLayout), C.POINTER(PageStatePtrs)
    lib.psi_cache_append.restype = C.c_int
    lib.psi_cache_append.argtypes = [lay, vp, vp, vp, i32, vp, i32, i32, i32, vp, i64, i64, vp,
                                     i64, i64, vp, i64, i64, vp, vp, f32, vp, i32, i32, f32, vp,
                                     vp, vp, vp]
    lib.psi_attend_block_workspace_bytes.restype = sz
    lib.psi_attend_block_workspace_bytes.argtypes = [lay, i32, i32, i32, i32]
    lib.psi_attend_block.restype = C.c_int
    lib.psi_attend_block.argtypes = [lay, vp, vp, vp, i32, vp, i32, i32, i32, vp, i64, i64, vp,
                                     f32, vp, vp, vp, vp, sz, vp]
    lib.psi_cache_commit.restype = C.c_int
    lib.psi_cache_commit.argtypes = [lay, vp, vp, vp, i32, vp, i32, i32, vp, vp, vp, vp, vp]
    lib.psi_cache_resize.restype = C.c_int
    lib.psi_cache_resize.argtypes = [i32, i32, i32, i32, vp, i32, st, st, vp, vp]
    lib.psi_cache_fork_workspace_bytes.restype = sz
    lib.psi_cache_fork_workspace_bytes.argtypes = [i32]
    lib.psi_cache_fork.restype = C.c_int
    lib.psi_cache_fork.argtypes = [lay, vp, vp, i32, i32, vp, vp, st, st, i32, vp, vp, vp, vp, sz,
                                   vp]


# ---- raw ABI (device pointers as ints, structures as the classes above) ------------

def _ref(s):
    return None if s is None else C.byref(s)


def psi_cache_append(layout, k_pages, v_pages, page_table, max_pages, lens, N, R, q_heads, q,
                     q_row_stride, q_head_stride, k, k_row_stride, k_head_stride, v, v_row_stride,
                     v_head_stride, q_weight, k_weight, eps, inv_freq, rotary_dim, interleaved,
                     rope_scale, parents, out_q, dev_status, stream) -> int:
    return int(load_library().psi_cache_append(
        _ref(layout), k_pages, v_pages, page_table, max_pages, lens, N, R, q_heads, q,
        q_row_stride, q_head_stride, k, k_row_stride, k_head_stride, v, v_row_stride,
        v_head_stride, q_weight, k_weight, eps, inv_freq, rotary_dim, interleaved, rope_scale,
        parents, out_q, dev_status, stream))


def psi_attend_block_workspace_bytes(layout, N, R, q_heads, max_pages) -> int:
    return int(load_library().psi_attend_block_workspace_bytes(_ref(layout), N, R, q_heads,
                                                               max_pages))


def psi_attend_block(layout, k_pages, v_pages, page_table, max_pages, lens, N, R, q_heads, q,
                     q_row_stride, q_head_stride, parents, scale, out_o, out_lse, dev_status,
                     workspace, workspace_bytes, stream) -> int:
    return int(load_library().psi_attend_block(
        _ref(layout), k_pages, v_pages, page_table, max_pages, lens, N, R, q_heads, q,
        q_row_stride, q_head_stride, parents, scale, out_o, out_lse, dev_status, workspace,
        workspace_bytes, stream))


def psi_cache_commit(layout, k_pages, v_pages, page_table, max_pages, lens, N, M, path_nodes,
                     path_len, out_lens, dev_status, stream) -> int:
    return int(load_library().psi_cache_commit(_ref(layout), k_pages, v_pages, page_table,
                                               max_pages, lens, N, M, path_nodes, path_len,
                                               out_lens, dev_status, stream))


def psi_cache_resize(N, max_pages, num_pages, page_size, lens, extra, in_state, out_state,
                     dev_status, stream) -> int:
    return int(load_library().psi_cache_resize(N, max_pages, num_pages, page_size, lens, extra,
                                               _ref(in_state), _ref(out_state), dev_status,
                                               stream))


def psi_cache_fork_workspace_bytes(K) -> int:
    return int(load_library().psi_cache_fork_workspace_bytes(K))


def psi_cache_fork(layout, k_pages, v_pages, N, max_pages, lens, out_lens, in_state, out_state, K,
                   src, dst, dev_status, workspace, workspace_bytes, stream) -> int:
    return int(load_library().psi_cache_fork(_ref(layout), k_pages, v_pages, N, max_pages, lens,
                                             out_lens, _ref(in_state), _ref(out_state), K, src,
                                             dst, dev_status, workspace, workspace_bytes, stream))


# ---- torch tensor helpers --------------------------------------------------------------

@dataclass
class AppendResult:
    q: "torch.Tensor"       # [N, R, Hq, D]
    status: "torch.Tensor"  # int32 [1] device status word


@dataclass
class AttendResult:
    o: "torch.Tensor"            # [N, R, Hq, D]
    lse: "torch.Tensor | None"   # float32 [N, R, Hq]
    status: "torch.Tensor"


@dataclass
class CommitResult:
    lens: "torch.Tensor"    # int32 [N]
    status: "torch.Tensor"


@dataclass
class PageState:
    """Who holds which page (``psi_page_state``); int32 tensors."""
    table: "torch.Tensor"   # [N, max_pages], -1 where no page is held
    counts: "torch.Tensor"  # [N]
    refs: "torch.Tensor"    # [P]
    free: "torch.Tensor"    # [P] stack of free pages
    n_free: "torch.Tensor"  # [1]

    @classmethod
    def empty(cls, N: int, max_pages: int, num_pages: int, device="cuda") -> "PageState":
        """No sequence holds a page; page 0 is the first to be popped."""
        torch = _torch()
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.full((N, max_pages), -1, **i32), torch.zeros(N, **i32),
                   torch.zeros(num_pages, **i32),
                   torch.arange(num_pages - 1, -1, -1, **i32),
                   torch.full((1,), num_pages, **i32))


@dataclass
class ResizeResult:
    pages: PageState
    status: "torch.Tensor"


@dataclass
class ForkResult:
    pages: PageState
    lens: "torch.Tensor"
    status: "torch.Tensor"


def _check(status, where):
    if status != PSI_OK:
        raise PsiError(status, where)


def _int32(name, t, shape):
    torch = _torch()
    if t.dtype != torch.int32 or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)}")


def _layout(k_pages, v_pages, layered: bool) -> CacheLayout:
    """The pools' layout: [P, S, H, D] of one layer, or [L, P, S, H, D]."""
    dims = 5 if layered else 4
    if k_pages.dim() != dims or k_pages.shape != v_pages.shape or \
            k_pages.stride() != v_pages.stride() or k_pages.dtype != v_pages.dtype:
        raise ValueError(f"k_pages and v_pages must have {dims} dims "
                         f"({'layers, ' if layered else ''}pages, slots, heads, elements) and the "
                         f"same shape, strides and dtype")
    if k_pages.stride(-1) != 1:
        raise ValueError("pages must have a contiguous last dim")
    shape = tuple(k_pages.shape) if layered else (1, *k_pages.shape)
    strides = tuple(k_pages.stride()) if layered else (0, *k_pages.stride())
    strides = [0 if n == 1 else s for n, s in zip(shape, strides)]
    return CacheLayout(_dtype_code(k_pages), *shape, *strides[:4])


def _heads(name, t, N, R, heads, D, dtype):
    """(row stride, head stride) of a [N, R, heads, D] tensor with evenly spaced rows."""
    if tuple(t.shape) != (N, R, heads, D) or t.dtype != dtype or t.stride(3) != 1:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {(N, R, heads, D)} with a "
                         f"contiguous last dim, got {t.dtype} {tuple(t.shape)}")
    row = t.stride(1) if R > 1 else t.stride(0) if N > 1 else 0
    if N > 1 and R > 1 and t.stride(0) != R * row:
        raise ValueError(f"{name}: rows must be evenly spaced")
    return row, t.stride(2) if heads > 1 else 0


def _block(q, page_table, lens, parents):
    torch = _torch()
    if q.dim() != 4:
        raise ValueError("q must be [N, R, heads, D]")
    N, R = q.shape[:2]
    if page_table.dim() != 2:
        raise ValueError("page_table must be [N, max_pages]")
    _int32("page_table", page_table, (N, page_table.shape[1]))
    _int32("lens", lens, (N,))
    if parents is not None:
        _int32("parents", parents, (N, R - 1))
    return N, R


# The common form of each call (outputs and workspace not given, the current
# stream) goes through the compiled binding, which checks the tensors as the
# functions below do; what it does not take comes back here as None.
_binding = None


def _short():
    global _binding
    if _binding is None:
        _torch()  # (the extension's symbols are torch's)
        lib = load_library()
        from . import build
        if not os.path.exists(build.BINDING):
            build.build_binding()
        from . import _cache_binding
        _cache_binding.bind(*(C.cast(getattr(lib, name), C.c_void_p).value for name in (
            "psi_cache_append", "psi_attend_block_workspace_bytes", "psi_attend_block",
            "psi_cache_commit", "psi_cache_resize", "psi_cache_fork_workspace_bytes",
            "psi_cache_fork")))
        _binding = _cache_binding
    return _binding


# A call's shapes, strides and dtypes decide what it may do: they are checked
# once, and what was found (the layout, the strides) is kept under them; the
# attention's workspace also under the device, whose size decides it.
_MAX_PLANS = 512
_plans = {}


def _remember(key, plan):
    if len(_plans) >= _MAX_PLANS:
        _plans.clear()
    _plans[key] = plan
    return plan


def _sig(t):
    return None if t is None else (t.shape, t.stride(), t.dtype)


def _on_device(ref, named):
    """Index of the device of `ref`, which must be the current one and that of
    the other tensors (``_device_of`` says what is wrong)."""
    torch = _torch()
    dev = ref.get_device()
    same = dev >= 0 and dev == torch._C._cuda_getDevice()
    for t in named.values():
        if t is not None and t.get_device() != dev:
            same = False
    if not same:
        _device_of(ref, **named)
    return dev


def _new_status(dev: int):
    return _torch().zeros(1, dtype=_torch().int32, device=dev)


def rope_frequencies(rotary_dim: int, theta: float = 1e6, factor: float = 1.0,
                     scaling: str = "none", original_length: int = 32768,
                     beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """(inv_freq, rope_scale) for :func:`cache_append`: float64 [rotary_dim/2].

    scaling "none"; "linear" (positions divided by ``factor``); "ntk" (theta
    grown so that the longest wavelength stretches by ``factor``); "yarn"
    (Peng et al., "YaRN: Efficient Context Window Extension of Large Language
    Models", 2023: pairs that turn less than ``beta_slow`` times over
    ``original_length`` are stretched, those over ``beta_fast`` are kept, with
    a ramp between, and the scores' temperature goes into rope_scale).
    """
    torch = _torch()
    if rotary_dim < 2 or rotary_dim % 2 or factor < 1:
        raise ValueError("rotary_dim must be even and positive, factor at least 1")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    if scaling == "ntk" and rotary_dim > 2:
        theta = theta * factor ** (rotary_dim / (rotary_dim - 2))
    inv = theta ** (-2.0 * i / rotary_dim)
    scale = 1.0
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "yarn":
        def pair(turns):  # the pair that turns so often over the original length
            return rotary_dim * math.log(original_length / (turns * 2 * math.pi)) / \
                (2 * math.log(theta))
        low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)),
                                                             rotary_dim - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        inv = inv / factor * ramp + inv * (1 - ramp)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"scaling must be none, linear, ntk or yarn, got {scaling!r}")
    return inv.to(device), scale


def cache_append(q, k, v, k_pages, v_pages, page_table, lens, q_weight=None, k_weight=None,
                 eps: float = 1e-6, inv_freq=None, interleaved: bool = False,
                 rope_scale: float = 1.0, parents=None, stream=None,
                 out: AppendResult | None = None) -> AppendResult:
    """Norm, rotary positions and the write of a block's keys and values into
    one layer's pages (``psi_cache_append``).

    q [N, R, Hq, D], k and v [N, R, H, D] (slices of one projection will do);
    k_pages, v_pages [P, S, H, D] of any strides; page_table int32
    [N, max_pages]; lens int32 [N]; q_weight, k_weight [D] or None;
    inv_freq float64 [rotary_dim / 2] or None; parents int32 [N, R - 1] or
    None (a chain).  ``out.q`` may be ``q`` itself.
    """
    if stream is not None:
        with _torch().cuda.stream(stream):
            return cache_append(q, k, v, k_pages, v_pages, page_table, lens, q_weight, k_weight,
                                eps, inv_freq, interleaved, rope_scale, parents, out=out)
    if out is None:
        r = (_binding or _short()).append(q, k, v, k_pages, v_pages, page_table, lens, q_weight,
                                          k_weight, eps, inv_freq, interleaved, rope_scale,
                                          parents)
        if r is not None:
            _check(r[0], "psi_cache_append")
            return AppendResult(r[1], r[2])
    key = ("append", _sig(q), _sig(k), _sig(v), _sig(k_pages), _sig(v_pages), _sig(page_table),
           _sig(lens), _sig(q_weight), _sig(k_weight), _sig(inv_freq), _sig(parents))
    plan = _plans.get(key) or _remember(key, _plan_append(
        q, k, v, k_pages, v_pages, page_table, lens, q_weight, k_weight, inv_freq, parents))
    lay, N, R, Hq, strides, rot, max_pages = plan
    others = dict(k=k, v=v, k_pages=k_pages, v_pages=v_pages, page_table=page_table, lens=lens,
                  q_weight=q_weight, k_weight=k_weight, inv_freq=inv_freq, parents=parents)
    if out is not None:
        torch = _torch()
        _check_out("q", out.q, q.dtype, q.shape)
        _check_out("status", out.status, torch.int32, (1,))
        others.update(out_q=out.q, status=out.status)
    dev = _on_device(q, others)
    raw = _torch()._C._cuda_getCurrentRawStream(dev)
    if out is None:
        out = AppendResult(_torch().empty(q.shape, dtype=q.dtype, device=q.device),
                           _new_status(dev))
    st = psi_cache_append(
        lay, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), max_pages,
        lens.data_ptr(), N, R, Hq, q.data_ptr(), *strides[0], k.data_ptr(), *strides[1],
        v.data_ptr(), *strides[2], _ptr(q_weight), _ptr(k_weight), eps, _ptr(inv_freq), rot,
        1 if interleaved else 0, rope_scale, _ptr(parents), out.q.data_ptr(),
        out.status.data_ptr(), raw)
    _check(st, "psi_cache_append")
    return out


def _plan_append(q, k, v, k_pages, v_pages, page_table, lens, q_weight, k_weight, inv_freq,
                 parents):
    torch = _torch()
    N, R = _block(q, page_table, lens, parents)
    lay = _layout(k_pages, v_pages, layered=False)
    Hq, D, H = q.shape[2], lay.head_dim, lay.kv_heads
    strides = [_heads(name, t, N, R, h, D, k_pages.dtype)
               for name, t, h in (("q", q, Hq), ("k", k, H), ("v", v, H))]
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dtype != q.dtype or tuple(w.shape) != (D,) or
                              not w.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {q.dtype} tensor of shape ({D},)")
    if inv_freq is not None and (inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or
                                 not inv_freq.is_contiguous()):
        raise ValueError("inv_freq must be a contiguous float64 vector")
    return lay, N, R, Hq, strides, 0 if inv_freq is None else 2 * len(inv_freq), \
        page_table.shape[1]


def attend_block(q, k_pages, v_pages, page_table, lens, parents=None, scale: float | None = None,
                 want_lse: bool = False, workspace=None, stream=None,
                 out: AttendResult | None = None) -> AttendResult:
    """Attention of a block over one layer's pages (``psi_attend_block``).

    q [N, R, Hq, D]; the block's keys and values are in the pages at
    positions lens[n]..lens[n] + R - 1.  R = 1 is a step of one new token;
    parents None is a drafted chain, else a tree.  scale defaults to
    D ** -0.5.  With ``out`` and a large enough ``workspace`` the call only
    launches work on the stream.
    """
    if stream is not None:
        with _torch().cuda.stream(stream):
            return attend_block(q, k_pages, v_pages, page_table, lens, parents, scale, want_lse,
                                workspace, out=out)
    if out is None and workspace is None:
        r = (_binding or _short()).attend(q, k_pages, v_pages, page_table, lens, parents, scale,
                                          want_lse)
        if r is not None:
            _check(r[0], "psi_attend_block")
            return AttendResult(r[1], r[2], r[3])
    key = ("attend", _sig(q), _sig(k_pages), _sig(v_pages), _sig(page_table), _sig(lens),
           _sig(parents))
    plan = _plans.get(key) or _remember(key, _plan_attend(q, k_pages, v_pages, page_table, lens,
                                                          parents))
    lay, N, R, Hq, q_row, q_head, max_pages, default_scale = plan
    torch = _torch()
    others = dict(k_pages=k_pages, v_pages=v_pages, page_table=page_table, lens=lens,
                  parents=parents, workspace=workspace)
    if out is not None:
        _check_out("o", out.o, q.dtype, q.shape)
        _check_out("lse", out.lse, torch.float32, q.shape[:3], optional=True)
        _check_out("status", out.status, torch.int32, (1,))
        others.update(o=out.o, lse=out.lse, status=out.status)
    _check_workspace(workspace)
    dev = _on_device(q, others)
    raw = _torch()._C._cuda_getCurrentRawStream(dev)
    device = q.device
    if out is None:
        out = AttendResult(torch.empty(q.shape, dtype=q.dtype, device=device),
                           torch.empty(q.shape[:3], dtype=torch.float32, device=device)
                           if want_lse else None, _new_status(dev))
    ws_key = ("attend workspace", dev, key)
    ws_bytes = _plans.get(ws_key)
    if ws_bytes is None:  # (0 for sizes that the call itself refuses)
        ws_bytes = _remember(ws_key, psi_attend_block_workspace_bytes(lay, N, R, Hq, max_pages))
    if workspace is None or _nbytes(workspace) < ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
    st = psi_attend_block(lay, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
                          max_pages, lens.data_ptr(), N, R, Hq, q.data_ptr(), q_row, q_head,
                          _ptr(parents), default_scale if scale is None else scale,
                          out.o.data_ptr(), _ptr(out.lse), out.status.data_ptr(),
                          workspace.data_ptr(), _nbytes(workspace), raw)
    _check(st, "psi_attend_block")
    return out


def _plan_attend(q, k_pages, v_pages, page_table, lens, parents):
    N, R = _block(q, page_table, lens, parents)
    lay = _layout(k_pages, v_pages, layered=False)
    Hq, D = q.shape[2], lay.head_dim
    q_row, q_head = _heads("q", q, N, R, Hq, D, k_pages.dtype)
    max_pages = page_table.shape[1]
    return lay, N, R, Hq, q_row, q_head, max_pages, D ** -0.5


def cache_commit(k_pages, v_pages, page_table, lens, path_nodes, path_len, stream=None,
                 out: CommitResult | None = None) -> CommitResult:
    """Keep the accepted path of a tree verify (``psi_cache_commit``).

    k_pages, v_pages [L, P, S, H, D]; path_nodes int32 [N, M] and path_len
    int32 [N] as :func:`verify_tree_greedy` and :func:`verify_tree_sampled`
    return them.  Returns the new lengths (``out.lens`` is not ``lens``).
    """
    if stream is not None:
        with _torch().cuda.stream(stream):
            return cache_commit(k_pages, v_pages, page_table, lens, path_nodes, path_len, out=out)
    if out is None:
        r = (_binding or _short()).commit(k_pages, v_pages, page_table, lens, path_nodes,
                                          path_len)
        if r is not None:
            _check(r[0], "psi_cache_commit")
            return CommitResult(r[1], r[2])
    key = ("commit", _sig(k_pages), _sig(v_pages), _sig(page_table), _sig(lens), _sig(path_nodes),
           _sig(path_len))
    plan = _plans.get(key) or _remember(key, _plan_commit(k_pages, v_pages, page_table, lens,
                                                          path_nodes, path_len))
    lay, N, M, max_pages = plan
    torch = _torch()
    others = dict(v_pages=v_pages, page_table=page_table, lens=lens, path_nodes=path_nodes,
                  path_len=path_len)
    if out is not None:
        _check_out("lens", out.lens, torch.int32, (N,))
        _check_out("status", out.status, torch.int32, (1,))
        others.update(out_lens=out.lens, status=out.status)
    dev = _on_device(k_pages, others)
    raw = _torch()._C._cuda_getCurrentRawStream(dev)
    if out is None:
        out = CommitResult(torch.empty_like(lens), _new_status(dev))
    st = psi_cache_commit(lay, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
                          max_pages, lens.data_ptr(), N, M, path_nodes.data_ptr(),
                          path_len.data_ptr(), out.lens.data_ptr(), out.status.data_ptr(), raw)
    _check(st, "psi_cache_commit")
    return out


def _plan_commit(k_pages, v_pages, page_table, lens, path_nodes, path_len):
    lay = _layout(k_pages, v_pages, layered=True)
    if page_table.dim() != 2 or path_nodes.dim() != 2:
        raise ValueError("page_table must be [N, max_pages], path_nodes [N, M]")
    N, M = path_nodes.shape
    _int32("page_table", page_table, (N, page_table.shape[1]))
    _int32("lens", lens, (N,))
    _int32("path_nodes", path_nodes, (N, M))
    _int32("path_len", path_len, (N,))
    return lay, N, M, page_table.shape[1]


_STATE = ("table", "counts", "refs", "free", "n_free")


def _check_state(name, s: PageState, N, max_pages, P):
    for field, shape in zip(_STATE, ((N, max_pages), (N,), (P,), (P,), (1,))):
        _int32(f"{name}.{field}", getattr(s, field), shape)


def _state_ptrs(s: PageState):
    return PageStatePtrs(s.table.data_ptr(), s.counts.data_ptr(), s.refs.data_ptr(),
                         s.free.data_ptr(), s.n_free.data_ptr())


def _state_sig(s: PageState):
    return tuple(_sig(getattr(s, f)) for f in _STATE)


def _named(name, s: PageState):
    return {f"{name}.{f}": getattr(s, f) for f in _STATE}


def _like(s: PageState, N, max_pages, P) -> PageState:
    """A state of the same sizes, in one allocation."""
    torch = _torch()
    table, refs, free, counts, n_free = torch.empty(
        N * max_pages + 2 * P + N + 1, dtype=torch.int32, device=s.table.device).split(
            (N * max_pages, P, P, N, 1))
    return PageState(table.view(N, max_pages), counts, refs, free, n_free)


def cache_resize(pages: PageState, lens, extra: int, page_size: int, stream=None,
                 out: ResizeResult | None = None) -> ResizeResult:
    """Fit each sequence's pages to lens[n] + extra positions
    (``psi_cache_resize``).  Returns a new state; with ``out.pages = pages``
    the state is changed in place."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return cache_resize(pages, lens, extra, page_size, out=out)
    if out is None:
        r = (_binding or _short()).resize(pages.table, pages.counts, pages.refs, pages.free,
                                          pages.n_free, lens, extra, page_size)
        if r is not None:
            _check(r[0], "psi_cache_resize")
            return ResizeResult(PageState(r[1], r[2], r[3], r[4], r[5]), r[6])
    key = ("resize", _state_sig(pages), _sig(lens))
    N, max_pages, P = _plans.get(key) or _remember(key, _plan_resize(pages, lens))
    others = dict(lens=lens, **_named("pages", pages))
    if out is not None:
        _check_state("out.pages", out.pages, N, max_pages, P)
        _check_out("status", out.status, _torch().int32, (1,))
        others.update(_named("out.pages", out.pages), status=out.status)
    dev = _on_device(pages.table, others)
    raw = _torch()._C._cuda_getCurrentRawStream(dev)
    if out is None:
        out = ResizeResult(_like(pages, N, max_pages, P), _new_status(dev))
    st = psi_cache_resize(N, max_pages, P, page_size, lens.data_ptr(), extra, _state_ptrs(pages),
                          _state_ptrs(out.pages), out.status.data_ptr(), raw)
    _check(st, "psi_cache_resize")
    return out


def _plan_resize(pages, lens):
    if pages.table.dim() != 2:
        raise ValueError("pages.table must be [N, max_pages]")
    N, max_pages = pages.table.shape
    P = pages.refs.numel()
    _check_state("pages", pages, N, max_pages, P)
    _int32("lens", lens, (N,))
    return N, max_pages, P


def cache_fork(k_pages, v_pages, pages: PageState, lens, src, dst, workspace=None, stream=None,
               out: ForkResult | None = None) -> ForkResult:
    """Row dst[k] becomes a copy of row src[k] (``psi_cache_fork``): whole
    pages are shared, the last, partly filled one is copied in every layer.

    k_pages, v_pages [L, P, S, H, D]; src, dst int32 [K].  Returns a new
    state and lengths; ``out`` may name the given ones (in place).
    """
    if stream is not None:
        with _torch().cuda.stream(stream):
            return cache_fork(k_pages, v_pages, pages, lens, src, dst, workspace, out=out)
    if out is None and workspace is None:
        r = (_binding or _short()).fork(k_pages, v_pages, pages.table, pages.counts, pages.refs,
                                        pages.free, pages.n_free, lens, src, dst)
        if r is not None:
            _check(r[0], "psi_cache_fork")
            return ForkResult(PageState(r[1], r[2], r[3], r[4], r[5]), r[6], r[7])
    key = ("fork", _sig(k_pages), _sig(v_pages), _state_sig(pages), _sig(lens), _sig(src),
           _sig(dst))
    plan = _plans.get(key) or _remember(key, _plan_fork(k_pages, v_pages, pages, lens, src, dst))
    lay, N, max_pages, P, K, ws_bytes = plan
    torch = _torch()
    others = dict(v_pages=v_pages, lens=lens, src=src, dst=dst, workspace=workspace,
                  **_named("pages", pages))
    if out is not None:
        _check_state("out.pages", out.pages, N, max_pages, P)
        _check_out("lens", out.lens, torch.int32, (N,))
        _check_out("status", out.status, torch.int32, (1,))
        others.update(_named("out.pages", out.pages), out_lens=out.lens, status=out.status)
    _check_workspace(workspace)
    dev = _on_device(k_pages, others)
    raw = _torch()._C._cuda_getCurrentRawStream(dev)
    if out is None:
        out = ForkResult(_like(pages, N, max_pages, P), torch.empty_like(lens),
                         _new_status(dev))
    if workspace is None or _nbytes(workspace) < ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=k_pages.device)
    st = psi_cache_fork(lay, k_pages.data_ptr(), v_pages.data_ptr(), N, max_pages,
                        lens.data_ptr(), out.lens.data_ptr(), _state_ptrs(pages),
                        _state_ptrs(out.pages), K, src.data_ptr(), dst.data_ptr(),
                        out.status.data_ptr(), workspace.data_ptr(), _nbytes(workspace), raw)
    _check(st, "psi_cache_fork")
    return out


def _plan_fork(k_pages, v_pages, pages, lens, src, dst):
    lay = _layout(k_pages, v_pages, layered=True)
    if pages.table.dim() != 2 or src.dim() != 1:
        raise ValueError("pages.table must be [N, max_pages], src and dst [K]")
    N, max_pages = pages.table.shape
    P, K = lay.num_pages, src.shape[0]
    _check_state("pages", pages, N, max_pages, P)
    _int32("lens", lens, (N,))
    _int32("src", src, (K,))
    _int32("dst", dst, (K,))
    return lay, N, max_pages, P, K, psi_cache_fork_workspace_bytes(K)
