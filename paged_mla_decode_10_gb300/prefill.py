"""Python surface of the calls around the decode: rotary positions, the append to
the paged cache, and the attention of ragged chunks of new tokens.

Each function checks its tensors, marshals pointers and sizes into one C call
(include/libmla.h) and enqueues it on the tensors' device: on ``stream``, or on
that device's current stream.

None of the calls records an autograd graph; the one whose gradient is offered, :func:`mla_rope`, refuses a tensor that
would need it.

The checks and the C structs depend on shapes, strides, types and devices alone
("layout"), so they are made once for each layout and kept; addresses are read at
every call.  On the host processor of a GB300 the checks take 30 to 60 us, longer
than most of the kernels.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import MlaAppendShape, MlaChunkRopeStrides, MlaChunkShape, MlaRopePlan, MlaRopeScaling, MlaRopeShape, check
from .api import HEAD_DIM, HEAD_DIM_V, _require

_ROPE_KINDS = {"linear": _lib.MLA_ROPE_LINEAR, "yarn": _lib.MLA_ROPE_YARN}
_DTYPES = {torch.bfloat16: _lib.MLA_DTYPE_BF16, torch.float16: _lib.MLA_DTYPE_F16, torch.float32: _lib.MLA_DTYPE_F32,
           torch.float8_e4m3fn: _lib.MLA_DTYPE_E4M3}
_E4M3 = (torch.float8_e4m3fn, torch.uint8)
_L = _lib.load()

# torch's own short ways to the current device's index and stream handle, where it has them
_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_stream_now = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


class _On:
    """Device `index` made current, and `stream` (None: its current one) with it, for the time of a call;
    tensors that the call allocates belong to that stream.  Gives the stream's handle."""

    def __init__(self, index, stream):
        self.scopes = [torch.cuda.device(index)] if index != _device_now() else []
        self.index, self.handle = index, None
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=index)
            _require(stream.device.index == index, "stream must be on the tensors' device")
            self.scopes.append(torch.cuda.stream(stream))
            self.handle = stream.cuda_stream

    def __enter__(self):
        for s in self.scopes:
            s.__enter__()
        return _stream_now(self.index) if self.handle is None else self.handle

    def __exit__(self, *exc):
        for s in reversed(self.scopes):
            s.__exit__(*exc)


def _call(run, layout, stream, *args):
    """run(layout, stream handle, *args) with the layout's device and the stream current."""
    if stream is None and layout.device == _device_now():
        return run(layout, _stream_now(layout.device), *args)
    with _On(layout.device, stream) as handle:
        return run(layout, handle, *args)


class _Layout:
    """What a call needs beside addresses: the C structs, the device, what to allocate there (torch.empty: new_empty
    takes twice as long)."""

    def __init__(self, device, **kw):
        self.__dict__.update(kw, device=device, where=torch.device("cuda", device))


class _Layouts(dict):
    """Layouts by everything they depend on; a program meets few, and the table is emptied rather than grown
    without end."""

    def add(self, key, layout):
        if len(self) >= 4096:
            self.clear()
        self[key] = layout
        return layout


def _sig(t):
    """A tensor's part of a layout's key."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _one_device(*tensors):
    tensors = [t for t in tensors if t is not None]
    _require(all(t.is_cuda for t in tensors), "all tensors must be CUDA tensors")
    _require(len({t.get_device() for t in tensors}) == 1, "all tensors must be on one device")
    return tensors[0].get_device()


def _last_contiguous(**tensors):
    for name, t in tensors.items():
        if t is not None:
            _require(t.shape[-1] <= 1 or t.stride(-1) == 1, f"{name}: the last dimension must be contiguous")


def _int32(**tensors):
    for name, t in tensors.items():
        if t is not None:
            _require(t.dtype == torch.int32, f"{name} must be int32")


def _strides(t: torch.Tensor, n: int):
    """Strides of the first n dimensions; a dimension of size one, whose stride no address depends
    on, is given a whole row's."""
    return [t.stride(i) if t.shape[i] != 1 else _row(t, i) for i in range(n)]


def _row(t, i):
    size = 1
    for k in range(i + 1, t.dim()):
        size = max(size, t.shape[k] * max(t.stride(k), 1))
    return size


# ---- rotary positions -------------------------------------------------------------------

def mla_rope_plan(rotary_dim: int, theta: float = 10000.0, interleaved: bool = True,
                  scaling: Optional[dict] = None) -> MlaRopePlan:
    """Frequencies of a rotary embedding over ``rotary_dim`` dims, for :func:`mla_rope` and
    :func:`mla_cache_append`.  ``interleaved``: pairs of neighbours, else of halves.  ``scaling``: None,
    ``{"kind": "linear", "factor": f}`` or ``{"kind": "yarn", "factor": f, "original_max_position": n,
    "beta_fast": 32, "beta_slow": 1, "mscale": 1, "mscale_all_dim": 0}`` (the last four optional)."""
    sc = None
    if scaling is not None:
        given = dict(scaling)
        kind = given.pop("kind", None)
        _require(kind in _ROPE_KINDS, f"scaling kind must be one of {sorted(_ROPE_KINDS)}")
        vals = {"factor": 1.0} if kind == "linear" else {
            "factor": 1.0, "original_max_position": 0.0, "beta_fast": 32.0, "beta_slow": 1.0, "mscale": 1.0,
            "mscale_all_dim": 0.0}
        _require(set(given) <= set(vals), f"unknown {kind} scaling entries {sorted(set(given) - set(vals))}")
        vals.update(given)
        sc = MlaRopeScaling(kind=_ROPE_KINDS[kind], **{k: float(v) for k, v in vals.items()})
    plan = MlaRopePlan()
    check(_L.mla_rope_init(plan._ref, int(rotary_dim), int(bool(interleaved)), float(theta),
                           ctypes.byref(sc) if sc is not None else None), "mla_rope_init")
    return plan


_rope_layouts = _Layouts()


def _rope_layout(key, x, positions, rotary_dim, rope_offset, out, out_dtype):
    _require(x.dim() in (3, 4), "x must be (tokens, heads, head_dim) or (batch, tokens, heads, head_dim)")
    _require(positions.shape == x.shape[:-2], "positions must have x's shape without heads and head_dim")
    _int32(positions=positions)
    if out is not None:
        _require(out.shape == x.shape, "out must have x's shape")
        _require(out_dtype is None or out.dtype == out_dtype, "out must be of out_dtype")
        out_dtype = out.dtype
    out_dtype = out_dtype or x.dtype
    _require(x.dtype in _DTYPES and out_dtype in _DTYPES, "x must be bf16, fp16 or fp32, out the same or float8_e4m3fn")
    _last_contiguous(x=x, out=out)
    device = _one_device(x, positions, out)
    x4 = x if x.dim() == 4 else x[None]
    sh = MlaRopeShape()
    sh.batch, sh.tokens, sh.heads, sh.head_dim = x4.shape
    sh.rope_offset = sh.head_dim - rotary_dim if rope_offset is None else int(rope_offset)
    sh.dtype, sh.out_dtype = _DTYPES[x.dtype], _DTYPES[out_dtype]
    sh.x_stride[:] = x4.stride()[:3]
    if out is not None:
        sh.out_stride[:] = (out if out.dim() == 4 else out[None]).stride()[:3]
    else:   # allocated contiguous
        row = sh.heads * sh.head_dim
        sh.out_stride[:] = (sh.tokens * row, row, sh.head_dim)
    return _rope_layouts.add(key, _Layout(shape=sh, ref=ctypes.byref(sh), device=device, out_dtype=out_dtype,
                                          copy_positions=not positions.is_contiguous()))


def _rope_run(lay, stream, x, positions, plan, inverse, out, out_scale):
    if out is None:
        out = torch.empty(x.shape, dtype=lay.out_dtype, device=lay.where)
    if lay.copy_positions:
        positions = positions.contiguous()
    rc = _L.mla_rope(plan._ref, lay.ref, x.data_ptr(), positions.data_ptr(), inverse, out.data_ptr(), out_scale, stream)
    if rc:
        check(rc, "mla_rope")
    return out


def mla_rope(x: torch.Tensor, positions: torch.Tensor, plan: MlaRopePlan, rope_offset: Optional[int] = None,
             inverse: bool = False, out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
             out_scale: float = 1.0, stream=None) -> torch.Tensor:
    """x (..., heads, head_dim) bf16, fp16 or fp32 with ``plan.rotary_dim`` dims of every head rotated by
    positions (int32, x's shape without its last two dimensions).  The rotated dims start at
    ``rope_offset`` (default: they are the last ones); the others are copied.  ``inverse`` turns the other way, with the
    same factor (it rotates back where the plan's factor is 1): the gradient of a call is the inverse call on the
    output's gradient.  The call records no graph, so that a tensor that requires one is refused while gradients are
    enabled; make both calls in a ``torch.autograd.Function``.  ``out``: where to write, ``x`` itself to rotate in place;
    ``out_dtype`` float8_e4m3fn rounds ``out_scale`` times the values to e4m3.  One or two leading dimensions."""
    if (x.requires_grad or (out is not None and out.requires_grad)) and torch.is_grad_enabled():
        raise ValueError("mla_rope records no graph: call it under torch.no_grad() or in a torch.autograd.Function, "
                         "with inverse=True for the gradient")
    key = (_sig(x), _sig(positions), _sig(out), plan.rotary_dim, rope_offset, out_dtype)
    lay = _rope_layouts.get(key) or _rope_layout(key, x, positions, plan.rotary_dim, rope_offset, out, out_dtype)
    return _call(_rope_run, lay, stream, x, positions, plan, bool(inverse), out, float(out_scale))


# ---- append to the paged cache ----------------------------------------------------------

_append_layouts = _Layouts()


def _append_layout(key, latent, k_rope, k_cache, block_table, cu_seqlens_q, cache_seqlens, krope_cache, positions):
    _require(latent.dim() == 3 and k_rope.dim() == 3 and k_cache.dim() == 4, "latent, k_rope (T, h_k, dims), k_cache 4-D")
    T, h_k = latent.shape[:2]
    _require(tuple(k_rope.shape[:2]) == (T, h_k) and latent.shape[2] == HEAD_DIM_V and
             k_rope.shape[2] == HEAD_DIM - HEAD_DIM_V, "latent must be (T, h_k, 512), k_rope (T, h_k, 64)")
    _require(latent.dtype == torch.bfloat16 and k_rope.dtype == torch.bfloat16, "latent and k_rope must be bf16")
    _require(k_cache.dtype in (torch.bfloat16,) + _E4M3, "k_cache must be bf16 or e4m3")
    _require(k_cache.shape[2] == h_k and k_cache.shape[3] == (HEAD_DIM_V if krope_cache is not None else HEAD_DIM),
             "k_cache must be (num_blocks, 64, h_k, 576), or 512 dims beside krope_cache")
    if krope_cache is not None:
        _require(krope_cache.dtype == k_cache.dtype and tuple(krope_cache.shape) ==
                 (*k_cache.shape[:3], HEAD_DIM - HEAD_DIM_V), "krope_cache must be (num_blocks, 64, h_k, 64) of k_cache's type")
    _require(block_table.dim() == 2 and cache_seqlens.dim() == 1 and block_table.shape[0] == cache_seqlens.shape[0],
             "block_table (batch, blocks) and cache_seqlens (batch,) must agree")
    B = cache_seqlens.shape[0]
    _require(cu_seqlens_q is None or tuple(cu_seqlens_q.shape) == (B + 1,), "cu_seqlens_q must be (batch + 1,)")
    _require(positions is None or tuple(positions.shape) == (T,), "positions must be (T,)")
    _int32(block_table=block_table, cu_seqlens_q=cu_seqlens_q, cache_seqlens=cache_seqlens, positions=positions)
    _last_contiguous(latent=latent, k_rope=k_rope, k_cache=k_cache, krope_cache=krope_cache, block_table=block_table)
    device = _one_device(latent, k_rope, k_cache, krope_cache, block_table, cu_seqlens_q, cache_seqlens, positions)
    sh = MlaAppendShape()
    sh.batch, sh.total_tokens, sh.h_k = B, T, h_k
    sh.page_block_size, sh.num_blocks, sh.max_blocks_per_seq = k_cache.shape[1], k_cache.shape[0], block_table.shape[1]
    sh.kv_dtype = _lib.MLA_DTYPE_BF16 if k_cache.dtype == torch.bfloat16 else _lib.MLA_DTYPE_E4M3
    sh.latent_stride[:], sh.k_rope_stride[:] = _strides(latent, 2), _strides(k_rope, 2)
    sh.k_stride[:] = _strides(k_cache, 3)
    if krope_cache is not None:
        sh.krope_stride[:] = _strides(krope_cache, 3)
    sh.bt_stride = block_table.stride(0) if block_table.shape[0] > 1 else block_table.shape[1]
    flat = all(t is None or t.is_contiguous() for t in (cu_seqlens_q, cache_seqlens, positions))
    return _append_layouts.add(key, _Layout(shape=sh, ref=ctypes.byref(sh), device=device, flat=flat))


def _append_run(lay, stream, latent, k_rope, plan, k_cache, block_table, cu_seqlens_q, cache_seqlens, krope_cache, positions,
                kv_scale):
    if not lay.flat:
        cu_seqlens_q, cache_seqlens, positions = (t if t is None else t.contiguous()
                                                  for t in (cu_seqlens_q, cache_seqlens, positions))
    rc = _L.mla_cache_append(lay.ref, plan._ref, latent.data_ptr(), k_rope.data_ptr(), block_table.data_ptr(),
                             _ptr(cu_seqlens_q), cache_seqlens.data_ptr(), _ptr(positions), k_cache.data_ptr(),
                             _ptr(krope_cache), kv_scale, stream)
    if rc:
        check(rc, "mla_cache_append")


def mla_cache_append(latent: torch.Tensor, k_rope: torch.Tensor, plan: MlaRopePlan, k_cache: torch.Tensor,
                     block_table: torch.Tensor, cu_seqlens_q: Optional[torch.Tensor], cache_seqlens: torch.Tensor,
                     krope_cache: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                     kv_scale: float = 1.0, stream=None) -> None:
    """Writes the cache rows of new tokens: latent (T, h_k, 512) as it is, k_rope (T, h_k, 64) rotated
    (both bf16), into k_cache (num_blocks, 64, h_k, 576), or, with krope_cache (num_blocks, 64, h_k, 64), into
    k_cache (num_blocks, 64, h_k, 512) and krope_cache.  Caches are bf16 or e4m3 (float8_e4m3fn or uint8,
    holding kv_scale times the values).  Sequence b's tokens cu_seqlens_q[b] .. cu_seqlens_q[b + 1] (None: the
    same number for each) are the last of its cache_seqlens[b] positions; ``positions`` (T) int32 overrides the
    position that the key is rotated by."""
    key = (_sig(latent), _sig(k_rope), _sig(k_cache), _sig(block_table), _sig(cu_seqlens_q), _sig(cache_seqlens),
           _sig(krope_cache), _sig(positions))
    lay = _append_layouts.get(key) or _append_layout(key, latent, k_rope, k_cache, block_table, cu_seqlens_q, cache_seqlens,
                                                     krope_cache, positions)
    _call(_append_run, lay, stream, latent, k_rope, plan, k_cache, block_table, cu_seqlens_q, cache_seqlens, krope_cache,
          positions, float(kv_scale))


# ---- attention of chunks ------------------------------------------------------------------

def mla_chunk_get_num_parts(device=None) -> int:
    index = None if device is None else torch.device(device).index
    out = ctypes.c_int(0)
    check(_L.mla_chunk_get_num_parts(torch.cuda.current_device() if index is None else index, ctypes.byref(out)),
          "mla_chunk_get_num_parts")
    return out.value


def mla_chunk_get_metadata(cu_seqlens_q: torch.Tensor, cache_seqlens: torch.Tensor, total_q: int, num_heads_q: int,
                           num_heads_k: int, causal: bool = True, num_parts: Optional[int] = None,
                           stream=None) -> torch.Tensor:
    """Schedule of :func:`mla_chunk_fwd` for these lengths: chunk_metadata (num_parts, 8) int32.  One call per step
    serves every layer."""
    _require(cache_seqlens.dim() == 1 and tuple(cu_seqlens_q.shape) == (cache_seqlens.shape[0] + 1,),
             "cu_seqlens_q must be (batch + 1,), cache_seqlens (batch,)")
    _int32(cu_seqlens_q=cu_seqlens_q, cache_seqlens=cache_seqlens)
    device = _one_device(cu_seqlens_q, cache_seqlens)
    with _On(device, stream) as handle:
        cu_seqlens_q, cache_seqlens = cu_seqlens_q.contiguous(), cache_seqlens.contiguous()
        if num_parts is None:
            num_parts = mla_chunk_get_num_parts(cache_seqlens.device)
        md = torch.empty((num_parts, _lib.MLA_METADATA_SIZE), dtype=torch.int32, device=cache_seqlens.device)
        check(_L.mla_chunk_get_metadata(_ptr(cu_seqlens_q), _ptr(cache_seqlens), cache_seqlens.shape[0], int(total_q),
                                        int(num_heads_q), int(num_heads_k), int(bool(causal)), int(num_parts), _ptr(md),
                                        handle), "mla_chunk_get_metadata")
    return md


def mla_chunk_workspace_size(shape: MlaChunkShape) -> int:
    n = ctypes.c_size_t(0)
    check(_L.mla_chunk_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "mla_chunk_workspace_size")
    return n.value


_chunk_layouts = _Layouts()


def _chunk_layout(key, name, q, q_rope, k_cache, krope, block_table, cu_seqlens_q, cache_seqlens, head_dim_v,
                  chunk_metadata, out, softmax_lse, workspace):
    if name == "mla_chunk_fwd":
        _require(q.dtype == torch.bfloat16 and k_cache.dtype == torch.bfloat16, "q and k_cache must be bf16")
        _require(q.shape[-1] == k_cache.shape[-1], "q and k_cache must have the same number of dims")
    elif name == "mla_chunk_fwd_fp8":
        _require(q.dtype in _E4M3 and k_cache.dtype in _E4M3, "q and k_cache must be float8_e4m3fn or uint8")
        _require(q.shape[-1] == k_cache.shape[-1], "q and k_cache must have the same number of dims")
    else:
        _require(all(t.dtype == torch.bfloat16 for t in (q, q_rope, k_cache, krope)), "q_nope, q_rope, ctkv, krope must be bf16")
        _require(q.dim() == 3 and q_rope.dim() == 3 and k_cache.dim() == 4 and krope.dim() == 4 and
                 q.shape[:2] == q_rope.shape[:2] and k_cache.shape[:3] == krope.shape[:3],
                 "nope and rope parts must agree in their leading dimensions")
        _require(q.shape[-1] == HEAD_DIM_V and k_cache.shape[-1] == HEAD_DIM_V and q_rope.shape[-1] == HEAD_DIM - HEAD_DIM_V and
                 krope.shape[-1] == HEAD_DIM - HEAD_DIM_V, "last dimensions must be 512 (nope) and 64 (rope)")
    _require(q.dim() == 3 and k_cache.dim() == 4, "q must be (tokens, heads, dims), k_cache (num_blocks, 64, h_k, dims)")
    _require(cache_seqlens.dim() == 1 and block_table.dim() == 2 and block_table.shape[0] == cache_seqlens.shape[0] and
             tuple(cu_seqlens_q.shape) == (cache_seqlens.shape[0] + 1,),
             "cu_seqlens_q (batch + 1,), cache_seqlens (batch,) and block_table (batch, blocks) must agree")
    _require(chunk_metadata.dim() == 2 and chunk_metadata.shape[1] == _lib.MLA_METADATA_SIZE and
             chunk_metadata.is_contiguous(), "chunk_metadata must be (num_parts, 8), contiguous")
    _int32(block_table=block_table, cu_seqlens_q=cu_seqlens_q, cache_seqlens=cache_seqlens, chunk_metadata=chunk_metadata)
    _last_contiguous(q=q, q_rope=q_rope, k_cache=k_cache, krope=krope, block_table=block_table, out=out)
    T, h_q, dims = q.shape
    if out is not None:
        _require(out.dtype == torch.bfloat16 and tuple(out.shape) == (T, h_q, head_dim_v),
                 "out must be (tokens, heads, head_dim_v) bf16")
    if softmax_lse is not None:
        _require(softmax_lse.dtype == torch.float32 and tuple(softmax_lse.shape) == (T, h_q) and softmax_lse.is_contiguous(),
                 "softmax_lse must be (tokens, heads) fp32, contiguous")
    if workspace is not None:
        _require(workspace.is_contiguous(), "workspace must be contiguous")
    device = _one_device(q, q_rope, k_cache, krope, block_table, cu_seqlens_q, cache_seqlens, chunk_metadata, out, softmax_lse,
                         workspace)
    sh = MlaChunkShape()
    sh.batch, sh.total_q, sh.h_q, sh.h_k = cache_seqlens.shape[0], T, h_q, k_cache.shape[2]
    sh.head_dim = dims if q_rope is None else HEAD_DIM
    sh.head_dim_v = int(head_dim_v)
    sh.page_block_size, sh.num_blocks, sh.max_blocks_per_seq = k_cache.shape[1], k_cache.shape[0], block_table.shape[1]
    sh.num_parts = chunk_metadata.shape[0]
    sh.q_stride[:], sh.k_stride[:] = _strides(q, 2), _strides(k_cache, 3)
    sh.out_stride[:] = (h_q * head_dim_v, head_dim_v) if out is None else _strides(out, 2)
    sh.bt_stride = block_table.stride(0) if block_table.shape[0] > 1 else block_table.shape[1]
    refs = [ctypes.byref(sh)]
    if q_rope is not None:
        rs = MlaChunkRopeStrides()
        rs.q_rope_stride[:], rs.krope_stride[:] = _strides(q_rope, 2), _strides(krope, 3)
        refs.append(ctypes.byref(rs))
    return _chunk_layouts.add(key, _Layout(
        fn=getattr(_L, name), name=name, refs=refs, device=device, out_shape=(T, h_q, head_dim_v), lse_shape=(T, h_q),
        flat=cu_seqlens_q.is_contiguous() and cache_seqlens.is_contiguous(), workspace_bytes=mla_chunk_workspace_size(sh),
        given_bytes=0 if workspace is None else workspace.numel() * workspace.element_size()))


def _chunk_run(lay, stream, q, q_rope, k_cache, krope, block_table, cu_seqlens_q, cache_seqlens, chunk_metadata, scales, causal,
               out, softmax_lse, workspace):
    if not lay.flat:
        cu_seqlens_q, cache_seqlens = cu_seqlens_q.contiguous(), cache_seqlens.contiguous()
    if out is None:
        out = torch.empty(lay.out_shape, dtype=torch.bfloat16, device=lay.where)
    if softmax_lse is None:
        softmax_lse = torch.empty(lay.lse_shape, dtype=torch.float32, device=lay.where)
    if workspace is None:
        # of this call alone: calls on other streams and other captured graphs get their own
        workspace, nbytes = torch.empty(lay.workspace_bytes, dtype=torch.uint8, device=lay.where), lay.workspace_bytes
    else:
        nbytes = lay.given_bytes
    data = (q.data_ptr(), k_cache.data_ptr()) if q_rope is None else \
        (q.data_ptr(), q_rope.data_ptr(), k_cache.data_ptr(), krope.data_ptr())
    rc = lay.fn(*lay.refs, *data, block_table.data_ptr(), cu_seqlens_q.data_ptr(), cache_seqlens.data_ptr(),
                chunk_metadata.data_ptr(), *scales, causal, out.data_ptr(), softmax_lse.data_ptr(), workspace.data_ptr(),
                nbytes, stream)
    if rc:
        check(rc, lay.name)
    return out, softmax_lse


def _chunk_call(name, q, q_rope, k_cache, krope, block_table, cu_seqlens_q, cache_seqlens, head_dim_v, chunk_metadata,
                scales, causal, out, softmax_lse, workspace, stream):
    key = (name, head_dim_v, _sig(q), _sig(k_cache), _sig(block_table), _sig(cu_seqlens_q), _sig(cache_seqlens),
           _sig(chunk_metadata), _sig(q_rope), _sig(krope), _sig(out), _sig(softmax_lse), _sig(workspace))
    lay = _chunk_layouts.get(key) or _chunk_layout(key, name, q, q_rope, k_cache, krope, block_table, cu_seqlens_q, cache_seqlens,
                                                   head_dim_v, chunk_metadata, out, softmax_lse, workspace)
    return _call(_chunk_run, lay, stream, q, q_rope, k_cache, krope, block_table, cu_seqlens_q, cache_seqlens, chunk_metadata,
                 scales, bool(causal), out, softmax_lse, workspace)


def mla_chunk_fwd(q, k_cache, block_table, cu_seqlens_q, cache_seqlens, head_dim_v, chunk_metadata, softmax_scale=None,
                  causal=True, out=None, softmax_lse=None, workspace=None, stream=None):
    """Attention of a ragged batch of new tokens, q (total_q, h_q, 576) bf16, over the paged cache that
    already holds their keys.  Returns (out (total_q, h_q, head_dim_v) bf16, softmax_lse (total_q, h_q) fp32);
    rows of tokens outside cu_seqlens_q are not written."""
    scale = HEAD_DIM ** (-0.5) if softmax_scale is None else float(softmax_scale)
    return _chunk_call("mla_chunk_fwd", q, None, k_cache, None, block_table, cu_seqlens_q, cache_seqlens, head_dim_v,
                       chunk_metadata, (scale,), causal, out, softmax_lse, workspace, stream)


def mla_chunk_fwd_split(q_nope, q_rope, ctkv, krope, block_table, cu_seqlens_q, cache_seqlens, head_dim_v, chunk_metadata,
                        softmax_scale=None, causal=True, out=None, softmax_lse=None, workspace=None, stream=None):
    """mla_chunk_fwd on split inputs: q_nope (total_q, h_q, 512), q_rope (total_q, h_q, 64), ctkv (num_blocks, 64, h_k, 512),
    krope (num_blocks, 64, h_k, 64), all bf16."""
    scale = HEAD_DIM ** (-0.5) if softmax_scale is None else float(softmax_scale)
    return _chunk_call("mla_chunk_fwd_split", q_nope, q_rope, ctkv, krope, block_table, cu_seqlens_q, cache_seqlens,
                       head_dim_v, chunk_metadata, (scale,), causal, out, softmax_lse, workspace, stream)


def mla_chunk_fwd_fp8(q, k_cache, block_table, cu_seqlens_q, cache_seqlens, head_dim_v, chunk_metadata, bmm1_scale,
                      bmm2_scale=1.0, causal=True, out=None, softmax_lse=None, workspace=None, stream=None):
    """mla_chunk_fwd over an e4m3 query and cache (float8_e4m3fn or uint8), with the product scales of
    mla_decode_fwd_fp8.  Returns (out bf16, softmax_lse fp32)."""
    return _chunk_call("mla_chunk_fwd_fp8", q, None, k_cache, None, block_table, cu_seqlens_q, cache_seqlens, head_dim_v,
                       chunk_metadata, (float(bmm1_scale), float(bmm2_scale)), causal, out, softmax_lse, workspace, stream)
