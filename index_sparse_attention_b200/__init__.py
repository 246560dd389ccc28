"""Block-sparse and index-sparse softmax attention for NVIDIA B200 (sm_100a).

Thin Python binding over the C ABI of ``libsparse_attn.so`` (include/sparse_attn.h).
PyTorch supplies device memory and the current CUDA stream; every step of the
computation (tile-list conversion, forward, backward) runs in the library's CUDA
kernels.  The functions carry the names of the C entry points.
"""
import ctypes
import functools
import math

import torch

from . import _lib
from ._lib import SA_MODE_BLOCK, SA_MODE_DENSE, SA_MODE_INDEX, SA_TILE, SparseAttnError

__all__ = ["BlockSparse", "block_mask_to_block_sparse", "index_to_block_sparse",
           "sparse_attn_fwd", "sparse_attn_fwd_gather", "sparse_attn_bwd",
           "sparse_attn_bwd_workspace_size", "sparse_attn_bwd_noalloc", "topk_select",
           "cache_attn_fwd", "cache_attn_workspace_size", "sparse_attn_key_weights",
           "cache_evict",
           "sparse_attn_set_wait_limit_ns", "sparse_attn_set_forward_form",
           "sparse_attn_set_backward_form", "SparseAttnError", "SA_TILE"]


def _stream(device):
    index = device.index if device.index is not None else torch.cuda.current_device()
    return torch._C._cuda_getCurrentRawStream(index)


def _on_device(arg):
    """Runs the wrapped entry point with the device of its tensor argument `arg` (name)
    made current: the C ABI launches on the current device and refuses a stream of
    another device, so a tensor on cuda:1 must not be handed over while cuda:0 is
    current."""
    def deco(fn):
        import inspect
        pos = list(inspect.signature(fn).parameters).index(arg)

        @functools.wraps(fn)
        def wrapper(*args, **kw):
            t = kw.get(arg) if arg in kw else (args[pos] if pos < len(args) else None)
            if isinstance(t, torch.Tensor) and t.is_cuda:
                if type(t) is torch.Tensor and t.get_device() == torch._C._cuda_getDevice():
                    return fn(*args, **kw)
                with torch.cuda.device(t.device):
                    return fn(*args, **kw)
            return fn(*args, **kw)

        wrapper.device_arg = arg
        return wrapper
    return deco


def _addr(t):
    return None if t is None else t.data_ptr()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _require(cond, msg, exc=ValueError):
    if not cond:
        raise exc(msg)


def _check(name, t, dtype, shape=None, ndim=None, device=None, contiguous=True):
    """Argument checks done here because the C ABI sees pointers and sizes only: a
    tensor of the wrong shape would be read or written out of bounds by the kernels."""
    # a tensor that passes is let through before any message is put together: the messages
    # take longer than the checks (a call of ten tensors: 60 us of host time against 10)
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.is_cuda
            and (shape is None or t.shape == shape) and (ndim is None or t.dim() == ndim)
            and (not contiguous or t.is_contiguous())
            and (device is None or t.device == device)):
        return
    _require(isinstance(t, torch.Tensor), f"{name} must be a torch.Tensor", TypeError)
    _require(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}", TypeError)
    if ndim is not None:
        _require(t.dim() == ndim, f"{name} must have {ndim} dimensions, got {t.dim()}")
    if shape is not None:
        _require(tuple(t.shape) == tuple(shape),
                 f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    _require(t.is_cuda, f"{name} must be a CUDA tensor")
    if contiguous:
        _require(t.is_contiguous(), f"{name} must be contiguous")
    if device is not None:
        _require(t.device == device, f"{name} is on {t.device}, expected {device}")


def _fits(t, dtype, shape, index):
    """Whether a tensor passes _check with these on CUDA device `index` (the fast way through a
    call's checks: one expression per tensor, and _check to say what is wrong where one fails)."""
    return (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype
            and t.shape == shape and t.is_contiguous())


def _check_status(dev_status, device):
    if dev_status is not None:
        _check("dev_status", dev_status, torch.int32, device=device)
        _require(dev_status.numel() >= 1, "dev_status must hold at least one int32")


def _check_qkv(q, k, v):
    _check("q", q, torch.bfloat16, ndim=4)
    B, Sq, HQ, Dqk = q.shape
    _check("k", k, torch.bfloat16, ndim=4, device=q.device)
    _require(k.shape[0] == B and k.shape[3] == Dqk,
             f"k must be [B={B}, Sk, HK, Dqk={Dqk}], got {tuple(k.shape)}")
    _check("v", v, torch.bfloat16, ndim=4, device=q.device)
    _require(tuple(v.shape[:3]) == tuple(k.shape[:3]),
             f"v must be [B, Sk, HK, Dv] with k's first three sizes {tuple(k.shape[:3])}, "
             f"got {tuple(v.shape)}")


class BlockSparse:
    """Tile lists (and the partial-tile mask data) of one sparsity pattern.

    Holds the device tensors the C struct ``sa_block_sparse`` points to:
    cnt [B,HK,Tm,2], idx [B,HK,Tm,Tn], tcnt [B,HK,Tn,2], tidx [B,HK,Tn,Tm] (int32),
    and ``bitmap`` [B,HK,Sq,ceil(Sk/32)] (uint32 as int32) in index mode or ``mask``
    [B,HK,Mb,Nb] (uint8) in block mode.
    """

    def __init__(self, mode, B, HK, Sq, Sk, causal, device, bs=SA_TILE, mask=None, bitmap=None):
        Tm, Tn = -(-Sq // SA_TILE), -(-Sk // SA_TILE)
        i32 = dict(dtype=torch.int32, device=device)
        self.mode, self.B, self.HK, self.Sq, self.Sk = mode, B, HK, Sq, Sk
        self.causal, self.bs, self.Tm, self.Tn = bool(causal), bs, Tm, Tn
        self.cnt = torch.empty((B, HK, Tm, 2), **i32)
        self.idx = torch.empty((B, HK, Tm, Tn), **i32)
        self.tcnt = torch.empty((B, HK, Tn, 2), **i32)
        self.tidx = torch.empty((B, HK, Tn, Tm), **i32)
        self.mask = mask
        self.bitmap = bitmap
        Mb = Nb = 0
        if mask is not None:
            Mb, Nb = mask.shape[2], mask.shape[3]
        self.c = _lib.BlockSparseStruct(
            mode, int(bool(causal)), B, HK, Sq, Sk, bs, Mb, Nb,
            None if mask is None else mask.data_ptr(),
            None if bitmap is None else bitmap.data_ptr(),
            self.cnt.data_ptr(), self.idx.data_ptr(), self.tcnt.data_ptr(), self.tidx.data_ptr())

    def active_tiles(self):
        """Active (query tile, key tile) pairs per (b, KV head), summed: full + partial."""
        return int(self.cnt.sum().item())


@_on_device("mask")
def block_mask_to_block_sparse(mask, B, HK, Sq, Sk, bs=SA_TILE, causal=False, device=None):
    """Tile lists from a block mask uint8 [B,HK,Mb,Nb] at granularity bs (64 or 128).

    ``mask=None`` means every block (dense attention, optionally causal).
    """
    L = _lib.load()
    if mask is not None:
        _check("mask", mask, torch.uint8, ndim=4)
        _require(tuple(mask.shape[:2]) == (B, HK),
                 f"mask must be [B={B}, HK={HK}, Mb, Nb], got {tuple(mask.shape)}")
        device = mask.device
        mode = SA_MODE_BLOCK
    else:
        mode = SA_MODE_DENSE
        device = torch.device("cuda") if device is None else torch.device(device)
        _require(device.type == "cuda", "device must be a CUDA device")
    with torch.cuda.device(device):
        bsp = BlockSparse(mode, B, HK, Sq, Sk, causal, device, bs=bs, mask=mask)
        _lib.check("block_mask_to_block_sparse",
                   L.block_mask_to_block_sparse(ctypes.byref(bsp.c), _stream(device)))
    return bsp


@_on_device("idx")
def index_to_block_sparse(idx, Sk, causal=False, dev_status=None):
    """Tile lists and presence bitmap from top-k indices int32 [B,Sq,HK,topk] (-1 = pad)."""
    L = _lib.load()
    _check("idx", idx, torch.int32, ndim=4)
    _check_status(dev_status, idx.device)
    B, Sq, HK, topk = idx.shape
    W = -(-Sk // 32)
    bitmap = torch.empty((B, HK, Sq, W), dtype=torch.int32, device=idx.device)
    bsp = BlockSparse(SA_MODE_INDEX, B, HK, Sq, Sk, causal, idx.device, bitmap=bitmap)
    _lib.check("index_to_block_sparse",
               L.index_to_block_sparse(_ptr(idx), topk, ctypes.byref(bsp.c), _ptr(dev_status),
                                       _stream(idx.device)))
    return bsp


def _params(q, k, v, o, lse, sparse, scale, dout=None, dq=None, dk=None, dv=None,
            dev_status=None):
    _check_qkv(q, k, v)
    B, Sq, HQ, Dqk = q.shape
    _, Sk, HK, _ = k.shape
    Dv = v.shape[3]
    _require(isinstance(sparse, BlockSparse), "sparse must be a BlockSparse", TypeError)
    dev = q.device
    _check("o", o, torch.bfloat16, shape=(B, Sq, HQ, Dv), device=dev)
    _check("lse", lse, torch.float32, shape=(B, HQ, Sq), device=dev)
    for name, t, like in (("dout", dout, o), ("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None:
            _check(name, t, torch.bfloat16, shape=like.shape, device=dev)
    _check_status(dev_status, dev)
    return _params_struct(q, k, v, o, lse, sparse, scale, dout, dq, dk, dv, dev_status)


def _params_struct(q, k, v, o, lse, sparse, scale, dout=None, dq=None, dk=None, dv=None,
                   dev_status=None):
    B, Sq, HQ, Dqk = q.shape
    _, Sk, HK, _ = k.shape
    Dv = v.shape[3]
    return _lib.ParamsStruct(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
        None if dout is None else dout.data_ptr(), None if dq is None else dq.data_ptr(),
        None if dk is None else dk.data_ptr(), None if dv is None else dv.data_ptr(),
        B, HQ, HK, Dqk, Dv, Sq, Sk, float(scale), ctypes.pointer(sparse.c),
        None if dev_status is None else dev_status.data_ptr())


@_on_device("q")
def sparse_attn_fwd(q, k, v, sparse, softmax_scale=None, o=None, lse=None, dev_status=None):
    """O [B,Sq,HQ,Dv] (bf16) and LSE [B,HQ,Sq] (fp32) of sparse attention."""
    L = _lib.load()
    B, Sq, HQ, Dqk = q.shape
    Dv = v.shape[3]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(Dqk)
    if o is None:
        o = torch.empty((B, Sq, HQ, Dv), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, HQ, Sq), dtype=torch.float32, device=q.device)
    p = _params(q, k, v, o, lse, sparse, softmax_scale, dev_status=dev_status)
    _lib.check("sparse_attn_fwd", L.sparse_attn_fwd(ctypes.byref(p), _stream(q.device)))
    return o, lse


@_on_device("q")
def sparse_attn_fwd_gather(q, k, v, sparse, softmax_scale=None, o=None, lse=None,
                           dev_status=None):
    """The forward of sparse_attn_fwd by per-query gathers of the selected K/V rows
    (index mode only; HQ / HK <= 8; Dv <= 128): a comparison path, same O and LSE."""
    L = _lib.load()
    B, Sq, HQ, Dqk = q.shape
    Dv = v.shape[3]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(Dqk)
    if o is None:
        o = torch.empty((B, Sq, HQ, Dv), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, HQ, Sq), dtype=torch.float32, device=q.device)
    p = _params(q, k, v, o, lse, sparse, softmax_scale, dev_status=dev_status)
    _lib.check("sparse_attn_fwd_gather", L.sparse_attn_fwd_gather(ctypes.byref(p), _stream(q.device)))
    return o, lse


@_on_device("q")
def sparse_attn_bwd_workspace_size(q, k, v, sparse):
    """Bytes of device workspace sparse_attn_bwd needs for these shapes."""
    L = _lib.load()
    _check_qkv(q, k, v)
    o = q.new_empty((1,))
    p = _params_struct(q, k, v, o, o, sparse, 1.0)
    return int(L.sparse_attn_bwd_workspace_size(ctypes.byref(p)))


@_on_device("q")
def sparse_attn_bwd(q, k, v, o, lse, dout, sparse, softmax_scale=None, dq=None, dk=None,
                    dv=None, workspace=None, dev_status=None, deterministic=False):
    """dQ, dK, dV (bf16, layouts of q, k, v) of sparse attention; with
    ``deterministic`` dQ is accumulated in a fixed order (bitwise reproducible)."""
    L = _lib.load()
    Dqk = q.shape[3]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(Dqk)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _require(dout is not None, "dout is required")
    p = _params(q, k, v, o, lse, sparse, softmax_scale, dout, dq, dk, dv, dev_status)
    need = int(L.sparse_attn_bwd_workspace_size(ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check("workspace", workspace, torch.uint8, device=q.device)
    fn = L.sparse_attn_bwd_deterministic if deterministic else L.sparse_attn_bwd
    _lib.check("sparse_attn_bwd",
               fn(ctypes.byref(p), _ptr(workspace), workspace.numel(), _stream(q.device)))
    return dq, dk, dv


@_on_device("q")
def sparse_attn_bwd_noalloc(q, k, v, o, lse, dout, sparse, softmax_scale=None, dq=None, dk=None,
                            dv=None, dev_status=None):
    """dQ, dK, dV like sparse_attn_bwd, with the scratch taken from the library's fixed
    device array instead of a workspace (for callers that cannot allocate device memory;
    see include/sparse_attn.h).  Calls on one device share that array: do not overlap
    them on the GPU."""
    L = _lib.load()
    Dqk = q.shape[3]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(Dqk)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _require(dout is not None, "dout is required")
    p = _params(q, k, v, o, lse, sparse, softmax_scale, dout, dq, dk, dv, dev_status)
    _lib.check("sparse_attn_bwd_noalloc", L.sparse_attn_bwd_noalloc(ctypes.byref(p),
                                                                    _stream(q.device)))
    return dq, dk, dv


@_on_device("scores")
def topk_select(scores, k, starts=None, ends=None, with_values=False, out_idx=None, out_val=None,
                dev_status=None):
    """Column indices (int32 [rows, k]) of the k largest fp32 scores of each row's range
    [starts[r], ends[r]), largest first, ties to the smaller column, -1 past the number
    of valid columns; with ``with_values`` also the selected scores (fp32 [rows, k])."""
    L = _lib.load()
    _check("scores", scores, torch.float32, ndim=2, contiguous=False)
    _require(scores.stride(1) == 1, "scores rows must be contiguous (stride(1) == 1)")
    rows, cols = scores.shape
    dev = scores.device
    for name, t in (("starts", starts), ("ends", ends)):
        if t is not None:
            _check(name, t, torch.int32, shape=(rows,), device=dev)
    _check_status(dev_status, dev)
    if out_idx is None:
        out_idx = torch.empty((rows, k), dtype=torch.int32, device=dev)
    _check("out_idx", out_idx, torch.int32, shape=(rows, k), device=dev)
    if with_values and out_val is None:
        out_val = torch.empty((rows, k), dtype=torch.float32, device=dev)
    if out_val is not None:
        _check("out_val", out_val, torch.float32, shape=(rows, k), device=dev)
    _lib.check("topk_select",
               L.topk_select(_ptr(scores), rows, cols, scores.stride(0), _ptr(starts), _ptr(ends),
                             k, _ptr(out_idx), _ptr(out_val), _ptr(dev_status),
                             _stream(scores.device)))
    return (out_idx, out_val) if with_values else out_idx


def _check_cache_args(q, k_cache, v_cache, lens, k_prefix, v_prefix, weights, weights_out, o, lse,
                      dev_status):
    _check("q", q, torch.bfloat16, ndim=4)
    B, T, HQ, Dqk = q.shape
    _require(T == 1, f"q must hold one token per sequence [B, 1, HQ, Dqk], got {tuple(q.shape)}")
    dev = q.device
    _check("k_cache", k_cache, torch.bfloat16, ndim=4, device=dev)
    _check("v_cache", v_cache, torch.bfloat16, ndim=4, device=dev)
    S, HK, Dv = k_cache.shape[1], k_cache.shape[2], v_cache.shape[3]
    _require(k_cache.shape[0] == B and k_cache.shape[3] == Dqk,
             f"k_cache must be [B={B}, S, HK, Dqk={Dqk}], got {tuple(k_cache.shape)}")
    _require(tuple(v_cache.shape[:3]) == (B, S, HK),
             f"v_cache must be [B, S, HK, Dv] with k_cache's first three sizes {(B, S, HK)}, "
             f"got {tuple(v_cache.shape)}")
    _check("lens", lens, torch.int32, shape=(B,), device=dev)
    _require((k_prefix is None) == (v_prefix is None), "k_prefix and v_prefix go together")
    if k_prefix is not None:
        _check("k_prefix", k_prefix, torch.bfloat16, ndim=3, device=dev)
        P = k_prefix.shape[0]
        _check("k_prefix", k_prefix, torch.bfloat16, shape=(P, HK, Dqk), device=dev)
        _check("v_prefix", v_prefix, torch.bfloat16, shape=(P, HK, Dv), device=dev)
    for name, t in (("weights", weights), ("weights_out", weights_out)):
        if t is not None:
            _check(name, t, torch.float32, shape=(B, HK, S), device=dev)
    if o is not None:
        _check("o", o, torch.bfloat16, shape=(B, 1, HQ, Dv), device=dev)
    if lse is not None:
        _check("lse", lse, torch.float32, shape=(B, HQ, 1), device=dev)
    _check_status(dev_status, dev)


def _cache_args_fit(q, k_cache, v_cache, lens, k_prefix, v_prefix, weights, weights_out, o, lse,
                    dev_status):
    """Whether everything _check_cache_args looks at is as it should be."""
    if not (isinstance(q, torch.Tensor) and q.dim() == 4 and isinstance(v_cache, torch.Tensor)
            and v_cache.dim() == 4 and dev_status is None):
        return False
    bf16, dev = torch.bfloat16, q.get_device()
    if dev < 0:
        return False
    B, T, HQ, Dqk = q.shape
    _, S, HK, Dv = v_cache.shape
    if not (_fits(q, bf16, (B, 1, HQ, Dqk), dev) and _fits(k_cache, bf16, (B, S, HK, Dqk), dev)
            and _fits(v_cache, bf16, (B, S, HK, Dv), dev) and _fits(lens, torch.int32, (B,), dev)):
        return False
    if k_prefix is not None:
        if not (isinstance(k_prefix, torch.Tensor) and k_prefix.dim() == 3):
            return False
        P = k_prefix.shape[0]
        if not (_fits(k_prefix, bf16, (P, HK, Dqk), dev) and _fits(v_prefix, bf16, (P, HK, Dv), dev)):
            return False
    elif v_prefix is not None:
        return False
    return ((weights is None or _fits(weights, torch.float32, (B, HK, S), dev))
            and (weights_out is None or _fits(weights_out, torch.float32, (B, HK, S), dev))
            and (o is None or _fits(o, bf16, (B, 1, HQ, Dv), dev))
            and (lse is None or _fits(lse, torch.float32, (B, HQ, 1), dev)))


def _cache_params(q, k_cache, v_cache, lens, k_prefix, v_prefix, scale, weights, weights_out, o,
                  lse, dev_status):
    if not _cache_args_fit(q, k_cache, v_cache, lens, k_prefix, v_prefix, weights, weights_out, o,
                           lse, dev_status):
        _check_cache_args(q, k_cache, v_cache, lens, k_prefix, v_prefix, weights, weights_out, o,
                          lse, dev_status)
    B, _, HQ, Dqk = q.shape
    _, S, HK, Dv = v_cache.shape
    P = 0 if k_prefix is None else k_prefix.shape[0]
    if P == 0:
        k_prefix = v_prefix = None
    return _lib.CacheAttnStruct(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), lens.data_ptr(), _addr(k_prefix),
        _addr(v_prefix), _addr(o), _addr(lse), _addr(weights), _addr(weights_out), B, HQ, HK, Dqk,
        Dv, S, P, 1.0 / math.sqrt(Dqk) if scale is None else float(scale), _addr(dev_status))


@_on_device("q")
def cache_attn_workspace_size(q, k_cache, v_cache, lens, k_prefix=None, v_prefix=None,
                              with_weights=False):
    """Bytes of device workspace cache_attn_fwd needs for these shapes."""
    L = _lib.load()
    p = _cache_params(q, k_cache, v_cache, lens, k_prefix, v_prefix, None, None, None, None, None,
                      None)
    p.weights_out = 16 if with_weights else None  # (only whether it is given matters)
    return int(L.cache_attn_workspace_size(ctypes.byref(p)))


@_on_device("q")
def cache_attn_fwd(q, k_cache, v_cache, lens, k_prefix=None, v_prefix=None, softmax_scale=None,
                   weights=None, with_weights=False, weights_out=None, o=None, lse=None,
                   workspace=None, dev_status=None):
    """O [B,1,HQ,Dv] (bf16) and LSE [B,HQ,1] (fp32) of one new token per sequence over the
    prefix k_prefix / v_prefix [P,HK,D] that the batch shares (read once for every
    128 / (HQ / HK) sequences) and the first lens[b] (int32 [B]) keys of each sequence's
    cache k_cache / v_cache [B,S,HK,D].

    With ``with_weights`` (or a ``weights_out``) also weights_out [B,HK,S] (fp32):
    ``weights`` (zeros when omitted) plus the attention weight that each of the sequence's
    own keys gets from this token, summed over the group's query heads; ``weights_out`` may
    be ``weights`` itself, which adds in place."""
    L = _lib.load()
    p = _cache_params(q, k_cache, v_cache, lens, k_prefix, v_prefix, softmax_scale, weights,
                      weights_out, o, lse, dev_status)
    if weights is not None and not with_weights and weights_out is None:
        raise ValueError("weights needs with_weights or a weights_out")
    B, HQ, HK, Dv, S, dev = p.B, p.HQ, p.HK, p.Dv, p.S, q.device
    if o is None:
        # (empty_like, where the shape is the same, takes three quarters of empty's host time)
        o = (torch.empty_like(q) if Dv == p.Dqk
             else torch.empty(B, 1, HQ, Dv, dtype=torch.bfloat16, device=dev))
        p.o = o.data_ptr()
    if lse is None:
        lse = torch.empty(B, HQ, 1, dtype=torch.float32, device=dev)
        p.lse = lse.data_ptr()
    if with_weights and weights_out is None:
        weights_out = torch.empty(B, HK, S, dtype=torch.float32, device=dev)
        p.weights_out = weights_out.data_ptr()
    ref = ctypes.byref(p)
    if workspace is None:
        workspace = torch.empty(L.cache_attn_workspace_size(ref), dtype=torch.uint8, device=dev)
    else:
        _check("workspace", workspace, torch.uint8, device=dev)
    code = L.cache_attn_fwd(ref, workspace.data_ptr(), workspace.numel(), _stream(dev))
    if code:
        _require_same_or_apart(weights, weights_out)
        _lib.check("cache_attn_fwd", code)
    return (o, lse) if weights_out is None else (o, lse, weights_out)


@_on_device("q")
def sparse_attn_key_weights(q, k, lse, sparse, softmax_scale=None, weights=None, weights_out=None,
                            workspace=None, dev_status=None):
    """The attention weight each key received in a forward pass, fp32 [B,HK,Sk]: the sum
    over the group's query heads and all queries that see the key of exp(scale q.k - lse),
    with the lse [B,HQ,Sq] that sparse_attn_fwd returned for the same q, k, lists and scale.
    Added to ``weights`` when given; ``weights_out`` may be ``weights`` itself."""
    L = _lib.load()
    _check("q", q, torch.bfloat16, ndim=4)
    B, Sq, HQ, Dqk = q.shape
    dev = q.device
    _check("k", k, torch.bfloat16, ndim=4, device=dev)
    _require(k.shape[0] == B and k.shape[3] == Dqk,
             f"k must be [B={B}, Sk, HK, Dqk={Dqk}], got {tuple(k.shape)}")
    Sk, HK = k.shape[1], k.shape[2]
    _check("lse", lse, torch.float32, shape=(B, HQ, Sq), device=dev)
    _require(isinstance(sparse, BlockSparse), "sparse must be a BlockSparse", TypeError)
    for name, t in (("weights", weights), ("weights_out", weights_out)):
        if t is not None:
            _check(name, t, torch.float32, shape=(B, HK, Sk), device=dev)
    _check_status(dev_status, dev)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(Dqk)
    if weights_out is None:
        weights_out = torch.empty((B, HK, Sk), dtype=torch.float32, device=dev)
    Dv = {64: 64, 128: 128, 192: 128, 256: 256}.get(Dqk, Dqk)  # (not read; selects the pair)
    p = _lib.ParamsStruct(
        q.data_ptr(), k.data_ptr(), None, None, lse.data_ptr(), None, None, None, None, B, HQ, HK,
        Dqk, Dv, Sq, Sk, float(softmax_scale), ctypes.pointer(sparse.c),
        None if dev_status is None else dev_status.data_ptr())
    ref = ctypes.byref(p)
    if workspace is None:
        workspace = torch.empty(L.sparse_attn_key_weights_workspace_size(ref), dtype=torch.uint8,
                                device=dev)
    else:
        _check("workspace", workspace, torch.uint8, device=dev)
    code = L.sparse_attn_key_weights(ref, _addr(weights), weights_out.data_ptr(),
                                     workspace.data_ptr(), workspace.numel(), _stream(dev))
    if code:
        _require_same_or_apart(weights, weights_out)
        _lib.check("sparse_attn_key_weights", code)
    return weights_out


@_on_device("k_cache")
def cache_evict(k_cache, v_cache, weights, lens, budget, sinks=0, recent=0, k_out=None, v_out=None,
                weights_out=None, lens_out=None, keep=None, dev_status=None):
    """Cuts every sequence's cache to at most ``budget`` keys per KV head: its first
    ``sinks`` keys, its last ``recent`` keys and the heaviest of the keys between them by
    ``weights`` [B,HK,S] (ties to the smaller position), in their order.

    Returns k_out, v_out [B,S_out,HK,D] (rows behind the kept ones left as they were; S_out
    is the capacity of a given k_out, else that of k_cache), weights_out [B,HK,S_out] (zeros
    behind the kept keys), lens_out int32 [B] and keep int32 [B,HK,budget] (the kept
    positions, then -1).  The outputs must not overlap the inputs."""
    L = _lib.load()
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    _check("k_cache", k_cache, bf16, ndim=4)
    B, S, HK, Dqk = k_cache.shape
    dev = k_cache.device
    _check("v_cache", v_cache, bf16, ndim=4, device=dev)
    Dv = v_cache.shape[3]
    index = dev.index
    if not (_fits(v_cache, bf16, (B, S, HK, Dv), index) and _fits(weights, f32, (B, HK, S), index)
            and _fits(lens, i32, (B,), index)):
        _check("v_cache", v_cache, bf16, shape=(B, S, HK, Dv), device=dev)
        _check("weights", weights, f32, shape=(B, HK, S), device=dev)
        _check("lens", lens, i32, shape=(B,), device=dev)
    _check_status(dev_status, dev)
    budget, sinks, recent = int(budget), int(sinks), int(recent)
    S_out = S
    if k_out is not None:
        _check("k_out", k_out, bf16, ndim=4, device=dev)
        S_out = k_out.shape[1]
        _check("k_out", k_out, bf16, shape=(B, S_out, HK, Dqk), device=dev)
    elif v_out is not None:
        _check("v_out", v_out, bf16, ndim=4, device=dev)
        S_out = v_out.shape[1]
    if not 1 <= budget <= S_out:
        raise ValueError(f"budget must be in [1, {S_out}] (k_out's rows), got {budget}")
    if sinks < 0 or recent < 0 or sinks + recent > budget:
        raise ValueError("sinks and recent must be non-negative with a sum of at most "
                         f"budget={budget}, got {sinks} and {recent}")
    # (empty_like, where the shape is the same, takes three quarters of empty's host time)
    if k_out is None:
        k_out = (torch.empty_like(k_cache) if S_out == S
                 else torch.empty(B, S_out, HK, Dqk, dtype=bf16, device=dev))
    if v_out is None:
        v_out = (torch.empty_like(v_cache) if S_out == S
                 else torch.empty(B, S_out, HK, Dv, dtype=bf16, device=dev))
    else:
        _check("v_out", v_out, bf16, shape=(B, S_out, HK, Dv), device=dev)
    if weights_out is None:
        weights_out = (torch.empty_like(weights) if S_out == S
                       else torch.empty(B, HK, S_out, dtype=f32, device=dev))
    else:
        _check("weights_out", weights_out, f32, shape=(B, HK, S_out), device=dev)
    if lens_out is None:
        lens_out = torch.empty_like(lens)
    else:
        _check("lens_out", lens_out, i32, shape=(B,), device=dev)
    if keep is None:
        keep = torch.empty(B, HK, budget, dtype=i32, device=dev)
    else:
        _check("keep", keep, i32, shape=(B, HK, budget), device=dev)
    p = _lib.CacheEvictStruct(
        k_cache.data_ptr(), v_cache.data_ptr(), weights.data_ptr(), lens.data_ptr(),
        k_out.data_ptr(), v_out.data_ptr(), weights_out.data_ptr(), lens_out.data_ptr(),
        keep.data_ptr(), B, HK, Dqk, Dv, S, S_out, budget, sinks, recent, _addr(dev_status))
    code = L.cache_evict(ctypes.byref(p), _stream(dev))
    if code == _lib.SA_ERR_INVALID:  # (every other cause has been checked above)
        _require_apart((k_cache, v_cache, weights, lens),
                       (k_out, v_out, weights_out, lens_out, keep))
    if code:
        _lib.check("cache_evict", code)
    return k_out, v_out, weights_out, lens_out, keep


def _require_same_or_apart(weights, weights_out):
    """weights_out is weights itself or shares no memory with it."""
    if weights is not None and weights_out is not None:
        step = abs(weights_out.data_ptr() - weights.data_ptr())
        _require(step == 0 or step >= 4 * weights.numel(),
                 "weights_out overlaps weights without being the same tensor")


def _require_apart(inputs, outputs):
    """No output shares memory with an input or with another output."""
    def span(t):
        return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()

    taken = [span(t) for t in inputs]
    for t in outputs:
        lo, hi = span(t)
        _require(all(hi <= a or b <= lo for a, b in taken),
                 "an output overlaps an input or another output")
        taken.append((lo, hi))


def sparse_attn_set_wait_limit_ns(ns):
    """Test instrumentation: the limit (ns) of every pipeline wait of the attention
    kernels enqueued after this call (0 restores the default of 2 s).  A wait that runs
    out sets the timeout flag (SA_STATUS_TIMEOUT, value 2) in the device status word and
    its CTA leaves; see include/sparse_attn.h."""
    _lib.check("sparse_attn_set_wait_limit_ns", _lib.load().sparse_attn_set_wait_limit_ns(int(ns)))


_FWD_FORMS = {"auto": _lib.SA_FWD_FORM_AUTO, "one_head": _lib.SA_FWD_FORM_ONE_HEAD,
              "cta_pair": _lib.SA_FWD_FORM_CTA_PAIR, "two_heads": _lib.SA_FWD_FORM_TWO_HEADS,
              "two_tiles": _lib.SA_FWD_FORM_TWO_TILES}


def sparse_attn_set_forward_form(form):
    """How the forward maps query heads and tiles to CTAs: "auto" (the library's
    choice), "one_head" (one CTA per query tile and head), "cta_pair" (two heads of a GQA
    group on a 2-CTA cluster with cta_group::2 MMAs sharing each K/V tile), "two_heads"
    (two heads of a group in one CTA, one softmax warpgroup each) or "two_tiles" (two
    consecutive query tiles of one head in one CTA, walking the union of their lists).  A
    form that does not apply to a call falls back to one head per CTA.  Applies to the forward calls made after it,
    process-wide; see include/sparse_attn.h."""
    code = _FWD_FORMS.get(form, form) if isinstance(form, str) else int(form)
    if isinstance(code, str):
        raise ValueError(f"form must be one of {sorted(_FWD_FORMS)}, got {form!r}")
    _lib.check("sparse_attn_set_forward_form", _lib.load().sparse_attn_set_forward_form(code))


_BWD_FORMS = {"auto": _lib.SA_BWD_FORM_AUTO, "split": _lib.SA_BWD_FORM_SPLIT,
              "whole": _lib.SA_BWD_FORM_WHOLE}


def sparse_attn_set_backward_form(form):
    """How the backward covers a key tile at head dims (192,128): "auto" (the library's
    choice by grid size), "split" (two CTAs per key tile, each with part of the head dim,
    both recomputing S^T and dP^T) or "whole" (one CTA per key tile, single-buffered).
    The deterministic backward always splits.  Applies to the backward calls made after
    it, process-wide; see include/sparse_attn.h."""
    code = _BWD_FORMS.get(form, form) if isinstance(form, str) else int(form)
    if isinstance(code, str):
        raise ValueError(f"form must be one of {sorted(_BWD_FORMS)}, got {form!r}")
    _lib.check("sparse_attn_set_backward_form", _lib.load().sparse_attn_set_backward_form(code))
