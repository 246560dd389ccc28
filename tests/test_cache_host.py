"""Refusals of the cache operators that need no GPU: the C ABI's host checks (fake pointers, never
dereferenced) and the binding's argument checks; and the references' own consistency."""
import ctypes

import numpy as np
import pytest
import torch

import cache_ref as R
import index_sparse_attention_b200 as sa
from index_sparse_attention_b200 import _lib
from index_sparse_attention_b200.build import build

BAD, UNSUP = _lib.SA_ERR_INVALID, _lib.SA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def attn(**kw):
    p = _lib.CacheAttnStruct(0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 0x7000, 0x8000, None,
                             None, 2, 8, 2, 128, 128, 100, 50, 0.1, None)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def call_attn(lib, p, ws=0x100000, n=1 << 40):
    return lib.cache_attn_fwd(ctypes.byref(p), ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), BAD), (dict(HQ=0), BAD), (dict(HK=0), BAD), (dict(S=0), BAD), (dict(P=-1), BAD),
    (dict(HQ=7), BAD), (dict(q=None), BAD), (dict(k_cache=None), BAD), (dict(v_cache=None), BAD),
    (dict(lens=None), BAD), (dict(o=None), BAD), (dict(lse=None), BAD), (dict(k_prefix=None), BAD),
    (dict(v_prefix=None), BAD), (dict(P=0), BAD), (dict(weights=0x9000), BAD),
    (dict(softmax_scale=0.0), BAD), (dict(softmax_scale=float("nan")), BAD),
    (dict(softmax_scale=-1.0), BAD), (dict(Dqk=96), UNSUP), (dict(Dv=64), UNSUP),
    (dict(HQ=258, HK=2), UNSUP), (dict(S=1 << 40), UNSUP), (dict(P=1 << 40), UNSUP),
    (dict(B=65536), UNSUP), (dict(B=65535, HQ=65535, HK=65535), UNSUP),
    (dict(q=0x1008), _lib.SA_ERR_ALIGN), (dict(k_prefix=0x5008), _lib.SA_ERR_ALIGN),
    (dict(o=0x7004), _lib.SA_ERR_ALIGN), (dict(lens=0x4002), _lib.SA_ERR_ALIGN),
    (dict(lse=0x8001), _lib.SA_ERR_ALIGN), (dict(weights_out=0x9002), _lib.SA_ERR_ALIGN),
], ids=str)
def test_attention_refusals(lib, kw, code):
    assert call_attn(lib, attn(**kw)) == code
    assert lib.cache_attn_fwd(None, None, 0, None) == BAD


def test_attention_workspace_is_checked(lib):
    p = attn()
    need = lib.cache_attn_workspace_size(ctypes.byref(p))
    assert need > 0
    assert call_attn(lib, p, None, 0) == _lib.SA_ERR_WORKSPACE
    assert call_attn(lib, p, 0x100000, need - 1) == _lib.SA_ERR_WORKSPACE
    assert call_attn(lib, p, 0x100008, need) == _lib.SA_ERR_WORKSPACE
    more = lib.cache_attn_workspace_size(ctypes.byref(attn(weights_out=0x9000)))
    assert more == need + 2 * 8 * 128 * 4  # the scores [B][HQ][ceil(S / 128) * 128]
    assert lib.cache_attn_workspace_size(ctypes.byref(attn(B=0))) == 0
    # sizes whose products pass 64 bits are refused before any of them is taken
    huge = attn(B=65535, HQ=65535, HK=65535, S=0x7FFFFF00, weights_out=0x9000)
    assert lib.cache_attn_workspace_size(ctypes.byref(huge)) == 0
    assert lib.cache_attn_fwd(ctypes.byref(huge), 0x10000, 1 << 40, None) == UNSUP


def test_key_weights_refusals(lib):
    s = _lib.BlockSparseStruct(_lib.SA_MODE_DENSE, 0, 1, 2, 256, 256, 128, 0, 0, None, None,
                               0x1000, 0x1000, 0x1000, 0x1000)

    def call(out=0x9000, **kw):
        p = _lib.ParamsStruct(0x1000, 0x1000, None, None, 0x1000, None, None, None, None, 1, 4, 2,
                              128, 128, 256, 256, 0.125, ctypes.pointer(s), None)
        for k, v in kw.items():
            setattr(p, k, v)
        return lib.sparse_attn_key_weights(ctypes.byref(p), None, out, None, 0, None)

    assert call(out=None) == BAD
    for kw in (dict(q=None), dict(k=None), dict(lse=None), dict(HQ=5), dict(Sq=300), dict(B=0),
               dict(softmax_scale=0.0)):
        assert call(**kw) == BAD, kw
    assert call(Dqk=96) == UNSUP
    assert call(q=0x1008) == _lib.SA_ERR_ALIGN
    assert call(lse=0x1002) == _lib.SA_ERR_ALIGN and call(out=0x9001) == _lib.SA_ERR_ALIGN
    assert lib.sparse_attn_key_weights(None, None, 0x9000, None, 0, None) == BAD
    p = _lib.ParamsStruct(0x1000, 0x1000, None, None, 0x1000, None, None, None, None, 1, 4, 2, 128,
                          128, 256, 256, 0.125, ctypes.pointer(s), None)
    need = lib.sparse_attn_key_weights_workspace_size(ctypes.byref(p))
    assert need > 0
    for ws, n in ((None, 0), (0x2000, need - 1), (0x2008, need)):
        assert lib.sparse_attn_key_weights(ctypes.byref(p), None, 0x9000, ws, n,
                                           None) == _lib.SA_ERR_WORKSPACE
    p.B = 0
    assert lib.sparse_attn_key_weights_workspace_size(ctypes.byref(p)) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), BAD), (dict(HK=0), BAD), (dict(S=0), BAD), (dict(budget=0), BAD),
    (dict(sinks=-1), BAD), (dict(recent=-1), BAD), (dict(sinks=30, recent=21), BAD),
    (dict(sinks=2147483647, recent=2147483647), BAD), (dict(budget=101), BAD),
    (dict(k_cache=None), BAD), (dict(weights=None), BAD), (dict(lens=None), BAD),
    (dict(k_out=None), BAD), (dict(keep=None), BAD), (dict(lens_out=None), BAD),
    (dict(k_out=0x100000), BAD), (dict(v_out=0x200000), BAD), (dict(weights_out=0x300000), BAD),
    (dict(lens_out=0x400000), BAD), (dict(k_out=0x100000 + 102384), BAD),
    (dict(v_out=0x500000 - 102384), BAD), (dict(keep=0x700010), BAD), (dict(Dqk=80), UNSUP), (dict(B=65536), UNSUP),
    (dict(S=1 << 40), UNSUP), (dict(k_cache=0x100008), _lib.SA_ERR_ALIGN),
    (dict(weights=0x300002), _lib.SA_ERR_ALIGN), (dict(keep=0x900001), _lib.SA_ERR_ALIGN),
], ids=str)
def test_eviction_refusals(lib, kw, code):
    p = _lib.CacheEvictStruct(0x100000, 0x200000, 0x300000, 0x400000, 0x500000, 0x600000, 0x700000,
                              0x800000, 0x900000, 2, 2, 128, 128, 100, 100, 50, 4, 8, None)
    for k, v in kw.items():
        setattr(p, k, v)
    assert lib.cache_evict(ctypes.byref(p), None) == code
    assert lib.cache_evict(None, None) == BAD


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_refuses_cpu_tensors_and_wrong_types(lib):
    lens = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        sa.cache_attn_fwd(bf(2, 1, 4, 64), bf(2, 8, 2, 64), bf(2, 8, 2, 64), lens)
    with pytest.raises(TypeError, match="q must be torch.bfloat16"):
        sa.cache_attn_fwd(torch.zeros(2, 1, 4, 64), bf(2, 8, 2, 64), bf(2, 8, 2, 64), lens)
    with pytest.raises(ValueError, match="k_cache must be a CUDA tensor"):
        sa.cache_evict(bf(2, 8, 2, 64), bf(2, 8, 2, 64), torch.zeros(2, 2, 8), lens, 4)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        sa.sparse_attn_key_weights(bf(1, 8, 2, 64), bf(1, 8, 2, 64), torch.zeros(1, 2, 8), None)


@pytest.fixture
def cuda_check_off(monkeypatch):
    """The shape logic of the checks on CPU tensors (nothing here reaches a kernel)."""
    strict = sa._require

    def lenient(cond, msg, exc=ValueError):
        if "CUDA tensor" not in msg:
            strict(cond, msg, exc)

    monkeypatch.setattr(sa, "_require", lenient)


def test_binding_refuses_wrong_shapes(lib, cuda_check_off):
    q, k, v = bf(2, 1, 4, 128), bf(2, 8, 2, 128), bf(2, 8, 2, 128)
    lens, w = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2, 8)
    assert sa.cache_attn_workspace_size(q, k, v, lens) > 0
    for match, args, kw in [
        ("one token", (bf(2, 2, 4, 128), k, v, lens), {}),
        ("k_cache must be", (q, bf(3, 8, 2, 128), v, lens), {}),
        ("v_cache must be", (q, k, bf(2, 9, 2, 128), lens), {}),
        ("lens must have shape", (q, k, v, torch.zeros(3, dtype=torch.int32)), {}),
        ("lens must be torch.int32", (q, k, v, torch.zeros(2)), {}),
        ("go together", (q, k, v, lens), dict(k_prefix=bf(5, 2, 128))),
        ("v_prefix must have shape", (q, k, v, lens),
         dict(k_prefix=bf(5, 2, 128), v_prefix=bf(6, 2, 128))),
        ("weights must have shape", (q, k, v, lens), dict(weights=w[:, :, :7].contiguous(), with_weights=True)),
        ("weights needs", (q, k, v, lens), dict(weights=w)),
        ("o must have shape", (q, k, v, lens), dict(o=bf(2, 4, 128))),
        ("k_cache must be contiguous", (q, bf(2, 8, 4, 128)[:, :, ::2], v, lens), {}),
    ]:
        with pytest.raises((ValueError, TypeError), match=match):
            sa.cache_attn_fwd(*args, **kw)
    for match, args, kw in [
        ("v_cache must have shape", (k, bf(2, 7, 2, 128), w, lens, 4), {}),
        ("weights must have shape", (k, v, w[:1], lens, 4), {}),
        ("budget must be", (k, v, w, lens, 0), {}),
        ("budget must be", (k, v, w, lens, 9), {}),
        ("sinks and recent", (k, v, w, lens, 4), dict(sinks=3, recent=2)),
        ("sinks and recent", (k, v, w, lens, 4), dict(sinks=-1)),
        ("k_out must have shape", (k, v, w, lens, 4), dict(k_out=bf(2, 8, 2, 64))),
        ("v_out must have shape", (k, v, w, lens, 4), dict(k_out=bf(2, 8, 2, 128), v_out=bf(2, 9, 2, 128))),
        ("keep must have shape", (k, v, w, lens, 4), dict(keep=torch.zeros(2, 2, 5, dtype=torch.int32))),
    ]:
        with pytest.raises((ValueError, TypeError), match=match):
            sa.cache_evict(*args, **kw)


def test_entry_points_run_on_their_tensors_device():
    for name in ("cache_attn_fwd", "cache_attn_workspace_size", "sparse_attn_key_weights",
                 "cache_evict"):
        assert getattr(getattr(sa, name), "device_arg", None), name


def test_references_agree_with_dense_softmax():
    """cache_attn over prefix + cache equals softmax over the joined keys, its weights sum to one
    per head with the prefix's share; evict keeps what a stable sort of the middle keeps."""
    rng = np.random.default_rng(0)
    B, HQ, HK, D, S, P = 2, 4, 2, 16, 12, 5
    q, kc, vc = (rng.standard_normal(s) for s in ((B, 1, HQ, D), (B, S, HK, D), (B, S, HK, D)))
    kp, vp = rng.standard_normal((P, HK, D)), rng.standard_normal((P, HK, D))
    lens = np.array([12, 0])
    (o, lse, w), _ = R.cache_attn(q, kc, vc, lens, kp, vp, 0.25)
    for b, h in np.ndindex(B, HQ):
        g = h // 2
        k = np.concatenate([kp[:, g], kc[b, :lens[b], g]])
        v = np.concatenate([vp[:, g], vc[b, :lens[b], g]])
        e = np.exp(0.25 * k @ q[b, 0, h])
        assert np.allclose(o[b, 0, h], e @ v / e.sum())
        assert np.isclose(lse[b, h, 0], np.log(e.sum()))
    assert (w[1] == 0).all() and (w[0] > 0).all()
    wts = rng.integers(0, 4, (B, HK, S)).astype(np.float32)
    keep = R.evict(kc, vc, wts, np.array([12, 3]), 6, 1, 2)
    for g in range(HK):
        order = 1 + np.argsort(-wts[0, g, 1:10], kind="stable")[:3]
        assert keep[0, g].tolist() == sorted([0, *order.tolist(), 10, 11])
        assert keep[1, g].tolist() == [0, 1, 2, -1, -1, -1]


@pytest.mark.parametrize("step", [4, 4 * (2 * 2 * 100 - 1)])
def test_weights_that_overlap_in_part_are_refused(lib, step):
    """Element j of one array is another element of the other: what is read would depend on which
    thread has written."""
    for a, b in ((0x100000, 0x100000 + step), (0x100000 + step, 0x100000)):
        assert call_attn(lib, attn(weights=a, weights_out=b)) == BAD
        s = _lib.BlockSparseStruct(_lib.SA_MODE_DENSE, 0, 2, 2, 256, 100, 128, 0, 0, None, None,
                                   0x1000, 0x1000, 0x1000, 0x1000)
        p = _lib.ParamsStruct(0x1000, 0x1000, None, None, 0x1000, None, None, None, None, 2, 4, 2,
                              128, 128, 256, 100, 0.125, ctypes.pointer(s), None)
        assert lib.sparse_attn_key_weights(ctypes.byref(p), a, b, None, 0, None) == BAD
    # the same array, and arrays that touch, get as far as the workspace
    for a, b in ((0x100000, 0x100000), (0x100000, 0x100000 + 4 * 400), (0x100000 + 4 * 400, 0x100000)):
        assert call_attn(lib, attn(weights=a, weights_out=b), None, 0) == _lib.SA_ERR_WORKSPACE
        assert lib.sparse_attn_key_weights(ctypes.byref(p), a, b, None, 0,
                                           None) == _lib.SA_ERR_WORKSPACE


def test_binding_names_weights_that_overlap_in_part(lib, cuda_check_off, monkeypatch):
    monkeypatch.setattr(sa, "_stream", lambda device: None)
    q, k = bf(2, 1, 4, 128), bf(2, 8, 2, 128)
    lens, pool = torch.zeros(2, dtype=torch.int32), torch.zeros(64)
    w, out = pool[:32].view(2, 2, 8), pool[16:48].view(2, 2, 8)
    with pytest.raises(ValueError, match="weights_out overlaps"):
        sa.cache_attn_fwd(q, k, k, lens, weights=w, weights_out=out)
