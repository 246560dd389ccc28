"""Streams under capture: an entry point takes the current device's own and refuses another
context's with SA_ERR_DEVICE before anything is enqueued, which leaves that capture as it was.
(A second context of the same device stands in for another device: its streams cannot be
launched on either.)"""
import ctypes

import pytest

from index_sparse_attention_b200 import _lib

pytestmark = pytest.mark.gpu


class Other:
    """A stream of a second context on device 0, under capture; the context that was current stays
    current outside."""

    def __enter__(self):
        self.d = d = ctypes.CDLL("libcuda.so.1")
        self.ctx, self.stream = ctypes.c_void_p(), ctypes.c_void_p()
        self.ok(d.cuCtxCreate_v2(ctypes.byref(self.ctx), 0, 0))  # (becomes current)
        try:
            self.ok(d.cuStreamCreate(ctypes.byref(self.stream), 1))
            self.ok(d.cuStreamBeginCapture_v2(self.stream, 2))
        finally:
            self.ok(d.cuCtxPopCurrent_v2(ctypes.byref(ctypes.c_void_p())))
        return self

    @staticmethod
    def ok(rc):
        assert rc == 0, f"driver call returned {rc}"

    def capturing(self):
        status = ctypes.c_int(-1)
        self.ok(self.d.cuStreamIsCapturing(self.stream, ctypes.byref(status)))
        return status.value == 1

    def __exit__(self, *exc):
        graph = ctypes.c_void_p()
        self.d.cuCtxPushCurrent_v2(self.ctx)
        rc = self.d.cuStreamEndCapture(self.stream, ctypes.byref(graph))
        n = ctypes.c_size_t(99)
        if rc == 0:
            self.d.cuGraphGetNodes(graph, None, ctypes.byref(n))
            self.d.cuGraphDestroy(graph)
        self.d.cuStreamDestroy_v2(self.stream)
        self.d.cuCtxPopCurrent_v2(ctypes.byref(ctypes.c_void_p()))
        self.d.cuCtxDestroy_v2(self.ctx)
        if exc[0] is None:
            assert rc == 0 and n.value == 0


def _calls():
    """(name, function of a stream) of the entry points' C symbols, on real tensors."""
    import torch
    import index_sparse_attention_b200 as sa
    L = _lib.load()
    B, S, HK, HQ, D = 1, 64, 1, 2, 64
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    f32 = lambda *s: torch.zeros(s, dtype=torch.float32, device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    q1, k, v, lens, w = bf(B, 1, HQ, D), bf(B, S, HK, D), bf(B, S, HK, D), i32(B), f32(B, HK, S)
    q, o, lse = bf(B, S, HQ, D), bf(B, S, HQ, D), f32(B, HQ, S)
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    lists = sa.block_mask_to_block_sparse(None, B, HK, S, S)
    scores, top = f32(4, 32), i32(4, 8)
    torch.cuda.synchronize()
    keep = (q1, k, v, lens, w, q, o, lse, ws, lists, scores, top, bf(B, S, HK, D), bf(B, S, HK, D),
            f32(B, HK, S), i32(B), i32(B, HK, 8), bf(B, 1, HQ, D), f32(B, HQ, 1))
    p = sa._params_struct(q, k, v, o, lse, lists, 0.125)
    pa = _lib.CacheAttnStruct(q1.data_ptr(), k.data_ptr(), v.data_ptr(), lens.data_ptr(), None, None,
                              keep[17].data_ptr(), keep[18].data_ptr(), None, None, B, HQ, HK, D, D,
                              S, 0, 0.125, None)
    pe = _lib.CacheEvictStruct(k.data_ptr(), v.data_ptr(), w.data_ptr(), lens.data_ptr(),
                               *(t.data_ptr() for t in keep[12:17]), B, HK, D, D, S, S, 8, 1, 1, None)
    R = ctypes.byref
    return keep, {
        "block_mask_to_block_sparse": lambda s: L.block_mask_to_block_sparse(R(lists.c), s),
        "sparse_attn_fwd": lambda s: L.sparse_attn_fwd(R(p), s),
        "topk_select": lambda s: L.topk_select(scores.data_ptr(), 4, 32, 32, None, None, 8,
                                               top.data_ptr(), None, None, s),
        "cache_attn_fwd": lambda s: L.cache_attn_fwd(R(pa), ws.data_ptr(), ws.numel(), s),
        "sparse_attn_key_weights": lambda s: L.sparse_attn_key_weights(
            R(p), None, w.data_ptr(), ws.data_ptr(), ws.numel(), s),
        "cache_evict": lambda s: L.cache_evict(R(pe), s),
    }


NAMES = ("block_mask_to_block_sparse", "sparse_attn_fwd", "topk_select", "cache_attn_fwd",
         "sparse_attn_key_weights", "cache_evict")


@pytest.mark.parametrize("name", NAMES)
def test_another_contexts_capture_is_refused_and_left_alone(name):
    import torch
    keep, calls = _calls()
    with Other() as other:
        assert other.capturing()
        assert calls[name](other.stream) == _lib.SA_ERR_DEVICE
        assert other.capturing()
    assert calls[name](ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_the_own_devices_capture_is_taken(name):
    import torch
    keep, calls = _calls()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        assert calls[name](ctypes.c_void_p(side.cuda_stream)) == 0
    graph.replay()
    torch.cuda.synchronize()
