"""cache_attn_fwd against its 64-bit reference: every head-dim pair, group sizes 1 to 128, lengths
around the tile edges (0 and 1 among them), no prefix to several tiles of it, weights in place and
out of place, whatever lies behind the lengths; streams, graph replay, wait limits."""
import numpy as np
import pytest

import cache_ref as R
from index_sparse_attention_b200 import _lib
from index_sparse_attention_b200 import inputs as I

pytestmark = pytest.mark.gpu


def _bf(seed, shape):
    bits = I.normal_bf16(seed, shape)
    return bits, I.bf16_bits_to_f32(bits).astype(np.float64)


def _gpu(bits):
    import torch
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).cuda()


class Case:
    def __init__(self, lens, HQ, HK, D, P=0, S=None, seed=0, kscale=1.0):
        import torch
        self.lens, B = np.array(lens, np.int32), len(lens)
        S = S or max(1, max(lens))
        Dqk, Dv = D
        self.scale = Dqk ** -0.5
        qb, self.q = _bf(seed, (B, 1, HQ, Dqk))
        kb, self.k = _bf(seed + 1, (B, S, HK, Dqk))
        vb, self.v = _bf(seed + 2, (B, S, HK, Dv))
        if kscale != 1.0:
            kb = I.f32_to_bf16_bits((self.k * kscale).astype(np.float32))
            self.k = I.bf16_bits_to_f32(kb).astype(np.float64)
        self.g = dict(q=_gpu(qb), k_cache=_gpu(kb), v_cache=_gpu(vb),
                      lens=torch.from_numpy(self.lens).cuda())
        self.kp = self.vp = None
        if P:
            kpb, self.kp = _bf(seed + 3, (P, HK, Dqk))
            vpb, self.vp = _bf(seed + 4, (P, HK, Dv))
            self.g.update(k_prefix=_gpu(kpb), v_prefix=_gpu(vpb))
        rng = np.random.default_rng(seed + 5)
        self.w = np.abs(rng.standard_normal((B, HK, S))).astype(np.float32)

    def poison(self):
        """NaN in K and infinities in V behind every length."""
        for b, n in enumerate(self.lens):
            self.g["k_cache"][b, max(n, 0):] = float("nan")
            self.g["v_cache"][b, max(n, 0):] = float("inf")

    def reference(self, weights=True):
        return R.cache_attn(self.q, self.k, self.v, self.lens, self.kp, self.vp, self.scale,
                            self.w.astype(np.float64) if weights else None)


def _compare(got, ref, tol):
    for name, x, r, t in zip(("o", "lse", "weights"), got, ref, tol):
        x = x.double().cpu().numpy()
        assert x.shape == r.shape, name
        inf = np.isneginf(r)
        assert np.array_equal(np.isneginf(x), inf), f"{name}: -inf pattern"
        assert np.isfinite(x[~inf]).all(), f"{name}: non-finite values"
        over = np.abs(x[~inf] - r[~inf]) - t[~inf]
        assert over.size == 0 or over.max() <= 0, f"{name}: {over.max():.3e} over its bound"


D64, D128, D192, D256 = (64, 64), (128, 128), (192, 128), (256, 256)
CASES = {
    "one_key": dict(lens=[1], HQ=1, HK=1, D=D64),
    "tile_edges_d64": dict(lens=[63, 64, 65, 127, 128, 129, 0, 1], HQ=4, HK=2, D=D64, P=130),
    "tile_edges_d128": dict(lens=[127, 128, 129, 255, 256, 257, 0, 1, 2], HQ=8, HK=2, D=D128, P=1),
    "tile_edges_d192": dict(lens=[63, 64, 65, 127, 128, 129, 0, 1], HQ=8, HK=1, D=D192, P=257),
    "tile_edges_d256": dict(lens=[31, 32, 33, 63, 64, 65, 0, 1], HQ=3, HK=3, D=D256, P=127),
    "no_prefix_long": dict(lens=[5000], HQ=8, HK=2, D=D128),
    "prefix_alone": dict(lens=[0, 0, 0], HQ=6, HK=2, D=D128, P=700),
    "nothing_at_all": dict(lens=[0, 0], HQ=4, HK=2, D=D64, S=5),
    "some_empty_no_prefix": dict(lens=[0, 300, 0, 0, 7, 0], HQ=6, HK=2, D=D192),
    "group_3": dict(lens=[100, 300, 77], HQ=9, HK=3, D=D128, P=200),
    "group_16": dict(lens=[100, 300, 77], HQ=32, HK=2, D=D128, P=200),
    "group_33": dict(lens=[140, 20], HQ=33, HK=1, D=D64, P=150),
    "group_48_d192": dict(lens=[140, 20, 300], HQ=48, HK=1, D=D192, P=150),
    "group_128": dict(lens=[300, 5], HQ=128, HK=1, D=D128, P=131),
    "group_128_d256": dict(lens=[300, 5], HQ=128, HK=1, D=D256, P=131),
    "group_20_d256": dict(lens=[140, 20, 300, 7, 500], HQ=20, HK=1, D=D256, P=150),
    "group_20_d256_many_parts": dict(lens=[3, 70, 64, 1, 90] * 60, HQ=20, HK=1, D=D256),
    "small_parts_d256": dict(lens=[3, 70, 64, 1, 90] * 40, HQ=8, HK=2, D=D256, P=150),
    "small_parts_full_prefix_d256": dict(lens=[9, 65], HQ=40, HK=2, D=D256, P=1000),
    "many_rows": dict(lens=[5 + 3 * i for i in range(70)], HQ=16, HK=2, D=D128, P=515),
    "many_rows_d256": dict(lens=[5 + 3 * i for i in range(40)], HQ=8, HK=1, D=D256, P=260),
    "many_sequences": dict(lens=[(7 * i) % 50 for i in range(400)], HQ=2, HK=1, D=D64, P=33),
    "more_sequences_than_threads": dict(lens=[(i % 3) for i in range(1500)], HQ=1, HK=1, D=D64),
    "many_sequences_and_rows": dict(lens=[(37 * i) % 190 for i in range(300)], HQ=8, HK=2, D=D128,
                                    P=140),
    "many_rows_no_prefix_d192": dict(lens=[(i % 7) * 21 for i in range(520)], HQ=4, HK=4, D=D192),
    "sharp": dict(lens=[500, 333], HQ=8, HK=2, D=D128, P=300, kscale=12.0),
}

# many tiles in a row for every SM, on memory that no cache holds yet
LONG = {
    "long_d64": dict(lens=[30001, 20000, 25000], HQ=16, HK=4, D=D64),
    "long_d128": dict(lens=[30001, 20000, 25000], HQ=16, HK=4, D=D128),
    "long_d192": dict(lens=[10001, 9000, 12345], HQ=16, HK=4, D=D192),
    "long_d256": dict(lens=[10001, 9000, 12345], HQ=8, HK=4, D=D256),
    "long_prefix_d128": dict(lens=[1, 300, 7], HQ=16, HK=4, D=D128, P=40001),
    "long_prefix_d256": dict(lens=[1, 300, 7], HQ=32, HK=2, D=D256, P=20001),
    "long_prefix_d192": dict(lens=[100, 3000, 7], HQ=64, HK=2, D=D192, P=20001),
}


@pytest.mark.parametrize("name", LONG)
def test_long_rows_on_cold_memory(name):
    import torch
    import index_sparse_attention_b200 as sa
    c = Case(seed=300, **LONG[name])
    ref, tol = c.reference(weights=False)
    for _ in range(3):
        g = {k: x.clone() for k, x in c.g.items()}
        torch.empty(1 << 28, dtype=torch.uint8, device="cuda").zero_()  # (larger than L2)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = sa.cache_attn_fwd(**g, dev_status=status)
        _compare(got, ref[:2], tol[:2])
        assert int(status.item()) == 0


@pytest.mark.parametrize("name", CASES)
def test_matches_the_reference(name):
    import torch
    import index_sparse_attention_b200 as sa
    c = Case(seed=100, **CASES[name])
    c.poison()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.from_numpy(c.w).cuda()
    got = sa.cache_attn_fwd(**c.g, weights=w, with_weights=True, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    _compare(got, *c.reference())
    # without weights: the same bits; in place: the same weights
    o, lse = sa.cache_attn_fwd(**c.g)
    assert torch.equal(o, got[0]) and torch.equal(lse, got[1])
    sa.cache_attn_fwd(**c.g, weights=w, weights_out=w)
    assert torch.equal(w, got[2])


def test_weights_start_from_zero_and_are_kept_behind_the_lengths():
    import torch
    import index_sparse_attention_b200 as sa
    c = Case([10, 0, 200], HQ=4, HK=2, D=D128, P=50, S=260, seed=7)
    _, _, w0 = sa.cache_attn_fwd(**c.g, with_weights=True)
    ref, tol = c.reference(weights=False)
    _compare((w0,), (ref[2],), (tol[2],))
    for b, n in enumerate(c.lens):
        assert (w0[b, :, n:] == 0).all()
    old = torch.full_like(w0, float("nan"))
    old[0, :, :10] = 1.0
    _, _, w1 = sa.cache_attn_fwd(**c.g, weights=old, with_weights=True)
    assert torch.isnan(w1[0, :, 10:]).all() and torch.isfinite(w1[0, :, :10]).all()


def test_bad_lengths_are_clamped_and_reported():
    import torch
    import index_sparse_attention_b200 as sa
    c = Case([40, 40, 40], HQ=4, HK=2, D=D128, S=40, seed=3)
    c.lens = np.array([-5, 41, 1 << 30], np.int32)
    c.g["lens"] = torch.from_numpy(c.lens).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sa.cache_attn_fwd(**c.g, dev_status=status)
    assert int(status.item()) == _lib.SA_STATUS_INDEX
    ref, tol = c.reference(weights=False)
    _compare(got, ref[:2], tol[:2])


def test_nan_and_infinite_keys_inside_the_length_reach_the_output():
    import torch
    import index_sparse_attention_b200 as sa
    c = Case([300, 300], HQ=4, HK=2, D=D128, seed=5)
    c.g["k_cache"][0, 17, 1, 3] = float("nan")
    o, lse = sa.cache_attn_fwd(**c.g)
    assert torch.isnan(lse[0, 2:]).all() and torch.isnan(o[0, 0, 2:]).all()
    assert torch.isfinite(o[0, 0, :2]).all() and torch.isfinite(o[1]).all()


def test_large_batch_offsets_beyond_32_bits():
    """A cache of more than 2^32 elements: the last sequence's rows are found."""
    import torch
    import index_sparse_attention_b200 as sa
    B, S, HK, D = 3, 1 << 21, 8, 128  # 6.4e9 elements in K, as many in V
    free, _ = torch.cuda.mem_get_info()
    if free < 32 << 30:
        pytest.skip("needs 32 GB of free device memory")
    c = Case([200, 1, 300], HQ=16, HK=HK, D=D128, seed=11)
    k = torch.empty((B, S, HK, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty((B, S, HK, D), dtype=torch.bfloat16, device="cuda")
    k[:, :300], v[:, :300] = c.g["k_cache"], c.g["v_cache"]
    # the last sequence's 200 last keys at the far end of the buffer too
    g = dict(c.g, k_cache=k, v_cache=v)
    got = sa.cache_attn_fwd(**g)
    ref, tol = c.reference(weights=False)
    _compare(got, ref[:2], tol[:2])


def test_other_stream_graph_replay_and_changed_lengths():
    """Captured once, replayed with new contents: lengths are read on the device, so a graph
    follows the growing caches."""
    import torch
    import index_sparse_attention_b200 as sa
    c = Case([50, 129, 0], HQ=8, HK=2, D=D128, P=140, S=300, seed=21)
    B, S = 3, 300
    o = torch.empty_like(c.g["q"])
    lse = torch.empty((B, 8, 1), device="cuda")
    w = torch.zeros((B, 2, S), device="cuda")
    need = sa.cache_attn_workspace_size(c.g["q"], c.g["k_cache"], c.g["v_cache"], c.g["lens"],
                                        c.g["k_prefix"], c.g["v_prefix"], with_weights=True)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    call = lambda: sa.cache_attn_fwd(**c.g, weights=w, weights_out=w, o=o, lse=lse, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()  # on another stream
    side.synchronize()
    c.w = np.zeros((B, 2, S), np.float32)
    _compare((o, lse, w), *c.reference())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([51, 130, 1], [300, 0, 299]):
        c.lens = np.array(lens, np.int32)
        c.g["lens"].copy_(torch.from_numpy(c.lens))
        w.zero_()
        ws.fill_(255)  # the workspace need not be initialised
        graph.replay()
        torch.cuda.synchronize()
        _compare((o, lse, w), *c.reference())


def test_two_calls_at_once_on_two_streams():
    import torch
    import index_sparse_attention_b200 as sa
    cs = [Case([700, 1, 333], HQ=8, HK=2, D=D128, P=400, seed=31),
          Case([90, 800], HQ=8, HK=1, D=D192, P=900, seed=41)]
    want = [sa.cache_attn_fwd(**c.g, with_weights=True) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = []
    for _ in range(5):
        got = []
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(sa.cache_attn_fwd(**c.g, with_weights=True))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("D", [D64, D128, D192, D256], ids=str)
def test_short_wait_limit_reports_timeout_then_recovers(D):
    """A wait limit below 1 us makes ordinary waits run out: the call returns, reports it and
    leaves the context usable."""
    import torch
    import index_sparse_attention_b200 as sa
    c = Case([700, 1, 333], HQ=8, HK=2, D=D, P=400, seed=51)
    want = sa.cache_attn_fwd(**c.g, with_weights=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        sa.sparse_attn_set_wait_limit_ns(300)
        sa.cache_attn_fwd(**c.g, with_weights=True, dev_status=status)
        torch.cuda.synchronize()
    finally:
        sa.sparse_attn_set_wait_limit_ns(0)
    assert int(status.item()) & _lib.SA_STATUS_TIMEOUT
    status.zero_()
    got = sa.cache_attn_fwd(**c.g, with_weights=True, dev_status=status)
    assert int(status.item()) == 0
    assert all(torch.equal(x, y) for x, y in zip(got, want))
