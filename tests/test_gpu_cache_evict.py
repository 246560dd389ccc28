"""cache_evict against its reference (equal, not near: the operator copies), and the operators
together as a server runs them: prompt, weights, eviction, decoding, eviction."""
import numpy as np
import pytest

import cache_ref as R
from index_sparse_attention_b200 import _lib
from index_sparse_attention_b200 import inputs as I

from helpers import bf16_to_f64, build_lists, to_gpu

pytestmark = pytest.mark.gpu


def _make(lens, HK, D, S, seed, weights=None):
    import torch
    rng = np.random.default_rng(seed)
    B = len(lens)
    k = I.normal_bf16(seed + 1, (B, S, HK, D[0]))
    v = I.normal_bf16(seed + 2, (B, S, HK, D[1]))
    w = np.exp(2 * rng.standard_normal((B, HK, S))).astype(np.float32) if weights is None else weights(rng, (B, HK, S))

    def bf(a):
        return torch.from_numpy(a.view(np.int16).copy()).view(torch.bfloat16).cuda()

    return (k, v, w, np.array(lens, np.int32),
            (bf(k), bf(v), torch.from_numpy(w).cuda(), torch.from_numpy(np.array(lens, np.int32)).cuda()))


def _check(k, v, w, lens, got, budget, sinks, recent, k0=None):
    import torch
    ko, vo, wo, lo, keep = (t.cpu() for t in got)
    ref = R.evict(k, v, w, lens, budget, sinks, recent)
    assert np.array_equal(keep.numpy(), ref)
    S = k.shape[1]
    n_out = np.minimum(np.clip(lens, 0, S), budget)
    assert np.array_equal(lo.numpy(), n_out)
    ko, vo = ko.view(torch.int16).numpy(), vo.view(torch.int16).numpy()
    for b, n in enumerate(n_out):
        for h in range(k.shape[2]):
            at = ref[b, h, :n]
            assert np.array_equal(ko[b, :n, h], k[b, at, h].view(np.int16))
            assert np.array_equal(vo[b, :n, h], v[b, at, h].view(np.int16))
            assert np.array_equal(wo[b, h, :n].numpy(), w[b, h, at], equal_nan=True)
            assert (wo[b, h, n:] == 0).all()
        if k0 is not None:  # rows behind stay as they were
            assert (ko[b, n:] == k0).all() and (vo[b, n:] == k0).all()


def ties(rng, shape):
    return rng.integers(0, 3, shape).astype(np.float32)


def equal(rng, shape):
    return np.full(shape, 0.25, np.float32)


def zeros(rng, shape):
    w = np.zeros(shape, np.float32)
    w[rng.random(shape) < 0.5] = -0.0
    return w


def special(rng, shape):
    w = rng.standard_normal(shape).astype(np.float32)
    for x in (np.nan, -np.nan, np.inf, -np.inf, 1e-42, -1e-42, 3.4e38):
        w[rng.random(shape) < 0.02] = x
    return w


def close(rng, shape):  # keys that differ in the lowest bits only
    return (np.float32(1.0) + rng.integers(0, 200, shape).astype(np.float32) * np.float32(2.0 ** -23))


D64, D128, D192, D256 = (64, 64), (128, 128), (192, 128), (256, 256)
CASES = {
    "one": dict(lens=[1], HK=1, D=D64, S=1, budget=1),
    "cut_to_one": dict(lens=[9], HK=2, D=D64, S=9, budget=1),
    "sinks_only": dict(lens=[50, 3], HK=2, D=D64, S=50, budget=5, sinks=5),
    "recent_only": dict(lens=[50, 3], HK=2, D=D128, S=50, budget=5, recent=5),
    "sinks_and_recent_fill": dict(lens=[50, 9], HK=1, D=D192, S=50, budget=9, sinks=4, recent=5),
    "below_at_above": dict(lens=[99, 100, 101, 0, 1, 300], HK=3, D=D128, S=300, budget=100, sinks=4, recent=20),
    "odd_d192": dict(lens=[1999, 777, 1234], HK=4, D=D192, S=2001, budget=501, sinks=3, recent=77),
    "odd_d256": dict(lens=[1500, 1023, 1025], HK=2, D=D256, S=1500, budget=999, sinks=1, recent=0),
    "one_less": dict(lens=[4096, 4097], HK=1, D=D64, S=4097, budget=4096),
    "long": dict(lens=[70001, 140000], HK=1, D=D64, S=140000, budget=20011, sinks=4, recent=100),
    "spread_over_eight": dict(lens=[60001, 33000, 9], HK=2, D=D64, S=60001, budget=7001, sinks=4, recent=1001),
    "spread_over_four_ties": dict(lens=[16384, 14000], HK=2, D=D64, S=16384, budget=9001, sinks=0, recent=3,
                                  weights=lambda rng, s: ties(rng, s)),
    "longer_than_registers": dict(lens=[140001, 100000], HK=1, D=D64, S=150000, budget=30000, sinks=4, recent=100,
                                  weights=lambda rng, s: ties(rng, s)),
    "ties": dict(lens=[5000, 3333], HK=2, D=D64, S=5000, budget=1700, sinks=4, recent=64, weights=ties),
    "all_equal": dict(lens=[5000, 2000], HK=2, D=D64, S=5000, budget=700, sinks=2, recent=3, weights=equal),
    "signed_zeros": dict(lens=[900], HK=2, D=D64, S=900, budget=300, weights=zeros),
    "nan_inf": dict(lens=[3000, 2999], HK=2, D=D64, S=3000, budget=200, sinks=2, recent=5, weights=special),
    "low_bits": dict(lens=[3000, 2999], HK=2, D=D64, S=3000, budget=1200, weights=close),
    "many_rows": dict(lens=[20 + i for i in range(50)], HK=8, D=D64, S=70, budget=33, sinks=1, recent=8),
    # as many rows as SMs, so that the selection copies its own: short and long ones, every head dim
    "own_copy_d64": dict(lens=[300, 301, 0, 1, 299, 700, 512, 90] * 3, HK=5, D=D64, S=700, budget=300, sinks=4, recent=20),
    "own_copy_d128": dict(lens=[40 + 7 * i for i in range(18)], HK=8, D=D128, S=160, budget=101, recent=9),
    "own_copy_d192": dict(lens=[33, 200, 201, 57] * 8, HK=4, D=D192, S=201, budget=57, sinks=3),
    "own_copy_d256": dict(lens=[20 + i for i in range(140)], HK=1, D=D256, S=160, budget=37, sinks=1, recent=1),
    "own_copy_cluster": dict(lens=[9001 - 500 * i for i in range(16)], HK=4, D=D64, S=9001, budget=1203, sinks=4, recent=64),
    "own_copy_of_ties": dict(lens=[400 - i for i in range(72)], HK=2, D=D64, S=400, budget=150, sinks=2, recent=3, weights=ties),
}


@pytest.mark.parametrize("name", CASES)
def test_matches_the_reference(name):
    import torch
    import index_sparse_attention_b200 as sa
    c = dict(CASES[name])
    budget, sinks, recent = c.pop("budget"), c.pop("sinks", 0), c.pop("recent", 0)
    k, v, w, lens, g = _make(seed=50, **c)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ko = torch.full_like(g[0], 1.0)
    vo = torch.full_like(g[1], 1.0)
    got = sa.cache_evict(*g, budget, sinks=sinks, recent=recent, k_out=ko, v_out=vo, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    _check(k, v, w, lens, got, budget, sinks, recent, k0=0x3F80)


def test_other_capacity_and_bad_lengths():
    import torch
    import index_sparse_attention_b200 as sa
    k, v, w, lens, g = _make([-3, 200, 4000], 2, D128, 90, 60)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ko = torch.zeros((3, 40, 2, 128), dtype=torch.bfloat16, device="cuda")
    got = sa.cache_evict(*g, 37, sinks=2, recent=3, k_out=ko, dev_status=status)
    assert int(status.item()) == _lib.SA_STATUS_INDEX
    assert got[1].shape == (3, 40, 2, 128) and got[2].shape == (3, 2, 40)
    _check(k, v, w, lens, got, 37, 2, 3)


def test_graph_replay_with_other_contents():
    import torch
    import index_sparse_attention_b200 as sa
    k, v, w, lens, g = _make([900, 50, 400], 2, D128, 900, 70)
    out = sa.cache_evict(*g, 300, sinks=4, recent=32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.cache_evict(*g, 300, sinks=4, recent=32, k_out=out[0], v_out=out[1], weights_out=out[2],
                       lens_out=out[3], keep=out[4])
    k, v, w, lens, h = _make([899, 301, 1], 2, D128, 900, 80)
    for x, y in zip(g, h):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    _check(k, v, w, lens, out, 300, 4, 32)


def test_two_calls_at_once_on_two_streams():
    import torch
    import index_sparse_attention_b200 as sa
    cases = [_make([20000, 9000, 1], 2, D128, 20000, 71), _make([3000, 2999, 3000], 2, D64, 3000, 72)]
    torch.cuda.synchronize()
    streams, out = [torch.cuda.Stream() for _ in cases], [None, None]
    for _ in range(3):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                out[i] = sa.cache_evict(*c[4], 300, sinks=4, recent=32)
    torch.cuda.synchronize()
    for c, got in zip(cases, out):
        _check(*c[:4], got, 300, 4, 32)


def test_offsets_beyond_32_bits():
    """Caches of 2^32 elements: the rows of the last sequence are found at their far end."""
    import torch
    import index_sparse_attention_b200 as sa
    B, S, HK, D, budget = 2, 1 << 22, 4, 128, 200
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    k = torch.empty((B, S, HK, D), dtype=torch.bfloat16, device="cuda")
    k.view(torch.int16)[:] = torch.arange(S, device="cuda").to(torch.int16)[None, :, None, None]
    w = torch.rand((B, HK, S), device="cuda")
    w[1, :, -1000:] += 1.0  # (more of the largest than are kept)
    lens = torch.tensor([7, S], dtype=torch.int32, device="cuda")
    ko = torch.zeros((B, budget, HK, D), dtype=torch.bfloat16, device="cuda")
    ko, vo, wo, lo, keep = sa.cache_evict(k, k, w, lens, budget, k_out=ko)
    assert lo.tolist() == [7, budget]
    for h in range(HK):
        at = torch.argsort(w[1, h, -1000:], descending=True, stable=True)[:budget] + (S - 1000)
        at = at.sort().values
        assert torch.equal(keep[1, h].long(), at)
        assert torch.equal(wo[1, h], w[1, h, at])
        assert torch.equal(ko[1, :, h].view(torch.int16), k[1, at, h].view(torch.int16))
        assert torch.equal(vo[1, :, h].view(torch.int16), k[1, at, h].view(torch.int16))


def test_overlapping_outputs_are_refused():
    import torch
    import index_sparse_attention_b200 as sa
    _, _, _, _, g = _make([20, 20], 2, D64, 40, 90)
    with pytest.raises(ValueError, match="overlaps"):
        sa.cache_evict(*g, 10, k_out=g[0])
    with pytest.raises(ValueError, match="overlaps"):
        sa.cache_evict(*g, 10, weights_out=g[2])
    ko = torch.zeros_like(g[0])
    with pytest.raises(ValueError, match="overlaps"):
        sa.cache_evict(*g, 10, k_out=ko, v_out=ko)


@pytest.mark.parametrize("D", [D64, D128, D192, D256], ids=str)
def test_prompt_weights_eviction_and_decoding_together(D):
    """Two prompts behind a shared prefix go through sparse_attn_fwd; their keys' weights decide
    the first eviction; tokens are decoded over prefix and cache, their weights added; a second
    eviction follows.  The kept positions and every output equal a 64-bit simulation's."""
    import torch
    import index_sparse_attention_b200 as sa
    B, n0, HQ, HK, P, budget, sinks, recent, steps = 2, 300, 4, 2, 200, 150, 4, 16, 5
    cap = 320
    w0 = I.scaled(I.WORKLOADS["gqa_blocksparse_b2_hq32_hk8_s8192_d128"], B=B, Sq=n0, Sk=n0, HQ=HQ,
                  HK=HK, Dqk=D[0], Dv=D[1], density=1.0, name="prompt")
    inp = I.make_inputs(w0, with_grad=False)
    g = to_gpu(inp)
    bsp = build_lists(inp, g)
    _, lse = sa.sparse_attn_fwd(g["q"], g["k"], g["v"], bsp)
    k = torch.zeros((B, cap, HK, D[0]), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((B, cap, HK, D[1]), dtype=torch.bfloat16, device="cuda")
    k[:, :n0], v[:, :n0] = g["k"], g["v"]
    w = torch.zeros((B, HK, cap), device="cuda")
    w[:, :, :n0] = sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp)
    a = np.broadcast_to(np.tril(np.ones((n0, n0), bool)), (B, HK, n0, n0))
    ref, tol = R.key_weights(bf16_to_f64(g["q"]), bf16_to_f64(g["k"]), lse.double().cpu().numpy(),
                             a, w0.scale)
    assert (np.abs(w[:, :, :n0].double().cpu().numpy() - ref) <= tol).all()
    rng = torch.Generator(device="cuda")
    rng.manual_seed(3)
    kp = torch.randn((P, HK, D[0]), generator=rng, device="cuda").bfloat16()
    vp = torch.randn((P, HK, D[1]), generator=rng, device="cuda").bfloat16()
    lens = torch.full((B,), n0, dtype=torch.int32, device="cuda")
    for turn in range(2):
        kh = bf16_to_f64(k), bf16_to_f64(v), w.cpu().numpy(), lens.cpu().numpy()
        keep_ref = R.evict(*kh, budget, sinks, recent)
        k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
        k, v, w, lens, keep = sa.cache_evict(k, v, w, lens, budget, sinks=sinks, recent=recent,
                                             k_out=k2, v_out=v2)
        assert np.array_equal(keep.cpu().numpy(), keep_ref)
        for t in range(steps):
            at = lens.long()
            for b in range(B):
                k[b, at[b]] = torch.randn((HK, D[0]), generator=rng, device="cuda").bfloat16()
                v[b, at[b]] = torch.randn((HK, D[1]), generator=rng, device="cuda").bfloat16()
            lens = lens + 1
            q = torch.randn((B, 1, HQ, D[0]), generator=rng, device="cuda").bfloat16()
            ref, tol = R.cache_attn(bf16_to_f64(q), bf16_to_f64(k), bf16_to_f64(v),
                                    lens.cpu().numpy(), bf16_to_f64(kp), bf16_to_f64(vp),
                                    D[0] ** -0.5, w.double().cpu().numpy())
            got = sa.cache_attn_fwd(q, k, v, lens, k_prefix=kp, v_prefix=vp, weights=w,
                                    weights_out=w)
            for x, r, e in zip(got, ref, tol):
                assert (np.abs(x.double().cpu().numpy() - r) <= e).all()
