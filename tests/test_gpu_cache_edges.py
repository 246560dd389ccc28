"""cache_attn_fwd where its warps, its workspace and its arithmetic have their edges: row maxima
that move by turns in either half of a tile, workspaces at every alignment that is allowed."""
import numpy as np
import pytest

from index_sparse_attention_b200 import inputs as I

from test_gpu_cache_attn import Case, D64, D128, D192, D256, _compare, _gpu

pytestmark = pytest.mark.gpu


def _bf16(x):
    """x rounded to bf16, as bits and as float64."""
    bits = I.f32_to_bf16_bits(x.astype(np.float32))
    return bits, I.bf16_bits_to_f32(bits).astype(np.float64)


def _steep(c, seed):
    """K along one direction, with scores that jump from run to run of 16 keys: the maximum of a
    tile lies now in one half of its columns and now in the other, often far above the one
    before it."""
    rng = np.random.default_rng(seed)
    u = rng.standard_normal(c.q.shape[-1])
    u /= np.linalg.norm(u)
    qb, c.q = _bf16(4.0 * u + 0.1 * rng.standard_normal(c.q.shape))
    c.g["q"] = _gpu(qb)
    for name, key in (("k", "k_cache"), ("kp", "k_prefix")):
        k = getattr(c, name)
        if k is None:
            continue
        n = k.shape[-3]
        climb = np.linspace(0.0, 60.0, n)
        jump = np.repeat(rng.choice([-25.0, 0.0, 9.0], -(-n // 16)), 16)[:n]
        s = (climb + jump + rng.standard_normal(n)) / (4.0 * c.scale)
        kb, x = _bf16(s[:, None, None] * u + 0.1 * rng.standard_normal(k.shape))
        setattr(c, name, x)
        c.g[key] = _gpu(kb)
    return c


STEEP = {
    "copies_of_rows_d64": dict(lens=[9001, 4000], HQ=8, HK=2, D=D64),
    "copies_of_rows_d128": dict(lens=[9001, 4000], HQ=8, HK=2, D=D128, P=1000),
    "copies_of_rows_d192": dict(lens=[9001, 4000], HQ=32, HK=2, D=D192, P=1000),
    "copies_of_rows_d256": dict(lens=[9001, 4000], HQ=8, HK=2, D=D256, P=1000),
    "whole_buffers_d64": dict(lens=[300] * 20, HQ=16, HK=2, D=D64, P=9001),
    "whole_buffers_d128": dict(lens=[300] * 20, HQ=16, HK=2, D=D128, P=9001),
    "whole_buffers_d192": dict(lens=[300] * 20, HQ=16, HK=2, D=D192, P=9001),
    "whole_buffers_d256": dict(lens=[300] * 20, HQ=16, HK=2, D=D256, P=9001),
    "wide_groups": dict(lens=[5000, 4000, 129], HQ=64, HK=1, D=D128),
    "parts_of_one_tile": dict(lens=[1 + 37 * i % 128 for i in range(600)], HQ=8, HK=2, D=D128),
    "parts_of_one_tile_of_wide_groups": dict(lens=[1 + 37 * i % 128 for i in range(300)], HQ=48,
                                             HK=1, D=D64),
}


@pytest.mark.parametrize("name", STEEP)
def test_maxima_that_move_from_half_to_half(name):
    """The two warps that share a row agree on its maximum in every tile and on its sum at every
    part's end, whichever of them holds it: right against 64 bits, and the same bits each time."""
    import torch
    import index_sparse_attention_b200 as sa
    c = _steep(Case(seed=500, **STEEP[name]), seed=501)
    w = torch.from_numpy(c.w).cuda()
    got = sa.cache_attn_fwd(**c.g, weights=w, with_weights=True)
    _compare(got, *c.reference())
    for _ in range(20):
        again = sa.cache_attn_fwd(**c.g, weights=w, with_weights=True)
        assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("shift", [0, 16, 48, 240])
@pytest.mark.parametrize("D", [D64, D128, D192, D256], ids=str)
def test_a_workspace_of_exact_size_at_any_16_byte_boundary(D, shift):
    """A slice of a caller's pool: every part's output lies inside it, with row copies (the caches
    here) and without (the prefix), and few bytes in front of it and behind it stay as they were."""
    import torch
    import index_sparse_attention_b200 as sa
    c = Case([300, 40, 7, 129] * 10, HQ=8, HK=2, D=D, P=700, seed=520)
    w = torch.from_numpy(c.w).cuda()
    need = sa.cache_attn_workspace_size(c.g["q"], c.g["k_cache"], c.g["v_cache"], c.g["lens"],
                                        c.g["k_prefix"], c.g["v_prefix"], with_weights=True)
    pool = torch.full((need + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    assert pool.data_ptr() % 256 == 0
    at = 256 + shift
    got = sa.cache_attn_fwd(**c.g, weights=w, with_weights=True, workspace=pool[at:at + need])
    _compare(got, *c.reference())
    assert (pool[:at] == 0xA5).all() and (pool[at + need:] == 0xA5).all()
