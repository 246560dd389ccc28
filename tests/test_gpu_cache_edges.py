"""cache_attn_fwd where its warps, its workspace and its arithmetic have their edges: row maxima
that move by turns in either half of a tile, workspaces at every alignment that is allowed,
infinities and NaN among the keys and values that a row sees."""
import numpy as np
import pytest

import cache_ref as R
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


SPECIAL = {
    "copies_of_rows_d64": dict(lens=[700, 130], HQ=4, HK=2, D=D64),
    "copies_of_rows_d128": dict(lens=[700, 130], HQ=4, HK=2, D=D128, P=200),
    "copies_of_rows_d192": dict(lens=[700, 130], HQ=4, HK=2, D=D192, P=200),
    "copies_of_rows_d256": dict(lens=[700, 130], HQ=4, HK=2, D=D256, P=200),
    "whole_buffers_d64": dict(lens=[700, 130], HQ=80, HK=2, D=D64, P=200),
    "whole_buffers_d128": dict(lens=[700, 130], HQ=80, HK=2, D=D128, P=200),
    "whole_buffers_d192": dict(lens=[700, 130], HQ=80, HK=2, D=D192, P=200),
    "whole_buffers_d256": dict(lens=[700, 130], HQ=80, HK=2, D=D256, P=200),
    "a_warp_per_row_d64": dict(lens=[60 + i % 90 for i in range(520)], HQ=4, HK=2, D=D64, P=40),
    "a_warp_per_row_d128": dict(lens=[60 + i % 90 for i in range(520)], HQ=4, HK=2, D=D128),
    "a_warp_per_row_d192": dict(lens=[60 + i % 90 for i in range(520)], HQ=4, HK=2, D=D192, P=40),
    "a_warp_per_row_d256": dict(lens=[60 + i % 90 for i in range(520)], HQ=4, HK=2, D=D256),
}


@pytest.mark.parametrize("name", SPECIAL)
def test_infinite_values_that_a_row_sees(name):
    """o is infinite in the columns where a value is, NaN where one is NaN or both infinities
    meet, and right everywhere else; lse and weights know nothing of it.  Behind the lengths lie
    infinities and NaN as well."""
    import torch
    import index_sparse_attention_b200 as sa
    c = Case(seed=540, **SPECIAL[name])
    c.poison()
    inf, nan = float("inf"), float("nan")
    B, G, Dv = len(c.lens), c.q.shape[2] // c.k.shape[2], c.v.shape[3]
    want = np.zeros((B, 1, c.q.shape[2], Dv))  # what is added to a finite column

    def put(b, j, g, d, x):
        c.g["v_cache"][b, j, g, d] = x
        c.v[b, j, g, d] = 0.0
        with np.errstate(invalid="ignore"):  # (both infinities: NaN)
            want[b, 0, g * G:(g + 1) * G, d] += x

    put(0, 0, 0, 0, inf)                          # the first key, the first column
    put(0, int(c.lens[0]) - 1, 0, Dv - 1, -inf)   # the last ones
    for j, x in ((17, inf), (57, -inf)):          # both infinities, in different quarters of a tile
        put(0, j, 1, 5, x)
    for j in (3, 40, 59):                         # one infinity several times
        put(0, j, 1, Dv // 2 + 1, -inf)
    put(0, 33, 1, 9, nan)
    put(0, 34, 1, 9, inf)
    put(B - 1, 20, 1, 40, inf)
    if c.vp is not None:                          # every sequence sees the prefix
        for j, d, x in ((len(c.vp) - 1, 2, inf), (0, 3, -inf)):
            c.g["v_prefix"][j, 0, d] = x
            c.vp[j, 0, d] = 0.0
            want[:, 0, :G, d] += x
    w = torch.from_numpy(c.w).cuda()
    got = sa.cache_attn_fwd(**c.g, weights=w, with_weights=True)
    (o, *rest), (tol, *rest_tol) = c.reference()
    for what, x, r, t in zip(("lse", "weights"), got[1:], rest, rest_tol):
        assert (np.abs(x.double().cpu().numpy() - r) <= t).all(), what
    x, even = got[0].double().cpu().numpy(), want == 0
    assert (np.abs(x[even] - o[even]) <= tol[even]).all()
    assert np.array_equal(x[~even], want[~even], equal_nan=True)


@pytest.mark.parametrize("name", [n for n in SPECIAL if "d128" in n or "d256" in n])
def test_infinite_keys_that_a_row_sees(name):
    """A key with an infinite component: a score of -inf takes no part, one of +inf leaves NaN in
    its rows' outputs and no others."""
    import torch
    import index_sparse_attention_b200 as sa
    c = Case(seed=560, **SPECIAL[name])
    G = c.q.shape[2] // c.k.shape[2]
    c.g["k_cache"][0, 33, 1, 3] = float("inf")
    up = c.q[0, 0, G:, 3] > 0
    assert up.any() and not up.all() and (c.q[0, 0, G:, 3] != 0).all()
    o, lse, w = (t.double().cpu().numpy() for t in sa.cache_attn_fwd(**c.g, with_weights=True))
    assert np.isnan(o[0, 0, G:][up]).all() and not np.isfinite(lse[0, G:, 0][up]).any()
    for h in np.flatnonzero(~up):
        q = c.q[0, 0, G + h]
        keys = np.delete(c.k[0, :c.lens[0], 1], 33, 0)
        vals = np.delete(c.v[0, :c.lens[0], 1], 33, 0)
        if c.kp is not None:
            keys = np.concatenate([c.kp[:, 1], keys])
            vals = np.concatenate([c.vp[:, 1], vals])
        ro, rl, _, pv = R.softmax_rows(q[None], keys, vals, c.scale)
        ds = R.score_bound(q[None], keys, c.scale)
        assert abs(lse[0, G + h, 0] - rl[0]) <= ds
        tol = 2.0 ** -8 * (pv + np.abs(ro)) + (2 * ds + 2.0 ** -20) * pv
        assert (np.abs(o[0, 0, G + h] - ro[0]) <= tol[0]).all()
    assert np.isfinite(o[0, 0, :G]).all() and np.isfinite(o[1:]).all() and np.isfinite(w[1:]).all()


@pytest.mark.parametrize("limit", [100, 1000, 3000, 10000, 30000])
@pytest.mark.parametrize("D", [D64, D128, D192, D256], ids=str)
def test_a_call_given_up_ends_when_its_copies_have_landed(D, limit):
    """Whatever state a CTA gives up in, it waits for its own loads and MMAs and no longer: a wait
    for an arrival that nobody makes would take the two seconds of its limit."""
    import torch
    import index_sparse_attention_b200 as sa
    c = Case([700, 1, 333] * 9, HQ=8, HK=2, D=D, P=4000, seed=580)
    want = sa.cache_attn_fwd(**c.g, with_weights=True)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    try:
        sa.sparse_attn_set_wait_limit_ns(limit)
        start.record()
        for _ in range(10):
            sa.cache_attn_fwd(**c.g, with_weights=True)
        end.record()
        torch.cuda.synchronize()
    finally:
        sa.sparse_attn_set_wait_limit_ns(0)
    assert start.elapsed_time(end) < 500
    got = sa.cache_attn_fwd(**c.g, with_weights=True)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_the_most_sequences_and_the_most_heads():
    """65535 sequences, and 65535 heads of one sequence: the largest sizes that the call takes."""
    import torch
    import index_sparse_attention_b200 as sa
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    for B, H, P in ((65535, 1, 0), (65535, 1, 9), (1, 65535, 0), (1, 65535, 2)):
        S, D = 3, 64
        q, k, v = (torch.randn(s, generator=g, device="cuda").bfloat16()
                   for s in ((B, 1, H, D), (B, S, H, D), (B, S, H, D)))
        kp, vp = (torch.randn((P, H, D), generator=g, device="cuda").bfloat16() for _ in "kv")
        lens = torch.randint(0, S + 1, (B,), generator=g, device="cuda").int()
        o, lse, w = sa.cache_attn_fwd(q, k, v, lens, k_prefix=kp if P else None,
                                      v_prefix=vp if P else None, with_weights=True)
        s = torch.einsum("bqhd,bshd->bhs", q.double(), k.double()) / 8
        size = torch.einsum("bqhd,bshd->bhs", q.double().abs(), k.double().abs()).max() / 8
        live = (torch.arange(S, device="cuda") < lens[:, None])[:, None].expand_as(s)
        s = s.masked_fill(~live, -float("inf"))
        vals = v.double().transpose(1, 2)
        if P:
            sp = torch.einsum("bqhd,phd->bhp", q.double(), kp.double()) / 8
            size = max(size, torch.einsum("bqhd,phd->bhp", q.double().abs(), kp.double().abs()).max() / 8)
            s = torch.cat([sp, s], 2)
            vals = torch.cat([vp.double().transpose(0, 1).expand(B, H, P, D), vals], 2)
        ref_lse = s.logsumexp(2)
        p = torch.where(ref_lse[..., None] == -float("inf"), 0.0, (s - ref_lse[..., None]).exp())
        ref, mag = (torch.einsum("bhs,bhsd->bhd", p, x) for x in (vals, vals.abs()))
        # (the bounds of cache_ref.py)
        ds = (D + 8) * R.U24 * size + 2.0 ** -20 + 2.0 ** -22 * size
        none = ref_lse == -float("inf")
        assert torch.equal(lse[..., 0] == -float("inf"), none)
        assert ((lse[..., 0].double() - ref_lse)[~none].abs() <= ds).all()
        tol = 2.0 ** -8 * (mag + ref.abs()) + (2 * ds + 2.0 ** -20) * mag + 1e-30
        assert ((o[:, 0].double() - ref).abs() <= tol).all()
        own = p[..., P:]
        assert ((w.double() - own).abs() <= (2 * ds + 2.0 ** -20 + 2 * R.U24) * own).all()


def test_rows_at_the_far_end_of_a_cache_of_more_than_2_to_the_32_elements():
    """The last sequence fills its capacity: every one of its two million keys takes part."""
    import torch
    import index_sparse_attention_b200 as sa
    B, S, HK, HQ, D = 3, 1 << 21, 8, 16, 128
    free, _ = torch.cuda.mem_get_info()
    if free < 48 << 30:
        pytest.skip("needs 48 GB of free device memory")
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    q = torch.randn((B, 1, HQ, D), generator=g, device="cuda").bfloat16()
    k, v = (torch.empty((B, S, HK, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    for x in (k, v):
        x[:2, :512].normal_(generator=g)
        for at in range(0, S, 1 << 18):
            x[2, at:at + (1 << 18)].normal_(generator=g)
    lens = torch.tensor([200, 1, S], dtype=torch.int32, device="cuda")
    o, lse = sa.cache_attn_fwd(q, k, v, lens)
    for h in range(HQ):
        s, size = torch.empty(S, dtype=torch.float64, device="cuda"), 0.0
        row = q[2, 0, h].double()
        for at in range(0, S, 1 << 18):
            keys = k[2, at:at + (1 << 18), h // 2].double()
            s[at:at + (1 << 18)] = keys @ row * D ** -0.5
            size = max(size, (keys.abs() @ row.abs()).max().item() * D ** -0.5)
        ref_lse = s.logsumexp(0)
        p = (s - ref_lse).exp()
        ref, mag = (sum(p[at:at + (1 << 18)] @ f(v[2, at:at + (1 << 18), h // 2].double())
                        for at in range(0, S, 1 << 18)) for f in (lambda x: x, torch.abs))
        ds = (D + 8) * R.U24 * size + 2.0 ** -20 + 2.0 ** -22 * size
        # two million terms are added in 148 parts, by tiles of 128: at most 128 + 16384 / 148
        # additions in a row, and 148 of the parts, each off by 2^-24 of the sum
        ds += (128 + 16384 / 148 + 148) * R.U24
        assert abs(lse[2, h, 0].item() - ref_lse.item()) <= ds
        tol = 2.0 ** -8 * (mag + ref.abs()) + (2 * ds + 2.0 ** -20) * mag
        assert ((o[2, 0, h].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("shape", [dict(lens=[30001], P=0), dict(lens=[9, 2000, 777], P=5001),
                                   dict(lens=[40 + i for i in range(600)], P=0),
                                   dict(lens=[40 + i for i in range(600)], P=700)],
                         ids=["one_long", "prefix", "many", "many_and_prefix"])
@pytest.mark.parametrize("HQ", [4, 48], ids=["copies_of_rows", "wide_groups"])
@pytest.mark.parametrize("D", [D64, D128, D192, D256], ids=str)
def test_an_infinity_wherever_it_lies_is_found(D, HQ, shape):
    """Every column of o has one infinite value, at a key of its own: in the first part of a row,
    the last, beside the borders.  A quarter of the columns also have a NaN or the other infinity
    elsewhere, whole rows of NaN come last."""
    import torch
    import index_sparse_attention_b200 as sa
    g = torch.Generator(device="cuda")
    g.manual_seed(17)
    lens, P, Dv = shape["lens"], shape["P"], D[1]
    B, S = len(lens), max(lens)
    if B > 3 and HQ > 4:
        HQ = 33
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    q, k, v = bf(B, 1, HQ, D[0]), bf(B, S, 1, D[0]), bf(B, S, 1, Dv)
    kp, vp = (bf(P, 1, D[0]), bf(P, 1, Dv)) if P else (None, None)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(18)
    cols = torch.arange(Dv, device="cuda")
    gpu = lambda x: torch.from_numpy(x.astype(np.float32)).cuda().bfloat16()
    args = dict(q=q, k_cache=k, v_cache=v, lens=n, k_prefix=kp, v_prefix=vp)

    def check():
        """o is the sum of the infinities and NaN that a column's values hold, a number where they
        hold none."""
        live = torch.arange(S, device="cuda")[None] < n[:, None]
        special = lambda x: torch.where(x.isfinite(), 0.0, x.double())
        want = special(torch.where(live[..., None], v[:, :, 0], 0.0)).sum(1)
        if P:
            want = want + special(vp[:, 0]).sum(0)
        o = sa.cache_attn_fwd(**args)[0][:, 0].double()
        want = want[:, None].expand_as(o)
        even = want == 0
        assert o[even].isfinite().all()
        assert torch.equal(o[~even].nan_to_num(7.0, 8.0, 9.0), want[~even].nan_to_num(7.0, 8.0, 9.0))

    sign = np.where(rng.random(Dv) < 0.5, np.inf, -np.inf)
    if P:  # the same for every sequence
        vp[torch.from_numpy(rng.integers(0, P, Dv)).cuda(), 0, cols] = gpu(sign)
    else:
        for b in range(B):
            v[b, torch.from_numpy(rng.integers(0, lens[b], Dv)).cuda(), 0, cols] = gpu(sign)
    check()
    other = np.where(rng.random(Dv) < 0.5, np.nan, -sign)[: Dv // 4]
    v[:, min(lens) - 1, 0, :Dv // 4] = gpu(other)
    if not P:  # (and an infinity that lay in the others' columns is gone)
        v[:, min(lens) - 1, 0, Dv // 4:] = 0.0
    check()
    v[:, :min(lens)] = float("nan")
    check()
