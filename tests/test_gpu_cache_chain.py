"""The cache calls one behind another without a host in between, as a server makes them: each
starts while the one before it ends, and reads what that one wrote.  The results are those of the
same calls with the GPU waited for after each."""
import pytest

pytestmark = pytest.mark.gpu

D64, D128, D192, D256 = (64, 64), (128, 128), (192, 128), (256, 256)


def _caches(B, S, HK, D, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    k = torch.randn((B, S, HK, D[0]), generator=g, device="cuda").bfloat16()
    v = torch.randn((B, S, HK, D[1]), generator=g, device="cuda").bfloat16()
    w = torch.rand((B, HK, S), generator=g, device="cuda")
    lens = torch.randint(S // 2, S + 1, (B,), generator=g, device="cuda").int()
    return g, k, v, w, lens


# sizes that are no multiple of a sector or line, in every way that a row is selected and copied
CHAINS = {
    "one_cache": dict(B=1, S=333, HK=3, D=D64, budget=111, again=57),
    "batch": dict(B=5, S=1021, HK=3, D=D128, budget=401, again=77),
    "own_copies": dict(B=37, S=517, HK=4, D=D128, budget=201, again=99),
    "spread_rows": dict(B=2, S=33001, HK=2, D=D64, budget=9001, again=4003),
    "longer_than_registers": dict(B=1, S=150001, HK=1, D=D64, budget=20011, again=3001),
    "d192": dict(B=3, S=2049, HK=2, D=D192, budget=1023, again=511),
    "d256": dict(B=3, S=1537, HK=2, D=D256, budget=1537, again=1),
}


@pytest.mark.parametrize("name", CHAINS)
def test_decode_then_evict_then_evict_again(name):
    import torch
    import index_sparse_attention_b200 as sa
    c = CHAINS[name]
    g, k, v, w0, lens = _caches(c["B"], c["S"], c["HK"], c["D"], seed=9)
    qs = [torch.randn((c["B"], 1, 2 * c["HK"], c["D"][0]), generator=g, device="cuda").bfloat16()
          for _ in range(12)]

    def chain(q, wait):
        w = w0.clone()
        out = list(sa.cache_attn_fwd(q, k, v, lens, weights=w, weights_out=w))
        wait()
        a = sa.cache_evict(k, v, w, lens, c["budget"], sinks=1, recent=0,
                           k_out=torch.zeros_like(k), v_out=torch.zeros_like(v))
        wait()
        b = sa.cache_evict(a[0], a[1], a[2], a[3], c["again"], recent=1,
                           k_out=torch.zeros_like(k), v_out=torch.zeros_like(v))
        wait()
        return [*out, *a, *b]

    for q in qs:
        torch.cuda.synchronize()
        got = chain(q, lambda: None)
        want = chain(q, torch.cuda.synchronize)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("Sq", [129, 1000])
def test_key_weights_then_evict(Sq):
    """Weights of a prompt that the eviction behind them reads."""
    import torch
    import index_sparse_attention_b200 as sa
    B, S, HK, HQ = 2, 1027, 2, 8
    g, k, v, _, _ = _caches(B, S, HK, D128, seed=19)
    lens = torch.full((B,), S, dtype=torch.int32, device="cuda")
    lists = sa.block_mask_to_block_sparse(None, B, HK, Sq, S)
    qs = [torch.randn((B, Sq, HQ, 128), generator=g, device="cuda").bfloat16() for _ in range(12)]

    def chain(q, wait):
        o, lse = sa.sparse_attn_fwd(q, k, v, lists)
        wait()
        w = sa.sparse_attn_key_weights(q, k, lse, lists)
        wait()
        a = sa.cache_evict(k, v, w, lens, 301, sinks=1, recent=3, k_out=torch.zeros_like(k),
                           v_out=torch.zeros_like(v))
        wait()
        return [o, lse, w, *a]

    for q in qs:
        torch.cuda.synchronize()
        got = chain(q, lambda: None)
        want = chain(q, torch.cuda.synchronize)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("D", [D64, D128, D192, D256], ids=str)
def test_key_weights_of_the_token_that_cache_attn_fwd_decoded(D):
    """cache_attn_fwd's lse is read by sparse_attn_key_weights as soon as it is joined; the weights
    are those that cache_attn_fwd gives itself, to the rounding of both."""
    import torch
    import index_sparse_attention_b200 as sa
    B, S, HK, HQ = 3, 1027, 2, 8
    g, k, v, _, _ = _caches(B, S, HK, D, seed=29)
    lens = torch.full((B,), S, dtype=torch.int32, device="cuda")
    lists = sa.block_mask_to_block_sparse(None, B, HK, 1, S)
    qs = [torch.randn((B, 1, HQ, D[0]), generator=g, device="cuda").bfloat16() for _ in range(20)]
    torch.cuda.synchronize()
    got = []
    for q in qs:
        _, lse = sa.cache_attn_fwd(q, k, v, lens)
        got.append(sa.sparse_attn_key_weights(q, k, lse, lists))
    torch.cuda.synchronize()
    for q, w in zip(qs, got):
        o, lse, own = sa.cache_attn_fwd(q, k, v, lens, with_weights=True)
        torch.cuda.synchronize()
        assert torch.equal(w, sa.sparse_attn_key_weights(q, k, lse, lists))
        # two computations of a score less its lse, each off by twice score_bound of cache_ref.py
        # (s: the largest sum of a score's terms), two exponentials and the additions of four heads
        s = (D[0] ** -0.5 * torch.einsum("bqhd,bsgd->bhgs", q.double().abs(),
                                         k.double().abs())).max().item()
        rel = 2 * ((D[0] + 8) * 2.0 ** -24 * s + 2.0 ** -20 + 2.0 ** -22 * s) + 2.0 ** -20
        assert ((w - own).abs().double() <= 2 * rel * own.double()).all()


def test_all_calls_in_one_captured_graph_with_branches():
    """Forward, key weights, two decodes at once, evictions one behind another, with other kernels
    and branches that join between them: replays give what the same calls gave uncaptured."""
    import torch
    import index_sparse_attention_b200 as sa
    B, S, HQ, HK = 3, 700, 8, 2
    g, k, v, _, _ = _caches(B, S, HK, D128, seed=39)
    lens = torch.full((B,), S, dtype=torch.int32, device="cuda")
    q1 = torch.randn((B, 1, HQ, 128), generator=g, device="cuda").bfloat16()
    q = torch.randn((B, S, HQ, 128), generator=g, device="cuda").bfloat16()
    lists = sa.block_mask_to_block_sparse(None, B, HK, S, S)

    def body(side):
        cur = torch.cuda.current_stream()

        def fork(f):
            side.wait_stream(cur)
            with torch.cuda.stream(side):
                return f()

        k2, n = fork(lambda: (k * 1.0, lens.clone()))
        v2 = v * 1.0
        cur.wait_stream(side)
        _, lse = sa.sparse_attn_fwd(q, k2, v2, lists)
        q2 = fork(lambda: q * 1.0)
        k3 = k2 * 1.0
        cur.wait_stream(side)
        w = sa.sparse_attn_key_weights(q2, k3, lse, lists)
        a = fork(lambda: sa.cache_attn_fwd(q1, k2, v2, n))
        b = sa.cache_attn_fwd(q1, k3, v2, n, weights=w, with_weights=True)
        cur.wait_stream(side)
        c = sa.cache_evict(k2, v2, b[2], n, 100, sinks=3, recent=5, k_out=torch.zeros_like(k),
                           v_out=torch.zeros_like(v))
        d = fork(lambda: sa.cache_evict(*c[:4], 50, k_out=torch.zeros_like(k),
                                        v_out=torch.zeros_like(v)))
        cur.wait_stream(side)
        return [w, *a, *b, *c, *d]

    want = body(torch.cuda.Stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = body(torch.cuda.Stream())
    for _ in range(10):
        for x in out:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_the_most_sequences_and_heads_for_weights_and_eviction():
    """65535 sequences, and 65535 KV heads of one sequence."""
    import torch
    import index_sparse_attention_b200 as sa
    S, D, budget = 5, 64, 3
    for B, HK in ((65535, 1), (1, 65535)):
        g, k, v, w, lens = _caches(B, S, HK, D64, seed=49)
        ko, vo, wo, lo, keep = sa.cache_evict(k, v, w, lens, budget, sinks=1,
                                              k_out=torch.zeros_like(k), v_out=torch.zeros_like(v))
        at = torch.arange(S, device="cuda")
        rank = w.clone()
        rank[..., 0] = 2.0
        rank = rank.masked_fill(at >= lens[:, None, None], -1.0)
        best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
        best = torch.where(best < lens[:, None, None], best, S).sort(dim=-1).values
        assert torch.equal(keep, torch.where(best < S, best, -1).int())
        assert torch.equal(lo, lens.clamp(max=budget))
        rows = best.clamp(max=S - 1).transpose(1, 2)[..., None].expand(-1, -1, -1, D)
        live = (best < S).transpose(1, 2)[..., None]
        for x, y in ((ko, k), (vo, v)):
            assert torch.equal(x[:, :budget], torch.where(live, y.gather(1, rows), 0))
        lists = sa.block_mask_to_block_sparse(None, B, HK, 2, S)
        q = torch.randn((B, 2, HK, D), generator=g, device="cuda").bfloat16()
        _, lse = sa.sparse_attn_fwd(q, k, v, lists)
        got = sa.sparse_attn_key_weights(q, k, lse, lists)
        s = torch.einsum("bqhd,bshd->bhqs", q.double(), k.double()) / 8
        size = torch.einsum("bqhd,bshd->bhqs", q.double().abs(), k.double().abs()).max() / 8
        ref = (s - lse.double()[..., None]).exp().sum(2)
        # (the bounds of cache_ref.py)
        rel = 2 * ((D + 8) * 2.0 ** -24 * size + 2.0 ** -20 + 2.0 ** -22 * size)
        rel = rel + 2.0 ** -22 * lse.abs().max().double() + 130 * 2.0 ** -24
        assert ((got.double() - ref).abs() <= rel * ref).all()
