"""sparse_attn_key_weights against its 64-bit reference in every mode and head-dim pair, with the
lse of sparse_attn_fwd: partial tiles, rows that see no key, repeated indices, splits of the query
range, sums continued from earlier ones."""
import numpy as np
import pytest

import cache_ref as R
from index_sparse_attention_b200 import _lib
from index_sparse_attention_b200 import inputs as I

from helpers import bf16_to_f64, build_lists, to_gpu

pytestmark = pytest.mark.gpu

W = I.WORKLOADS
IDX = W["indexsparse_gqa_q16384_hq32_hk4_d192_128_top2048"]
GQA = W["gqa_blocksparse_b2_hq32_hk8_s8192_d128"]
CASES = [
    I.scaled(W["blocksparse_mha_s256_d64"], name="block64_d64"),
    I.scaled(W["blocksparse_mha_s256_d64"], Sq=200, Sk=331, causal=True, name="block64_odd_causal"),
    I.scaled(W["blocksparse_mha_s256_d64"], Sq=1, Sk=1, HQ=1, HK=1, name="one_by_one"),
    I.scaled(GQA, B=2, Sq=520, Sk=520, HQ=8, HK=2, density=0.4, name="gqa_causal_d128"),
    I.scaled(GQA, B=1, Sq=64, Sk=1500, HQ=12, HK=4, causal=False, density=1.0, name="few_queries"),
    I.scaled(GQA, B=1, Sq=1, Sk=700, HQ=4, HK=1, causal=False, density=1.0, name="one_query"),
    I.scaled(GQA, B=1, Sq=1500, Sk=100, HQ=6, HK=1, causal=False, density=1.0, name="split_queries"),
    I.scaled(GQA, B=1, Sq=700, Sk=700, HQ=4, HK=4, Dqk=128, bs=64, density=0.5, name="block64_d128"),
    I.scaled(IDX, Sq=520, Sk=520, HQ=8, HK=1, topk=64, name="index_d192"),
    I.scaled(IDX, Sq=300, Sk=700, HQ=8, HK=2, topk=90, span="all", causal=False, dup=0.3,
             name="index_dup_d192"),
    I.scaled(IDX, B=2, Sq=257, Sk=257, HQ=4, HK=2, Dqk=64, Dv=64, topk=40, name="index_d64"),
    I.scaled(IDX, Sq=200, Sk=200, HQ=4, HK=2, Dqk=256, Dv=256, topk=40, name="index_d256"),
    I.scaled(W["long_causal_blocksparse_h16_s32768_d256"], Sq=600, Sk=600, HQ=4, HK=4, density=0.5,
             name="causal_d256"),
    # many tiles for every SM
    I.scaled(GQA, B=1, Sq=1400, Sk=1400, HQ=32, HK=4, density=0.7, name="many_tiles_d128"),
    I.scaled(GQA, B=1, Sq=1409, Sk=1300, HQ=32, HK=4, Dqk=64, Dv=64, density=0.7,
             name="many_tiles_d64"),
    I.scaled(GQA, B=1, Sq=1400, Sk=1400, HQ=32, HK=4, Dqk=192, density=0.7,
             name="many_tiles_d192"),
    I.scaled(GQA, B=1, Sq=1400, Sk=1401, HQ=32, HK=8, Dqk=256, Dv=256, density=0.7, causal=False,
             name="many_tiles_d256"),
    I.scaled(IDX, Sq=1401, Sk=1401, HQ=32, HK=4, Dqk=128, topk=200, name="index_many_tiles_d128"),
    I.scaled(IDX, Sq=1401, Sk=1401, HQ=32, HK=4, topk=200, name="index_many_tiles_d192"),
    # many key tiles of one query tile each, or of none
    I.scaled(GQA, B=4, Sq=100, Sk=1500, HQ=8, HK=8, causal=False, density=1.0, name="short_lists"),
    I.scaled(GQA, B=2, Sq=130, Sk=3001, HQ=4, HK=4, causal=False, density=0.2, name="empty_lists"),
    I.scaled(GQA, B=2, Sq=257, Sk=6000, HQ=5, HK=5, Dqk=256, Dv=256, causal=False, density=0.5,
             name="short_lists_d256"),
]


def allowed_of(w, inp):
    a = np.zeros((w.B, w.HK, w.Sq, w.Sk), bool)
    i, j = np.arange(w.Sq), np.arange(w.Sk)
    if w.mode == "block":
        a[:] = inp.mask[:, :, i // w.bs][:, :, :, j // w.bs].astype(bool)
    else:
        for b, q, h in np.ndindex(w.B, w.Sq, w.HK):
            row = inp.idx[b, q, h]
            a[b, h, q, row[row >= 0]] = True
    if w.causal:
        a &= j[None, :] <= i[:, None]
    return a


def _run(w, empty_rows=()):
    import torch
    import index_sparse_attention_b200 as sa
    inp = I.make_inputs(w, with_grad=False)
    if empty_rows:
        inp.idx[:, list(empty_rows)] = -1
    g = to_gpu(inp)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsp = build_lists(inp, g, dev_status=status)
    _, lse = sa.sparse_attn_fwd(g["q"], g["k"], g["v"], bsp, w.scale, dev_status=status)
    got = sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp, w.scale, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    ref, tol = R.key_weights(bf16_to_f64(g["q"]), bf16_to_f64(g["k"]),
                             lse.double().cpu().numpy(), allowed_of(w, inp), w.scale)
    return g, bsp, lse, got, ref, tol


def _compare(got, ref, tol):
    x = got.double().cpu().numpy()
    assert np.isfinite(x).all()
    over = np.abs(x - ref) - tol
    assert over.max() <= 0, f"{over.max():.3e} over its bound"


@pytest.mark.parametrize("w", CASES, ids=[w.name for w in CASES])
def test_matches_the_reference(w):
    import torch
    import index_sparse_attention_b200 as sa
    g, bsp, lse, got, ref, tol = _run(w)
    _compare(got, ref, tol)
    # every query that sees a key hands out a total weight of one per head
    total = np.isfinite(lse.cpu().numpy()).sum()
    assert abs(got.double().sum().item() - total) <= 1e-3 * total
    # the same bits again; continued from earlier sums, in place too
    again = sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp, w.scale)
    assert torch.equal(got, again)
    start = torch.rand_like(got)
    out = sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp, w.scale, weights=start)
    assert torch.equal(out, start + got)
    sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp, w.scale, weights=start, weights_out=start)
    assert torch.equal(out, start)


def test_rows_without_keys_add_nothing():
    w = I.scaled(IDX, Sq=300, Sk=300, HQ=8, HK=1, topk=64, name="empty_rows")
    _, _, lse, got, ref, tol = _run(w, empty_rows=(0, 17, 128, 299))
    assert np.isneginf(lse.cpu().numpy()[:, :, [0, 17, 128, 299]]).all()
    _compare(got, ref, tol)


def test_dense_lists_without_a_mask():
    import torch
    import index_sparse_attention_b200 as sa
    w = I.scaled(GQA, B=2, Sq=333, Sk=444, HQ=4, HK=2, name="dense")
    inp = I.make_inputs(w, with_grad=False)
    g = to_gpu(inp)
    bsp = sa.block_mask_to_block_sparse(None, 2, 2, 333, 444, causal=True)
    _, lse = sa.sparse_attn_fwd(g["q"], g["k"], g["v"], bsp)
    got = sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp)
    a = np.broadcast_to(np.arange(444)[None] <= np.arange(333)[:, None], (2, 2, 333, 444))
    ref, tol = R.key_weights(bf16_to_f64(g["q"]), bf16_to_f64(g["k"]), lse.double().cpu().numpy(),
                             a, w.scale)
    _compare(got, ref, tol)
    assert (got[:, :, 333:] == 0).all()


@pytest.mark.parametrize("w", [CASES[3], CASES[8], CASES[12]], ids=lambda w: w.name)
def test_short_wait_limit_reports_timeout_then_recovers(w):
    import torch
    import index_sparse_attention_b200 as sa
    g, bsp, lse, got, ref, tol = _run(w)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        sa.sparse_attn_set_wait_limit_ns(300)
        sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp, w.scale, dev_status=status)
        torch.cuda.synchronize()
    finally:
        sa.sparse_attn_set_wait_limit_ns(0)
    assert int(status.item()) & _lib.STATUS_TIMEOUT
    status.zero_()
    again = sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp, w.scale, dev_status=status)
    assert int(status.item()) == 0 and torch.equal(again, got)


def test_other_stream_and_graph_replay():
    import torch
    import index_sparse_attention_b200 as sa
    g, bsp, lse, got, ref, tol = _run(CASES[3])
    q, k = g["q"], g["k"]
    side = torch.cuda.Stream()
    out = torch.full_like(got, float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sa.sparse_attn_key_weights(q, k, lse, bsp, CASES[3].scale, weights_out=out)
    side.synchronize()
    assert torch.equal(out, got)
    qs, ls = torch.zeros_like(q), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.sparse_attn_key_weights(qs, k, ls, bsp, CASES[3].scale, weights_out=out)
    for _ in range(2):
        qs.copy_(q)
        ls.copy_(lse)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got)


def test_offsets_beyond_32_bits():
    """Q of 2^32 elements: the last query tile of the second batch is found."""
    import torch
    import index_sparse_attention_b200 as sa
    B, Sq, HQ, HK, D, Sk = 2, 1 << 18, 32, 4, 256, 200
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    rng = np.random.default_rng(5)
    q = torch.zeros((B, Sq, HQ, D), dtype=torch.bfloat16, device="cuda")
    rows = [*range(64), *range(Sq - 128, Sq)]
    few = torch.from_numpy(rng.standard_normal((B, len(rows), HQ, D)).astype(np.float32))
    q[:, rows] = few.bfloat16().cuda()
    k = torch.from_numpy(rng.standard_normal((B, Sk, HK, D)).astype(np.float32)).bfloat16().cuda()
    mask = np.zeros((B, HK, Sq // 128, 2), np.uint8)
    mask[:, :, 0, 0] = mask[:, :, -1] = 1
    bsp = sa.block_mask_to_block_sparse(torch.from_numpy(mask).cuda(), B, HK, Sq, Sk, bs=128)
    rows = [*range(128), *range(Sq - 128, Sq)]
    allowed = np.zeros((B, HK, 256, Sk), bool)
    allowed[:, :, :128, :128] = allowed[:, :, 128:] = True
    qr = q[:, rows].double().unflatten(2, (HK, -1))
    s = torch.einsum("bqghd,bkgd->bghqk", qr, k.double()) * D ** -0.5
    s = s.masked_fill(~torch.from_numpy(allowed).cuda()[:, :, None], float("-inf"))
    lse = torch.full((B, HQ, Sq), float("-inf"), device="cuda")
    lse[:, :, rows] = s.logsumexp(-1).flatten(1, 2).float()
    got = sa.sparse_attn_key_weights(q, k, lse, bsp)
    ref, tol = R.key_weights(bf16_to_f64(q[:, rows].contiguous()), bf16_to_f64(k),
                             lse[:, :, rows].double().cpu().numpy(), allowed, D ** -0.5)
    _compare(got, ref, tol)
