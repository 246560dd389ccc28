"""sparse_attn_key_weights where queries or keys hold no numbers: padded queries (lse -inf) with
anything in them, rows behind a ragged end beside an infinite key."""
import numpy as np
import pytest

import cache_ref as R
from index_sparse_attention_b200 import inputs as I

from helpers import bf16_to_f64, build_lists, to_gpu
from test_gpu_key_weights import GQA, IDX, W, _compare, allowed_of

pytestmark = pytest.mark.gpu

CASES = [
    I.scaled(W["blocksparse_mha_s256_d64"], Sq=390, Sk=400, density=0.8, name="block64_d64"),
    I.scaled(GQA, B=2, Sq=520, Sk=520, HQ=8, HK=2, density=0.6, name="causal_d128"),
    I.scaled(GQA, B=2, Sq=400, Sk=700, HQ=8, HK=2, causal=False, density=1.0, name="full_d128"),
    I.scaled(GQA, B=1, Sq=300, Sk=500, HQ=8, HK=2, Dqk=256, Dv=256, causal=False, density=1.0,
             name="full_d256"),
    I.scaled(GQA, B=1, Sq=1400, Sk=1400, HQ=32, HK=4, Dqk=64, Dv=64, causal=False, density=1.0,
             name="many_tiles_d64"),
    I.scaled(IDX, Sq=300, Sk=700, HQ=8, HK=2, topk=90, span="all", causal=False, name="index_d192"),
]


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 3e38], ids=str)
@pytest.mark.parametrize("w", CASES, ids=[w.name for w in CASES])
def test_padded_queries_add_nothing_whatever_they_hold(w, fill):
    """The second half of each batch's queries less a few, and some in the middle of a tile, have
    no lse: the weights are those of the others, as if the lists did not name them."""
    import torch
    import index_sparse_attention_b200 as sa
    inp = I.make_inputs(w, with_grad=False)
    g = to_gpu(inp)
    bsp = build_lists(inp, g)
    _, lse = sa.sparse_attn_fwd(g["q"], g["k"], g["v"], bsp, w.scale)
    pad = np.zeros((w.B, w.Sq), bool)
    pad[:, 3] = pad[:, 40:45] = True
    for b in range(w.B):
        pad[b, w.Sq // 2 + 7 * b:] = True
    at = torch.from_numpy(pad).cuda()
    lse.masked_fill_(at[:, None], -float("inf"))
    q = bf16_to_f64(g["q"])
    q[pad] = 0.0
    g["q"][at] = fill
    got = sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp, w.scale)
    ref, tol = R.key_weights(q, bf16_to_f64(g["k"]), lse.double().cpu().numpy(),
                             allowed_of(w, inp), w.scale)
    _compare(got, ref, tol)


@pytest.mark.parametrize("w", CASES, ids=[w.name for w in CASES])
def test_a_key_that_no_query_weighs(w):
    """An infinite component turns a key's scores to -inf: no weight, however ragged the end of the
    queries is; the other keys' weights are right."""
    import torch
    import index_sparse_attention_b200 as sa
    inp = I.make_inputs(w, with_grad=False)
    g = to_gpu(inp)
    g["q"][..., 3] = g["q"][..., 3].abs() + 0.5
    bsp = build_lists(inp, g)
    k = bf16_to_f64(g["k"])
    g["k"][:, 5, :, 3] = -float("inf")
    _, lse = sa.sparse_attn_fwd(g["q"], g["k"], g["v"], bsp, w.scale)
    got = sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp, w.scale)
    assert (got[:, :, 5] == 0).all()
    allowed = allowed_of(w, inp)
    allowed[..., 5] = False
    ref, tol = R.key_weights(bf16_to_f64(g["q"]), k, lse.double().cpu().numpy(), allowed, w.scale)
    _compare(got, ref, tol)


@pytest.mark.parametrize("limit", [100, 1000, 3000, 10000, 30000, 100000])
@pytest.mark.parametrize("w", [CASES[4], CASES[5]], ids=lambda w: w.name)
def test_a_call_given_up_ends_when_its_copies_have_landed(w, limit):
    """Whatever state a CTA gives up in, it waits for its own loads and no longer: a wait for an
    arrival that nobody makes would take the two seconds of its limit."""
    import torch
    import index_sparse_attention_b200 as sa
    inp = I.make_inputs(w, with_grad=False)
    g = to_gpu(inp)
    bsp = build_lists(inp, g)
    _, lse = sa.sparse_attn_fwd(g["q"], g["k"], g["v"], bsp, w.scale)
    want = sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp, w.scale)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    try:
        sa.sparse_attn_set_wait_limit_ns(limit)
        start.record()
        for _ in range(10):
            sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp, w.scale)
        end.record()
        torch.cuda.synchronize()
    finally:
        sa.sparse_attn_set_wait_limit_ns(0)
    assert start.elapsed_time(end) < 500
    assert torch.equal(sa.sparse_attn_key_weights(g["q"], g["k"], lse, bsp, w.scale), want)
