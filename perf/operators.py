"""Cases of the cache operators: attention of one new token per sequence over a shared prefix and
each sequence's own cache (cache_attn_fwd), the attention weight every key has received
(sparse_attn_key_weights) and eviction from the cache by that weight (cache_evict).

``run`` computes a case in elementary torch operations, or with ``own`` set through the package's
entry points; ``exact`` computes it in 64 bits from the definitions.
"""
import math

import torch

own = False

DIMS = ((64, 64), (128, 128), (192, 128), (256, 256))


def listed():
    attn = dict(op="attn", weights=False)
    wts = dict(op="weights", topk=0, density=1.0, causal=False)
    evict = dict(op="evict")
    return [
        # one short sequence at the smallest head size: a call's latency
        dict(attn, name="attn_b1_h2_d64_len256", B=1, HQ=2, HK=2, Dqk=64, Dv=64, P=0, S=256),
        # one long conversation alone on the GPU: all SMs share one sequence's heads
        dict(attn, name="attn_b1_hq32_hk8_d128_len16384", B=1, HQ=32, HK=8, Dqk=128, Dv=128, P=0,
             S=16384),
        # a system prompt of 8192 tokens under 16 conversations of odd lengths, weights kept up
        dict(attn, name="attn_b16_p8192_s2049_d128_weights", weights=True, B=16, HQ=32, HK=8,
             Dqk=128, Dv=128, P=8192, S=2049),
        # the index workload's heads over a document that 32 questions share
        dict(attn, name="attn_b32_p16384_s1024_d192_128_weights", weights=True, B=32, HQ=32, HK=4,
             Dqk=192, Dv=128, P=16384, S=1024),
        # wide heads, one query head per KV head, ragged prefix
        dict(attn, name="attn_b8_h16_p4097_s777_d256", B=8, HQ=16, HK=16, Dqk=256, Dv=256, P=4097,
             S=777),
        # a full serving batch behind a long shared prompt
        dict(attn, name="attn_b64_p32768_s4096_d128", B=64, HQ=32, HK=8, Dqk=128, Dv=128, P=32768,
             S=4096),
        # the weights of a dense causal prompt
        dict(wts, name="weights_causal_b2_h16_s4096_d128", mode="dense", causal=True, B=2, Sq=4096,
             Sk=4096, HQ=16, HK=16, Dqk=128, Dv=128),
        # of a block-sparse prompt with shared KV heads
        dict(wts, name="weights_gqa_blocksparse_hq32_hk8_s8192_d128", mode="block", causal=True,
             density=0.25, B=1, Sq=8192, Sk=8192, HQ=32, HK=8, Dqk=128, Dv=128),
        # of an index-sparse prompt of odd length
        dict(wts, name="weights_index_hq32_hk4_s4001_d192_128", mode="index", causal=True, topk=512,
             B=1, Sq=4001, Sk=4001, HQ=32, HK=4, Dqk=192, Dv=128),
        # one small cache, as after each answer of a conversation
        dict(evict, name="evict_b1_hk8_s4096_to_1024_d128", B=1, HK=8, Dqk=128, Dv=128, S=4096,
             budget=1024, sinks=4, recent=128),
        # a batch of caches of odd lengths, some of them below the budget
        dict(evict, name="evict_b16_hk8_s8191_to_2048_d128", B=16, HK=8, Dqk=128, Dv=128, S=8191,
             budget=2048, sinks=4, recent=257),
        # long contexts cut to an eighth
        dict(evict, name="evict_b8_hk4_s65536_to_8192_d192_128", B=8, HK=4, Dqk=192, Dv=128,
             S=65536, budget=8192, sinks=16, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attn", "weights", "evict"))
    Dqk, Dv = rng.choice(DIMS)
    if op == "attn":
        while True:
            HK = rng.choice((1, 2, 4, 8, 16))
            c = dict(op=op, weights=rng.random() < 0.5, B=_log(rng, 1, 64),
                     HQ=HK * rng.choice((1, 2, 3, 4, 6, 8)), HK=HK, Dqk=Dqk, Dv=Dv,
                     P=rng.choice((0, _log(rng, 16, 32768))), S=_log(rng, 16, 16384))
            w = work(c)
            if w["bytes"] <= 1.0e9 and w["flops"] <= 4e10:
                return c
    if op == "weights":
        mode = rng.choice(("dense", "block", "index"))
        while True:
            HK = rng.choice((1, 2, 4, 8, 16))
            Sq = _log(rng, 64, 8192)
            c = dict(op=op, mode=mode, topk=_log(rng, 16, 1024) if mode == "index" else 0,
                     density=rng.uniform(0.1, 0.9) if mode == "block" else 1.0,
                     causal=rng.random() < 0.6, B=rng.choice((1, 1, 2, 3)), Sq=Sq, Sk=Sq,
                     HQ=HK * rng.choice((1, 2, 3, 4, 8)), HK=HK, Dqk=Dqk, Dv=Dv)
            if rng.random() < 0.3:  # the last queries alone look back over all keys
                c.update(Sq=_log(rng, 1, 256), causal=False)
            # the plain form holds every score at once
            if c["B"] * c["HQ"] * c["Sq"] * c["Sk"] <= 1 << 30:
                return c
    while True:
        S = _log(rng, 64, 65536)
        budget = max(1, int(S * rng.uniform(0.05, 1.0)))
        c = dict(op=op, B=_log(rng, 1, 32), HK=rng.choice((1, 2, 4, 8, 16)), Dqk=Dqk, Dv=Dv, S=S,
                 budget=budget, sinks=min(budget // 4, rng.choice((0, 1, 4, 16))),
                 recent=int(budget * rng.uniform(0.0, 0.5)))
        if c["B"] * S * c["HK"] * (Dqk + Dv) <= 1 << 30 and work(c)["bytes"] <= 4e8:
            return c


def _lens(c):
    """The lengths of a case's sequences, sorted: spread over the upper half of the capacity, the
    last one filling it; with many sequences also a few short ones."""
    B, S = c["B"], c["S"]
    lens = [max(1, S - (S // 2) * i // max(1, B)) for i in range(B)]
    if B >= 8:
        lens[-1] = max(1, S // 16)
    return sorted(lens)


def _tiles(c):
    """Expected active 128 x 128 tiles of one (batch, query head) of a weights case."""
    tm, tn = -(-c["Sq"] // 128), -(-c["Sk"] // 128)
    n = 0.0
    for m in range(tm):
        other = min(m, tn) if c["causal"] else tn - (1 if m < tn else 0)
        n += (1 if m < tn else 0) + c["density"] * other
    return n


def work(case):
    c = case
    d = c["Dqk"] + c["Dv"]
    if c["op"] == "attn":
        keys = sum(_lens(c))
        by = 2 * c["HK"] * d * (keys + c["P"]) + 2 * c["B"] * c["HQ"] * d + 4 * c["B"] * c["HQ"]
        if c["weights"]:
            by += 8 * c["HK"] * c["B"] * c["S"]
        return {"bytes": by, "flops": 2 * c["HQ"] * d * (keys + c["B"] * c["P"])}
    if c["op"] == "weights":
        by = (2 * c["Dqk"] * c["B"] * (c["Sq"] * c["HQ"] + c["Sk"] * c["HK"])
              + 4 * c["B"] * (c["HQ"] * c["Sq"] + c["HK"] * c["Sk"]))
        if c["mode"] == "index":
            pairs = sum(min(c["topk"], q + 1 if c["causal"] else c["Sk"]) for q in range(c["Sq"]))
            by += c["B"] * c["HK"] * c["Sq"] * c["Sk"] // 8  # the presence bitmap of the lists
        elif c["mode"] == "block":
            pairs = _tiles(c) * 128 * 128
        else:
            pairs = c["Sq"] * (c["Sk"] + 1) / 2 if c["causal"] else c["Sq"] * c["Sk"]
        return {"bytes": by, "flops": 2 * c["B"] * c["HQ"] * pairs * c["Dqk"]}
    kept = sum(min(n, c["budget"]) for n in _lens(c))
    by = c["HK"] * (4 * kept * d + 4 * sum(_lens(c)) + 4 * c["B"] * c["S"] + 4 * c["B"] * c["budget"])
    return {"bytes": by, "flops": 0}


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(c=c, scale=1.0 / math.sqrt(c["Dqk"]))
    B, HK, Dqk, Dv = c["B"], c["HK"], c["Dqk"], c["Dv"]
    if c["op"] in ("attn", "evict"):
        order = torch.randperm(B, generator=g, device="cuda")
        st["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")[order].contiguous()
        st["k"], st["v"] = _normal(g, B, c["S"], HK, Dqk), _normal(g, B, c["S"], HK, Dv)
        # what keys have received so far: a few heavy ones, many light ones, some none at all
        w = torch.exp(2.0 * torch.randn((B, HK, c["S"]), generator=g, device="cuda") - 3.0)
        w *= torch.rand(w.shape, generator=g, device="cuda") < 0.9
        w *= (torch.arange(c["S"], device="cuda") < st["lens"][:, None, None])
        st["weights"] = w
    if c["op"] == "attn":
        st["q"] = _normal(g, B, 1, c["HQ"], Dqk)
        if c["P"]:
            st["kp"], st["vp"] = _normal(g, c["P"], HK, Dqk), _normal(g, c["P"], HK, Dv)
    elif c["op"] == "evict":
        # the second buffer of a cache that is compacted from one into the other
        st["k_out"], st["v_out"] = torch.zeros_like(st["k"]), torch.zeros_like(st["v"])
    else:
        Sq, Sk, G = c["Sq"], c["Sk"], c["HQ"] // HK
        st["q"], st["k"] = _normal(g, B, Sq, c["HQ"], Dqk), _normal(g, B, Sk, HK, Dqk)
        if c["mode"] == "block":
            mb, nb = -(-Sq // 128), -(-Sk // 128)
            m = torch.rand((B, HK, mb, nb), generator=g, device="cuda") < c["density"]
            m |= torch.eye(mb, nb, dtype=torch.bool, device="cuda")
            st["mask"] = m.to(torch.uint8)
        elif c["mode"] == "index":
            # each query's `topk` distinct keys among those it may see, -1 behind the last one
            top = min(c["topk"], Sk)
            idx = torch.full((B, Sq, HK, c["topk"]), -1, dtype=torch.int32, device="cuda")
            reach = torch.arange(Sq, device="cuda")[:, None, None] if c["causal"] else Sk
            for b in range(B):
                u = torch.rand((Sq, HK, Sk), generator=g, device="cuda")
                u.masked_fill_(torch.arange(Sk, device="cuda") > reach, -1.0)
                best = u.topk(top, dim=-1)
                idx[b, :, :, :top] = torch.where(best.values >= 0, best.indices, -1).int()
            st["idx"] = idx
        # the forward's log-sum-exp, which the program has from the prompt's pass
        lse = torch.empty((B, c["HQ"], Sq), device="cuda")
        allowed = _allowed(st)
        for b in range(B):
            for h in range(c["HQ"]):
                s = st["q"][b, :, h].float() @ st["k"][b, :, h // G].float().T * st["scale"]
                if allowed is not None:
                    s.masked_fill_(~allowed[b % allowed.shape[0], (h // G) % allowed.shape[1]],
                                   -math.inf)
                lse[b, h] = torch.logsumexp(s, -1)
        st["lse"] = lse
        if own:  # the lists that the prompt's forward ran on
            import index_sparse_attention_b200 as sa
            if c["mode"] == "index":
                st["lists"] = sa.index_to_block_sparse(st["idx"], Sk, causal=c["causal"])
            else:
                st["lists"] = sa.block_mask_to_block_sparse(st.get("mask"), B, HK, Sq, Sk,
                                                            causal=c["causal"])
    return st


def _allowed(st):
    """Which keys each query may see: bool, broadcastable to [B, HK, Sq, Sk]; None for all."""
    c = st["c"]
    Sq, Sk = c["Sq"], c["Sk"]
    a = None
    if c["mode"] == "block":
        a = st["mask"].bool().repeat_interleave(128, 2).repeat_interleave(128, 3)[:, :, :Sq, :Sk]
    elif c["mode"] == "index":
        at = torch.where(st["idx"] < 0, Sk, st["idx"]).long().transpose(1, 2)
        a = torch.zeros((c["B"], c["HK"], Sq, Sk + 1), dtype=torch.bool, device=at.device)
        a = a.scatter_(3, at, True)[..., :Sk]
    if c["causal"]:
        tri = (torch.arange(Sk, device="cuda") <= torch.arange(Sq, device="cuda")[:, None])[None, None]
        a = tri if a is None else a & tri
    return a


def _plain_attn(st):
    c = st["c"]
    B, HQ, HK = c["B"], c["HQ"], c["HK"]
    G = HQ // HK
    q = st["q"].float().reshape(B, HK, G, c["Dqk"]) * st["scale"]
    k, v = st["k"].float().transpose(1, 2), st["v"].float().transpose(1, 2)  # [B, HK, S, D]
    s = q @ k.transpose(2, 3)  # [B, HK, G, S]
    behind = torch.arange(c["S"], device=s.device) >= st["lens"][:, None, None, None]
    s = s.masked_fill(behind, -math.inf)
    if c["P"]:
        kp, vp = st["kp"].float().transpose(0, 1), st["vp"].float().transpose(0, 1)
        rows = q.transpose(0, 1).reshape(HK, B * G, c["Dqk"])  # every sequence's heads at once
        sp = (rows @ kp.transpose(1, 2)).reshape(HK, B, G, c["P"]).transpose(0, 1)
        s = torch.cat([sp, s], -1)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    p = p / total
    pc = p[..., c["P"]:]
    o = pc @ v
    if c["P"]:
        pp = p[..., :c["P"]].transpose(0, 1).reshape(HK, B * G, c["P"])
        o = o + (pp @ vp).reshape(HK, B, G, c["Dv"]).transpose(0, 1)
    o = o.reshape(B, 1, HQ, c["Dv"]).bfloat16()
    lse = (m + torch.log(total)).reshape(B, HQ, 1)
    return (o, lse, st["weights"] + pc.sum(2)) if c["weights"] else (o, lse)


def _plain_weights(st):
    c = st["c"]
    B, HK = c["B"], c["HK"]
    G = c["HQ"] // HK
    q = st["q"].float().transpose(1, 2).reshape(B, HK, G * c["Sq"], c["Dqk"])
    k = st["k"].float().permute(0, 2, 3, 1)
    p = (q @ k).reshape(B, HK, G, c["Sq"], c["Sk"])
    p.mul_(st["scale"]).sub_(st["lse"].reshape(B, HK, G, c["Sq"], 1)).exp_()
    allowed = _allowed(st)
    if allowed is not None:
        p.masked_fill_(~allowed[:, :, None], 0.0)
    return p.sum((2, 3))


def _plain_evict(st):
    c = st["c"]
    n = st["lens"][:, None, None].long()
    at = torch.arange(c["S"], device=n.device)
    inside = at < n
    forced = inside & ((at < c["sinks"]) | (at >= n - c["recent"]))
    rank = st["weights"].masked_fill(~inside, -math.inf).masked_fill(forced, math.inf)
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :c["budget"]]
    best = torch.sort(torch.where(best < n, best, c["S"]), dim=-1).values  # in the cache's order
    valid = best < c["S"]
    best = best.clamp(max=c["S"] - 1)
    keep = torch.where(valid, best, -1).int()
    w = torch.zeros_like(st["weights"])
    w[..., :c["budget"]] = torch.where(valid, st["weights"].gather(2, best), 0.0)
    rows, live = best.transpose(1, 2)[..., None], valid.transpose(1, 2)[..., None]
    k, v = st["k_out"], st["v_out"]
    m = c["budget"]
    k[:, :m] = torch.where(live, st["k"].gather(1, rows.expand(-1, -1, -1, c["Dqk"])), k[:, :m])
    v[:, :m] = torch.where(live, st["v"].gather(1, rows.expand(-1, -1, -1, c["Dv"])), v[:, :m])
    return k, v, w, st["lens"].clamp(max=m), keep


def run(state):
    st = state
    c = st["c"]
    if not own:
        return {"attn": _plain_attn, "weights": _plain_weights, "evict": _plain_evict}[c["op"]](st)
    import index_sparse_attention_b200 as sa
    if c["op"] == "attn":
        return sa.cache_attn_fwd(st["q"], st["k"], st["v"], st["lens"], k_prefix=st.get("kp"),
                                 v_prefix=st.get("vp"), with_weights=c["weights"],
                                 weights=st["weights"] if c["weights"] else None)
    if c["op"] == "weights":
        return sa.sparse_attn_key_weights(st["q"], st["k"], st["lse"], st["lists"])
    return sa.cache_evict(st["k"], st["v"], st["weights"], st["lens"], c["budget"],
                          sinks=c["sinks"], recent=c["recent"], k_out=st["k_out"],
                          v_out=st["v_out"])


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    B, HK, f64 = c["B"], c["HK"], torch.float64
    if c["op"] == "attn":
        G = c["HQ"] // HK
        o = torch.empty((B, 1, c["HQ"], c["Dv"]), dtype=f64, device="cuda")
        lse = torch.empty((B, c["HQ"], 1), dtype=f64, device="cuda")
        w = st["weights"].to(f64)
        for b in range(B):
            n = int(st["lens"][b])
            for g in range(HK):
                keys, vals = st["k"][b, :n, g].to(f64), st["v"][b, :n, g].to(f64)
                if c["P"]:
                    keys = torch.cat([st["kp"][:, g].to(f64), keys])
                    vals = torch.cat([st["vp"][:, g].to(f64), vals])
                q = st["q"][b, 0, g * G:(g + 1) * G].to(f64)
                s = torch.einsum("hd,jd->hj", q, keys) / math.sqrt(c["Dqk"])
                total = torch.logsumexp(s, 1)
                p = torch.exp(s - total[:, None])
                o[b, 0, g * G:(g + 1) * G] = torch.einsum("hj,jd->hd", p, vals)
                lse[b, g * G:(g + 1) * G, 0] = total
                w[b, g, :n] += p[:, c["P"]:].sum(0)
        return (o, lse, w) if c["weights"] else (o, lse)
    if c["op"] == "weights":
        G = c["HQ"] // HK
        w = torch.zeros((B, HK, c["Sk"]), dtype=f64, device="cuda")
        i, j = torch.arange(c["Sq"], device="cuda"), torch.arange(c["Sk"], device="cuda")
        for b in range(B):
            for g in range(HK):
                see = torch.ones((c["Sq"], c["Sk"]), dtype=torch.bool, device="cuda")
                if c["mode"] == "block":
                    see = st["mask"][b, g].bool()[i // 128][:, j // 128]
                elif c["mode"] == "index":
                    rows, slots = torch.nonzero(st["idx"][b, :, g] >= 0, as_tuple=True)
                    see.fill_(False)
                    see[rows, st["idx"][b, rows, g, slots].long()] = True
                if c["causal"]:
                    see &= j[None, :] <= i[:, None]
                for h in range(g * G, (g + 1) * G):
                    s = torch.einsum("id,jd->ij", st["q"][b, :, h].to(f64), st["k"][b, :, g].to(f64))
                    s = s / math.sqrt(c["Dqk"]) - st["lse"][b, h].to(f64)[:, None]
                    w[b, g] += torch.where(see, torch.exp(s), 0.0).sum(0)
        return w
    lens = st["lens"].tolist()
    k, v = torch.zeros(st["k"].shape, dtype=f64), torch.zeros(st["v"].shape, dtype=f64)
    w = torch.zeros(st["weights"].shape, dtype=f64)
    keep = torch.full((B, HK, c["budget"]), -1, dtype=torch.int32)
    kc, vc, wc = st["k"].cpu(), st["v"].cpu(), st["weights"].cpu()
    for b, n in enumerate(lens):
        first, last = min(c["sinks"], n), max(min(c["sinks"], n), n - c["recent"])
        for g in range(HK):
            if n <= c["budget"]:
                got = list(range(n))
            else:
                row = wc[b, g].tolist()
                middle = sorted(range(first, last), key=lambda x: (-row[x], x))
                got = sorted([*range(first), *middle[:c["budget"] - first - (n - last)],
                              *range(last, n)])
            at = torch.tensor(got, dtype=torch.long)
            keep[b, g, :len(got)] = at.int()
            k[b, :len(got), g], v[b, :len(got), g] = kc[b, at, g].to(f64), vc[b, at, g].to(f64)
            w[b, g, :len(got)] = wc[b, g, at].to(f64)
    return k, v, w, torch.tensor([min(n, c["budget"]) for n in lens], dtype=torch.int32), keep
