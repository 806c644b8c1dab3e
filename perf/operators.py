"""Cases of the attention-cache operators: attention of drafted tokens (a tree, or one token) over a
paged key/value cache, the commit of an accepted path, the accumulation of attention weight per cache
entry, and the eviction of the entries with the least of it.

`own` false runs each operator in its plain form (elementary torch operations in 32 bits); `own` true
through hybrid_ssm_gated_gb300.kv.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one user, a chain of four drafted tokens after a short prompt: latency decides
        dict(name="tree_chain4_b1_d256", op="tree", B=1, T=4, Hq=16, Hkv=2, d=256, L=700, page=16, dtype="bf16",
             chain=True, ragged=False, pad=0),
        # ordinary decode: one token each for a batch of sequences of unequal lengths
        dict(name="decode_b64_l8192", op="tree", B=64, T=1, Hq=32, Hkv=8, d=128, L=8192, page=64, dtype="bf16",
             chain=True, ragged=True, pad=0),
        # a served batch verifying draft trees of 16 nodes, small pages, one padded row of the batch
        dict(name="tree16_b32_l4096_f16", op="tree", B=32, T=16, Hq=32, Hkv=8, d=128, L=4096, page=16, dtype="f16",
             chain=False, ragged=True, pad=1),
        # one very long context and a wide tree: 256 query rows a key head, the largest call
        dict(name="tree64_b1_l131072", op="tree", B=1, T=64, Hq=32, Hkv=8, d=128, L=131072, page=64, dtype="bf16",
             chain=False, ragged=False, pad=0),
        # a single-precision cache with an odd head size and odd pages (an evaluation run)
        dict(name="tree7_b5_f32_d80", op="tree", B=5, T=7, Hq=8, Hkv=4, d=80, L=1501, page=24, dtype="f32",
             chain=False, ragged=True, pad=0),
        # the accepted path of one user's chain is written to the cache
        dict(name="commit_b1", op="commit", B=1, T=4, P=4, Hq=16, Hkv=2, d=256, L=700, page=16, dtype="bf16", pad=0),
        # the same for a large served batch
        dict(name="commit_b256", op="commit", B=256, T=16, P=6, Hq=32, Hkv=8, d=128, L=500, page=16, dtype="f16",
             pad=2),
        # weights of one user's accepted tokens
        dict(name="weights_b2_l1500", op="weights", B=2, T=4, P=3, Hq=16, Hkv=2, d=256, L=1500, page=32,
             dtype="bf16", decay=1.0, pad=0),
        # weights of a served batch's accepted paths, with forgetting
        dict(name="weights_b64_l8192_f16", op="weights", B=64, T=16, P=4, Hq=32, Hkv=8, d=128, L=8192, page=64,
             dtype="f16", decay=0.98, pad=1),
        # one user's short cache is brought back to its budget
        dict(name="evict_b2_600", op="evict", B=2, Hq=16, Hkv=2, d=256, L=600, page=16, budget=512, recent=64,
             dtype="bf16", pad=0),
        # a served batch that ran 256 tokens past its budget
        dict(name="evict_b64_4352", op="evict", B=64, Hq=32, Hkv=8, d=128, L=4352, page=64, budget=4096, recent=512,
             dtype="f16", pad=1),
        # one long prompt cut to half after its prefill
        dict(name="evict_b1_131072", op="evict", B=1, Hq=32, Hkv=8, d=128, L=131072, page=64, budget=65536,
             recent=1024, dtype="bf16", pad=0),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "commit", "weights", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"]) if op in ("tree", "weights") else \
        rng.choice(["bf16", "f16", "f32"])
    d = rng.choice([64, 80, 96, 128, 128, 192, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 16, 32, 48, 64, 128])
    # entries of the whole batch: a pool of up to 256 MB a side (64 MB in single precision)
    most = (1 << (26 if dtype == "f32" else 28)) // (Hkv * d * SIZE[dtype])
    L = min(_logu(rng, 24, 60000), most)
    B = min(_logu(rng, 1, 64), max(1, most // L))
    pad = rng.choice([0, 0, 1]) if B > 1 else 0
    c = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, L=L, page=page, dtype=dtype, pad=pad)
    if op == "tree":
        c.update(T=rng.choice([1, _logu(rng, 1, 64), _logu(rng, 2, 64)]), chain=rng.random() < 0.3,
                 ragged=rng.random() < 0.7)
        while c["T"] > 1 and dtype == "f32" and c["T"] * L * B * Hq > 1 << 26:
            c["T"] = max(1, c["T"] // 2)
        while c["T"] * L * B * Hq > 1 << 28 and c["T"] > 1:
            c["T"] = max(1, c["T"] // 2)
    elif op == "commit":
        T = _logu(rng, 1, 64)
        c.update(T=T, P=min(T, _logu(rng, 1, 16)))
    elif op == "weights":
        T = _logu(rng, 1, 32)
        c.update(T=T, P=min(T, _logu(rng, 1, 10)), decay=rng.choice([1.0, 0.9, 0.98]))
        while c["P"] > 1 and c["P"] * L * B * Hq > 1 << 26:
            c["P"] = max(1, c["P"] // 2)
        c["L"] = max(L, c["P"])
    else:
        budget = max(1, int(L * rng.uniform(0.3, 0.97)))
        c.update(budget=budget, recent=int(budget * rng.uniform(0.0, 0.5)))
    return c


def _lengths(case):
    """Entries of each sequence (all L where not ragged; a spread of 0.2 L .. L otherwise)."""
    B, L = case["B"], case["L"]
    if not case.get("ragged", case["op"] in ("commit", "weights")):
        return [L] * B
    return [max(1, int(L * (0.2 + 0.8 * ((b * 0.6180339887) % 1.0)))) if b else L for b in range(B)]


def _nodes(case):
    """Drafted nodes of each sequence: all T for most, fewer for some."""
    return [case["T"] if b % 3 != 2 else max(1, case["T"] - case["T"] // 3) for b in range(case["B"])]


def _npath(case):
    return [1 + (b * 5 + case["P"] - 1) % case["P"] for b in range(case["B"])]


def prepare(case, seed):
    """A paged cache with its slots and what the call takes beside it."""
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    r = np.random.default_rng(seed)
    op, B, Hq, Hkv, d, page = case["op"], case["B"], case["Hq"], case["Hkv"], case["d"], case["page"]
    dt = DT[case["dtype"]]
    lens = _lengths(case)
    need = [-(-(n + (case.get("P", 0) if op == "commit" else 0)) // page) for n in lens]
    maxp, num_pages, slots_n = max(need) + 1, sum(need) + 3, B + 2
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    # keys of a head share a direction, as trained heads' do; queries lean along it for some rows
    lean = rnd(1, Hkv, 1, d)
    k = rnd(num_pages, Hkv, page, d).add_(lean, alpha=0.5).to(dt)
    v = rnd(num_pages, Hkv, page, d).to(dt)
    slots = r.permutation(slots_n)[:B].astype(np.int32)
    order, table, at = r.permutation(num_pages).astype(np.int32), np.full((slots_n, maxp), -1, np.int32), 0
    lengths = np.zeros(slots_n, np.int32)
    for b in range(B):
        table[slots[b], :need[b]] = order[at:at + need[b]]
        at += need[b]
        lengths[slots[b]] = lens[b]
    counts = lengths + (997 if op != "tree" else 0)  # tokens committed so far, evicted ones among them
    if case["pad"]:
        slots[-case["pad"]:] = -1
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    n = num_pages * Hkv * page
    # weights, stamps, lengths and counts in one buffer, so that a pass can start from the same bookkeeping again
    book = torch.zeros(2 * n + 2 * ((slots_n + 3) // 4 * 4), dtype=torch.int32, device="cuda")
    s4 = (slots_n + 3) // 4 * 4
    s = dict(case=case, k=k, v=v, page_table=dev(table), slots=dev(slots), book=book,
             weights=book[:n].view(torch.float32).view(num_pages, Hkv, page),
             stamps=book[n:2 * n].view(num_pages, Hkv, page), lengths=book[2 * n:2 * n + slots_n],
             counts=book[2 * n + s4:2 * n + s4 + slots_n], err=torch.zeros(1, dtype=torch.int32, device="cuda"),
             scale=1.0 / math.sqrt(d))
    s["ctl"] = book[2 * n:]
    s["lengths"].copy_(dev(lengths))
    s["counts"].copy_(dev(counts.astype(np.int32)))
    if op in ("weights", "evict"):
        # what earlier tokens left: a few entries hold most of the weight
        s["weights"].copy_(rnd(num_pages, Hkv, page).mul_(1.5).exp_().mul_(Hq // Hkv / case["L"]))
    if op == "evict":
        # after earlier evictions the newest entries lie anywhere: a random order of stamps in each head
        for b in range(B):
            if slots[b] >= 0:
                m = need[b] * page
                e = torch.rand(Hkv, lens[b], device="cuda", generator=g).argsort(-1)
                full = torch.zeros(Hkv, m, dtype=torch.int32, device="cuda")
                full[:, :lens[b]] = (e + int(counts[slots[b]]) - lens[b]).int()
                s["stamps"][dev(table[slots[b], :need[b]]).long()] = full.view(Hkv, need[b], page).transpose(0, 1)
    if op in ("tree", "commit"):
        T = case["T"]
        s["k_new"] = rnd(B, T, Hkv, d).add_(lean.view(1, 1, Hkv, d), alpha=0.5).to(dt)
        s["v_new"] = rnd(B, T, Hkv, d).to(dt)
    if op in ("tree", "weights"):
        T = case["T"]
        tilt = rnd(B, T, Hq, 1) * lean.view(1, 1, Hkv, 1, d).expand(1, 1, Hkv, Hq // Hkv, d).reshape(1, 1, Hq, d)
        s["q"] = rnd(B, T, Hq, d).add_(tilt, alpha=0.3).to(dt)
    if op == "tree":
        T, nodes = case["T"], _nodes(case)
        mask = np.zeros((B, T), np.uint64)
        for i in range(T):
            mask[:, i] = np.uint64(1) << np.uint64(i)
            if i:
                parent = np.full(B, i - 1) if case["chain"] else r.integers(0, i, B)
                mask[:, i] |= mask[np.arange(B), parent]
        s.update(mask=dev(mask.view(np.int64)), nodes=dev(np.array(nodes, np.int32)),
                 out=torch.empty(B, T, Hq, d, dtype=dt, device="cuda"),
                 lse=torch.empty(B, T, Hq, dtype=torch.float32, device="cuda"))
    if op in ("commit", "weights"):
        T, P = case["T"], case["P"]
        path = np.sort(np.stack([r.permutation(T)[:P] for _ in range(B)]), 1).astype(np.int32)
        s.update(path=dev(path), npath=dev(np.array(_npath(case), np.int32)))
    if op == "weights":
        s["lse"] = _path_lse(s)
    s["book0"] = s["book"].clone()
    s["ctl0"], s["weights0"] = s["book0"][2 * n:], s["book0"][:n].view(torch.float32).view(num_pages, Hkv, page)
    if own:
        from hybrid_ssm_gated_gb300 import kv

        s["cache"] = kv.KVCache(s["k"], s["v"], s["page_table"], s["lengths"], s["counts"], s["weights"], s["stamps"])
        if op == "tree":
            s["ws"] = kv.kv_tree_workspace(s["cache"], s["q"])
        if op == "evict":
            s["ws"] = kv.kv_evict_workspace(s["cache"], B, case["budget"])
    return s


# ---------------------------------------------------------------- plain forms


def _rows(s, pool, length):
    """Cache rows of the batch's sequences in order, [B, Hkv, length, d] in 32 bits."""
    page = pool.shape[2]
    n = -(-length // page)
    pages = s["page_table"][s["slots"].clamp(min=0).long()][:, :n].clamp(min=0).long()
    x = pool[pages].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], n * page, *pool.shape[3:])[:, :, :length].float()


def _live(s):
    """Entries of each row of the batch (0 for a padded one)."""
    sl = s["slots"].long()
    return torch.where(sl >= 0, s["lengths"][sl.clamp(min=0)].long(), 0)


def _path_lse(s):
    """log-sum-exp of the accepted nodes over the cache, at their node places: what the attention of
    the step gave."""
    q, case = s["q"], s["case"]
    B, T, Hq, d = q.shape
    P, Hkv = case["P"], case["Hkv"]
    sc = _path_scores(s)
    lse_p = torch.logsumexp(sc, -1).view(B, Hkv, P, Hq // Hkv).transpose(1, 2).reshape(B, P, Hq)
    lse = torch.zeros(B, T, Hq, device="cuda")
    lse.scatter_(1, s["path"].long()[:, :, None].expand(B, P, Hq), torch.nan_to_num(lse_p, neginf=0.0))
    return lse


def _path_scores(s):
    """Scores of the accepted path's rows over the cache [B, Hkv, P * G, L], -inf where not seen."""
    q, case = s["q"], s["case"]
    B, T, Hq, d = q.shape
    P, Hkv, L = case["P"], case["Hkv"], case["L"]
    G = Hq // Hkv
    rows = q.float().gather(1, s["path"].long()[:, :, None, None].expand(B, P, Hq, d))
    rows = rows.view(B, P, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, P * G, d)
    sc = rows @ _rows(s, s["k"], L).transpose(-1, -2) * s["scale"]
    n, live = s["npath"].long(), _live(s)
    j = torch.arange(P, device="cuda").repeat_interleave(G)
    last = (live - n)[:, None] + j  # the entry that holds the row's own token
    seen = (torch.arange(L, device="cuda") <= last[:, :, None]) & (j < n[:, None])[:, :, None] & \
        (live > 0)[:, None, None]
    return sc.masked_fill(~seen[:, None], float("-inf"))


def _plain_tree(s):
    q, case = s["q"], s["case"]
    B, T, Hq, d = q.shape
    Hkv, L = case["Hkv"], case["L"]
    G = Hq // Hkv
    live = _live(s)
    nodes = torch.where(s["slots"] >= 0, s["nodes"], 0).long()
    qf = q.float().view(B, T, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, T * G, d)
    sc = qf @ _rows(s, s["k"], L).transpose(-1, -2) * s["scale"]
    sc.masked_fill_(torch.arange(L, device="cuda") >= live[:, None, None, None], float("-inf"))
    st = qf @ s["k_new"].float().permute(0, 2, 3, 1) * s["scale"]
    t = torch.arange(T, device="cuda")
    bits = ((s["mask"][:, :, None] >> t) & 1).bool() & (t < nodes[:, None])[:, None, :]
    st.masked_fill_(~bits.repeat_interleave(G, 1)[:, None], float("-inf"))
    sc = torch.cat([sc, st], -1)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = (sc - m).exp_()
    total = p.sum(-1, keepdim=True)
    o = p[..., :L] @ _rows(s, s["v"], L) + p[..., L:] @ s["v_new"].float().transpose(1, 2)
    row = (t < nodes[:, None]).repeat_interleave(G, 1)[:, None, :, None]
    o = torch.where((total > 0) & row, o / total, 0.0)
    lse = torch.where(row, m + total.log(), float("-inf"))
    back = lambda x: x.view(B, Hkv, T, G, -1).transpose(1, 2).reshape(B, T, Hq, -1)
    return {"out": back(o).to(q.dtype), "lse": back(lse)[..., 0]}


def _plain_commit(s):
    case = s["case"]
    B, P, page = case["B"], case["P"], case["page"]
    j = torch.arange(P, device="cuda")
    take = (s["slots"] >= 0)[:, None] & (j < s["npath"][:, None])
    b, jj = take.nonzero(as_tuple=True)
    slot = s["slots"].long()[b]
    at = s["lengths"].long()[slot] + jj
    pages = s["page_table"][slot, at // page].long()
    node = s["path"].long()[b, jj]
    s["k"][pages, :, at % page] = s["k_new"][b, node]
    s["v"][pages, :, at % page] = s["v_new"][b, node]
    s["weights"][pages, :, at % page] = 0.0
    s["stamps"][pages, :, at % page] = (s["counts"].long()[slot] + jj).int()[:, None]
    valid = s["slots"] >= 0
    add = torch.zeros_like(s["lengths"]).index_add_(0, s["slots"].clamp(min=0).long(),
                                                    torch.where(valid, s["npath"], 0))
    s["lengths"].add_(add)
    s["counts"].add_(add)


def _places(s, L):
    """(page, place in it, entry exists) of the batch's entries, [B, L] each."""
    page = s["case"]["page"]
    e = torch.arange(L, device="cuda")
    pages = s["page_table"][s["slots"].clamp(min=0).long()][:, e // page].long()
    return pages, (e % page).expand_as(pages), e < _live(s)[:, None]


def _plain_weights(s):
    case = s["case"]
    B, Hkv, L, P = case["B"], case["Hkv"], case["L"], case["P"]
    Hq = case["Hq"]
    G = Hq // Hkv
    lse = s["lse"].gather(1, s["path"].long()[:, :, None].expand(B, P, Hq))
    lse = lse.view(B, P, Hkv, G).transpose(1, 2).reshape(B, Hkv, P * G, 1)
    w = (_path_scores(s) - lse).exp_().sum(2)
    pages, at, live = _places(s, L)
    b, e = live.nonzero(as_tuple=True)
    pe, ae = pages[b, e], at[b, e]
    s["weights"][pe, :, ae] = s["weights"][pe, :, ae] * case["decay"] + w[b, :, e]


def _plain_evict(s):
    case = s["case"]
    budget, L, Hkv = case["budget"], case["L"], case["Hkv"]
    pages, at, live = _places(s, L)
    full = _live(s) > budget
    sel = full.nonzero(as_tuple=True)[0]  # the sequences over their budget
    pages, at, live = pages[sel], at[sel], live[sel]
    slot = s["slots"].long()[sel]
    w = s["weights"][pages, :, at].transpose(1, 2)  # [n, Hkv, L]
    st = s["stamps"][pages, :, at].transpose(1, 2)
    kept_by_age = st >= (s["counts"][slot] - case["recent"])[:, None, None]
    w = torch.where(kept_by_age, float("inf"), w).masked_fill(~live[:, None], -1.0)
    order = w.sort(dim=-1, descending=True, stable=True).indices
    keep = torch.zeros_like(w, dtype=torch.bool).scatter_(-1, order[..., :budget], True)
    e = torch.arange(L, device="cuda")
    hole, filler = ~keep & (e < budget), keep & (e >= budget)
    n, h, dst = hole.nonzero(as_tuple=True)  # in order of sequence, head, entry: the pairs line up
    _, _, src = filler.nonzero(as_tuple=True)
    pd, ad, ps, as_ = pages[n, dst], at[n, dst], pages[n, src], at[n, src]
    for name in ("k", "v", "weights", "stamps"):
        s[name][pd, h, ad] = s[name][ps, h, as_]
    s["lengths"][slot] = budget


def run(state):
    s = state
    op, case = s["case"]["op"], s["case"]
    if own:
        from hybrid_ssm_gated_gb300 import kv
    if op == "tree":
        if not own:
            return _plain_tree(s)
        kv.kv_tree_attention(s["cache"], s["slots"], s["q"], s["k_new"], s["v_new"], s["mask"], s["out"], s["err"],
                             s["ws"], num_nodes=s["nodes"], lse=s["lse"], scale=s["scale"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "commit":
        s["ctl"].copy_(s["ctl0"])  # every pass commits to the same lengths
        if own:
            kv.kv_commit(s["cache"], s["slots"], s["k_new"], s["v_new"], s["path"], s["npath"], s["err"])
        else:
            _plain_commit(s)
        return {n: s[n] for n in ("k", "v", "weights", "stamps", "lengths", "counts")}
    if op == "weights":
        s["weights"].copy_(s["weights0"])  # every pass adds to the same weights
        if own:
            kv.kv_accumulate(s["cache"], s["slots"], s["q"], s["lse"], s["path"], s["npath"], s["err"],
                             decay=case["decay"], scale=s["scale"])
        else:
            _plain_weights(s)
        return {"weights": s["weights"]}
    s["book"].copy_(s["book0"])  # every pass evicts from the same bookkeeping (the moved rows are the same ones)
    if own:
        kv.kv_evict(s["cache"], s["slots"], case["budget"], case["recent"], s["err"], s["ws"])
    else:
        _plain_evict(s)
    return {n: s[n] for n in ("k", "v", "weights", "stamps", "lengths")}


def work(case):
    op, B, Hq, Hkv, d = case["op"], case["B"], case["Hq"], case["Hkv"], case["d"]
    sz, lens = SIZE[case["dtype"]], _lengths(case)
    if case["pad"]:
        lens = lens[:-case["pad"]]
    B1 = len(lens)
    if op == "tree":
        T, nodes = case["T"], _nodes(case)[:B1]
        keys = sum(lens)
        small = B1 * T * (2 * Hkv * d * sz + 8) + B * T * Hq * (2 * d * sz + 4)
        return {"bytes": 2 * keys * Hkv * d * sz + small,
                "flops": sum(4 * Hq * d * t * (n + (t + 1) / 2) for n, t in zip(lens, nodes))}
    if op == "commit":
        rows = sum(_npath(case)[:B1])
        return {"bytes": rows * Hkv * (4 * d * sz + 8) + 16 * B1, "flops": 0}
    if op == "weights":
        npath = _npath(case)[:B1]
        keys = sum(lens)
        return {"bytes": keys * Hkv * (d * sz + 8) + sum(npath) * Hq * (d * sz + 4),
                "flops": sum(2 * Hq * d * t * n for t, n in zip(npath, lens))}
    over = [n for n in lens if n > case["budget"]]
    moves = sum((n - case["budget"]) * case["budget"] / n for n in over) * Hkv  # the mean over random weights
    return {"bytes": sum(over) * Hkv * 8 + moves * (4 * d * sz + 16), "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    """The operators from their definitions, one sequence and head at a time, in 64 bits."""
    s = prepare(case, seed)
    op, Hq, Hkv, d, page = case["op"], case["Hq"], case["Hkv"], case["d"], case["page"]
    G = Hq // Hkv
    slots, table = s["slots"].tolist(), s["page_table"]
    lengths = s["lengths"].tolist()

    def entries(pool, slot, h, n):
        pages = table[slot, :-(-n // page)].long()
        return pool[pages, h].reshape(-1, *pool.shape[3:])[:n].double()

    if op == "tree":
        B, T = case["B"], case["T"]
        nodes, masks = s["nodes"].tolist(), s["mask"].tolist()
        out = torch.zeros(B, T, Hq, d, dtype=torch.float64, device="cuda")
        lse = torch.full((B, T, Hq), float("-inf"), dtype=torch.float64, device="cuda")
        for b, slot in enumerate(slots):
            if slot < 0:
                continue
            n, t = lengths[slot], nodes[b]
            attends = torch.tensor([[(masks[b][i] >> j) & 1 for j in range(t)] for i in range(t)], device="cuda") == 1
            allowed = torch.cat([torch.ones(t, n, dtype=torch.bool, device="cuda"), attends], 1)
            for h in range(Hkv):
                keys = torch.cat([entries(s["k"], slot, h, n), s["k_new"][b, :t, h].double()])
                vals = torch.cat([entries(s["v"], slot, h, n), s["v_new"][b, :t, h].double()])
                for x in range(h * G, (h + 1) * G):
                    a = torch.where(allowed, s["q"][b, :t, x].double() @ keys.T / math.sqrt(d), float("-inf"))
                    z = torch.logsumexp(a, 1)
                    lse[b, :t, x] = z
                    out[b, :t, x] = torch.where(z[:, None] > float("-inf"), (a - z[:, None]).exp() @ vals, 0.0)
        return {"out": out, "lse": lse}
    if op == "weights":
        w = s["weights"].double()
        path, npath = s["path"].tolist(), s["npath"].tolist()
        for b, slot in enumerate(slots):
            if slot < 0:
                continue
            n, t = lengths[slot], npath[b]
            rows = torch.tensor(path[b][:t], device="cuda")
            seen = torch.ones(t, n, dtype=torch.bool, device="cuda").tril(n - t)
            pages = table[slot, :-(-n // page)].long()
            for h in range(Hkv):
                keys, add = entries(s["k"], slot, h, n), torch.zeros(n, dtype=torch.float64, device="cuda")
                for x in range(h * G, (h + 1) * G):
                    a = s["q"][b, rows, x].double() @ keys.T / math.sqrt(d) - s["lse"][b, rows, x].double()[:, None]
                    add += torch.where(seen, a.exp(), 0.0).sum(0)
                old = w[pages, h].reshape(-1)
                old[:n] = old[:n] * case["decay"] + add
                w[pages, h] = old.view(-1, page)
        return {"weights": w}
    return None  # the others move values and compute none
