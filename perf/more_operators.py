"""Cases of a prompt's way through the attention layers, and of shared pages: norms of queries and keys with
the position rotation, the prompt's entries in the paged cache, causal attention of packed prompts over it,
forks of sequences, and the compaction of the pool's pages.

`own` false runs each operator in its plain form (elementary torch operations in 32 bits, angles in 64);
`own` true through hybrid_ssm_gated_gb300.kv.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # one user's prompt with large heads: latency and the causal corner
        dict(name="prompt_b1_n700_d256", op="prompt", B=1, n=700, prefix=0, Hq=16, Hkv=2, d=256, page=16, dtype="bf16",
             ragged=False, pad=0),
        # a served batch: packed chunks of unequal lengths behind cached prefixes of unequal lengths, one padded
        dict(name="prompt_b16_n512_over8192_f16", op="prompt", B=16, n=512, prefix=8192, Hq=32, Hkv=8, d=128, page=16,
             dtype="f16", ragged=True, pad=1),
        # one long document, the largest call
        dict(name="prompt_b1_n20000", op="prompt", B=1, n=20000, prefix=0, Hq=32, Hkv=8, d=128, page=64, dtype="bf16",
             ragged=False, pad=0),
        # an evaluation run in single precision with an odd head size and odd pages
        dict(name="prompt_b3_n1200_f32_d80", op="prompt", B=3, n=1200, prefix=100, Hq=8, Hkv=4, d=80, page=24,
             dtype="f32", ragged=True, pad=0),
        # the keys and values of one user's prompt, rotated in a quarter of their elements
        dict(name="append_b1_n700_d256", op="append", B=1, n=700, prefix=0, Hq=16, Hkv=2, d=256, page=16, dtype="bf16",
             ragged=False, pad=0, rot=64, axes=1, interleaved=False),
        # a batch of long prompts with images in them: positions in time, height and width
        dict(name="append_b8_n8192_axes3", op="append", B=8, n=8192, prefix=300, Hq=32, Hkv=8, d=128, page=64,
             dtype="f16", ragged=True, pad=1, rot=128, axes=3, interleaved=False),
        # the drafted tokens of a decode step
        dict(name="rotate_b64_t4_d256", op="rotate", B=64, T=4, Hq=16, Hkv=2, d=256, dtype="bf16", rot=64, axes=1,
             interleaved=False),
        # a long text's queries and keys, turned in neighbouring pairs
        dict(name="rotate_b1_t20000", op="rotate", B=1, T=20000, Hq=32, Hkv=8, d=128, dtype="bf16", rot=128, axes=1,
             interleaved=True),
        # four samples of one user's prompt: shared pages, a copied last one
        dict(name="fork_1to4_n700", op="fork", n=4, parents=1, L=700, Hq=16, Hkv=2, d=256, page=16, dtype="bf16",
             whole=False),
        # 32 sequences get pages of their own (their weights will part)
        dict(name="fork_8to32_n4096_whole", op="fork", n=32, parents=8, L=4096, Hq=32, Hkv=8, d=128, page=64,
             dtype="f16", whole=True),
        # a small pool after one of its users left
        dict(name="compact_b4_n700", op="compact", B=4, L=700, free=0.25, Hq=16, Hkv=2, d=256, page=16, dtype="bf16"),
        # a served pool in which a third of the sequences have ended
        dict(name="compact_b64_n4096", op="compact", B=64, L=4096, free=0.35, Hq=32, Hkv=8, d=128, page=64,
             dtype="f16"),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "prompt", "append", "append", "rotate", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
    d = rng.choice([64, 80, 96, 128, 128, 192, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 16, 24, 32, 48, 64, 128])
    c = dict(op=op, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype)
    entry = Hkv * d * SIZE[dtype]
    rot = rng.choice([d, d, d // 2, d // 4 // 2 * 2, 32])
    if op in ("prompt", "append"):
        n = _logu(rng, 1, 20000 if op == "prompt" else 16000)
        c.update(B=_logu(rng, 1, 32), n=n, prefix=rng.choice([0, 0, _logu(rng, 1, 20000)]), ragged=rng.random() < 0.7)
        # entries of the whole batch: a pool of up to 256 MB a side; pairs of a prompt's row and an entry as many as
        # the largest listed case has
        while c["B"] > 1 and c["B"] * (n + c["prefix"]) * entry > 1 << 28:
            c["B"] = max(1, c["B"] // 2)
        most = 20000 * 20000 * 16 * 128 * (1 if dtype != "f32" else 0.1)
        while op == "prompt" and c["B"] * c["n"] * (c["n"] / 2 + c["prefix"]) * Hq * d > most:
            c["B"], c["n"] = max(1, c["B"] // 2), max(1, c["n"] * 3 // 4)
        c["pad"] = rng.choice([0, 0, 1]) if c["B"] > 1 else 0
    if op == "rotate":
        c.update(B=_logu(rng, 1, 64), T=_logu(rng, 1, 20000))
        while c["B"] * c["T"] * (Hq + Hkv) * d > 20000 * 40 * 128:
            c["B"], c["T"] = max(1, c["B"] // 2), max(1, c["T"] * 3 // 4)
        del c["page"]
    if op in ("append", "rotate"):
        c.update(rot=rot, axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4)
    if op == "fork":
        L, parents = _logu(rng, 1, 30000), _logu(rng, 1, 8)
        n = parents * rng.choice([1, 2, 3, 4])
        while n * L * entry > 1 << 28:
            L = L // 2
        c.update(n=n, parents=parents, L=max(1, L), whole=rng.random() < 0.4)
    if op == "compact":
        B, L = _logu(rng, 1, 64), _logu(rng, 1, 30000)
        while B * L * entry > 1 << 28:
            B, L = max(1, B * 3 // 4), max(1, L * 3 // 4)
        c.update(B=B, L=L, free=rng.uniform(0.0, 0.8))
    return c


def _spread(x, B, ragged):
    """x for each of B sequences, or a spread of 0.2 x .. x."""
    return [x if not ragged or b == 0 else max(1, int(x * (0.2 + 0.8 * ((b * 0.6180339887) % 1.0)))) for b in range(B)]


def _prompts(case):
    """(new tokens, entries before them) of each sequence."""
    n = _spread(case["n"], case["B"], case["ragged"])
    p = _spread(case["prefix"], case["B"], case["ragged"])[::-1] if case["prefix"] else [0] * case["B"]
    return list(zip(n, p))


def _frequencies(case):
    """Radians a position of each turned pair (64 bits), and the axis that it follows."""
    h = case["rot"] // 2
    f = 1000000.0 ** (-torch.arange(h, dtype=torch.float64) / h)
    cut = [h * (i + 1) // case["axes"] for i in range(case["axes"])]  # sections of the frequencies, one an axis
    axis = [next(a for a, c in enumerate(cut) if i < c) for i in range(h)]
    return f, axis


def _positions(case, starts, counts):
    """Positions [axes, tokens] of sequences that begin at `starts`: text, or rows and columns of an image."""
    pos = np.zeros((case["axes"], sum(counts)), np.int32)
    at = 0
    for s, n in zip(starts, counts):
        t = np.arange(n)
        pos[0, at:at + n] = s + (t if case["axes"] == 1 else t // 64)
        if case["axes"] > 1:
            pos[1, at:at + n] = s + t // 8 % 8
        if case["axes"] > 2:
            pos[2, at:at + n] = s + t % 8
        at += n
    return pos


def prepare(case, seed):
    """What a program has in hand: the cache's tensors (or activations alone), the call's rows, its handles."""
    g = torch.Generator(device="cuda").manual_seed(seed * 6151 + 29)
    r = np.random.default_rng(seed + 1)
    op, Hq, Hkv, d, dt = case["op"], case["Hq"], case["Hkv"], case["d"], DT[case["dtype"]]
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    s = dict(case=case, scale=1.0 / math.sqrt(d), err=torch.zeros(1, dtype=torch.int32, device="cuda"))

    if op in ("append", "rotate"):
        s["freq"], s["axis"] = _frequencies(case)
        s["q_norm"], s["k_norm"] = 0.2 * rnd(d), 0.2 * rnd(d)  # stored about zero: the weight is 1 + this
    if op == "rotate":
        B, T = case["B"], case["T"]
        s["q"] = (rnd(B, T, Hq, d) * 3.0).to(dt)
        s["k"] = (rnd(B, T, Hkv, d) * 3.0).to(dt)
        starts = r.integers(0, 100000, B)
        s["positions"] = dev(_positions(case, starts, [T] * B).reshape(case["axes"], B, T))
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        if own:
            from hybrid_ssm_gated_gb300 import kv

            s["rotary"] = kv.Rotary(s["freq"], axis=s["axis"], axes=case["axes"], interleaved=case["interleaved"],
                                    q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, offset=1.0)
        return s

    page = case["page"]
    if op in ("prompt", "append"):
        lens = [n + p for n, p in _prompts(case)]
    elif op == "fork":
        lens = _spread(case["L"], case["parents"], True)
    else:
        lens = _spread(case["L"], case["B"], True)
    need = [-(-n // page) for n in lens]
    copies = 0
    if op == "fork":
        child = [i % case["parents"] for i in range(case["n"])]
        # a page of its own for every page of a whole copy, else for one that is not full
        fresh = [need[p] if case["whole"] else int(lens[p] % page != 0) for p in child]
        copies = sum(fresh)
    slots_n = len(lens) + (case["n"] if op == "fork" else 2)
    maxp, num_pages = max(need) + 1, sum(need) + copies + 3
    # keys of a head share a direction, as trained heads' do; queries lean along it
    lean = rnd(1, Hkv, 1, d)
    k = rnd(num_pages, Hkv, page, d).add_(lean, alpha=0.5).to(dt)
    v = rnd(num_pages, Hkv, page, d).to(dt)
    order, at = r.permutation(num_pages).astype(np.int32), 0
    table, lengths = np.full((slots_n, maxp), -1, np.int32), np.zeros(slots_n, np.int32)
    slots = r.permutation(slots_n).astype(np.int32)
    for b, n in enumerate(lens):
        table[slots[b], :need[b]] = order[at:at + need[b]]
        at += need[b]
        lengths[slots[b]] = n
    s4 = (slots_n + 3) // 4 * 4
    ctl = torch.zeros(2 * s4 + slots_n * maxp, dtype=torch.int32, device="cuda")
    s.update(k=k, v=v, ctl=ctl, lengths=ctl[:slots_n], counts=ctl[s4:s4 + slots_n],
             page_table=ctl[2 * s4:].view(slots_n, maxp),
             weights=rnd(num_pages, Hkv, page).exp_(),
             stamps=torch.randint(0, 1 << 20, (num_pages, Hkv, page), device="cuda", generator=g, dtype=torch.int32))

    if op in ("prompt", "append"):
        B, prompts = case["B"], _prompts(case)
        total = sum(n for n, _ in prompts)
        cu = np.concatenate([[0], np.cumsum([n for n, _ in prompts])]).astype(np.int32)
        batch = slots[:B].copy()
        if op == "append":
            for b, (n, p) in enumerate(prompts):
                lengths[slots[b]] = p
        if case["pad"]:
            batch[-case["pad"]:] = -1
        s.update(slots=dev(batch), cu=dev(cu), total=total)
        tilt = rnd(total, Hq, 1) * lean.view(1, Hkv, 1, d).expand(1, Hkv, Hq // Hkv, d).reshape(1, Hq, d)
        s["q"] = rnd(total, Hq, d).add_(tilt, alpha=0.3).to(dt)
        if op == "append":
            s["k_new"], s["v_new"] = (rnd(total, Hkv, d) * 3.0).to(dt), rnd(total, Hkv, d).to(dt)
            s["q_out"] = torch.zeros_like(s["q"])
            s["positions"] = dev(_positions(case, [p + 11 for _, p in prompts], [n for n, _ in prompts]))
        else:
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(total, Hq, device="cuda")
    elif op == "fork":
        new, P = np.full((case["n"], maxp), -1, np.int32), case["parents"]
        for i, p in enumerate(child):
            first = need[p] - fresh[i]
            new[i, first:need[p]] = order[at:at + fresh[i]]
            at += fresh[i]
        s.update(src=dev(slots[child]), dst=dev(slots[P:P + case["n"]]), new_pages=dev(new))
    else:
        lengths[slots[:len(lens)][r.random(len(lens)) < case["free"]]] = 0  # sequences that have ended
        s["used"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["lengths"].copy_(dev(lengths))
    s["counts"].copy_(dev((lengths + 11).astype(np.int32)))
    s["page_table"].copy_(dev(table))
    s["ctl0"] = ctl.clone()
    if own:
        from hybrid_ssm_gated_gb300 import kv

        s["cache"] = kv.KVCache(s["k"], s["v"], s["page_table"], s["lengths"], s["counts"], s["weights"], s["stamps"])
        if op == "prompt":
            s["ws"] = kv.kv_prompt_workspace(s["cache"], s["slots"].shape[0], s["q"])
        if op == "append":
            s["rotary"] = kv.Rotary(s["freq"], axis=s["axis"], axes=case["axes"], interleaved=case["interleaved"],
                                    q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, offset=1.0)
        if op == "compact":
            s["ws"] = kv.kv_compact_workspace(s["cache"])
    return s


# ---------------------------------------------------------------- plain forms


def _plain_turn(s, x, norm, positions):
    """x [tokens, heads, d] normed by head and turned at positions [axes, tokens], in 32 bits."""
    case = s["case"]
    rot, h = case["rot"], case["rot"] // 2
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (norm + 1.0)
    angle = positions.double()[torch.tensor(s["axis"], device="cuda")].T * s["freq"].cuda()
    c, sn = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * c - b * sn, a * sn + b * c), -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:rot]
        turned = torch.cat((a * c - b * sn, a * sn + b * c), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rotate(s):
    case = s["case"]
    pos = s["positions"].view(case["axes"], -1)
    for x, norm, out in ((s["q"], s["q_norm"], s["q_out"]), (s["k"], s["k_norm"], s["k_out"])):
        out.copy_(_plain_turn(s, x.flatten(0, 1), norm, pos).view(x.shape))


def _tokens(s):
    """Of every token of a live sequence: its row, its sequence's slot, its place among the new ones."""
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    b = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=s["total"])
    row = torch.arange(s["total"], device="cuda")
    j = row - s["cu"].long()[b]
    slot = s["slots"].long()[b]
    live = slot >= 0
    return row[live], slot[live], j[live]


def _plain_append(s):
    page, dt = s["case"]["page"], s["k"].dtype
    row, slot, j = _tokens(s)
    e = s["lengths"].long()[slot] + j
    pages, at = s["page_table"][slot, e // page].long(), e % page
    pos = s["positions"][:, row]
    s["k"][pages, :, at] = _plain_turn(s, s["k_new"][row], s["k_norm"], pos).to(dt)
    s["v"][pages, :, at] = s["v_new"][row]
    s["q_out"][row] = _plain_turn(s, s["q"][row], s["q_norm"], pos).to(dt)
    s["weights"][pages, :, at] = 0.0
    s["stamps"][pages, :, at] = (s["counts"].long()[slot] + j).int()[:, None]
    add = torch.zeros_like(s["lengths"]).index_add_(0, slot, torch.ones_like(slot, dtype=torch.int32))
    s["lengths"].add_(add)
    s["counts"].add_(add)


def _rows(s, pool, b, length):
    """A sequence's cache rows in order, [Hkv, length, d] in 32 bits."""
    page = pool.shape[2]
    pages = s["page_table"][s["slots"][b].clamp(min=0).long()][:-(-length // page)].clamp(min=0).long()
    x = pool[pages].transpose(0, 1)
    return x.reshape(x.shape[0], -1, x.shape[-1])[:, :length].float()


def _plain_prompt(s):
    case, out, lse = s["case"], s["out"], s["lse"]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    G, at = Hq // Hkv, 0
    for b, (n, p) in enumerate(_prompts(case)):
        if b >= case["B"] - case["pad"]:
            out[at:at + n] = 0.0
            lse[at:at + n] = float("-inf")
            at += n
            continue
        L = n + p
        k, v = _rows(s, s["k"], b, L), _rows(s, s["v"], b, L)
        e = torch.arange(L, device="cuda")
        step = max(1, (1 << 28) // (L * Hq))  # rows whose scores are formed at once
        for j0 in range(0, n, step):
            j1 = min(n, j0 + step)
            q = s["q"][at + j0:at + j1].float().view(j1 - j0, Hkv, G, d).permute(1, 0, 2, 3).reshape(Hkv, -1, d)
            sc = q @ k.transpose(1, 2) * s["scale"]
            last = (p + torch.arange(j0, j1, device="cuda")).repeat_interleave(G)
            sc.masked_fill_(e > last[:, None], float("-inf"))
            m = sc.amax(-1, keepdim=True)
            w = sc.sub_(m).exp_()
            total = w.sum(-1, keepdim=True)
            o = (w @ v) / total
            back = lambda x: x.view(Hkv, j1 - j0, G, -1).transpose(0, 1).reshape(j1 - j0, Hq, -1)
            out[at + j0:at + j1] = back(o).to(out.dtype)
            lse[at + j0:at + j1] = back(m + total.log())[..., 0]
        at += n


def _plain_fork(s):
    page = s["case"]["page"]
    src, dst, new = s["src"].long(), s["dst"].long(), s["new_pages"]
    maxp = new.shape[1]
    length = s["lengths"][src].long()
    j = torch.arange(maxp, device="cuda")
    held = j < (-(-length // page))[:, None]
    old = s["page_table"][src]
    copied = held & (new >= 0)
    i, jj = copied.nonzero(as_tuple=True)
    entry = jj[:, None] * page + torch.arange(page, device="cuda")
    n, at = (entry < length[i][:, None]).nonzero(as_tuple=True)  # entries past the length are not copied
    a, b = old[i, jj][n].long(), new[i, jj][n].long()
    for name in ("k", "v", "weights", "stamps"):
        s[name][b, :, at] = s[name][a, :, at]
    s["page_table"][dst] = torch.where(copied, new, torch.where(held, old, s["page_table"][dst]))
    s["lengths"][dst] = s["lengths"][src]
    s["counts"][dst] = s["counts"][src]


def _plain_compact(s):
    page, num_pages = s["case"]["page"], s["k"].shape[0]
    table, lengths = s["page_table"], s["lengths"].long()
    held = torch.arange(table.shape[1], device="cuda") < (-(-lengths // page))[:, None]
    live = torch.zeros(num_pages, dtype=torch.bool, device="cuda")
    live[table[held].long()] = True
    used = live.sum()
    index = torch.arange(num_pages, device="cuda")
    hole = (~live & (index < used)).nonzero(as_tuple=True)[0]
    mover = (live & (index >= used)).nonzero(as_tuple=True)[0]
    for name in ("k", "v", "weights", "stamps"):
        s[name][hole] = s[name][mover]
    to = index.clone()
    to[mover] = hole
    table[held] = to[table[held].long()].int()
    s["used"].copy_(used.int())


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from hybrid_ssm_gated_gb300 import kv
    if op == "prompt":
        if own:
            kv.kv_prompt_attention(s["cache"], s["slots"], s["cu"], s["q"], s["out"], s["err"], s["ws"], lse=s["lse"],
                                   scale=s["scale"])
        else:
            _plain_prompt(s)
        return {"out": s["out"], "lse": s["lse"]}
    if op == "rotate":
        if own:
            kv.kv_norm_rotate(s["rotary"], s["positions"], q=s["q"], k=s["k"], q_out=s["q_out"], k_out=s["k_out"])
        else:
            _plain_rotate(s)
        return {"q_out": s["q_out"], "k_out": s["k_out"]}
    s["ctl"].copy_(s["ctl0"])  # every pass begins with the same tables, lengths and counts
    if op == "append":
        if own:
            kv.kv_append(s["cache"], s["slots"], s["cu"], s["k_new"], s["v_new"], s["err"], rotary=s["rotary"],
                         positions=s["positions"], q=s["q"], q_out=s["q_out"])
        else:
            _plain_append(s)
        return {n: s[n] for n in ("k", "v", "q_out", "weights", "stamps", "lengths", "counts")}
    if op == "fork":
        if own:
            kv.kv_fork(s["cache"], s["src"], s["dst"], s["new_pages"], s["err"])
        else:
            _plain_fork(s)
        return {n: s[n] for n in ("k", "v", "weights", "stamps", "page_table", "lengths", "counts")}
    if own:
        kv.kv_compact(s["cache"], s["used"], s["err"], s["ws"])
    else:
        _plain_compact(s)
    return {n: s[n] for n in ("k", "v", "weights", "stamps", "page_table", "used")}


def work(case):
    op, Hq, Hkv, d, sz = case["op"], case["Hq"], case["Hkv"], case["d"], SIZE[case["dtype"]]
    if op == "rotate":
        rows = case["B"] * case["T"]
        return {"bytes": rows * (2 * (Hq + Hkv) * d * sz + 4 * case["axes"]), "flops": 7 * rows * (Hq + Hkv) * d}
    if op in ("prompt", "append"):
        prompts = _prompts(case)
        prompts = prompts[:len(prompts) - case["pad"]]
        rows = sum(n for n, _ in prompts)
    if op == "append":
        return {"bytes": rows * (2 * (Hq + 2 * Hkv) * d * sz + 4 * case["axes"] + 8 * Hkv) + 24 * len(prompts),
                "flops": 7 * rows * (Hq + Hkv) * d}
    if op == "prompt":
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in prompts)
        entries = sum(n + p for n, p in prompts)
        return {"bytes": rows * Hq * (2 * d * sz + 4) + 2 * entries * Hkv * d * sz, "flops": 4 * Hq * d * pairs}
    page = case["page"]
    one = Hkv * (2 * d * sz + 8)  # an entry's key, value, weight and stamp
    if op == "fork":
        lens = [_spread(case["L"], case["parents"], True)[i % case["parents"]] for i in range(case["n"])]
        copied = sum(n if case["whole"] else n % page for n in lens)
        return {"bytes": 2 * copied * one + sum(12 * -(-n // page) for n in lens), "flops": 0}
    lens = _spread(case["L"], case["B"], True)
    held = sum(-(-n // page) for n in lens) * (1 - case["free"])  # in the mean over who has ended
    total = sum(-(-n // page) for n in lens) + 3
    moves = held * (1 - held / total)  # live pages at or above `held`, where they lie at random
    return {"bytes": 2 * moves * page * one + 8 * held, "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits


def _turned(x, weight, angle, interleaved):
    """One head's rows x [tokens, d] in 64 bits: norm, then each pair turned as a complex number."""
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * (1.0 + weight.double())
    h = angle.shape[1]
    i = torch.arange(h, device="cuda")
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    z = torch.complex(y[:, first], y[:, second]) * torch.polar(torch.ones_like(angle), angle)
    y[:, first], y[:, second] = z.real, z.imag
    return y


def exact(case, seed):
    """The operators from their definitions, one sequence and head at a time, in 64 bits."""
    op, Hq, Hkv, d = case["op"], case["Hq"], case["Hkv"], case["d"]
    if op in ("fork", "compact"):
        return None  # they move values and compute none
    s = prepare(case, seed)
    if op in ("rotate", "append"):
        freq = s["freq"].cuda()
        pos = s["positions"].view(case["axes"], -1).double()
        angle = torch.stack([pos[a] * freq[i] for i, a in enumerate(s["axis"])], 1)
    if op == "rotate":
        res = {}
        for name, w in (("q", "q_norm"), ("k", "k_norm")):
            x = s[name].flatten(0, 1)
            y = torch.stack([_turned(x[:, h], s[w], angle, case["interleaved"]) for h in range(x.shape[1])], 1)
            res[name + "_out"] = y.view(s[name].shape)
        return res
    page, at = case["page"], 0
    slots, table = s["slots"].tolist(), s["page_table"]
    if op == "append":
        k, q = s["k"].double(), s["q_out"].double()
        for b, (n, p) in enumerate(_prompts(case)):
            if slots[b] >= 0:
                e = torch.arange(p, p + n, device="cuda")
                pages = table[slots[b]].long()[e // page]
                for h in range(Hkv):
                    k[pages, h, e % page] = _turned(s["k_new"][at:at + n, h], s["k_norm"], angle[at:at + n],
                                                    case["interleaved"])
                for h in range(Hq):
                    q[at:at + n, h] = _turned(s["q"][at:at + n, h], s["q_norm"], angle[at:at + n], case["interleaved"])
            at += n
        return {"k": k, "v": None, "q_out": q, "weights": None, "stamps": None, "lengths": None, "counts": None}
    out = torch.zeros(s["total"], Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((s["total"], Hq), float("-inf"), dtype=torch.float64, device="cuda")
    for b, (n, p) in enumerate(_prompts(case)):
        if slots[b] >= 0:
            pages = table[slots[b], :-(-(n + p) // page)].long()
            for h in range(Hkv):
                keys = s["k"][pages, h].reshape(-1, d)[:n + p].double()
                vals = s["v"][pages, h].reshape(-1, d)[:n + p].double()
                for x in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                    for j0 in range(0, n, 2048):
                        j1 = min(n, j0 + 2048)
                        top = p + j1  # no row of these sees an entry past it
                        a = s["q"][at + j0:at + j1, x].double() @ keys[:top].T / math.sqrt(d)
                        seen = torch.ones(j1 - j0, top, dtype=torch.bool, device="cuda").tril(p + j0)
                        a = torch.where(seen, a, float("-inf"))
                        z = torch.logsumexp(a, 1)
                        lse[at + j0:at + j1, x] = z
                        out[at + j0:at + j1, x] = a.sub_(z[:, None]).exp_() @ vals[:top]
        at += n
    return {"out": out, "lse": lse}
