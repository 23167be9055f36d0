"""Cases of the speculative-decoding operators, for timing and comparison.

One speculative step over a paged KV cache takes four operators: the block
tables and slot maps of the step, the ancestor masks of the drafted trees, the
attention of every drafted token, and the move of the accepted path's keys and
values to the places of ordinary tokens.  ``run`` computes each either in
plain torch operations (``own = False``) or through the package's entry points.

Lengths of a case come from the case alone, values, trees and page orders from
the seed.
"""
import math
import random

import torch

own = False

_TREE = dict(op="tree", B=1, T=8, Hq=40, Hkv=8, D=128, ps=16, lo=1, hi=1, kv8=False, ragged=False, lens=1)
_TABLES = dict(op="tables", B=1, L=0, ps=16, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=0, lens=1)
_MASK = dict(op="mask", B=1, T=8, ragged=False, lens=1)
_COMMIT = dict(op="commit", B=1, A=4, layers=1, Hkv=8, D=128, ps=16, lo=1, hi=1, kv8=False, lens=1)


def listed():
    return [
        # One request with a short draft: what a single user waits for.
        dict(_TREE, name="tree_one_user", B=1, T=8, ps=16, lo=700, hi=700, lens=11),
        # A chat batch: mid-sized trees, ragged contexts and ragged drafts.
        dict(_TREE, name="tree_chat", B=16, T=16, ps=128, lo=512, hi=8192, ragged=True, lens=12),
        # The long-context batch of the decode benchmark with 32 drafts each: all of the cache is read.
        dict(_TREE, name="tree_long", B=64, T=32, ps=128, lo=512, hi=32768, lens=13),
        # Wide trees: the products, not the cache, take the time.
        dict(_TREE, name="tree_wide", B=16, T=121, Hq=32, ps=64, lo=256, hi=8192, lens=14),
        # Head dim 256, one query head per KV head.
        dict(_TREE, name="tree_hd256", B=8, T=24, Hq=16, Hkv=16, D=256, ps=32, lo=256, hi=8192, ragged=True, lens=15),
        # An 8-bit cache.
        dict(_TREE, name="tree_fp8", B=32, T=16, ps=64, lo=512, hi=16384, kv8=True, lens=16),
        # The tables of one decode step: every request brings a few drafts, some cross into a new page.
        dict(_TABLES, name="tables_step", B=32, L=8, ps=16, new_lo=0, new_hi=8, ctx_lo=0, ctx_hi=4096, lens=21),
        # The tables of a prompt pass of a large server, tokens packed.
        dict(_TABLES, name="tables_prompts", B=2048, L=0, ps=16, new_lo=1, new_hi=8192, ctx_lo=0, ctx_hi=2048, lens=22),
        # Masks of a small and of a large batch of trees.
        dict(_MASK, name="mask_small", B=4, T=24, lens=31),
        dict(_MASK, name="mask_large", B=1024, T=121, ragged=True, lens=32),
        # Accepted paths of a small batch in one layer, and of a large one in every layer of a packed cache.
        dict(_COMMIT, name="commit_one_layer", B=8, A=4, layers=1, ps=128, lo=64, hi=500, lens=41),
        dict(_COMMIT, name="commit_all_layers", B=192, A=6, layers=32, ps=16, lo=1, hi=64, lens=42),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "tables", "mask", "commit"])
    lens = rng.randrange(1, 1 << 30)
    if op == "tree":
        D = rng.choice([128, 128, 256])
        hq, hkv = rng.choice([(40, 8), (32, 8), (16, 16), (8, 2), (24, 3), (32, 1), (12, 12), (7, 1)])
        T = _log_int(rng, 1, 128)
        B = _log_int(rng, 1, 64)
        kv8 = D == 128 and rng.random() < 0.35
        hi = _log_int(rng, 16, 32768)
        per_key = hkv * 2 * D * (1 if kv8 else 2)
        hi = max(T + 1, min(hi, int(5.5e9 / (B * per_key)), int(9e11 / (B * T * hq * 4 * D))))
        return dict(_TREE, B=B, T=T, Hq=hq, Hkv=hkv, D=D, ps=rng.choice([8, 16, 32, 64, 128, 256]),
                    lo=rng.randint(0, hi // 2), hi=hi, kv8=kv8, ragged=rng.random() < 0.5, lens=lens)
    if op == "tables":
        if rng.random() < 0.5:
            L = _log_int(rng, 1, 128)
            return dict(_TABLES, B=_log_int(rng, 1, 2048), L=L, ps=rng.choice([8, 16, 32, 64, 128]), new_lo=0,
                        new_hi=L, ctx_lo=0, ctx_hi=_log_int(rng, 16, 4096), lens=lens)
        hi = _log_int(rng, 4, 5400)
        return dict(_TABLES, B=_log_int(rng, 1, 2048), ps=rng.choice([16, 32, 64, 128]), new_lo=rng.randint(0, hi // 2),
                    new_hi=hi, ctx_lo=0, ctx_hi=_log_int(rng, 16, 2048), lens=lens)
    if op == "mask":
        return dict(_MASK, B=_log_int(rng, 1, 1024), T=_log_int(rng, 1, 121), ragged=rng.random() < 0.5, lens=lens)
    hkv, D = rng.choice([(8, 128), (2, 128), (4, 256), (1, 128), (3, 64)])
    return dict(_COMMIT, B=_log_int(rng, 1, 96), A=_log_int(rng, 1, 8), layers=_log_int(rng, 1, 32), Hkv=hkv, D=D,
                ps=rng.choice([8, 16, 64, 128]), lo=1, hi=_log_int(rng, 8, 64), kv8=rng.random() < 0.3, lens=lens)


# ------------------------------------------------------------------ lengths

def _lens(case):
    """Everything of a case that is a length, as host lists."""
    r = random.Random(case["lens"])
    op, B = case["op"], case["B"]
    if op == "tree":
        n = [max(case["T"], r.randint(case["lo"], case["hi"])) for _ in range(B)]
        d = [r.randint(1, case["T"]) if case["ragged"] else case["T"] for _ in range(B)]
        return dict(n=n, d=d)
    if op == "mask":
        return dict(d=[r.randint(1, case["T"]) if case["ragged"] else case["T"] for _ in range(B)])
    if op == "tables":
        ps = case["ps"]
        ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(B)]
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
        held = [-(-c // ps) for c in ctx]
        seq = []
        for b in range(B):
            if r.random() < 0.05:                     # the request has left: its pages go back
                ctx[b] = new[b] = 0
            elif case["L"] and r.random() < 0.3:      # pages that rejected drafts took are still held
                held[b] += r.randint(0, 2)
            seq.append(ctx[b] + new[b])
        return dict(seq=seq, new=new, held=held)
    base = [r.randint(case["lo"], case["hi"]) for _ in range(B)]
    m = [r.randint(0, case["A"]) for _ in range(B)]
    return dict(base=base, m=m, T=case["A"] + 24)


def work(case):
    x = _lens(case)
    op, B = case["op"], case["B"]
    if op == "tree":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        kv = sum(x["n"]) * Hkv * 2 * D * (1 if case["kv8"] else 2)
        rows = sum(x["d"]) * Hq
        words = sum(x["d"]) * ((T + 31) // 32) * 4
        table = sum(-(-n // case["ps"]) for n in x["n"]) * 4
        io = rows * D * 2 + B * T * Hq * (D * 2 + 4)
        flops = sum((n - d + 1) * d for n, d in zip(x["n"], x["d"])) * Hq * 4 * D
        return dict(bytes=kv + io + words + table + 8 * B, flops=flops)
    if op == "mask":
        W = (case["T"] + 31) // 32
        return dict(bytes=4 * B * case["T"] * (W + 1) + 4 * sum(x["d"]) + 4 * B, flops=sum(x["d"]))
    if op == "tables":
        ps = case["ps"]
        want = [-(-s // ps) for s in x["seq"]]
        moved = sum(abs(w - h) for w, h in zip(want, x["held"]))
        under = 0                                     # table entries under new tokens of pages held before
        for s, n, h in zip(x["seq"], x["new"], x["held"]):
            if n:
                under += max(0, min(h, -(-s // ps)) - (s - n) // ps)
        slots = B * case["L"] if case["L"] else sum(x["new"])
        return dict(bytes=4 * (3 * B + 2 * moved + under + slots + 2 * B + 5), flops=slots)
    row = case["Hkv"] * case["D"] * (1 if case["kv8"] else 2) * 2 * case["layers"]
    # A path entry that is already in place (the first child accepted first) costs nothing; at least the others do.
    moves = sum(max(0, m - 1) for m in x["m"])
    return dict(bytes=2 * moves * row + 4 * (sum(x["m"]) + 3 * B), flops=moves)


# ------------------------------------------------------------------- inputs

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pages(g, counts, ps, spare=3):
    """A pool in random order and the block table that hands it out."""
    total = sum(counts)
    perm = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(counts))
    off = torch.tensor([0] + counts, device="cuda").cumsum(0)[:-1]
    col = torch.arange(width, device="cuda")
    idx = (off[:, None] + col[None, :]).clamp(max=total + spare - 1)
    return perm[idx].contiguous(), total + spare


def _values(g, shape, kv8):
    x = torch.empty(shape, dtype=torch.float8_e4m3fn if kv8 else torch.bfloat16, device="cuda")
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        part = torch.randn(min(1 << 27, flat.numel() - i), generator=g, device="cuda")
        flat[i:i + part.numel()] = ((part * 60.0).clamp_(-448.0, 448.0) if kv8 else part).to(x.dtype)
    return x


def _parents(g, B, T):
    """Random trees in topological order: a node hangs below one of the nodes
    before it, mostly a recent one, or starts a branch of its own."""
    t = torch.arange(T, device="cuda")[None, :].expand(B, T)
    u = torch.rand(B, T, generator=g, device="cuda")
    back = 1 + (u * u * 12).long()
    return torch.where(u < 0.08, -1, torch.clamp(t - back, min=-1)).to(torch.int32).contiguous()


def _ancestors(parents):
    """[B, T, T] truth values: column j is t itself or one of its ancestors."""
    B, T = parents.shape
    m = torch.zeros(B, T, T, dtype=torch.bool, device=parents.device)
    rows = torch.arange(B, device=parents.device)
    for t in range(T):
        p = parents[:, t].long()
        m[:, t] = m[rows, p.clamp(min=0)] & (p >= 0)[:, None]
        m[:, t, t] = True
    return m


def _pack(m):
    """Truth values [B, T, T] as bits [B, T, ceil(T / 32)] int32."""
    B, T, _ = m.shape
    W = (T + 31) // 32
    pad = torch.zeros(B, T, W * 32, dtype=torch.int64, device=m.device)
    pad[:, :, :T] = m
    bits = pad.view(B, T, W, 32) << torch.arange(32, device=m.device)
    v = bits.sum(-1)
    return torch.where(v >= 1 << 31, v - (1 << 32), v).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = _lens(case)
    op, B = case["op"], case["B"]
    s = dict(case=case, x=x)
    if op == "tree":
        T, Hq, Hkv, D, ps, kv8 = (case[k] for k in ("T", "Hq", "Hkv", "D", "ps", "kv8"))
        s["block_table"], pages = _pages(g, [-(-n // ps) for n in x["n"]], ps)
        s["k_cache"] = _values(g, (pages, ps, Hkv, D), kv8)
        s["v_cache"] = _values(g, (pages, ps, Hkv, D), kv8)
        s["q"] = _values(g, (B, T, Hq, D), False)
        s["seq_lens"] = _i32(x["n"])
        s["draft_lens"] = _i32(x["d"]) if case["ragged"] else None
        live = torch.arange(T, device="cuda")[None, :] < _i32(x["d"])[:, None]
        s["tree_mask"] = _pack(_ancestors(_parents(g, B, T)) & live[:, :, None] & live[:, None, :])
        s["scale"] = 1.0 / math.sqrt(D)
        s["k_scale"], s["v_scale"] = (1.0 / 60.0, 0.013) if kv8 else (1.0, 1.0)
    elif op == "mask":
        s["parents"] = _parents(g, B, case["T"])
        s["draft_lens"] = _i32(x["d"]) if case["ragged"] else None
    elif op == "tables":
        ps = case["ps"]
        width = max(1, max(max(-(-a // ps), h) for a, h in zip(x["seq"], x["held"])))
        held = sum(x["held"])
        want = sum(-(-a // ps) for a in x["seq"])
        pool = held + want + 17
        perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        col = torch.arange(width, device="cuda")
        h = _i32(x["held"]).long()
        off = h.cumsum(0) - h
        mine = col[None, :] < h[:, None]
        s["block_table"] = torch.where(mine, perm[(off[:, None] + col).clamp(max=pool - 1)], -1).to(torch.int32)
        free = pool - held
        head = int(torch.randint(0, pool, (1,), generator=g, device="cuda").item())
        s["free_queue"] = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
        s["free_queue"][(head + torch.arange(free, device="cuda")) % pool] = perm[held:]
        s["free_range"] = _i32([head, free])
        s["seq_lens"], s["new_lens"], s["held"] = _i32(x["seq"]), _i32(x["new"]), _i32(x["held"])
        s["slot_shape"] = (B, case["L"]) if case["L"] else (max(1, sum(x["new"])),)
    else:
        ps, Hkv, D, layers, kv8 = (case[k] for k in ("ps", "Hkv", "D", "layers", "kv8"))
        s["block_table"], pages = _pages(g, [-(-(b + x["T"]) // ps) for b in x["base"]], ps)
        s["k_cache"] = _values(g, (layers * pages, ps, Hkv, D), kv8)
        s["v_cache"] = _values(g, (layers * pages, ps, Hkv, D), kv8)
        s["base_lens"], s["path_lens"] = _i32(x["base"]), _i32(x["m"])
        # The first child at index 0 (accepted most often), later ones from the deeper levels; a path never leaves
        # through an index that the move fills, so that the same move can be made again on the same cache.
        A = case["A"]
        deep = torch.rand(B, 24, generator=g, device="cuda").argsort(1)[:, :A].sort(1).values + A
        deep[:, 0] = torch.where(torch.rand(B, generator=g, device="cuda") < 0.7, 0, deep[:, 0])
        s["path"] = deep.to(torch.int32).contiguous()
        s["layers"] = layers
    return s


# --------------------------------------------------------------- plain forms

def _tree_plain(s):
    c, x = s["case"], s["x"]
    B, T, Hq, Hkv, D, ps = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "ps"))
    G = Hq // Hkv
    out = torch.zeros(B, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T, Hq), -math.inf, device="cuda")
    words = s["tree_mask"].long()
    bits = ((words[..., None] >> torch.arange(32, device="cuda")) & 1).bool().flatten(2)
    for b in range(B):
        n, d = x["n"][b], x["d"][b]
        pages = s["block_table"][b, :-(-n // ps)].long()
        k = s["k_cache"][pages].reshape(-1, Hkv, D)[:n].float().permute(1, 2, 0) * s["k_scale"]
        v = s["v_cache"][pages].reshape(-1, Hkv, D)[:n].float().permute(1, 0, 2) * s["v_scale"]
        q = s["q"][b, :d].float().view(d, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, d * G, D)
        sc = (q @ k).mul_(s["scale"]).view(Hkv, d, G, n)
        seen = torch.ones(d, n, dtype=torch.bool, device="cuda")
        seen[:, n - d:] = bits[b, :d, :d]
        sc.masked_fill_(~seen[None, :, None, :], -math.inf)
        m = sc.amax(-1, keepdim=True)
        e = sc.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
        z = e.sum(-1, keepdim=True)
        o = (e.view(Hkv, d * G, n) @ v).view(Hkv, d, G, D) / torch.where(z == 0, 1.0, z)
        out[b, :d] = o.permute(1, 0, 2, 3).reshape(d, Hq, D).to(torch.bfloat16)
        lse[b, :d] = (m + z.log()).squeeze(-1).permute(1, 0, 2).reshape(d, Hq)
    return out, lse


def _mask_plain(s):
    par = s["parents"]
    B, T = par.shape
    anc = _ancestors(par)
    depth = anc.sum(-1).to(torch.int32) - 1
    if s["draft_lens"] is not None:
        live = torch.arange(T, device="cuda")[None, :] < s["draft_lens"][:, None]
        anc = anc & live[:, :, None]
        depth = torch.where(live, depth, -1)
    return _pack(anc), depth


def _tables_plain(s):
    ps = s["case"]["ps"]
    bt, queue = s["block_table"], s["free_queue"]
    F, width = queue.numel(), bt.shape[1]
    seq, new, held = s["seq_lens"].long(), s["new_lens"].long(), s["held"].long()
    head, count = s["free_range"].long().unbind()
    want = (seq + ps - 1) // ps
    need, back = (want - held).clamp(min=0), (held - want).clamp(min=0)
    upto = need.cumsum(0)
    served = (need == 0) | (upto <= count)
    taken = torch.where(served & (need > 0), upto, 0).amax()
    col = torch.arange(width, device="cuda")[None, :]
    got = queue[(head + (upto - need)[:, None] + col - held[:, None]) % F]
    grow = served[:, None] & (col >= held[:, None]) & (col < want[:, None])
    shrink = (col >= want[:, None]) & (col < held[:, None])
    to = (head + count + (back.cumsum(0) - back)[:, None] + col - want[:, None]) % F
    spare = torch.cat([queue, queue[:1]])
    spare.scatter_(0, torch.where(shrink, to, F).flatten(), bt.flatten())
    queue.copy_(spare[:F])
    bt.copy_(torch.where(grow, got, bt))
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), new.cumsum(0)])
    if len(s["slot_shape"]) == 2:
        j = torch.arange(s["slot_shape"][1], device="cuda")[None, :].expand(s["slot_shape"])
        row = torch.arange(seq.numel(), device="cuda")[:, None].expand(s["slot_shape"])
        live = j < new[:, None]
    else:
        i = torch.arange(s["slot_shape"][0], device="cuda")
        row = torch.searchsorted(cu[1:].contiguous(), i, right=True)
        live = row < seq.numel()
        row = row.clamp(max=seq.numel() - 1)
        j = i - cu[row]
    pos = ((seq - new)[row] + j).clamp(min=0)
    page = bt[row, (pos // ps).clamp(max=width - 1)].long()
    slots = torch.where(live & served[row], page * ps + pos % ps, -1).to(torch.int32)
    left = torch.stack([(head + taken) % F, count - taken + back.sum()]).to(torch.int32)
    return dict(block_table=bt, slot_mapping=slots, cu_new=cu.to(torch.int32),
                held=torch.where(served, want, held).to(torch.int32), free_queue=queue, free_range=left)


def _commit_plain(s):
    c, x = s["case"], s["x"]
    ps, layers = c["ps"], s["layers"]
    B, A = s["path"].shape
    total = sum(x["m"])
    m = s["path_lens"].long()
    row = torch.repeat_interleave(torch.arange(B, device="cuda"), m, output_size=total)
    i = torch.arange(total, device="cuda") - (m.cumsum(0) - m)[row]
    base = s["base_lens"].long()[row]

    def place(pos):
        return s["block_table"][row, pos // ps].long() * ps + pos % ps

    dst, src = place(base + i), place(base + s["path"][row, i].long())
    for cache in (s["k_cache"], s["v_cache"]):
        raw = cache.view(torch.uint8 if cache.dtype == torch.float8_e4m3fn else torch.int16)
        rows = raw.view(layers, -1, raw.shape[2] * raw.shape[3])
        rows[:, dst] = rows[:, src]
    return _as_values(s, s["base_lens"] + s["path_lens"])


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"tree": _tree_plain, "mask": _mask_plain, "tables": _tables_plain, "commit": _commit_plain}[op](s)
    import ragged_softmax_attention_gb300 as fw
    if op == "tree":
        return fw.paged_decode_tree(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"],
                                    s["tree_mask"], s["scale"], draft_lens=s["draft_lens"], k_scale=s["k_scale"],
                                    v_scale=s["v_scale"])
    if op == "mask":
        return fw.tree_mask(s["parents"], draft_lens=s["draft_lens"])
    if op == "tables":
        slots = torch.empty(s["slot_shape"], dtype=torch.int32, device="cuda")
        cu, held, left = fw.build_page_tables(s["seq_lens"], s["new_lens"], s["held"], s["free_queue"],
                                              s["free_range"], s["case"]["ps"], s["block_table"], slots)
        return dict(block_table=s["block_table"], slot_mapping=slots, cu_new=cu, held=held,
                    free_queue=s["free_queue"], free_range=left)
    new_lens = fw.kv_commit(s["path"], s["path_lens"], s["base_lens"], s["block_table"], s["k_cache"], s["v_cache"],
                            num_layers=s["layers"])
    return _as_values(s, new_lens)


def _as_values(s, new_lens):
    """The caches as values: 8-bit ones widened (BF16 holds every one)."""
    k, v = s["k_cache"], s["v_cache"]
    return (k.to(torch.bfloat16), v.to(torch.bfloat16), new_lens) if s["case"]["kv8"] else (k, v, new_lens)


# --------------------------------------------------------------- exact values

def exact(case, seed):
    """Attention outputs in 64 bits, from the definition, one request and one
    KV head at a time.  The other operators move and count whole numbers."""
    if case["op"] != "tree":
        return None
    s = prepare(case, seed)
    B, T, Hq, Hkv, D, ps = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "ps"))
    G = Hq // Hkv
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    n_all = s["seq_lens"].tolist()
    d_all = s["draft_lens"].tolist() if s["draft_lens"] is not None else [T] * B
    words = s["tree_mask"].tolist()
    for b, (n, d) in enumerate(zip(n_all, d_all)):
        barred = torch.zeros(d, n, dtype=torch.float64)
        for t in range(d):
            for j in range(d):
                if not (words[b][t][j >> 5] >> (j & 31)) & 1:
                    barred[t, n - d + j] = -math.inf
        barred = barred.cuda().repeat_interleave(G, 0)
        pos = torch.arange(n, device="cuda")
        where = s["block_table"][b].long()[pos // ps], pos % ps
        for g in range(Hkv):
            k = s["k_cache"].select(2, g)[where].double()
            v = s["v_cache"].select(2, g)[where].double()
            q = s["q"][b, :d, g * G:(g + 1) * G].double().reshape(d * G, D)
            score = torch.matmul(q, k.t()) * (float(s["scale"]) * float(s["k_scale"])) + barred
            z = torch.logsumexp(score, 1)
            w = torch.exp(score - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
            out[b, :d, g * G:(g + 1) * G] = (torch.matmul(w, v) * float(s["v_scale"])).view(d, G, D)
            lse[b, :d, g * G:(g + 1) * G] = z.view(d, G)
    return out, lse
