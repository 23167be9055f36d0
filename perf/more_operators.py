"""Cases of the serving-step operators around the paged cache, for timing and
comparison.

A step over a paged KV cache norms and rotates the new tokens' queries and keys
(and puts keys and values into their cache slots), attends a chunk of new tokens
per request over cache and chunk, and, when tokens were drafted, verifies the
drafts against the target's probabilities.  ``run`` computes each either in
plain torch operations (``own = False``) or through the package's entry points.

Lengths of a case come from the case alone, values, trees and page orders from
the seed.
"""
import math
import random

import torch

own = False

_CHUNK = dict(op="chunk", B=1, Hq=40, Hkv=8, D=128, ps=64, lo=0, hi=0, dlo=1, dhi=1, ones=0.0, kv8=False, causal=True,
              window=-1, lens=1)
_ROPE = dict(op="rope", N=1, Hq=40, Hkv=8, D=128, rot=128, axes=1, interleaved=False, norm=True, append=True, kv8=False,
             ps=64, far=4096, lens=1)
_VERIFY = dict(op="verify", B=1, T=4, V=32000, branch=1, draft=True, context=False, noise=1.0, lens=1)


def listed():
    return [
        # The last few tokens of one user's prompt: latency of a small chunk.
        dict(_CHUNK, name="chunk_one_user", B=1, ps=16, lo=700, hi=700, dlo=24, dhi=24, lens=11),
        # A continuous batch: most requests bring one token, the others a chunk of their prompt.
        dict(_CHUNK, name="chunk_mixed", B=48, ps=64, lo=256, hi=8192, dlo=128, dhi=1024, ones=0.8, lens=12),
        # A later chunk of one long prompt.
        dict(_CHUNK, name="chunk_long", B=1, ps=128, lo=32768, hi=32768, dlo=2048, dhi=2048, lens=13),
        # First chunks of prompts, ragged, nothing cached before.
        dict(_CHUNK, name="chunk_prompts", B=16, Hq=32, ps=64, lo=0, hi=0, dlo=300, dhi=5000, lens=14),
        # Head dim 256, one query head per KV head.
        dict(_CHUNK, name="chunk_hd256", B=4, Hq=16, Hkv=16, D=256, ps=32, lo=1024, hi=6000, dlo=200, dhi=1100, lens=15),
        # An 8-bit cache.
        dict(_CHUNK, name="chunk_fp8", B=8, ps=64, lo=2048, hi=16384, dlo=256, dhi=1024, kv8=True, lens=16),
        # A sliding window: the work goes with the window, not with the cache.
        dict(_CHUNK, name="chunk_window", B=6, Hq=32, ps=16, lo=4000, hi=20000, dlo=500, dhi=2000, window=1023, lens=17),
        # A decode batch's new tokens, normed, rotated and put into the cache.
        dict(_ROPE, name="rope_decode", N=48, far=32768, lens=21),
        # A prompt pass, 8-bit cache.
        dict(_ROPE, name="rope_prompt", N=8191, kv8=True, far=131072, lens=22),
        # Positions with three axes (time, height, width) of image and video tokens, keys given back.
        dict(_ROPE, name="rope_axes", N=5000, Hq=32, axes=3, append=False, far=2048, lens=23),
        # One user's chain of drafts.
        dict(_VERIFY, name="verify_one_user", B=1, T=6, V=32000, lens=31),
        # A batch of trees with several children a node.
        dict(_VERIFY, name="verify_trees", B=64, T=24, V=152000, branch=3, lens=32),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "rope", "verify"])
    lens = rng.randrange(1, 1 << 30)
    if op == "chunk":
        D = rng.choice([128, 128, 128, 256])
        hq, hkv = rng.choice([(40, 8), (32, 8), (16, 16), (8, 2), (28, 4), (32, 1), (12, 12), (7, 1)])
        B = _log_int(rng, 1, 64)
        kv8 = D == 128 and rng.random() < 0.35
        dhi = _log_int(rng, 2, 4096)
        hi = _log_int(rng, 16, 32768)
        per_key = hkv * 2 * D * (1 if kv8 else 2)
        dhi = max(1, min(dhi, int(3e8 / (B * hq * D * 4))))
        hi = max(1, min(hi, int(2.5e9 / (B * per_key)), int(8e11 / (B * dhi * hq * 4 * D))))
        return dict(_CHUNK, B=B, Hq=hq, Hkv=hkv, D=D, ps=rng.choice([8, 16, 32, 64, 128, 256]), lo=rng.randint(0, hi // 2),
                    hi=hi, dlo=rng.randint(1, dhi), dhi=dhi, ones=rng.choice([0.0, 0.0, 0.7]), kv8=kv8,
                    causal=rng.random() < 0.85, window=_log_int(rng, 1, 4096) if rng.random() < 0.25 else -1, lens=lens)
    if op == "rope":
        D = rng.choice([64, 128, 128, 128, 256])
        hq, hkv = rng.choice([(40, 8), (32, 8), (16, 16), (8, 2), (28, 4), (32, 1), (7, 1)])
        append = rng.random() < 0.6
        return dict(_ROPE, N=_log_int(rng, 1, int(8191 * 48 * 128 / ((hq + hkv) * D))), Hq=hq, Hkv=hkv, D=D,
                    rot=rng.choice([D, D, D // 2]), axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.3,
                    norm=rng.random() < 0.8, append=append, kv8=append and rng.random() < 0.4,
                    ps=rng.choice([8, 16, 64, 128]), far=_log_int(rng, 16, 1000000), lens=lens)
    V = rng.choice([32000, 50257, 100003, 128000, 152000])
    T = _log_int(rng, 1, 32)
    return dict(_VERIFY, B=_log_int(rng, 1, max(1, int(64 * 24 * 152000 / (V * (T + 1))))), T=T, V=V,
                branch=rng.choice([1, 1, 2, 4]), draft=rng.random() < 0.7, context=rng.random() < 0.4,
                noise=rng.choice([0.2, 1.0, 2.0]), lens=lens)


# ------------------------------------------------------------------ lengths

def _lens(case):
    """Chunk lengths d and key counts n (the chunk included) of a chunk case, as host lists."""
    r = random.Random(case["lens"])
    d, n = [], []
    for _ in range(case["B"]):
        c = r.randint(case["lo"], case["hi"])
        x = 1 if r.random() < case["ones"] else r.randint(case["dlo"], case["dhi"])
        d.append(x)
        n.append(c + x)
    return d, n


def _visible(case, d, n):
    """(query, key) pairs of one request and the keys that some query sees."""
    W = case["window"]
    pairs, first = 0, n
    for t in range(d):
        hi = n - d + t + 1 if case["causal"] else n
        lo = max(0, n - d + t - W) if W >= 0 else 0
        pairs += hi - lo
        first = min(first, lo)
    return pairs, n - first


def work(case):
    op = case["op"]
    if op == "chunk":
        d, n = _lens(case)
        seen = [_visible(case, a, b) for a, b in zip(d, n)]
        keys = sum(k for _, k in seen)
        rows = sum(d) * case["Hq"]
        kv = keys * case["Hkv"] * 2 * case["D"] * (1 if case["kv8"] else 2)
        table = 4 * sum(-(-k // case["ps"]) for _, k in seen)
        return dict(bytes=kv + rows * (4 * case["D"] + 4) + table + 8 * len(d), flops=sum(p for p, _ in seen) * case["Hq"] * 4 * case["D"])
    if op == "rope":
        N, Hq, Hkv, D = (case[k] for k in ("N", "Hq", "Hkv", "D"))
        kv = 2 if case["append"] else 1                       # keys, and values on their way into the cache
        out = 1 if case["kv8"] else 2
        return dict(bytes=N * D * (4 * Hq + Hkv * kv * (2 + out)) + 4 * N * (case["axes"] + case["append"]),
                    flops=N * (Hq + Hkv) * D * (4 * case["norm"] + 3))
    # One row is needed whole, where the path ends, of the drafts' probabilities too where one was rejected.
    return dict(bytes=case["B"] * (4 * case["V"] + 4 * (4 * case["T"] + 3)), flops=case["B"] * 2 * case["V"])


# ------------------------------------------------------------------- inputs

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _values(g, shape, kv8):
    x = torch.empty(shape, dtype=torch.float8_e4m3fn if kv8 else torch.bfloat16, device="cuda")
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        part = torch.randn(min(1 << 27, flat.numel() - i), generator=g, device="cuda")
        flat[i:i + part.numel()] = ((part * 60.0).clamp_(-448.0, 448.0) if kv8 else part).to(x.dtype)
    return x


def _prepare_chunk(case, g):
    B, Hq, Hkv, D, ps, kv8 = (case[k] for k in ("B", "Hq", "Hkv", "D", "ps", "kv8"))
    d, n = _lens(case)
    counts = [-(-x // ps) for x in n]
    pages = sum(counts) + 3
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    off = torch.tensor([0] + counts, device="cuda").cumsum(0)[:-1]
    col = torch.arange(max(counts), device="cuda")
    cu = [0]
    for x in d:
        cu.append(cu[-1] + x)
    return dict(block_table=perm[(off[:, None] + col).clamp(max=pages - 1)].contiguous(),
                k_cache=_values(g, (pages, ps, Hkv, D), kv8), v_cache=_values(g, (pages, ps, Hkv, D), kv8),
                q=_values(g, (cu[-1], Hq, D), False), cu=_i32(cu), seq_lens=_i32(n), d=d, n=n,
                scale=1.0 / math.sqrt(D), k_scale=1.0 / 60.0 if kv8 else 1.0, v_scale=0.013 if kv8 else 1.0)


def _prepare_rope(case, g):
    N, Hq, Hkv, D, rot, ps = (case[k] for k in ("N", "Hq", "Hkv", "D", "rot", "ps"))
    # One projection's output, of which queries, keys and values are views; its columns differ in size.
    qkv = torch.randn(N, Hq + 2 * Hkv, D, generator=g, device="cuda") * \
        (0.2 + 3.0 * torch.rand(Hq + 2 * Hkv, 1, generator=g, device="cuda"))
    qkv = qkv.to(torch.bfloat16)
    s = dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:])
    weight = lambda: (1.0 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
    s["q_weight"], s["k_weight"] = (weight(), weight()) if case["norm"] else (None, None)
    s["inv_freq"] = (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    if case["axes"] == 1:
        s["positions"] = torch.randint(0, case["far"], (N,), generator=g, device="cuda", dtype=torch.int32)
        s["axis_map"] = None
    else:
        s["positions"] = torch.randint(0, case["far"], (case["axes"], N), generator=g, device="cuda", dtype=torch.int32)
        # The frequencies in turn to the axes.
        s["axis_map"] = torch.arange(rot // 2, device="cuda").remainder(case["axes"]).to(torch.int32)
    if case["append"]:
        pages = -(-N // ps) + 2
        s["k_cache"], s["v_cache"] = (_values(g, (pages, ps, Hkv, D), case["kv8"]) for _ in range(2))
        s["slots"] = torch.randperm(pages * ps, generator=g, device="cuda")[:N].to(torch.int32)
        s["k_scale"], s["v_scale"] = (0.02, 0.05) if case["kv8"] else (1.0, 1.0)
    s["eps"] = 1e-6
    return s


def _prepare_verify(case, g):
    B, T, V = (case[k] for k in ("B", "T", "V"))
    rows = T + 1 if case["context"] else T
    t = torch.arange(T, device="cuda")
    if case["branch"] == 1:
        parents = (t - 1).expand(B, T)
    else:
        back = 1 + (torch.rand(B, T, generator=g, device="cuda") * case["branch"] * 1.7).long()
        parents = torch.clamp(t - back, min=-1 if case["context"] else 0)
        parents[:, 0] = -1
    parents = parents.to(torch.int32).contiguous()
    # Peaked rows as of a vocabulary, the draft model's a disturbed copy of the target's.
    target = torch.empty(B, rows, V, device="cuda")
    draft = torch.empty(B, rows, V, device="cuda")
    tokens = torch.empty(B, T, dtype=torch.int32, device="cuda")
    par_row = parents.long() + (rows - T)
    for b in range(B):
        logits = 2.5 * torch.randn(rows, V, generator=g, device="cuda")
        target[b] = torch.softmax(logits, -1)
        draft[b] = torch.softmax(logits + case["noise"] * torch.randn(rows, V, generator=g, device="cuda"), -1)
        # Drafts are drawn from the draft model's row of their parent.
        e = torch.empty(T, V, device="cuda").exponential_(generator=g)
        tokens[b] = (draft[b][par_row[b].clamp(min=0)] / e).argmax(-1).to(torch.int32)
    return dict(tokens=tokens, parents=parents, target=target, draft=draft if case["draft"] else None,
                uniforms=torch.rand(B, T + 1, generator=g, device="cuda"), B=B, T=T, V=V, extra=rows - T)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"chunk": _prepare_chunk, "rope": _prepare_rope, "verify": _prepare_verify}[case["op"]](case, g)
    s["case"] = case
    return s


# --------------------------------------------------------------- plain forms

def _chunk_plain(s):
    c = s["case"]
    Hq, Hkv, D, ps, W = (c[k] for k in ("Hq", "Hkv", "D", "ps", "window"))
    G = Hq // Hkv
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    t0 = 0
    for b, (d, n) in enumerate(zip(s["d"], s["n"])):
        pos = torch.arange(n - d, n, device="cuda")
        first = 0 if W < 0 else max(0, n - d - W)
        key = torch.arange(first, n, device="cuda")
        hidden = None
        if c["causal"] and d > 1:
            hidden = key[None, :] > pos[:, None]
        if W >= 0:
            early = key[None, :] < pos[:, None] - W
            hidden = early if hidden is None else hidden | early
        pages = s["block_table"][b, first // ps:-(-n // ps)].long()
        cut = slice(first - first // ps * ps, first - first // ps * ps + n - first)
        for g in range(Hkv):
            k = s["k_cache"][pages, :, g].reshape(-1, D)[cut].float() * s["k_scale"]
            v = s["v_cache"][pages, :, g].reshape(-1, D)[cut].float() * s["v_scale"]
            q = s["q"][t0:t0 + d, g * G:(g + 1) * G].float().reshape(d * G, D)
            sc = (q @ k.t()).mul_(s["scale"])
            if hidden is not None:
                sc.view(d, G, -1).masked_fill_(hidden[:, None, :], -math.inf)
            m = sc.amax(-1, keepdim=True)
            e = sc.sub_(m).exp_()
            z = e.sum(-1, keepdim=True)
            out[t0:t0 + d, g * G:(g + 1) * G] = ((e @ v) / z).view(d, G, D).to(torch.bfloat16)
            lse[t0:t0 + d, g * G:(g + 1) * G] = (m + z.log()).view(d, G)
        t0 += d
    return out, lse


def _rotate(s, x, weight):
    c = s["case"]
    rot = c["rot"]
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * weight.float()
    pos = s["positions"]
    pos = pos[:, None] if s["axis_map"] is None else pos[s["axis_map"].long()].t()
    angle = pos.double() * s["inv_freq"].double()             # far positions: 32 bits lose the angle
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = y[..., :rot]
    if c["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, y[..., rot:]], -1)


def _rope_plain(s):
    c = s["case"]
    q = _rotate(s, s["q"], s["q_weight"]).to(torch.bfloat16)
    k = _rotate(s, s["k"], s["k_weight"])
    if not c["append"]:
        return q, k.to(torch.bfloat16)
    at = s["slots"].long()
    for cache, x, scale in ((s["k_cache"], k, s["k_scale"]), (s["v_cache"], s["v"].float(), s["v_scale"])):
        if c["kv8"]:
            x = (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
            cache.view(torch.uint8).view(-1, *x.shape[1:])[at] = x
        else:
            cache.view(-1, *x.shape[1:])[at] = x.to(torch.bfloat16)
    return q, _as_values(s, s["k_cache"]), _as_values(s, s["v_cache"])


def _as_values(s, cache):
    """A cache as values: 8-bit ones widened (BF16 holds every one)."""
    return cache.to(torch.bfloat16) if s["case"]["kv8"] else cache


def _verify_plain(s):
    B, T, V, extra = (s[k] for k in ("B", "T", "V", "extra"))
    row = torch.arange(B, device="cuda")
    u = s["uniforms"].double()
    tokens, parents = s["tokens"].long(), s["parents"].long()
    target, draft = s["target"], s["draft"]
    one = torch.ones(B, dtype=torch.float64, device="cuda")
    path = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    if extra:
        cur, count = torch.full_like(row, -1), torch.zeros_like(row)
    else:                                                     # draft 0 is the token sampled in the last step
        cur, count = torch.zeros_like(row), torch.ones_like(row)
        path[:, 0] = 0
    left = target[row, cur + extra].double()                  # what is left of the target's row
    total = one.clone()
    for t in range(0 if extra else 1, T):
        here = parents[:, t] == cur
        tok = tokens[:, t]
        p = left[row, tok] / total
        q = draft[row, cur + extra, tok].double() if draft is not None else one
        yes = here & (u[:, t] * q < p)
        no = here & ~yes
        if draft is not None:
            less = (left - total[:, None] * draft[row, cur + extra].double()).clamp_(min=0)
        else:
            less = left.clone()
            less[row, tok] = 0
        some = less.sum(-1)
        cur = torch.where(yes, t, cur)
        count = count + yes
        path.scatter_(1, (count - 1).clamp(min=0)[:, None],
                      torch.where(yes, t, path[row, (count - 1).clamp(min=0)].long())[:, None].to(torch.int32))
        keep = ~yes & ~(no & (some > 0))
        left = torch.where(yes[:, None], target[row, cur + extra].double(), torch.where(keep[:, None], left, less))
        total = torch.where(yes, one, torch.where(keep, total, some))
    run = left.cumsum(-1)
    want = u[:, T] * run[:, -1]
    return path, count.to(torch.int32), (run <= want[:, None]).sum(-1).clamp(max=V - 1).to(torch.int32)


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"chunk": _chunk_plain, "rope": _rope_plain, "verify": _verify_plain}[c["op"]](s)
    import ragged_softmax_attention_gb300 as fw
    if c["op"] == "chunk":
        return fw.paged_prefill(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu"], s["seq_lens"], s["scale"],
                                causal=c["causal"], window_left=c["window"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if c["op"] == "rope":
        how = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], axis_map=s["axis_map"],
                   interleaved=c["interleaved"])
        if not c["append"]:
            return fw.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], **how)
        q = fw.qk_norm_rope_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"], 0, s["k_cache"],
                                   s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"], **how)
        return q, _as_values(s, s["k_cache"]), _as_values(s, s["v_cache"])
    return fw.verify_drafts(s["tokens"], s["parents"], s["target"], s["uniforms"], draft_probs=s["draft"])


# --------------------------------------------------------------- exact values

def _exact_chunk(case, s):
    Hq, Hkv, D, ps, W = (case[k] for k in ("Hq", "Hkv", "D", "ps", "window"))
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    cu, lens = s["cu"].tolist(), s["seq_lens"].tolist()
    for b in range(case["B"]):
        n, d = lens[b], cu[b + 1] - cu[b]
        at = torch.arange(n, device="cuda")
        where = s["block_table"][b].long()[at // ps], at % ps
        barred = torch.zeros(d, n, dtype=torch.float64, device="cuda")
        own_pos = n - d + torch.arange(d, device="cuda").unsqueeze(1)
        if case["causal"]:
            barred[at > own_pos] = -math.inf
        if W >= 0:
            barred[at < own_pos - W] = -math.inf
        for h in range(Hq):
            g = h * Hkv // Hq
            if h * Hkv % Hq == 0:
                k = s["k_cache"].select(2, g)[where].double()
                v = s["v_cache"].select(2, g)[where].double() * float(s["v_scale"])
            score = torch.matmul(s["q"][cu[b]:cu[b + 1], h].double(), k.t()) * (float(s["scale"]) * float(s["k_scale"]))
            score += barred
            z = torch.logsumexp(score, 1)
            lse[cu[b]:cu[b + 1], h] = z
            out[cu[b]:cu[b + 1], h] = torch.matmul(torch.exp(score - z[:, None]), v)
    return out, lse


def _e4m3(x):
    """The stored value: the nearest of E4M3 (ties to even), 448 at most.  Three bits follow the leading one, down
    to exponent -6."""
    x = x.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_rope(case, s):
    rot = case["rot"]
    half = rot // 2
    axis = [0] * half if s["axis_map"] is None else s["axis_map"].tolist()
    pos = s["positions"].reshape(case["axes"], -1).double()
    turn = torch.stack([torch.polar(torch.ones_like(pos[a]), pos[a] * s["inv_freq"][i].double()) for i, a in enumerate(axis)], -1)

    def one(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + s["eps"]) * w.double()
        y = y.clone()
        i = torch.arange(half, device="cuda")
        re, im = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        z = torch.complex(y[..., re], y[..., im]) * turn[:, None, :]
        y[..., re], y[..., im] = z.real, z.imag
        return y

    q, k = one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])
    if not case["append"]:
        return q, k
    caches = []
    for cache, x, scale in ((s["k_cache"], k, s["k_scale"]), (s["v_cache"], s["v"].double(), s["v_scale"])):
        full = cache.double().flatten(0, 1)
        full[s["slots"].long()] = _e4m3(x / scale) if case["kv8"] else x
        caches.append(full.view(cache.shape))
    return q, *caches


def exact(case, seed):
    """Attention, norms and rotations in 64 bits, from their definitions.
    Verification gives whole numbers."""
    if case["op"] == "verify":
        return None
    s = prepare(case, seed)
    return _exact_chunk(case, s) if case["op"] == "chunk" else _exact_rope(case, s)
