"""Tree masks, page tables and path commits on the GPU, against plain loops:
whole numbers and moved bytes, equal bit for bit."""
import math
import random

import pytest
import torch

import oracle
from oracle import spec
from tests.gpu_common import built_library
from tests.test_tree_decode_gpu import check, make, on_gpu, parents_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    return built_library()


def raw(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


# ---------------------------------------------------------------- tree masks

@pytest.mark.parametrize("kind", ["chain", "star", "tree"])
@pytest.mark.parametrize("B,T", [(1, 1), (3, 7), (2, 31), (5, 32), (2, 33), (130, 64), (4, 121), (3, 256)])
def test_masks_equal_the_definition(fw, kind, B, T):
    par = parents_of(kind, B, T, seed=B + T)
    drafts = [(T * (i + 1)) // B if i else 0 for i in range(B)]
    for dl in (None, i32(drafts)):
        mask, depths = fw.tree_mask(par.cuda(), draft_lens=None if dl is None else dl.cuda())
        torch.cuda.synchronize()
        assert fw.device_status() == 0
        m_ref, d_ref = spec.tree_mask(par, dl)
        assert torch.equal(mask.cpu(), m_ref) and torch.equal(depths.cpu(), d_ref)


def test_mask_views_and_clamped_counts(fw):
    par = parents_of("tree", 4, 40, seed=1)
    wide = torch.full((4, 60), 99, dtype=torch.int32)
    wide[:, 10:50] = par
    buf = torch.full((4, 42, 6), 7, dtype=torch.int32, device="cuda")
    dep = torch.full((4, 50), 7, dtype=torch.int32, device="cuda")
    fw.tree_mask(wide.cuda()[:, 10:50], draft_lens=i32([50, -3, 17, 40]).cuda(), mask=buf[:, 1:41, 1:4],
                 depths=dep[:, 5:45])
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    m_ref, d_ref = spec.tree_mask(par, i32([40, 0, 17, 40]))
    assert torch.equal(buf[:, 1:41, 1:3].cpu(), m_ref) and torch.equal(dep[:, 5:45].cpu(), d_ref)
    assert (buf[:, 1:41, 3] == 0).all()                      # words past the tree are cleared
    assert (buf[:, 0] == 7).all() and (buf[:, 41] == 7).all() and (buf[:, :, 0] == 7).all()
    assert (buf[:, :, 4:] == 7).all() and (dep[:, :5] == 7).all() and (dep[:, 45:] == 7).all()


def test_one_tree_for_every_request(fw):
    """Parents as an expanded view, counts of their own."""
    parents = parents_of("tree", 1, 50, 3)
    drafts = i32([50, 0, 31, 32, 33, 1])
    mask, depths = fw.tree_mask(parents.cuda().expand(6, -1), draft_lens=drafts.cuda())
    torch.cuda.synchronize()
    m, d = spec.tree_mask(parents.expand(6, -1), drafts)
    assert fw.device_status() == 0 and torch.equal(mask.cpu(), m) and torch.equal(depths.cpu(), d)


def test_bad_parents_are_reported_and_become_roots(fw):
    par = i32([[-1, 1, 0, 7, -2, 4], [-1, 0, 1, 2, 3, 99]])
    mask, depths = fw.tree_mask(par.cuda(), draft_lens=i32([6, 5]).cuda())
    torch.cuda.synchronize()
    assert fw.device_status() == 1
    m_ref, d_ref = spec.tree_mask(par, i32([6, 5]))
    assert torch.equal(mask.cpu(), m_ref) and torch.equal(depths.cpu(), d_ref)
    fw.tree_mask(par[1:].cuda(), draft_lens=i32([5]).cuda())   # a bad parent of padding is nobody's
    torch.cuda.synchronize()
    assert fw.device_status() == 0


# --------------------------------------------------------------- page tables

def table_case(B, ps, L, seed, ctx=300, new=40, spare=9, leave=0.1, shrink=0.3):
    """A consistent step: pools, rings and rows of B requests."""
    r = random.Random(seed)
    seq, fresh, held = [], [], []
    for _ in range(B):
        c, f = r.randint(0, ctx), r.randint(0, L if L else new)
        h = -(-c // ps)
        if r.random() < leave:
            c = f = 0
        elif r.random() < shrink:
            h += r.randint(0, 3)
        seq.append(c + f)
        fresh.append(f)
        held.append(h)
    width = max([1] + [max(h, -(-s // ps)) for h, s in zip(held, seq)])
    want = sum(max(0, -(-s // ps) - h) for s, h in zip(seq, held))
    F = sum(held) + want + spare
    pages = list(range(F))
    r.shuffle(pages)
    bt = torch.full((B, width), -1, dtype=torch.int32)
    for b in range(B):
        for i in range(held[b]):
            bt[b, i] = pages.pop()
    head = r.randrange(F)
    queue = [-1] * F
    for i, p in enumerate(pages):
        queue[(head + i) % F] = p
    slots = torch.full((B, L) if L else (sum(fresh) + 3,), 77, dtype=torch.int32)
    return dict(seq_lens=i32(seq), new_lens=i32(fresh), held=i32(held), free_queue=i32(queue),
                free_range=i32([head, len(pages)]), page_size=ps, block_table=bt, slot_mapping=slots)


def run_tables(fw, x, status=None, in_place=False):
    bt, slots, cu, held, queue, left, codes = spec.page_tables(**x)
    g = on_gpu(x)
    kw = dict(held_out=g["held"], range_out=g["free_range"]) if in_place else {}
    before = {k: g[k].clone() for k in ("seq_lens", "new_lens", "held", "free_range")}
    c, h, f = fw.build_page_tables(**g, **kw)
    torch.cuda.synchronize()
    got = fw.device_status()
    assert got in codes if codes else got == 0, (got, codes)
    if status is not None:
        assert got == status
    assert torch.equal(c.cpu(), cu), "cu_new"
    assert torch.equal(h.cpu(), held), "held_out"
    assert torch.equal(f.cpu(), left), "range_out"
    assert torch.equal(g["block_table"].cpu(), bt), "block_table"
    assert torch.equal(g["free_queue"].cpu(), queue), "free_queue"
    assert torch.equal(g["slot_mapping"].cpu(), slots), "slot_mapping"
    if not in_place:
        for k, v in before.items():
            assert torch.equal(g[k], v), f"{k} was written"
    return c, h, f


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,ps,L", [(1, 16, 1), (1, 16, 0), (5, 8, 3), (33, 16, 8), (64, 128, 0), (64, 1, 0), (257, 24, 5),
                                    (1025, 16, 0), (3000, 16, 4), (8192, 16, 1), (2048, 7, 0), (4000, 2, 100), (3000, 16, 96)])
def test_tables_equal_the_definition(fw, B, ps, L, in_place):
    run_tables(fw, table_case(B, ps, L, seed=B + ps + L), in_place=in_place)


def test_long_prompts_packed(fw):
    run_tables(fw, table_case(40, 16, 0, seed=5, ctx=5000, new=9000))
    run_tables(fw, table_case(1, 16, 0, seed=6, ctx=0, new=100000), in_place=True)


def test_pool_runs_out(fw):
    """Requests are served in order until one asks for more than is left."""
    x = table_case(20, 16, 0, seed=7, spare=0, leave=0.0, shrink=0.0, ctx=50, new=200)
    x["free_range"][1] -= 15
    run_tables(fw, x, status=3)
    run_tables(fw, x, status=3, in_place=True)
    x["free_range"][1] = 0
    run_tables(fw, x, status=3)


def test_steps_follow_each_other(fw):
    """Forty steps on one ring: requests grow, shrink, leave and return; no page
    is ever in two places."""
    r = random.Random(11)
    B, ps, F, width = 24, 16, 90, 12
    x = dict(seq_lens=i32([0] * B), new_lens=i32([0] * B), held=i32([0] * B),
             free_queue=i32(r.sample(range(F), F)), free_range=i32([0, F]), page_size=ps,
             block_table=torch.full((B, width), -1, dtype=torch.int32),
             slot_mapping=torch.zeros(B, 40, dtype=torch.int32))
    g = on_gpu(x)
    cur = [0] * B
    for step in range(40):
        seq, fresh = [], []
        for b in range(B):
            u = r.random()
            if u < 0.1:
                cur[b], f = 0, 0
            else:
                cur[b] = max(0, cur[b] - (r.randint(0, 20) if u < 0.4 else 0))
                f = min(r.randint(0, 40), width * ps - cur[b])
                cur[b] += f
            seq.append(cur[b])
            fresh.append(f)
        x["seq_lens"], x["new_lens"] = i32(seq), i32(fresh)
        g["seq_lens"], g["new_lens"] = x["seq_lens"].cuda(), x["new_lens"].cuda()
        bt, slots, cu, held, queue, left, codes = spec.page_tables(**x)
        fw.build_page_tables(**g, held_out=g["held"], range_out=g["free_range"])
        torch.cuda.synchronize()
        status = fw.device_status()
        assert status in codes if codes else status == 0
        x.update(block_table=bt, held=held, free_queue=queue, free_range=left)
        for k in ("block_table", "held", "free_queue", "free_range"):
            assert torch.equal(g[k].cpu(), x[k]), (step, k)
        assert torch.equal(g["slot_mapping"].cpu(), slots), step
        for b in range(B):                        # a request that was not served keeps what it had
            cur[b] = min(cur[b], int(held[b]) * ps)
        have = [int(p) for b in range(B) for p in bt[b, :held[b]]]
        free = [int(queue[(left[0] + i) % F]) for i in range(int(left[1]))]
        assert sorted(have + free) == list(range(F)), step


@pytest.mark.parametrize("what", ["seq", "new", "held", "range", "count", "places", "width", "page", "room", "negative"])
def test_contradictions_are_reported(fw, what):
    x = table_case(12, 16, 0 if what == "places" else 6, seed=13, leave=0.0)
    if what == "seq":
        x["seq_lens"][3] = x["block_table"].shape[1] * 16 + 1
    elif what == "new":
        x["new_lens"][5] = x["seq_lens"][5] + 1
    elif what == "held":
        x["held"][2] = x["block_table"].shape[1] + 1
    elif what == "range":
        x["free_range"][0] = x["free_queue"].numel()
    elif what == "count":
        x["free_range"][1] = -1
    elif what == "places":
        x["slot_mapping"] = x["slot_mapping"][:10].clone()
    elif what == "width":
        x["slot_mapping"] = x["slot_mapping"][:, :2].contiguous()
    elif what == "page":
        x["free_queue"][:] = 2 ** 31 - 1
        x["block_table"][:] = -3
    elif what == "room":
        x["seq_lens"][:] = 0
        x["new_lens"][:] = 0
        x["free_range"][1] = x["free_queue"].numel() - 2
    elif what == "negative":
        x["seq_lens"][0], x["new_lens"][1], x["held"][4] = -1, -2, -3
    run_tables(fw, x, status=1)
    run_tables(fw, x, status=1, in_place=True)


def test_tables_of_nobody(fw):
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    q = torch.arange(5, dtype=torch.int32, device="cuda")
    slots = torch.zeros(6, dtype=torch.int32, device="cuda")
    cu, held, left = fw.build_page_tables(z, z, z, q, i32([2, 3]).cuda(), 16, z.view(0, 4), slots)
    torch.cuda.synchronize()
    assert cu.tolist() == [0] and left.tolist() == [2, 3] and (slots == -1).all() and fw.device_status() == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("leave", [False, True])
def test_many_pages_for_few_places(fw, in_place, leave):
    """Rows that take, or give back, hundreds of pages for a token each."""
    B, width, ps = 150, 1400, 8
    F = B * width + 5
    held = [width if leave else 0] * B
    bt = torch.full((B, width), -1, dtype=torch.int32)
    if leave:
        bt[:] = torch.arange(B * width, dtype=torch.int32).flip(0).view(B, width)
    seq = [0 if leave and b % 3 else width * ps - b for b in range(B)]
    x = dict(seq_lens=i32(seq), new_lens=i32([min(1, s) for s in seq]), held=i32(held),
             free_queue=torch.arange(F, dtype=torch.int32), free_range=i32([F - 3, 4 if leave else F]), page_size=ps,
             block_table=bt, slot_mapping=torch.zeros(B, 1, dtype=torch.int32))
    run_tables(fw, x, status=0, in_place=in_place)


def test_tables_on_two_streams(fw):
    cases = [table_case(300, 16, 0, seed=21 + i, new=300) for i in range(2)]
    refs = [spec.page_tables(**x) for x in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    runs = []
    for _ in range(6):
        gs = [on_gpu(x) for x in cases]
        torch.cuda.synchronize()
        for g, s in zip(gs, streams):
            runs.append((g, fw.build_page_tables(**g, held_out=g["held"], range_out=g["free_range"], stream=s)))
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    for i, (g, (cu, held, left)) in enumerate(runs):
        bt, slots, cu_r, held_r, queue, left_r, _ = refs[i % 2]
        assert torch.equal(cu.cpu(), cu_r) and torch.equal(held.cpu(), held_r) and torch.equal(left.cpu(), left_r)
        assert torch.equal(g["block_table"].cpu(), bt) and torch.equal(g["slot_mapping"].cpu(), slots)
        assert torch.equal(g["free_queue"].cpu(), queue)


def test_pages_without_new_tokens(fw):
    """Pages reserved ahead: no new token, no place."""
    B, width, ps = 5, 8, 16
    x = dict(seq_lens=i32([100, 0, 17, 128, 1]), new_lens=i32([0] * B), held=i32([0, 2, 0, 3, 1]),
             free_queue=torch.arange(100, 140, dtype=torch.int32), free_range=i32([35, 30]), page_size=ps,
             block_table=torch.arange(B * width, dtype=torch.int32).view(B, width),
             slot_mapping=torch.empty(0, dtype=torch.int32))
    run_tables(fw, x, status=0)
    x["slot_mapping"] = torch.empty(B, 0, dtype=torch.int32)
    run_tables(fw, x, status=0, in_place=True)


# ---------------------------------------------------------------- path commit

def commit_case(B, A, T, layers, Hkv, Dk, Dv, ps, kv8, seed, spare=2):
    r = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    base = [r.randint(0, 3 * ps + 5) for _ in range(B)]
    counts = [-(-(n + T) // ps) for n in base]
    P = sum(counts) + spare
    perm = torch.randperm(P, generator=g).to(torch.int32)
    bt = torch.full((B, max(counts)), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        bt[b, :c] = perm[at:at + c]
        at += c
    path = torch.stack([torch.randperm(T, generator=g)[:A].sort().values for _ in range(B)]).to(torch.int32)
    lens = i32([A if i == 0 else r.randint(0, A) for i in range(B)])
    dt = torch.float8_e4m3fn if kv8 else torch.bfloat16
    k = torch.randn(layers * P, ps, Hkv, Dk, generator=g).to(dt)
    v = torch.randn(layers * P, ps, Hkv, Dv, generator=g).to(dt) if Dv else None
    return path, lens, i32(base), bt, k, v


@pytest.mark.parametrize("B,A,T,layers,Hkv,Dk,Dv,ps,kv8", [
    (1, 1, 1, 1, 1, 128, 128, 16, False),
    (3, 4, 16, 1, 8, 128, 128, 128, False),
    (5, 7, 9, 3, 2, 128, 128, 8, False),           # most sources are destinations too, paths cross pages
    (2, 64, 100, 2, 2, 64, 128, 16, False),
    (2, 256, 256, 1, 1, 128, 128, 64, False),      # every draft accepted: nothing moves
    (4, 6, 33, 5, 4, 256, 256, 32, False),
    (4, 6, 33, 3, 3, 128, 128, 24, True),
    (9, 5, 20, 2, 1, 576, 0, 64, False),           # keys alone
    (40, 3, 12, 30, 8, 128, 128, 16, False),
    (2, 3, 12, 2, 60, 128, 128, 16, False),
])
def test_commit_moves_rows(fw, B, A, T, layers, Hkv, Dk, Dv, ps, kv8):
    path, lens, base, bt, k, v = commit_case(B, A, T, layers, Hkv, Dk, Dv, ps, kv8, seed=B + A)
    refs, new_ref = spec.commit(path, lens, base, bt, [k, v] if Dv else [k], layers)
    dk, dv = k.cuda(), (v.cuda() if Dv else None)
    new = fw.kv_commit(path.cuda(), lens.cuda(), base.cuda(), bt.cuda(), dk, dv, num_layers=layers)
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    assert torch.equal(new.cpu(), new_ref)
    assert torch.equal(raw(dk.cpu()), raw(refs[0]))
    if Dv:
        assert torch.equal(raw(dv.cpu()), raw(refs[1]))


def test_commit_of_interleaved_caches(fw):
    """K and V as the halves of every page of one buffer."""
    path, lens, base, bt, k, v = commit_case(4, 5, 14, 2, 2, 128, 128, 16, False, seed=3)
    refs, _ = spec.commit(path, lens, base, bt, [k, v], 2)
    kv = torch.stack([k, v], 1).contiguous().cuda()
    fw.kv_commit(path.cuda(), lens.cuda(), base.cuda(), bt.cuda(), kv[:, 0], kv[:, 1], num_layers=2)
    torch.cuda.synchronize()
    assert torch.equal(kv[:, 0].cpu(), refs[0]) and torch.equal(kv[:, 1].cpu(), refs[1])


def test_bad_paths_leave_the_cache(fw):
    path, lens, base, bt, k, v = commit_case(6, 4, 12, 1, 2, 128, 128, 16, False, seed=4)
    lens[:] = 4
    path[1] = i32([3, 2, 5, 6])                    # does not increase
    path[2] = i32([-1, 2, 5, 6])
    path[3, 3] = bt.shape[1] * 16                  # past the table row
    lens[4] = 5                                    # longer than the array
    path[5] = i32([0, 2, 5, 9])
    bt[5, (int(base[5]) + 9) // 16] = k.shape[0]   # a page outside the layer
    good = [0]
    refs, new_ref = spec.commit(path[good], lens[good], base[good], bt[good], [k, v])
    dk, dv = k.cuda(), v.cuda()
    new = fw.kv_commit(path.cuda(), lens.cuda(), base.cuda(), bt.cuda(), dk, dv)
    torch.cuda.synchronize()
    assert fw.device_status() == 1
    assert new.tolist() == [int(new_ref[0])] + base[1:].tolist()
    assert torch.equal(dk.cpu(), refs[0]) and torch.equal(dv.cpu(), refs[1])


def test_commit_of_nothing(fw):
    path, lens, base, bt, k, v = commit_case(4, 3, 9, 2, 2, 128, 128, 16, False, seed=9)
    dk, dv = k.cuda(), v.cuda()
    new = fw.kv_commit(path[:, :0].cuda(), torch.zeros_like(lens).cuda(), base.cuda(), bt.cuda(), dk, dv, num_layers=2)
    torch.cuda.synchronize()
    assert fw.device_status() == 0 and torch.equal(new.cpu(), base)
    assert torch.equal(raw(dk).cpu(), raw(k)) and torch.equal(raw(dv).cpu(), raw(v))


# ------------------------------------------------------------- a whole step

@pytest.mark.parametrize("kv8", [False, True])
def test_speculative_steps_end_to_end(fw, kv8):
    """Three steps of a two-layer cache, drafted, attended, accepted, committed;
    after each, every layer's rows and the attention over them are those of a
    plain model that keeps contiguous sequences."""
    r = random.Random(5)
    g = torch.Generator().manual_seed(9)
    B, T, Hq, Hkv, D, ps, layers, width, F = 3, 9, 8, 2, 128, 16, 2, 12, 40
    dt = torch.float8_e4m3fn if kv8 else torch.bfloat16
    ks, vs = (0.04, 0.05) if kv8 else (1.0, 1.0)
    kc = torch.zeros(layers * F, ps, Hkv, D, device="cuda").to(dt)
    vc = torch.zeros_like(kc)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    held = torch.zeros(B, dtype=torch.int32, device="cuda")
    ring = torch.randperm(F - 1, generator=g).to(torch.int32).cuda() + 1          # page 0 takes what has no slot
    ring_state = i32([0, F - 1]).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    history = [[[] for _ in range(B)] for _ in range(layers)]                     # (k, v) rows as stored

    def append(slots, k, v):
        for l in range(layers):
            fw.kv_append(k[l].cuda(), v[l].cuda(), slots, l * F * ps, kc, vc, k_scale=ks, v_scale=vs)

    def stored(x, s):
        if not kv8 or x.shape[0] == 0:
            return x.to(dt)
        c = torch.zeros(1, x.shape[0], Hkv, D).to(dt)
        return oracle.kv_append(x[None], x[None], torch.arange(x.shape[0], dtype=torch.int32), 0, c, c, k_scale=s,
                                v_scale=s)[0][0]

    # the prompts, tokens packed
    prompt = [20, 3, 45]
    new = i32(prompt).cuda()
    slots = torch.empty(sum(prompt), dtype=torch.int32, device="cuda")
    cu, held, ring_state = fw.build_page_tables(new, new, held, ring, ring_state, ps, table, slots)
    k = torch.randn(layers, sum(prompt), 1, Hkv, D, generator=g).to(torch.bfloat16)
    v = torch.randn(layers, sum(prompt), 1, Hkv, D, generator=g).to(torch.bfloat16)
    append(slots, k, v)
    for l in range(layers):
        for b in range(B):
            lo, hi = int(cu[b]), int(cu[b + 1])
            history[l][b] = [(stored(k[l, lo:hi, 0], ks), stored(v[l, lo:hi, 0], vs))]
    lens = lens + new

    for step in range(3):
        drafts = [T, r.randint(1, T), r.randint(1, T)]
        dl = i32(drafts).cuda()
        par = parents_of("tree", B, T, seed=step)
        mask, depths = fw.tree_mask(par.cuda(), draft_lens=dl)
        slots = torch.empty(B, T, dtype=torch.int32, device="cuda")
        seq = lens + dl
        _, held, ring_state = fw.build_page_tables(seq, dl, held, ring, ring_state, ps, table, slots)
        k = torch.randn(layers, B, T, Hkv, D, generator=g).to(torch.bfloat16)
        v = torch.randn(layers, B, T, Hkv, D, generator=g).to(torch.bfloat16)
        append(slots, k, v)
        q = torch.randn(B, T, Hq, D, generator=g).to(torch.bfloat16)
        for l in range(layers):
            out, lse = fw.paged_decode_tree(q.cuda(), kc[l * F:(l + 1) * F], vc[l * F:(l + 1) * F], table, seq, mask,
                                            1 / math.sqrt(D), draft_lens=dl, k_scale=ks, v_scale=vs)
            torch.cuda.synchronize()
            longest = max(int(lens[b]) + drafts[b] for b in range(B))
            flat_k = torch.zeros(B, longest, Hkv, D).to(dt)
            flat_v = torch.zeros_like(flat_k)
            for b in range(B):
                hk = torch.cat([raw(a) for a, _ in history[l][b]] + [raw(stored(k[l, b, :drafts[b]], ks))])
                hv = torch.cat([raw(a) for _, a in history[l][b]] + [raw(stored(v[l, b, :drafts[b]], vs))])
                raw(flat_k)[b, :hk.shape[0]] = hk
                raw(flat_v)[b, :hv.shape[0]] = hv
            ref = spec.tree_attention(q, flat_k, flat_v, torch.arange(B, dtype=torch.int32)[:, None], seq.cpu(),
                                      mask.cpu(), 1 / math.sqrt(D), dl.cpu(), ks, vs)
            check(out, lse, ref, D, f"step {step} layer {l}")
        # accept a path: from some draft up to its root
        path, m = torch.zeros(B, T, dtype=torch.int32), []
        for b in range(B):
            u, way = r.randrange(drafts[b]), []
            while u >= 0:
                way.append(u)
                u = int(par[b, u])
            way = way[::-1][:r.randint(0, T)]
            path[b, :len(way)] = i32(way)
            m.append(len(way))
            assert depths[b, way].tolist() == list(range(len(way))) if way else True
            for l in range(layers):
                history[l][b].append((stored(k[l, b, way], ks), stored(v[l, b, way], vs)))
        lens = fw.kv_commit(path.cuda(), i32(m).cuda(), lens, table, kc, vc, num_layers=layers)
        torch.cuda.synchronize()
        assert fw.device_status() == 0
        for l in range(layers):
            for b in range(B):
                n = int(lens[b])
                pages = table[b, :-(-n // ps)].long() + l * F
                rows = raw(kc)[pages].reshape(-1, Hkv, D)[:n].cpu(), raw(vc)[pages].reshape(-1, Hkv, D)[:n].cpu()
                want = [torch.cat([raw(h[i]) for h in history[l][b]]) for i in (0, 1)]
                assert n == want[0].shape[0]
                assert torch.equal(rows[0], want[0]) and torch.equal(rows[1], want[1]), (step, l, b)


def test_a_captured_step_equals_the_eager_one(fw):
    """One graph of a whole step, state updated in place, replayed for steps of
    other lengths, trees and queries, against eager calls on state of their own;
    the cache, the tables and the outputs are equal bit for bit."""
    r = random.Random(15)
    g = torch.Generator().manual_seed(19)
    B, T, Hq, Hkv, D, ps, layers, width, F = 6, 20, 8, 2, 128, 16, 2, 40, 260
    bf = torch.bfloat16

    def state():
        return dict(kc=torch.zeros(layers * F, ps, Hkv, D, dtype=bf, device="cuda"),
                    vc=torch.zeros(layers * F, ps, Hkv, D, dtype=bf, device="cuda"),
                    table=torch.full((B, width), -1, dtype=torch.int32, device="cuda"),
                    held=torch.zeros(B, dtype=torch.int32, device="cuda"),
                    ring=torch.arange(1, F, dtype=torch.int32, device="cuda"),
                    left=i32([0, F - 1]).cuda(), slots=torch.zeros(B, T, dtype=torch.int32, device="cuda"),
                    lens=torch.zeros(B, dtype=torch.int32, device="cuda"))

    def step(s, x):
        seq = s["lens"] + x["dl"]
        mask, depths = fw.tree_mask(x["par"], draft_lens=x["dl"])
        fw.build_page_tables(seq, x["dl"], s["held"], s["ring"], s["left"], ps, s["table"], s["slots"],
                             held_out=s["held"], range_out=s["left"])
        outs = [mask, depths]
        for l in range(layers):
            fw.kv_append(x["k"][l], x["v"][l], s["slots"], l * F * ps, s["kc"], s["vc"])
            outs += fw.paged_decode_tree(x["q"], s["kc"][l * F:(l + 1) * F], s["vc"][l * F:(l + 1) * F], s["table"], seq,
                                         mask, 0.09, draft_lens=x["dl"])
        s["lens"].copy_(fw.kv_commit(x["path"], x["m"], s["lens"], s["table"], s["kc"], s["vc"], num_layers=layers))
        return outs

    def inputs(seed):
        drafts = [r.randint(0, T) for _ in range(B)]
        par = parents_of("tree", B, T, seed=seed)
        path, m = torch.zeros(B, T, dtype=torch.int32), []
        for b in range(B):
            u, way = drafts[b] - 1, []
            while u >= 0:
                way.append(u)
                u = int(par[b, u])
            path[b, :len(way)] = i32(way[::-1])
            m.append(len(way))
        rnd = lambda *s: torch.randn(*s, generator=g).to(bf)
        return {k: v.cuda() for k, v in dict(
            par=par, dl=i32(drafts), path=path, m=i32(m), q=rnd(B, T, Hq, D), k=rnd(layers, B, T, Hkv, D),
            v=rnd(layers, B, T, Hkv, D)).items()}

    static = inputs(0)
    warm, graph_state, eager_state = state(), state(), state()
    step(warm, static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(graph_state, static)
    for n in range(5):
        x = inputs(n + 1)
        for k in static:
            static[k].copy_(x[k])
        graph.replay()
        want = step(eager_state, x)
        torch.cuda.synchronize()
        assert fw.device_status() == 0
        for a, b in zip(captured, want):
            assert torch.equal(a, b), n
        for s in (graph_state, eager_state):
            for k in ("kc", "vc"):                # row 0 of a layer takes every place without a token, in any order
                s[k].view(layers, F, ps, Hkv, D)[:, 0, 0] = 0
        for k in eager_state:
            assert torch.equal(graph_state[k], eager_state[k]), (n, k)
