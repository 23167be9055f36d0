"""Tree decode on the GPU against the 64-bit definition.

The bound of an output element, from the arithmetic alone: every probability is
rounded to BF16 for the product (half a step, u = 2^-8 relative; against a row
sum of unrounded ones that moves the output by at most u * absv, and 2u covers
either way of summing); an FP32 score of D products is off by at most
(D + 8) * 2^-24 * sum |q_i k_i| * scale, which moves every weight by that much
relative, numerator and denominator; exponentials, sums and the merge of pieces
by less than 2^-18 relative; the result is rounded to BF16, 2^-8 of its value.
LSE: the score's error plus 2^-20 of its magnitude plus 2^-18.  Over an 8-bit
cache a query element below 2^-10 of its row's largest is carried to within
2^-17 of that largest, so a score may be off by another 2^-17 * max |q_i| *
sum |k_i| * scale.
"""
import math

import numpy as np
import pytest
import torch

from oracle import spec
from tests.gpu_common import built_library

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


@pytest.fixture(scope="module")
def fw():
    return built_library()


def parents_of(kind, B, T, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "chain":
        return (torch.arange(T) - 1).to(torch.int32).repeat(B, 1)
    if kind == "star":
        return torch.full((B, T), -1, dtype=torch.int32)
    t = torch.arange(T).repeat(B, 1)
    back = 1 + (torch.rand(B, T, generator=g) ** 2 * 10).long()
    return torch.clamp(t - back, min=-1).to(torch.int32)


def mask_of(kind, B, T, seed):
    W = -(-T // 32)
    g = torch.Generator().manual_seed(seed)
    if kind == "none":
        return torch.zeros(B, T, W, dtype=torch.int32)
    if kind == "all":
        return torch.full((B, T, W), -1, dtype=torch.int32)
    if kind == "noise":                    # any relation: later drafts, missing diagonals, empty rows
        m = torch.randint(-2 ** 31, 2 ** 31, (B, T, W), generator=g, dtype=torch.int64).to(torch.int32)
        m[:, ::5] = 0
        return m
    return spec.tree_mask(parents_of(kind, B, T, seed))[0]


def make(B, T, Hq, Hkv, D, ps, lens, drafts=None, mask="tree", kv8=False, seed=0, spare=2, width=None, amp=1.0):
    """Inputs on the CPU: pages in random order, entries past a row's last page
    -1, spare pages and the slots past a row's end NaN."""
    g = torch.Generator().manual_seed(1000 + seed)
    counts = [-(-n // ps) for n in lens]
    P = sum(counts) + spare
    perm = torch.randperm(P, generator=g).to(torch.int32)
    width = width or max(1, max(counts))
    bt = torch.full((B, width), -1, dtype=torch.int32)
    dt = torch.float8_e4m3fn if kv8 else torch.bfloat16
    k = (torch.randn(P, ps, Hkv, D, generator=g) * (30.0 if kv8 else 1.0)).clamp(-448, 448)
    v = (torch.randn(P, ps, Hkv, D, generator=g) * (30.0 if kv8 else 1.0)).clamp(-448, 448)
    used = torch.zeros(P, ps, dtype=torch.bool)
    at = 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        bt[b, :c] = perm[at:at + c]
        for i in range(c):
            used[perm[at + i].long(), :min(ps, n - i * ps)] = True
        at += c
    k[~used] = math.nan
    v[~used] = math.nan
    q = (torch.randn(B, T, Hq, D, generator=g) * amp).to(torch.bfloat16)
    return dict(q=q, k_cache=k.to(dt), v_cache=v.to(dt), block_table=bt,
                seq_lens=torch.tensor(lens, dtype=torch.int32),
                draft_lens=None if drafts is None else torch.tensor(drafts, dtype=torch.int32),
                tree_mask=mask_of(mask, B, T, seed), scale=1.0 / math.sqrt(D),
                k_scale=0.031 if kv8 else 1.0, v_scale=0.02 if kv8 else 1.0)


def on_gpu(x):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}


def check(out, lse, ref, D, what):
    o_ref, l_ref, absv, reach, spread = ref
    o = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(o).all(), f"{what}: non-finite output"
    delta = (D + 8) * 2.0 ** -24 * reach + 2.0 ** -17 * spread
    d = (2 * U + 2 * delta[..., None] + 2.0 ** -18) * absv
    bound = d + U * (np.abs(o_ref) + d) + 1e-30
    diff = np.abs(o - o_ref)
    worst = np.unravel_index(np.argmax(diff / bound), diff.shape)
    assert diff[worst] <= bound[worst], (what, worst, diff[worst], bound[worst], o_ref[worst])
    if lse is not None:
        l = lse.cpu().numpy().astype(np.float64)
        empty = np.isneginf(l_ref)
        assert np.array_equal(np.isneginf(l), empty), f"{what}: empty rows differ"
        assert (o[empty] == 0).all(), f"{what}: an empty row is not zero"
        tol = delta + 2.0 ** -20 * np.abs(np.where(empty, 0, l_ref)) + 2.0 ** -18
        assert (np.abs(l - np.where(empty, 0, l_ref))[~empty] <= tol[~empty]).all(), f"{what}: lse"


def run_and_check(fw, x, what, **kw):
    g = on_gpu(x)
    out, lse = fw.paged_decode_tree(**g, **kw)
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    check(out, lse, spec.tree_attention(**x), x["q"].shape[-1], what)
    return out, lse


# batch, drafts, heads, KV heads, head dim, page size, lengths, draft counts, mask
CASES = [
    (1, 1, 8, 2, 128, 16, [1], None, "tree"),
    (2, 1, 8, 2, 128, 16, [37, 200], None, "all"),
    (3, 5, 40, 8, 128, 16, [5, 128, 133], None, "tree"),
    (4, 8, 8, 2, 128, 8, [0, 8, 9, 257], [8, 8, 3, 0], "tree"),
    (2, 16, 40, 8, 128, 128, [1000, 131], [16, 7], "tree"),
    (1, 31, 24, 3, 128, 32, [700], None, "chain"),
    (2, 32, 16, 16, 128, 64, [160, 33], None, "star"),
    (2, 33, 7, 1, 128, 16, [33, 1500], [33, 20], "noise"),
    (1, 64, 32, 8, 128, 64, [2000], None, "noise"),
    (2, 65, 12, 12, 128, 256, [300, 65], None, "none"),
    (1, 121, 8, 2, 128, 16, [1111], None, "tree"),
    (1, 256, 4, 2, 128, 32, [800], None, "tree"),
    (2, 256, 8, 8, 128, 128, [256, 700], [256, 255], "noise"),
    (1, 3, 160, 1, 128, 64, [500], None, "tree"),
    (1, 2, 300, 2, 128, 64, [260], None, "all"),
    (2, 6, 128, 1, 128, 64, [390, 129], None, "tree"),
    (2, 4, 16, 16, 256, 32, [100, 515], None, "tree"),
    (3, 24, 16, 16, 256, 64, [24, 1300, 400], [24, 24, 9], "noise"),
    (1, 40, 8, 1, 256, 128, [900], None, "tree"),
    (1, 5, 200, 1, 256, 16, [333], None, "chain"),
    (70, 2, 4, 1, 128, 16, [(37 * i) % 300 for i in range(70)], None, "chain"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(i) for i in c[:6]) + "-" + c[8])
def test_matches_definition(fw, case):
    B, T, Hq, Hkv, D, ps, lens, drafts, mask = case
    run_and_check(fw, make(B, T, Hq, Hkv, D, ps, lens, drafts, mask, seed=T + Hq), f"case {case}")


@pytest.mark.parametrize("case", [c for c in CASES if c[4] == 128][::2],
                         ids=lambda c: "-".join(str(i) for i in c[:6]) + "-" + c[8])
def test_fp8_cache_matches_definition(fw, case):
    B, T, Hq, Hkv, D, ps, lens, drafts, mask = case
    run_and_check(fw, make(B, T, Hq, Hkv, D, ps, lens, drafts, mask, kv8=True, seed=T), f"fp8 {case}")


@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
def test_every_offset_of_the_drafts_inside_a_tile(fw, D, kv8):
    """The drafts begin at every place of a 128-key tile, some reach over its end."""
    lens = [40 + n for n in range(0, 260, 13)]
    run_and_check(fw, make(len(lens), 40, 4, 2, D, 16, lens, None, "noise", kv8=kv8, seed=3), "offsets")


@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
def test_long_rows_are_split_and_merged(fw, D, kv8):
    run_and_check(fw, make(2, 9, 8, 2, D, 64, [9000, 77], None, "tree", kv8=kv8, seed=5), "long")


@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
@pytest.mark.parametrize("T,Hq,Hkv", [(24, 16, 16), (40, 16, 4)])
def test_many_pieces_per_cta(fw, D, kv8, T, Hq, Hkv):
    """Several units to a CTA, every one with a tile that holds drafts while the
    copies of the next tiles and units are in flight."""
    lens = [150 + 211 * i % 1800 for i in range(10)]
    x = make(10, T, Hq, Hkv, D, 32, lens, [T - i for i in range(10)], "tree", kv8=kv8, seed=43)
    first = run_and_check(fw, x, "many pieces")
    g = on_gpu(x)
    for _ in range(20):
        again = fw.paged_decode_tree(**g)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("scale", [-0.7, 0.0, 1.5])
def test_scales_that_move_the_maximum(fw, scale):
    """A large scale makes later tiles outgrow what the first ones showed; a
    negative one turns the order round; zero makes every weight equal."""
    x = make(2, 12, 8, 2, 128, 32, [900, 390], None, "tree", seed=9)
    x["scale"] = scale
    run_and_check(fw, x, f"scale {scale}")


def test_scores_that_rise_along_the_cache(fw):
    """Keys aligned with the query grow along the row, so the row maximum moves in every tile."""
    x = make(1, 4, 2, 1, 128, 64, [1400], None, "tree", seed=11)
    grow = torch.linspace(0, 6, 1400)
    pages = x["block_table"][0, :-(-1400 // 64)].long()
    k = x["k_cache"][pages].float().reshape(-1, 1, 128)
    k[:1400] = (x["q"][0, 0, 0].float()[None, None, :] * grow[:, None, None] + 0.1 * k[:1400])
    x["k_cache"][pages] = k.to(torch.bfloat16).reshape(len(pages), 64, 1, 128)
    run_and_check(fw, x, "rising scores")


def test_nothing_hidden_is_read(fw):
    """Keys no row sees are NaN or infinite in K and V, padding queries NaN."""
    x = make(2, 10, 8, 2, 128, 16, [150, 40], [10, 6], "chain", seed=13)
    for b, (n, d) in enumerate(((150, 10), (40, 6))):
        dead = n - d + d // 2                                 # nobody sees this draft, not even itself
        page, off = int(x["block_table"][b, dead // 16]), dead % 16
        x["k_cache"][page, off] = math.nan if b else math.inf
        x["v_cache"][page, off] = math.inf if b else math.nan
        j = d // 2
        x["tree_mask"][b, :, 0] &= ~(1 << j)
    x["q"][1, 6:] = math.nan
    g = on_gpu(x)
    out, lse = fw.paged_decode_tree(**g)
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    clean = dict(x)
    for name in ("k_cache", "v_cache"):
        clean[name] = torch.nan_to_num(x[name].float(), nan=0.0, posinf=0.0).to(torch.bfloat16)
    clean["q"] = torch.nan_to_num(x["q"])
    check(out, lse, spec.tree_attention(**clean), 128, "hidden keys")


def test_strided_views(fw):
    """Q, out and lse as views of wider buffers, K and V the halves of one
    cache, a table with spare columns, a mask inside a wider one."""
    x = make(2, 7, 8, 2, 128, 32, [100, 260], [7, 5], "tree", seed=17, width=20)
    g = on_gpu(x)
    q = torch.full((2, 9, 16, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    q[:, 1:8, 4:12] = g["q"]
    kv = torch.stack([g["k_cache"].float(), g["v_cache"].float()], 1).to(torch.bfloat16).contiguous()
    wide = torch.full((2, 7, 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :, :1] = g["tree_mask"]
    table = torch.full((2, 33), -7, dtype=torch.int32, device="cuda")
    table[:, :20] = g["block_table"]
    obuf = torch.full((2, 9, 10, 160), 7.0, dtype=torch.bfloat16, device="cuda")
    lbuf = torch.full((2, 7, 11), 7.0, device="cuda")
    out, lse = fw.paged_decode_tree(q[:, 1:8, 4:12], kv[:, 0], kv[:, 1], table[:, :20], g["seq_lens"], wide,
                                    x["scale"], draft_lens=g["draft_lens"], out=obuf[:, 1:8, 1:9, 16:144],
                                    lse=lbuf[:, :, 2:10])
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    check(out, lse, spec.tree_attention(**x), 128, "views")
    keep = torch.ones_like(obuf, dtype=torch.bool)
    keep[:, 1:8, 1:9, 16:144] = False
    assert (obuf[keep] == 7).all(), "written outside the output view"
    assert (lbuf[:, :, :2] == 7).all() and (lbuf[:, :, 10:] == 7).all()


def test_chain_equals_the_causal_decode(fw):
    """A chain of up to four drafts is what the causal decode computes."""
    x = make(3, 4, 40, 8, 128, 64, [4, 300, 2000], None, "chain", seed=19)
    g = on_gpu(x)
    out, lse = fw.paged_decode_tree(**g)
    o2, l2 = fw.paged_decode(g["q"], g["k_cache"], g["v_cache"], g["block_table"], g["seq_lens"], x["scale"])
    torch.cuda.synchronize()
    ref = spec.tree_attention(**x)
    check(out, lse, ref, 128, "tree chain")
    check(o2, l2, ref, 128, "causal decode")


def test_lengths_outside_the_table_are_clamped(fw):
    x = make(2, 4, 8, 2, 128, 16, [64, 30], None, "tree", seed=21)
    g = on_gpu(x)
    g["seq_lens"] = torch.tensor([10 ** 6, -5], dtype=torch.int32, device="cuda")
    g["draft_lens"] = torch.tensor([9, 4], dtype=torch.int32, device="cuda")
    out, lse = fw.paged_decode_tree(**g)
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    y = dict(x, seq_lens=torch.tensor([64, 0], dtype=torch.int32), draft_lens=torch.tensor([4, 0], dtype=torch.int32))
    check(out, lse, spec.tree_attention(**y), 128, "clamped")


def test_a_bad_page_is_reported(fw):
    x = make(1, 4, 8, 2, 128, 16, [64], None, "tree", seed=23)
    g = on_gpu(x)
    g["block_table"][0, 1] = 10 ** 6
    fw.paged_decode_tree(**g)
    torch.cuda.synchronize()
    assert fw.device_status() == 1                 # FW_ERR_INVALID_ARG


def test_repeats_are_bitwise_equal(fw):
    x = on_gpu(make(8, 20, 40, 8, 128, 64, [300 + 517 * i for i in range(8)], None, "tree", seed=25))
    first = fw.paged_decode_tree(**x)
    for _ in range(5):
        again = fw.paged_decode_tree(**x)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("ctas", [1, 2, 5])
@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
def test_few_ctas(fw, ctas, D, kv8):
    x = make(3, 50, 10, 2, D, 32, [500, 50, 1200], [50, 50, 13], "tree", kv8=kv8, seed=27)
    fw.set_option(fw.FW_OPT_MAX_CTAS, ctas)
    try:
        run_and_check(fw, x, f"{ctas} CTAs")
    finally:
        fw.set_option(fw.FW_OPT_MAX_CTAS, 0)


def test_two_streams_and_a_graph(fw):
    """Calls in flight on two streams and a captured one keep their own
    workspaces: each gives what it gives alone."""
    xs = [on_gpu(make(4, 30, 40, 8, 128, 64, [3000 + 100 * i, 200, 900, 4000], None, "tree", seed=30 + i))
          for i in range(3)]
    alone = [fw.paged_decode_tree(**x) for x in xs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = fw.paged_decode_tree(**xs[2])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        a = fw.paged_decode_tree(**xs[0], stream=s1)
        b = fw.paged_decode_tree(**xs[1], stream=s2)
        graph.replay()
        got.append((a, b))
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    for a, b in got:
        assert torch.equal(a[0], alone[0][0]) and torch.equal(a[1], alone[0][1])
        assert torch.equal(b[0], alone[1][0]) and torch.equal(b[1], alone[1][1])
    assert torch.equal(captured[0], alone[2][0]) and torch.equal(captured[1], alone[2][1])


def test_callers_workspace_and_no_lse(fw):
    x = make(2, 9, 8, 2, 128, 64, [3000, 77], None, "tree", seed=35)
    g = on_gpu(x)
    ws = torch.empty(max(256, fw.paged_decode_tree_workspace_size(128)), dtype=torch.uint8, device="cuda")
    out, lse = fw.paged_decode_tree(**g, workspace=ws)
    o2, l2 = fw.paged_decode_tree(**g, return_lse=False)
    torch.cuda.synchronize()
    assert l2 is None and torch.equal(out, o2)
    check(out, lse, spec.tree_attention(**x), 128, "own workspace")


def test_empty_batch(fw):
    q = torch.empty(0, 4, 8, 128, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(1, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    out, lse = fw.paged_decode_tree(q, c, c.clone(), z.view(0, 1), z, z.view(0, 4, 1), 0.1)
    assert out.shape == (0, 4, 8, 128) and lse.shape == (0, 4, 8)


def test_a_cache_past_32_bit_offsets(fw):
    """Pages whose element offsets pass 2^32: the row's pages lie at both ends of an 8.6 GB cache."""
    Hkv, D, ps = 8, 128, 128
    P = (2 ** 32) // (ps * Hkv * D) + 3
    x = make(1, 6, 16, Hkv, D, ps, [4 * ps + 11], None, "tree", seed=37, spare=0)
    pages = torch.tensor([0, P - 1, 1, P - 2, P - 3], dtype=torch.int32)
    g = on_gpu(x)
    for name in ("k_cache", "v_cache"):
        big = torch.empty(P, ps, Hkv, D, dtype=torch.bfloat16, device="cuda")
        big[pages.cuda().long()] = g[name][g["block_table"][0].long()]
        g[name] = big
    g["block_table"] = pages[None].cuda()
    out, lse = fw.paged_decode_tree(**g)
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    check(out, lse, spec.tree_attention(**x), D, "large cache")


@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
@pytest.mark.parametrize("T,Hq", [(9, 8), (70, 8)])
def test_nan_stays_in_the_rows_that_see_it(fw, D, kv8, T, Hq):
    """NaN in a query row, in a committed key (one KV head of one request) and in
    the key of a draft some rows see: those rows are NaN, LSE too, all others
    what they are without it; in rows of one piece and of many."""
    Hkv, ps = 2, 64
    x = make(3, T, Hq, Hkv, D, ps, [9000, 300, 5000], [T, T - 2, T], "tree", kv8=kv8, seed=41)
    ref = spec.tree_attention(**x)
    hit = torch.zeros(3, T, Hq, dtype=torch.bool)
    y = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}

    def spoil(b, pos, g):
        k = y["k_cache"].view(torch.uint8 if kv8 else torch.int16)
        k[int(x["block_table"][b, pos // ps]), pos % ps, g, 3] = 0x7f if kv8 else 0x7fff

    y["q"][0, 1, 2, 7] = math.nan
    y["q"][1, 3, 5, 0] = math.nan
    hit[0, 1, 2] = hit[1, 3, 5] = True
    spoil(1, 100, 1)
    hit[1, :T - 2, Hq // 2:] = True
    j = 4                                                     # a draft of request 2
    spoil(2, 5000 - T + j, 0)
    sees = (x["tree_mask"][2, :, j // 32].numpy().astype(np.int64) >> (j % 32)) & 1
    hit[2, :, :Hq // 2] |= torch.from_numpy(sees.astype(bool))[:, None]
    assert sees.any() and not sees.all()
    out, lse = fw.paged_decode_tree(**on_gpu(y))
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    out, lse = out.cpu(), lse.cpu()
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    out[hit] = torch.from_numpy(ref[0])[hit].to(torch.bfloat16)
    lse[hit] = torch.from_numpy(ref[1])[hit].float()
    check(out, lse, ref, D, "rows without NaN")


def test_the_largest_batch(fw):
    lens = [(7 * i) % 41 for i in range(4096)]
    x = make(4096, 2, 2, 1, 128, 16, lens, [i % 3 for i in range(4096)], "chain", seed=43)
    run_and_check(fw, x, "4096 requests")


@pytest.mark.parametrize("kv8", [False, True])
def test_pages_shared_by_requests(fw, kv8):
    """One prompt's pages in several rows, and the same page twice in a row."""
    x = make(4, 12, 8, 2, 128, 32, [500, 500, 700, 300], None, "tree", kv8=kv8, seed=45)
    x["block_table"][1, :10] = x["block_table"][0, :10]
    x["block_table"][2, :10] = x["block_table"][0, :10]
    x["block_table"][3, 5] = x["block_table"][3, 2]
    run_and_check(fw, x, "shared pages")


def test_two_graphs_on_one_workspace(fw):
    """Graphs captured with the same workspace, replayed one after another."""
    xs = [on_gpu(make(3, 20, 40, 8, 128, 64, [2500 + 700 * i, 90, 3100], None, "tree", seed=47 + i)) for i in range(2)]
    alone = [fw.paged_decode_tree(**x) for x in xs]
    ws = torch.empty(fw.paged_decode_tree_workspace_size(128), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graphs, got = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(fw.paged_decode_tree(**x, workspace=ws))
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(got[i][0], alone[i][0]) and torch.equal(got[i][1], alone[i][1])
        for o, l in got:
            o.zero_(), l.zero_()
    assert fw.device_status() == 0


@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
@pytest.mark.parametrize("T", [5, 70])
def test_pages_that_are_no_power_of_two(fw, D, kv8, T):
    x = make(2, T, 8, 2, D, 384, [1500, 385], [T, T - 1], "tree", kv8=kv8, seed=51)
    run_and_check(fw, x, "384-slot pages")


@pytest.mark.parametrize("Hq,Hkv,T", [(160, 1, 3), (300, 2, 2), (128, 1, 6), (7, 1, 40)])
def test_fp8_odd_groups(fw, Hq, Hkv, T):
    run_and_check(fw, make(2, T, Hq, Hkv, 128, 16, [700, 130], None, "noise", kv8=True, seed=53), "odd groups")


def test_fp8_strided_views(fw):
    """K and V the halves of one 8-bit cache, Q and out inside wider buffers."""
    x = make(2, 7, 8, 2, 128, 32, [100, 260], [7, 5], "tree", kv8=True, seed=55)
    g = on_gpu(x)
    kv = torch.stack([g["k_cache"].view(torch.uint8), g["v_cache"].view(torch.uint8)], 3).view(torch.float8_e4m3fn)
    q = torch.full((2, 9, 16, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    q[:, 1:8, 4:12] = g["q"]
    obuf = torch.full((2, 9, 10, 160), 7.0, dtype=torch.bfloat16, device="cuda")
    g.update(q=q[:, 1:8, 4:12], k_cache=kv[:, :, :, 0], v_cache=kv[:, :, :, 1])
    out, lse = fw.paged_decode_tree(**g, out=obuf[:, 1:8, 1:9, 16:144])
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    check(out, lse, spec.tree_attention(**x), 128, "FP8 views")
    keep = torch.ones_like(obuf, dtype=torch.bool)
    keep[:, 1:8, 1:9, 16:144] = False
    assert (obuf[keep] == 7).all(), "written outside the output view"


@pytest.mark.parametrize("kv8", [False, True])
def test_expanded_inputs(fw, kv8):
    """One tree and one table row for every request, as expanded views."""
    x = make(1, 12, 8, 2, 128, 32, [500], None, "tree", kv8=kv8, seed=57)
    B = 3
    y = dict(x)
    y["block_table"], y["tree_mask"] = x["block_table"].expand(B, -1), x["tree_mask"].expand(B, -1, -1)
    y["seq_lens"] = torch.tensor([500, 100, 12], dtype=torch.int32)
    y["q"] = torch.cat([x["q"], -x["q"], x["q"].flip(1)])
    g = on_gpu(y)
    g["block_table"], g["tree_mask"] = x["block_table"].cuda().expand(B, -1), x["tree_mask"].cuda().expand(B, -1, -1)
    assert g["tree_mask"].stride(0) == 0 and g["block_table"].stride(0) == 0
    out, lse = fw.paged_decode_tree(**g)
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    check(out, lse, spec.tree_attention(**y), 128, "expanded")


@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
def test_nobody_drafts(fw, D, kv8):
    x = on_gpu(make(3, 9, 8, 2, D, 16, [100, 0, 7], [0, 5, -3], "tree", kv8=kv8, seed=59))
    out = torch.full((3, 9, 8, D), 7.0, dtype=torch.bfloat16, device="cuda")
    _, lse = fw.paged_decode_tree(**x, out=out)
    torch.cuda.synchronize()
    assert fw.device_status() == 0 and (out == 0).all() and torch.isneginf(lse).all()


def test_workspaces_that_do_not_fit(fw):
    x = on_gpu(make(1, 4, 8, 2, 128, 16, [100], None, "tree", seed=61))
    n = fw.paged_decode_tree_workspace_size(128)
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    before = fw.launch_count()
    with pytest.raises(fw.FwError, match="workspace"):
        fw.paged_decode_tree(**x, workspace=ws[:n - 1])
    with pytest.raises(fw.FwError, match="aligned"):
        fw.paged_decode_tree(**x, workspace=ws[16:])
    with pytest.raises(ValueError, match="contiguous"):
        fw.paged_decode_tree(**x, workspace=ws[::2])
    with pytest.raises(ValueError, match="CUDA"):
        fw.paged_decode_tree(**x, workspace=torch.empty(n, dtype=torch.uint8))
    assert fw.launch_count() == before


@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
@pytest.mark.parametrize("T,Hq", [(9, 8), (70, 8), (200, 2)])
def test_values_that_are_not_finite(fw, D, kv8, T, Hq):
    """A draft's NaN or infinite value reaches the rows that see the draft, in one
    KV head, and nobody else; a committed key's reaches every row."""
    Hkv, ps = 2, 64
    lens, drafts = [9000, 300, 5003, 640], [T, T - 2, T, T - 1]
    x = make(4, T, Hq, Hkv, D, ps, lens, drafts, "tree", kv8=kv8, seed=63)
    ref = spec.tree_attention(**x)
    y = dict(x, v_cache=x["v_cache"].clone())
    hit = torch.zeros(4, T, Hq, dtype=torch.bool)
    G = Hq // Hkv

    def spoil(b, pos, g, col, bits):
        v = y["v_cache"].view(torch.uint8 if kv8 else torch.int16)
        v[int(x["block_table"][b, pos // ps]), pos % ps, g, col] = bits

    def sees(b, j):
        return torch.from_numpy(((x["tree_mask"][b, :, j // 32].numpy().astype(np.int64) >> (j % 32)) & 1).astype(bool))

    nan, inf = (0x7f, 0xff) if kv8 else (0x7fc1, 0x7f80)     # E4M3 has no infinity: both NaNs
    for b, j, g, col, bits in ((0, 4, 0, 3, nan), (0, T - 1, 1, D - 1, inf), (2, 0, 1, 64, inf), (3, 2, 0, 0, nan)):
        spoil(b, lens[b] - drafts[b] + j, g, col, bits)
        if j < drafts[b]:
            s = sees(b, j)
            s[drafts[b]:] = False
            hit[b, :, g * G:(g + 1) * G] |= s[:, None]
    assert hit.any() and not hit[0].all()
    out, lse = fw.paged_decode_tree(**on_gpu(y))
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    out, lse = out.cpu(), lse.cpu()
    assert torch.isnan(out[hit]).all()
    out[hit] = torch.from_numpy(ref[0])[hit].to(torch.bfloat16)
    check(out, lse, ref, D, "rows without such values")

    spoil(1, 7, 1, 5, nan)                                    # committed
    out, _ = fw.paged_decode_tree(**on_gpu(y))
    torch.cuda.synchronize()
    assert torch.isnan(out[1, :T - 2, G:, 5]).all() and torch.isfinite(out[1, :, :G]).all()
    assert torch.isfinite(out[1, :T - 2, G:, :5]).all()
