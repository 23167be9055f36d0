"""Chunk attention over a paged cache against the 64-bit definition.

The bound of an output element, from the arithmetic alone, is that of the tree
decode over a BF16 cache (E4M3 values are widened exactly, and queries over them carried
exactly down to 2^-10 of a row's largest element; normal ones below, one in 400, are off by
2^-17 of it, a hundredth of the scores' bound): weights rounded to BF16
(2u absv, u = 2^-8, covers either way of summing), FP32 scores of D products off by
(D + 8) 2^-24 sum |q_i k_i| scale, exponentials, sums and the merge by less than 2^-18
relative, the result rounded to BF16.  LSE: the score's error plus 2^-20 of its
magnitude plus 2^-18."""
import math

import numpy as np
import pytest
import torch

from oracle import step
from tests.gpu_common import built_library

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def fw():
    return built_library()


def make(d, n, Hq, Hkv, D, ps, kv8=False, seed=0, spare=2, width=None, amp=1.0, behind=0, first=0):
    """Inputs on the CPU: pages in random order, entries past a row's last page -1,
    spare pages and the places past a row's end NaN; `behind` rows of no request,
    `first` rows before the first."""
    g = torch.Generator().manual_seed(2000 + seed)
    counts = [-(-x // ps) for x in n]
    P = sum(counts) + spare
    perm = torch.randperm(P, generator=g).to(torch.int32)
    bt = torch.full((len(n), width or max(1, max(counts))), -1, dtype=torch.int32)
    dt = torch.float8_e4m3fn if kv8 else torch.bfloat16
    k, v = ((torch.randn(P, ps, Hkv, D, generator=g) * (30.0 if kv8 else 1.0)).clamp(-448, 448) for _ in range(2))
    used = torch.zeros(P, ps, dtype=torch.bool)
    at = 0
    for b, (x, c) in enumerate(zip(n, counts)):
        bt[b, :c] = perm[at:at + c]
        for i in range(c):
            used[perm[at + i].long(), :min(ps, x - i * ps)] = True
        at += c
    k[~used] = math.nan
    v[~used] = math.nan
    cu = [first]
    for x in d:
        cu.append(cu[-1] + x)
    q = (torch.randn(cu[-1] + behind, Hq, D, generator=g) * amp).to(torch.bfloat16)
    return dict(q=q, k_cache=k.to(dt), v_cache=v.to(dt), block_table=bt, cu_seqlens_q=torch.tensor(cu, dtype=torch.int32),
                seq_lens=torch.tensor(n, dtype=torch.int32), scale=1.0 / math.sqrt(D), k_scale=0.031 if kv8 else 1.0,
                v_scale=0.02 if kv8 else 1.0)


def on_gpu(x):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}


def check(out, lse, ref, D, what):
    o_ref, l_ref, absv, reach = ref
    mine = ~np.isnan(l_ref)                               # rows of requests
    o = out.float().cpu().numpy().astype(np.float64)[mine]
    o_ref, l_ref, absv, reach = o_ref[mine], l_ref[mine], absv[mine], reach[mine]
    assert np.isfinite(o).all(), f"{what}: non-finite output"
    delta = (D + 8) * 2.0 ** -24 * reach
    d = (2 * U + 2 * delta[..., None] + 2.0 ** -18) * absv
    bound = d + U * (np.abs(o_ref) + d) + 1e-30
    diff = np.abs(o - o_ref)
    worst = np.unravel_index(np.argmax(diff / bound), diff.shape)
    assert diff[worst] <= bound[worst], (what, worst, diff[worst], bound[worst], o_ref[worst])
    if lse is not None:
        l = lse.cpu().numpy().astype(np.float64)[mine]
        empty = np.isneginf(l_ref)
        assert np.array_equal(np.isneginf(l), empty), f"{what}: empty rows differ"
        assert (o[empty] == 0).all(), f"{what}: an empty row is not zero"
        tol = delta + 2.0 ** -20 * np.abs(np.where(empty, 0, l_ref)) + 2.0 ** -18
        assert (np.abs(l - np.where(empty, 0, l_ref))[~empty] <= tol[~empty]).all(), f"{what}: lse"


def run_and_check(fw, x, what="", status=0, **kw):
    how = {k: kw[k] for k in ("causal", "window_left") if k in kw}
    g = on_gpu(x)
    out, lse = fw.paged_prefill(**g, **kw)
    torch.cuda.synchronize()
    assert fw.device_status() == status
    check(out, lse, step.paged_prefill(**x, **how), x["q"].shape[-1], what)
    return out, lse


# chunk lengths, key counts, heads, KV heads, head dim, page size
CASES = [
    ([1], [1], 8, 2, 128, 16),
    ([1, 1], [37, 200], 8, 2, 128, 16),
    ([5, 128, 3], [5, 128, 133], 40, 8, 128, 16),
    ([0, 8, 3, 0], [0, 8, 257, 40], 8, 2, 128, 8),
    ([16, 7], [1000, 131], 40, 8, 128, 128),
    ([31], [700], 28, 4, 128, 32),
    ([130, 257, 1], [130, 600, 1500], 16, 16, 128, 64),
    ([33, 300], [33, 1500], 7, 1, 128, 16),
    ([64], [2000], 32, 8, 128, 64),
    ([500], [500], 4, 1, 128, 256),
    ([300, 1, 2], [1000, 999, 3], 12, 12, 128, 256),
    ([129], [1111], 32, 1, 128, 16),
    ([3], [500], 160, 1, 128, 64),
    ([2, 5], [260, 5], 300, 2, 128, 64),
    ([6, 2], [390, 129], 128, 1, 128, 64),
    ([4, 1], [100, 515], 16, 16, 256, 32),
    ([24, 200, 9], [24, 1300, 400], 16, 16, 256, 64),
    ([90], [900], 8, 1, 256, 128),
    ([70, 1], [400, 77], 8, 4, 256, 8),
    ([1] * 9, [3, 128, 129, 500, 1, 64, 1000, 257, 12], 40, 8, 128, 16),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_against_the_definition(fw, case, causal):
    d, n, Hq, Hkv, D, ps = case
    run_and_check(fw, make(d, n, Hq, Hkv, D, ps, seed=len(d) + Hq), str(case), causal=causal)


@pytest.mark.parametrize("case", [c for c in CASES if c[4] == 128], ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_8_bit_caches(fw, case, causal):
    d, n, Hq, Hkv, D, ps = case
    run_and_check(fw, make(d, n, Hq, Hkv, D, ps, kv8=True, seed=len(d) + Hq), str(case), causal=causal)


@pytest.mark.parametrize("window", [0, 1, 127, 128, 300, 5000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,kv8", [(8, 2, 128, False), (8, 2, 128, True), (4, 4, 256, False), (7, 1, 128, False)])
def test_windows(fw, window, causal, Hq, Hkv, D, kv8):
    """Pages wholly before the window are gone: their entries name no page."""
    d, n, ps = [1, 40, 333, 64], [900, 41, 1400, 64], 16
    x = make(d, n, Hq, Hkv, D, ps, kv8=kv8, seed=window)
    for b in range(4):
        x["block_table"][b, :max(0, n[b] - d[b] - window) // ps] = -7
    run_and_check(fw, x, f"window {window}", causal=causal, window_left=window)


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("d,n", [([300], [20]), ([70, 5, 600], [0, 3, 599]), ([200, 200], [1, 0]), ([9], [0])])
def test_more_tokens_than_keys(fw, d, n, kv8):
    """Bottom-right alignment: the first tokens see nothing."""
    for Hq, Hkv, D in ((8, 2, 128), (160, 1, 128)) + (() if kv8 else ((4, 2, 256),)):
        for causal in (True, False):
            run_and_check(fw, make(d, n, Hq, Hkv, D, 16, kv8=kv8, width=40), f"{d} {n}", causal=causal)


@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
@pytest.mark.parametrize("ctas", [0, 1, 3, 16])
def test_units_cut_across_ctas(fw, D, kv8, ctas):
    """One request over many keys, and few CTAs over many pieces."""
    fw.set_option(fw.FW_OPT_MAX_CTAS, ctas)
    try:
        run_and_check(fw, make([20], [6000], 8, 2, D, 64, kv8=kv8, seed=3), "one request")
        run_and_check(fw, make([150, 1, 1, 400], [1500, 4000, 130, 400], 10, 2, D, 32, kv8=kv8, seed=4), "mixed")
    finally:
        fw.set_option(fw.FW_OPT_MAX_CTAS, 0)


def test_rows_of_no_request_are_left(fw):
    x = make([5, 200], [60, 300], 8, 2, 128, 16, behind=77, first=9)
    g = on_gpu(x)
    out = torch.full((291, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((291, 8), 3.0, device="cuda")
    run_and_check(fw, x, "packed", out=out, lse=lse)
    for t in (out, lse):
        assert (t[:9] == 3.0).all() and (t[214:] == 3.0).all() and not (t[9:214] == 3.0).all()


def test_contradictory_rows_are_skipped_and_told(fw):
    x = make([5, 20, 8], [60, 300, 50], 8, 2, 128, 16)
    good = run_and_check(fw, x)[0]
    for cu in ([0, 5, 3, 11], [-2, 5, 25, 33], [0, 5, 25, 34], [0, 2 ** 31 - 1, 25, 33]):
        y = dict(on_gpu(x), cu_seqlens_q=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        out = torch.full_like(good, 2.0)
        fw.paged_prefill(**y, out=out)
        assert fw.device_status() == 1
    y = dict(on_gpu(x), cu_seqlens_q=torch.tensor([0, 5, 25, 34], dtype=torch.int32, device="cuda"))
    out = torch.full_like(good, 2.0)
    fw.paged_prefill(**y, out=out)
    assert torch.equal(out[:25], good[:25]) and (out[25:] == 2.0).all() and fw.device_status() == 1


def test_lengths_beyond_the_table_are_clamped(fw):
    x = make([4, 4], [64, 30], 8, 2, 128, 16, width=4)
    good = run_and_check(fw, x)[0]
    y = dict(on_gpu(x), seq_lens=torch.tensor([1000, 30], dtype=torch.int32, device="cuda"))
    assert torch.equal(fw.paged_prefill(**y)[0], good)
    y["seq_lens"] = torch.tensor([-5, 30], dtype=torch.int32, device="cuda")
    out, lse = fw.paged_prefill(**y)
    assert (out[:4] == 0).all() and torch.isneginf(lse[:4]).all() and torch.equal(out[4:], good[4:])


def test_a_page_outside_the_pool_is_told(fw):
    x = make([4, 4], [64, 30], 8, 2, 128, 16)
    y = on_gpu(x)
    for page in (10 ** 6, -1):
        y["block_table"][0, 1] = page
        fw.paged_prefill(**y)
        assert fw.device_status() == 1


@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
@pytest.mark.parametrize("n,d", [(300, 150), (1000, 64), (260, 260)])
def test_values_that_are_not_finite(fw, D, kv8, n, d):
    """A bad value in the chunk: rows before it are as if it were not there, rows that
    see it are NaN (or, of units that see its tile whole, not finite in its column),
    their LSE is not touched."""
    x = make([d, 3], [n, 9], 8, 2, D, 16, kv8=kv8, seed=5)
    clean, clean_lse = run_and_check(fw, x)
    for key in (n - d + 1, n - d + d // 2, n - 1):
        for value in ((math.nan,) if kv8 else (math.nan, math.inf, -math.inf)):
            y = on_gpu(x)
            page = y["block_table"][0, key // 16].long()
            old = y["v_cache"].clone()
            v = y["v_cache"].float()
            v[page, key % 16, 1, 7] = value
            y["v_cache"] = v.to(old.dtype)
            out, lse = fw.paged_prefill(**y)
            t = key - (n - d)
            assert torch.equal(out[:t], clean[:t]) and torch.equal(lse, clean_lse)
            assert torch.equal(out[:, :4], clean[:, :4]) and torch.equal(out[d:], clean[d:])
            assert not torch.isfinite(out[t:d, 4:, 7]).any()
            assert torch.isnan(out[t, 4:]).all()          # its own row does not see the tile whole, or is the last to


@pytest.mark.parametrize("window", [3, 200])
def test_bad_values_at_both_ends_of_a_window(fw, window):
    d, n = 300, 1000
    x = make([d], [n], 4, 2, 128, 16, seed=6)
    clean, _ = run_and_check(fw, x, window_left=window)
    for key in (n - d - window, n - d - window + 130, n - d, n - 100):
        y = on_gpu(x)
        y["v_cache"][y["block_table"][0, key // 16].long(), key % 16, 0, 3] = math.nan
        out, _ = fw.paged_prefill(**y, window_left=window)
        t = torch.arange(d, device="cuda")
        sees = (key <= n - d + t) & (key >= n - d + t - window)
        assert torch.equal(out[~sees], clean[~sees]) and torch.equal(out[:, 2:], clean[:, 2:])
        assert torch.isnan(out[sees][:, :2, 3]).all()


@pytest.mark.parametrize("kv8", [False, True])
def test_nan_keys_and_queries(fw, kv8):
    x = make([100], [400], 8, 2, 128, 16, kv8=kv8, seed=7)
    clean, clean_lse = run_and_check(fw, x)
    y = on_gpu(x)
    k = y["k_cache"].float()
    k[y["block_table"][0, 350 // 16].long(), 350 % 16, 1, 0] = math.nan
    y["k_cache"] = k.to(y["k_cache"].dtype)
    out, lse = fw.paged_prefill(**y)
    assert torch.equal(out[:50], clean[:50]) and torch.equal(out[:, :4], clean[:, :4])
    assert torch.isnan(out[50:, 4:]).all() and torch.isnan(lse[50:, 4:]).all()
    y = on_gpu(x)
    y["q"][3, 2, 5] = math.nan
    out, lse = fw.paged_prefill(**y)
    keep = torch.ones(100, 8, dtype=torch.bool, device="cuda")
    keep[3, 2] = False
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[3, 2]).all() and torch.isnan(lse[3, 2])


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_queries_that_are_not_finite_over_8_bit_caches(fw, bad):
    """Both terms of such a row are NaN: the row and its LSE are, the others are as ever."""
    x = make([100, 3], [400, 50], 8, 2, 128, 16, kv8=True, seed=27)
    clean, clean_lse = run_and_check(fw, x)
    y = on_gpu(x)
    for at in ((3, 2, 5), (99, 7, 127), (101, 0, 0)):
        y["q"][at] = bad
    out, lse = fw.paged_prefill(**y)
    keep = torch.ones(103, 8, dtype=torch.bool, device="cuda")
    for at in ((3, 2), (99, 7), (101, 0)):
        keep[at] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
    assert torch.isnan(out[~keep]).all() and torch.isnan(lse[~keep]).all()


@pytest.mark.parametrize("ratio", [2.0 ** 9, 2.0 ** 12, 2.0 ** 17, 2.0 ** 30])
def test_queries_of_a_wide_range_over_8_bit_caches(fw, ratio):
    """An element far above the others of its row: two E4M3 terms are off by at most 2^-17 of
    it in each other element (and exact down to 2^-10 of it), so a score by 2^-17 max |q| sum
    |k_i| scale, on top of the other bounds."""
    x = make([70, 2], [300, 40], 8, 2, 128, 16, kv8=True, seed=28)
    x["q"][:, :, 17] *= ratio
    x["scale"] = 0.02 / ratio
    out, lse = fw.paged_prefill(**on_gpu(x))
    assert fw.device_status() == 0
    o_ref, l_ref, absv, reach = step.paged_prefill(**x)
    k = x["k_cache"].double().nan_to_num(0.0).abs().sum(-1).amax().item() * x["k_scale"]
    big = x["q"].double().abs().amax(-1).numpy()
    delta = 136 * 2.0 ** -24 * reach + 2.0 ** -17 * big * k * x["scale"]
    assert (np.abs(lse.double().cpu().numpy() - l_ref) <= delta + 2.0 ** -20 * np.abs(l_ref) + 2.0 ** -18).all()
    d = (2 * U + 2 * delta[..., None] + 2.0 ** -18) * absv
    assert (np.abs(out.double().cpu().numpy() - o_ref) <= d + U * (np.abs(o_ref) + d) + 1e-30).all()


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("ctas", [0, 1, 2])
def test_units_of_one_and_two_row_tiles_in_turn(fw, kv8, ctas):
    """A stream without a row tile keeps step: short units between long ones, one tile or many."""
    d = [200, 1, 1, 1, 130, 2, 64, 300, 1, 1, 1, 1, 1, 257, 3, 1]
    n = [200, 1, 300, 2, 131, 900, 64, 700, 5, 128, 129, 1, 640, 300, 3, 1500]
    fw.set_option(fw.FW_OPT_MAX_CTAS, ctas)
    try:
        run_and_check(fw, make(d, n, 8, 2, 128, 16, kv8=kv8, seed=29), "turns")
    finally:
        fw.set_option(fw.FW_OPT_MAX_CTAS, 0)


@pytest.mark.parametrize("amp,scale", [(1.0, -0.05), (1.0, 0.0), (40.0, 0.3), (1e-3, 0.088), (30.0, -0.2)])
@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
def test_scales(fw, amp, scale, D, kv8):
    x = make([40, 200], [500, 201], 8, 2, D, 16, kv8=kv8, amp=amp, seed=8)
    x["scale"] = scale
    run_and_check(fw, x, f"{amp} {scale}")


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("case", [([31], [700], 28, 4, 128, 32), ([64], [2000], 32, 8, 128, 64), ([5], [300], 8, 2, 128, 16),
                                  ([5, 128, 3], [5, 128, 133], 40, 8, 128, 16), ([40], [40], 4, 4, 256, 16)], ids=str)
def test_what_lay_in_shared_memory_does_not_matter(fw, case, kv8):
    """Pages that are not copied leave what an earlier call put there, NaN of any type."""
    if kv8 and case[4] == 256:
        pytest.skip("8-bit caches have head dim 128")
    x = make(*case, kv8=kv8, seed=18)
    for dt in (torch.bfloat16, torch.float8_e4m3fn):
        dirty = on_gpu(make([600] * 8, [900] * 8, 40, 8, 128, 16, kv8=dt != torch.bfloat16))
        for name in ("k_cache", "v_cache"):
            dirty[name].view(torch.uint8).fill_(255)
        fw.paged_prefill(**dirty)
        run_and_check(fw, x, str(case))


def test_rising_scores_move_the_base(fw):
    """Keys grow along the row, so that the maximum rises tile after tile."""
    for D, kv8 in ((128, False), (256, False)):
        x = make([150], [2000], 4, 2, D, 16, seed=9)
        pages = x["block_table"][0].long()
        ramp = torch.linspace(0.1, 30.0, pages.numel() * 16).view(-1, 16, 1, 1)
        x["k_cache"][pages] = (x["k_cache"][pages].float() * ramp).to(torch.bfloat16)
        run_and_check(fw, x, "ramp")


def test_one_token_equals_decode(fw):
    """Against the library's own decode, on lengths where both walk the same keys."""
    x = on_gpu(make([1] * 5, [700, 3, 128, 1000, 65], 40, 8, 128, 16, seed=10))
    out, lse = fw.paged_prefill(**x)
    ref, ref_lse = fw.paged_decode(x["q"][:, None], x["k_cache"].nan_to_num(0), x["v_cache"].nan_to_num(0), x["block_table"],
                                   x["seq_lens"], x["scale"])
    assert (out.float() - ref[:, 0].float()).abs().max() <= 2.0 ** -6 and (lse - ref_lse[:, 0]).abs().max() <= 1e-4


def test_strides_and_table_views(fw):
    x = make([30, 100], [400, 140], 8, 2, 128, 16, seed=11)
    want = run_and_check(fw, x)
    g = on_gpu(x)
    buf = torch.zeros(130, 24, 128, dtype=torch.bfloat16, device="cuda")            # columns of one projection
    buf[:, 8:16] = g["q"]
    kv = torch.zeros(g["k_cache"].shape[0], 2, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    kv[:, 0], kv[:, 1] = g["k_cache"], g["v_cache"]
    table = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    table[:, 5:5 + g["block_table"].shape[1]] = g["block_table"]
    out = torch.zeros(130, 8, 136, dtype=torch.bfloat16, device="cuda")[:, :, :128]
    lse = torch.zeros(8, 130, device="cuda")
    y = dict(g, q=buf[:, 8:16], k_cache=kv[:, 0], v_cache=kv[:, 1], block_table=table[:, 5:40])
    fw.paged_prefill(**y, out=out)
    assert torch.equal(out, want[0])
    with pytest.raises(fw.FwError):
        fw.paged_prefill(**y, lse=lse.t())                # the last dimension is not contiguous


def test_streams_workspaces_and_graphs(fw):
    a, b = on_gpu(make([200, 1], [900, 3000], 8, 2, 128, 16, seed=12)), on_gpu(make([50], [5000], 8, 2, 128, 64, seed=13))
    want_a, want_b = fw.paged_prefill(**a), fw.paged_prefill(**b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):                                    # two calls at once, workspaces of their own
        got = [fw.paged_prefill(**x, stream=s) for x, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got[0] + got[1], want_a + want_b))
    graphs, got = [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(fw.paged_prefill(**x))
        graphs.append(g)
    for o, l in got:
        o.zero_(), l.zero_()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got[0] + got[1], want_a + want_b))
    a["seq_lens"].copy_(torch.tensor([850, 2000]))        # a replayed step takes the lengths of its time
    graphs[0].replay()
    fresh = fw.paged_prefill(**a)
    torch.cuda.synchronize()
    assert torch.equal(got[0][0], fresh[0]) and fw.device_status() == 0
    n = fw.paged_prefill_workspace_size(128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert torch.equal(fw.paged_prefill(**b, workspace=ws)[0], want_b[0])
    for bad in (ws[:-256], ws[:0]):
        with pytest.raises(fw.FwError) as e:
            fw.paged_prefill(**b, workspace=bad)
        assert e.value.status == 3
    with pytest.raises(fw.FwError):
        fw.paged_prefill(**b, workspace=torch.empty(n + 256, dtype=torch.uint8, device="cuda")[128:])


def test_repeats_are_equal(fw):
    x = on_gpu(make([300, 1, 40], [1200, 5000, 40], 40, 8, 128, 16, seed=14))
    ref = fw.paged_prefill(**x)
    for _ in range(10):
        assert all(torch.equal(g, w) for g, w in zip(fw.paged_prefill(**x), ref))


def test_empty_batches(fw):
    x = on_gpu(make([3], [20], 8, 2, 128, 16))
    before = fw.launch_count()
    y = dict(x, q=x["q"][:0], cu_seqlens_q=torch.zeros(2, dtype=torch.int32, device="cuda"))
    out, lse = fw.paged_prefill(**y)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8) and fw.launch_count() == before
    y = dict(x, block_table=x["block_table"][:0], seq_lens=x["seq_lens"][:0],
             cu_seqlens_q=torch.zeros(1, dtype=torch.int32, device="cuda"))
    fw.paged_prefill(**y)
    out = torch.ones_like(x["q"])                         # requests without tokens
    y = dict(x, cu_seqlens_q=torch.zeros(2, dtype=torch.int32, device="cuda"))
    fw.paged_prefill(**y, out=out)
    assert (out == 1).all() and fw.device_status() == 0


def test_a_large_batch_of_short_requests(fw):
    r = np.random.RandomState(0)
    d = [int(x) for x in r.randint(0, 4, 1500)]
    n = [x + int(r.randint(0, 40)) for x in d]
    run_and_check(fw, make(d, n, 4, 2, 128, 16, seed=15), "many")


def test_outputs_over_anything_else_are_refused(fw):
    x = on_gpu(make([6, 6], [100, 60], 8, 2, 128, 16, seed=16))
    q, rows = x["q"], 12 * 8
    flat = lambda t, dt, m: t.view(torch.uint8).view(-1)[:m].view(dt)
    lse, out = torch.empty(12, 8, device="cuda"), torch.empty_like(q)
    n = fw.paged_prefill_workspace_size(128)
    ws = torch.empty(n + 4096, dtype=torch.uint8, device="cuda")
    before = fw.launch_count()
    for name, kw in {"q": dict(out=q), "k_cache": dict(out=flat(x["k_cache"], torch.bfloat16, 2 * rows * 128).view(q.shape)),
                     "v_cache": dict(lse=flat(x["v_cache"], torch.float32, 4 * rows).view(12, 8)),
                     "lse": dict(out=out, lse=flat(out, torch.float32, 4 * rows).view(12, 8)),
                     "the workspace": dict(out=ws[:2 * rows * 128].view(torch.bfloat16).view(q.shape), workspace=ws)}.items():
        with pytest.raises(fw.FwError, match=name):
            fw.paged_prefill(**x, **kw)
    assert fw.launch_count() == before


def test_a_wait_that_runs_out_is_told(fw):
    """The copying warp waits for nothing: the call reports it, and the next one is fine."""
    for D, kv8, d in ((128, False, [200]), (128, False, [2]), (128, True, [200]), (128, True, [2]), (256, False, [50])):
        x = on_gpu(make(d, [900], 8, 2, D, 16, kv8=kv8, seed=17))
        want = fw.paged_prefill(**x)[0]
        fw.set_option(fw.FW_OPT_WAIT_TIMEOUT_MS, 50)
        fw.set_option(fw.FW_OPT_TEST_STALL, 1)
        try:
            fw.paged_prefill(**x)
            torch.cuda.synchronize()
        finally:
            fw.set_option(fw.FW_OPT_TEST_STALL, 0)
            fw.set_option(fw.FW_OPT_WAIT_TIMEOUT_MS, 2000)
        assert fw.device_status() == 5
        assert torch.equal(fw.paged_prefill(**x)[0], want) and fw.device_status() == 0
