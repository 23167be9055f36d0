"""Verification of drafts against exact arithmetic: chains and trees, with and
without a draft model's rows, with and without a context row; borders, degenerate
rows and refused drafts; the distribution of what comes out."""
import numpy as np
import pytest
import torch

from oracle import step
from tests.gpu_common import built_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    return built_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


def make(B, T, V, branch, draft=True, context=False, seed=0, sharp=1.5, noise=0.7):
    g = torch.Generator().manual_seed(seed)
    rows = T + int(context)
    logits = sharp * torch.randn(B, rows, V, generator=g)
    target = torch.softmax(logits, -1)
    dp = torch.softmax(logits + noise * torch.randn(B, rows, V, generator=g), -1)
    t = torch.arange(T)
    par = t - 1 - (torch.rand(B, T, generator=g) * branch).long() if branch > 1 else (t - 1).expand(B, T).clone()
    par = par.clamp(min=-1 if context else 0)
    par[:, 0] = -1
    rows_of = (par + int(context)).clamp(min=0)
    pick = torch.gather(dp, 1, rows_of[..., None].expand(B, T, V))
    tokens = torch.multinomial(pick.reshape(-1, V), 1, generator=g).view(B, T).to(torch.int32)
    return dict(tokens=tokens, parents=par.to(torch.int32).contiguous(), target_probs=target, uniforms=torch.rand(B, T + 1, generator=g),
                draft_probs=dp if draft else None)


def run(fw, x, **kw):
    d = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in {**x, **kw}.items()}
    return [t.cpu() for t in fw.verify_drafts(**d)]


def check(fw, x, status=0, **kw):
    got = run(fw, x, **kw)
    assert fw.device_status() == status
    ref = step.verify(x["tokens"], x["parents"], x["target_probs"], x["uniforms"], x.get("draft_probs"),
                      kw.get("draft_lens", x.get("draft_lens")), kw.get("max_path"))
    assert got[0].tolist() == ref[0] and got[1].tolist() == ref[1] and got[2].tolist() == ref[2]
    return got


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("context", [True, False])
@pytest.mark.parametrize("B,T,V,branch", [(1, 1, 5, 1), (3, 6, 40, 1), (5, 12, 33, 3), (2, 24, 127, 4), (40, 5, 9, 2),
                                          (1, 3, 4, 3), (2, 40, 12, 40)])
def test_against_exact_arithmetic(fw, B, T, V, branch, draft, context):
    for seed in range(4):
        check(fw, make(B, T, V, branch, draft, context, seed=seed))


def test_many_rejections_at_one_node(fw):
    """Flat targets and drafts that rarely fit: up to 60 children of one node."""
    for draft in (True, False):
        for seed in range(3):
            x = make(3, 61, 50, 1, draft, False, seed=seed, sharp=0.3)
            x["parents"][:, 1:] = 0
            x["uniforms"][:, 1:61] = 1 - 2.0 ** -20
            check(fw, x)


@pytest.mark.parametrize("B", [1, 80, 200, 700])
def test_batches_of_every_cluster_size(fw, B):
    check(fw, make(B, 4, 130, 2, seed=B))


@pytest.mark.parametrize("V", [1, 2, 3, 4, 5, 1023, 4099])
def test_vocabularies_that_end_anywhere(fw, V):
    x = make(3, 3, V, 1, seed=V)
    check(fw, x)
    wide = torch.zeros(3, 3, V + 3)                    # rows that begin on no 16-byte boundary, q's on others than p's
    wide[:, :, 1:V + 1] = x["target_probs"]
    w2 = torch.zeros(3, 3, V + 6)
    w2[:, :, 2:V + 2] = x["draft_probs"]
    y = dict(x, target_probs=wide.cuda()[:, :, 1:V + 1], draft_probs=w2.cuda()[:, :, 2:V + 2])
    got = fw.verify_drafts(**{k: v.cuda() for k, v in y.items()})
    ref = run(fw, x)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, ref))


def test_borders_are_strict(fw):
    """u q < p and running sum > u: quarters are exact in every format."""
    p = torch.full((1, 1, 4), 0.25)
    for u, token in ((0.0, 0), (0.25, 1), (0.5, 2), (0.75, 3), (1 - 2.0 ** -24, 3), (0.25 - 2.0 ** -26, 0)):
        x = dict(tokens=i32([[0]]), parents=i32([[-1]]), target_probs=p, uniforms=torch.tensor([[0.0, u]]))
        assert check(fw, x)[2].tolist() == [token]
    q = torch.tensor([[[0.5, 0.5, 0.0, 0.0]]])
    for u, yes in ((0.5, False), (0.5 - 2.0 ** -25, True)):
        x = dict(tokens=i32([[1]]), parents=i32([[-1]]), target_probs=p.expand(1, 2, 4).contiguous(),
                 draft_probs=q.expand(1, 2, 4).contiguous(), uniforms=torch.tensor([[u, 0.0]]))
        assert check(fw, x)[1].tolist() == [int(yes)]


def test_rows_of_zeros_nan_negative_and_large(fw):
    bad = torch.tensor([float("nan"), -1.0, float("-inf"), 0.5, 0.0, 0.25, float("nan"), 0.25])
    x = dict(tokens=i32([[3]] * 5), parents=i32([[-1]] * 5), target_probs=bad.expand(5, 1, 8).contiguous(),
             uniforms=torch.tensor([[0.0, u] for u in (0.0, 0.49, 0.5, 0.75, 0.99)]))
    assert check(fw, x)[2].tolist() == [3, 3, 5, 7, 7]
    x["target_probs"] = torch.zeros(5, 1, 8)
    assert check(fw, x, status=1)[2].tolist() == [-1] * 5
    x["target_probs"] = torch.tensor([0, 7.0, 0, float("inf"), 0, 0, 0, 1.0]).expand(5, 1, 8).contiguous()     # ones
    assert check(fw, x)[2].tolist() == [1, 3, 3, 7, 7]
    x["target_probs"] = torch.ones(5, 1, 4096)         # adds up to more than 4: a token or -1, and told
    got = run(fw, x)[2]
    assert fw.device_status() == 1 and ((got >= -1) & (got < 4096)).all()


def test_uniforms_out_of_range(fw):
    x = make(4, 5, 20, 1, seed=3)
    x["uniforms"][0] = 1.0
    x["uniforms"][1] = float("nan")
    x["uniforms"][2] = -1.0
    x["uniforms"][3] = 5.0
    check(fw, x)


def test_nothing_left_keeps_the_row(fw):
    """Target and draft alike, a uniform that refuses all the same."""
    p = torch.tensor([[[0.5, 0.25, 0.25]]]).expand(1, 3, 3).contiguous()
    for draft in (p, None):
        x = dict(tokens=i32([[0, 0, 1]]), parents=i32([[-1, 0, 0]]), target_probs=p if draft is not None else
                 torch.tensor([[[1.0, 0.0, 0.0]]]).expand(1, 3, 3).contiguous(), draft_probs=draft,
                 uniforms=torch.tensor([[0.0, 1.0, 1.0, 0.6]]))
        check(fw, x)


def test_draft_lens_and_short_paths(fw):
    x = make(6, 9, 30, 2, seed=12, noise=0.1)
    x["uniforms"][:, :9] *= 0.2
    check(fw, x, draft_lens=i32([9, 5, 1, 12, 3, 9]))
    for most in (1, 2, 4, 200):
        check(fw, x, max_path=most)
    y = make(4, 5, 30, 1, context=True, seed=13)
    check(fw, y, draft_lens=i32([0, -3, 2, 5]))
    got = check(fw, x, status=1, draft_lens=i32([0, 0, 9, 9, 9, 9]))
    assert got[2].tolist()[:2] == [-1, -1] and got[1].tolist()[:2] == [0, 0]


def test_bad_tokens_and_parents(fw):
    x = make(4, 6, 30, 2, seed=14)
    x["tokens"][0, 2], x["tokens"][1, 1], x["tokens"][2, 3] = 30, -1, 2 ** 31 - 1
    check(fw, x, status=1)
    y = make(4, 6, 30, 2, context=True, seed=15)
    y["parents"][0, 2], y["parents"][1, 1], y["parents"][2, 3] = 2, 5, -7
    check(fw, y, status=1)


def test_same_token_twice_below_a_node(fw):
    for draft in (True, False):
        for seed in range(4):
            x = make(4, 8, 6, 1, draft, seed=seed)
            x["parents"][:, 1:] = 0
            x["tokens"][:, 1:] = x["tokens"][:, 1:] % 2
            x["uniforms"][:, 1:8] = 0.5 + 0.5 * x["uniforms"][:, 1:8]
            check(fw, x)


def test_strided_and_given_outputs(fw):
    x = make(5, 7, 64, 2, seed=16)
    ref = run(fw, x)
    big = {k: torch.zeros(5, *(2 * s for s in v.shape[1:]), dtype=v.dtype, device="cuda") for k, v in x.items()}
    y = {}
    for k, v in x.items():
        y[k] = big[k][tuple(slice(0, s) for s in v.shape)]
        y[k].copy_(v)
    path = torch.zeros(5, 20, dtype=torch.int32, device="cuda")
    lens, nxt = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    out = fw.verify_drafts(**y, path=path[:, 3:10], path_lens=lens, next_tokens=nxt)
    assert torch.equal(out[0].cpu(), ref[0]) and torch.equal(lens.cpu(), ref[1]) and torch.equal(nxt.cpu(), ref[2])
    assert (path[:, :3] == 0).all() and (path[:, 10:] == 0).all()


def test_large_rows_repeat_and_graph(fw):
    x = {k: v.cuda() for k, v in make(6, 7, 50257, 2, seed=17, sharp=2.5).items()}
    ref = fw.verify_drafts(**x)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(ref, fw.verify_drafts(**x)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fw.verify_drafts(**x)
    x["uniforms"].copy_(torch.rand(6, 8))
    graph.replay()
    ref = fw.verify_drafts(**x)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got)) and fw.device_status() == 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fw.verify_drafts(**x, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_rows_that_add_up_to_far_more_than_four_are_told(fw):
    """Halves of a row and its neighbours full of ones: sums of 64 bits must not go round."""
    for ones in (4096, 2048, 4095, 1024, 3000, 8192):
        p = torch.zeros(1, 1, 8192)
        p[..., :ones] = 1.0
        p[..., 4100] = 0.5
        x = dict(tokens=i32([[0]]), parents=i32([[-1]]), target_probs=p, uniforms=torch.tensor([[0.0, 0.3]]))
        for v in (4096, 8192):
            got = run(fw, dict(x, target_probs=p[..., :v].contiguous()))[2]
            assert fw.device_status() == 1 and -1 <= got.item() < v


def test_long_rows_in_large_batches(fw):
    """One CTA to a request, or eight: the same tokens, whatever a lane adds up."""
    x = make(4, 4, 300001, 1, seed=20, sharp=2.0, noise=1.2)
    x["parents"][:, 1:] = 0
    x["uniforms"][1:3, 1:4] = 1 - 2.0 ** -20
    x["uniforms"][0, 1:4] = 0.9
    few = {k: v.cuda() for k, v in x.items()}
    many = {k: v.repeat(160, *([1] * (v.dim() - 1))) if k not in ("target_probs", "draft_probs") else v for k, v in few.items()}
    for draft in (True, False):
        ref = fw.verify_drafts(**dict(few, draft_probs=few["draft_probs"] if draft else None))
        for b in range(4):                                 # 640 requests that read one request's rows
            y = dict(many, target_probs=few["target_probs"][b:b + 1].expand(640, -1, -1),
                     draft_probs=few["draft_probs"][b:b + 1].expand(640, -1, -1) if draft else None)
            got = fw.verify_drafts(**y)
            for a, r in zip(got, ref):
                assert torch.equal(a[b::4], r[b:b + 1].expand_as(a[b::4]))
    assert fw.device_status() == 0


@pytest.mark.parametrize("draft", [True, False])
def test_first_token_is_distributed_as_the_targets(fw, draft):
    """80,000 requests with two children drawn from the draft model (or fixed): the
    first token is the target's sample.  Five standard deviations of each count."""
    B, V = 80000, 6
    g = torch.Generator().manual_seed(18)
    p, q = torch.tensor([0.3, 0.05, 0.2, 0.25, 0.15, 0.05]), torch.tensor([0.1, 0.3, 0.1, 0.1, 0.1, 0.3])
    tokens = torch.multinomial(q.expand(B, V), 2, replacement=True, generator=g).to(torch.int32) if draft else \
        i32([[3, 1]]).expand(B, 2).contiguous()
    x = dict(tokens=tokens, parents=i32([[-1, -1]]).expand(B, 2).contiguous(), target_probs=p.expand(B, 3, V).contiguous(),
             draft_probs=q.expand(B, 3, V).contiguous() if draft else None, uniforms=torch.rand(B, 3, generator=g))
    path, n, nxt = run(fw, x)
    first = torch.where(n > 0, tokens.gather(1, path[:, :1].clamp(min=0).long())[:, 0], nxt)
    counts = torch.bincount(first.long(), minlength=V).double().numpy()
    pe = p.double().numpy()
    assert (np.abs(counts - B * pe) <= 5 * np.sqrt(B * pe * (1 - pe))).all(), counts
