"""Verification of drafts over rows long enough for every part of a sweep (several groups a
lane and stage, sums handed on after 1,024 elements, draws that look at many groups), against
exact sums in integers: probabilities are taken as multiples of 2^-149, products are kept to
2^-240, far below the 2^-60 that the kernel counts in.  Uniform numbers are as good as never
that close to a border."""
import numpy as np
import pytest
import torch

from tests.gpu_common import built_library

UNIT = 240


def whole(t):
    """FP32 probabilities as Python integers of 2^-240."""
    m, e = np.frexp(np.clip(t.double().numpy(), 0.0, 1.0))
    return (m * 2.0 ** 53).astype(np.int64).astype(object) << (e.astype(np.int64) + (UNIT - 53)).astype(object)


def verify(tokens, parents, target, uniforms, draft):
    """One request; the context has no row."""
    T = len(tokens)
    u = [int(x) for x in whole(uniforms)]
    path, node = [0], 0
    left, total, rejections = whole(target[0]), 1 << UNIT, 0
    for t in range(1, T):
        if parents[t] != node:
            continue
        tok = tokens[t]
        q = whole(draft[node]) if draft is not None else None
        if u[t] * (int(q[tok]) if q is not None else 1 << UNIT) * total < int(left[tok]) << 2 * UNIT:
            path.append(t)
            node = t
            left, total = whole(target[t]), 1 << UNIT
            continue
        rejections += 1
        if q is not None:
            rest = np.maximum(left - ((q * total) >> UNIT), 0)
        else:
            rest = left.copy()
            rest[tok] = 0
        s = int(rest.sum())
        if s > 0:
            left, total = rest, s
    run = np.cumsum(left)
    return path, int(np.argmax((run << UNIT) > u[T] * int(run[-1]))), rejections


def test_the_sums_of_the_test():
    """On quarters, worked out by hand."""
    p, q = torch.tensor([[0.5, 0.25, 0.25]] * 2), torch.tensor([[0.25, 0.75, 0.0]] * 2)
    for draft, want in ((q, [0, 0, 0, 2, 2]), (None, [0, 0, 0, 2, 2])):
        for draw, token in zip((0.0, 0.25, 0.499, 0.5 if draft is not None else 0.75, 0.99), want):
            got = verify([0, 1], [-1, 0], p, torch.tensor([0.0, 0.9, draw]), draft)
            assert got == ([0], token, 1)


def make(B, V, seed, sharp, noise, children):
    """`children` drafts below the first one, as many below some of those, drawn from the draft model."""
    g = torch.Generator().manual_seed(seed)
    T = 1 + 2 * children
    parents = [-1] + [0] * children + [1 + (seed + i) % children if i else 1 for i in range(children)]
    logits = sharp * torch.randn(B, T, V, generator=g)
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits + noise * torch.randn(B, T, V, generator=g), -1)
    tokens = torch.multinomial(draft[:, [max(p, 0) for p in parents]].reshape(-1, V), 1, generator=g).view(B, T)
    uniforms = torch.rand(B, T + 1, generator=g)
    uniforms[:, 1:children + 1] = 0.5 + 0.5 * uniforms[:, 1:children + 1]      # so that some are rejected
    return tokens.to(torch.int32), parents, target, draft, uniforms


@pytest.mark.gpu
@pytest.mark.parametrize("ctas", [8, 1])
@pytest.mark.parametrize("shift", [(0, 0), (1, 2), (3, 3)])          # rows behind 16-byte boundaries, by floats
@pytest.mark.parametrize("V,sharp", [(50257, 2.5), (300001, 1.0)])
def test_against_integers(V, sharp, shift, ctas):
    fw = built_library()
    B = 3
    tokens, parents, target, draft, uniforms = make(B, V, V % 97 + shift[0], sharp, 1.5, 3)
    T = len(parents)

    def place(t, by):
        buf = torch.zeros(B, T, V + by + 3 & ~3, device="cuda") if by else torch.empty(B, T, V + 3 & ~3, device="cuda")
        buf[:, :, by:by + V].copy_(t)
        return buf[:, :, by:by + V]
    x = dict(tokens=tokens.cuda(), parents=torch.tensor([parents] * B, dtype=torch.int32).cuda(), uniforms=uniforms.cuda(),
             target_probs=place(target, shift[0]))
    rows = place(draft, shift[1])
    rejected = 0
    for with_draft in (True, False):
        want = [verify(tokens[b].tolist(), parents, target[b], uniforms[b], draft[b] if with_draft else None) for b in range(B)]
        rejected += sum(w[2] for w in want)
        y = dict(x, draft_probs=rows if with_draft else None)
        if ctas == 8:
            path, n, nxt = fw.verify_drafts(**y)
            got = [(path[b, :n[b]].tolist(), int(nxt[b])) for b in range(B)]
        else:                                             # so many requests that a CTA takes one each
            got = []
            for b in range(B):
                z = {k: None if v is None else v[b:b + 1].expand(640, *v.shape[1:]) for k, v in y.items()}
                path, n, nxt = fw.verify_drafts(**z)
                assert (path == path[:1]).all() and (n == n[:1]).all() and (nxt == nxt[:1]).all()
                got.append((path[0, :n[0]].tolist(), int(nxt[0])))
        assert got == [w[:2] for w in want]
    assert rejected >= 4 and fw.device_status() == 0
