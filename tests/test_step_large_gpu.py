"""The operators around a step's attention where offsets pass 32 bits: caches, packed rows and
probabilities of more than 2^31 elements give, at their far ends, what the same rows give by
themselves or in 64 bits."""
import math

import pytest
import torch

from oracle import step
from tests import test_paged_prefill_gpu as chunk
from tests.gpu_common import built_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    return built_library()


@pytest.fixture(autouse=True)
def room():
    yield
    torch.cuda.empty_cache()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D,kv8", [(128, False), (128, True), (256, False)])
@pytest.mark.parametrize("d", [3, 200])
def test_chunk_at_the_end_of_a_large_pool(fw, D, kv8, d):
    ps, Hkv, pages = 16, 4, 6
    P = 2 ** 31 // (ps * Hkv * D) + 40                    # more than 2^31 elements
    dt = torch.float8_e4m3fn if kv8 else torch.bfloat16
    g = torch.Generator().manual_seed(3)
    small = [(torch.randn(pages, ps, Hkv, D, generator=g) * (20 if kv8 else 1)).to(dt).cuda() for _ in range(2)]
    big = [torch.zeros(P, ps, Hkv, D, dtype=dt, device="cuda") for _ in range(2)]
    at = [P - 1 - 3 * i for i in range(pages)]
    for b, s in zip(big, small):
        for i, page in enumerate(at):
            b[page] = s[i]
    q = torch.randn(d, 8, D, generator=g).to(torch.bfloat16).cuda()
    n = max(d, ps * pages - 5) if d < ps * pages else ps * pages
    args = (i32([0, d]), i32([n]), 1 / math.sqrt(D))
    kw = dict(k_scale=0.05, v_scale=0.05) if kv8 else {}
    want = fw.paged_prefill(q, *small, i32([list(range(pages))]), *args, **kw)
    got = fw.paged_prefill(q, *big, i32([at]), *args, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and want[0].abs().max() > 0 and fw.device_status() == 0
    # and what the append puts there
    x = torch.randn(2, 8 + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
    freq = torch.linspace(1, 0.1, D // 2, device="cuda")
    how = dict(positions=i32([5, 9]), inv_freq=freq, **kw)
    fw.qk_norm_rope_append(x[:, :8], x[:, 8:8 + Hkv], x[:, 8 + Hkv:], slot_mapping=i32([1, 17]), layer_base_rows=0,
                           k_cache=small[0], v_cache=small[1], **how)
    fw.qk_norm_rope_append(x[:, :8], x[:, 8:8 + Hkv], x[:, 8 + Hkv:], slot_mapping=i32([3 * ps + 1, 17 - ps]),
                           layer_base_rows=(P - 4) * ps, k_cache=big[0], v_cache=big[1], **how)
    raw = lambda t: t.view(torch.uint8)
    for b, s in zip(big, small):
        assert torch.equal(raw(b[P - 1, 1]), raw(s[0, 1])) and torch.equal(raw(b[P - 4, 1]), raw(s[1, 1]))


def test_chunk_of_many_rows(fw):
    """2^31 elements of queries and outputs: the last request against 64 bits (ranges cut its
    units at other keys than in a call by itself, so that sums are rounded differently)."""
    Hq, D, ps = 32, 128, 16
    N = 2 ** 31 // (Hq * D) + 300
    q = torch.zeros(N, Hq, D, dtype=torch.bfloat16, device="cuda")
    q[-300:].normal_()
    k, v = (torch.randn(20, ps, 1, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.randperm(20).to(torch.int32).cuda()[None]
    ref = step.paged_prefill(q[-300:], k, v, table, i32([0, 300]), i32([310]), 0.09)
    out, lse = fw.paged_prefill(q, k, v, table.expand(2, 20).contiguous(), i32([0, N - 300, N]), i32([64, 310]), 0.09,
                                window_left=400)
    chunk.check(out[-300:], lse[-300:], ref, D, "the last request")
    assert (out[:N - 300 - 64] == 0).all() and torch.isneginf(lse[:N - 300 - 64]).all()       # more tokens than keys
    # Queries of zeros see the mean of their keys.
    mean = v[table[0, :4].long()].float().view(64, D).mean(0)
    assert (out[N - 301].float() - mean).abs().max() <= 2.0 ** -7 and fw.device_status() == 0


@pytest.mark.parametrize("D", [64, 256])
def test_norms_of_many_rows(fw, D):
    H = 64
    N = 2 ** 31 // (H * D) + 100
    q = torch.zeros(N, H, D, dtype=torch.bfloat16, device="cuda")
    q[-100:].normal_()
    k = q[:, :1]
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    freq, w = torch.linspace(1, 0.01, D // 2, device="cuda"), torch.linspace(0.5, 2, D, device="cuda")
    want = fw.qk_norm_rope(q[-100:].clone(), k[-100:].clone(), pos[-100:].clone(), freq, w, w)
    got = fw.qk_norm_rope(q, k, pos, freq, w, w)
    assert torch.equal(got[0][-100:], want[0]) and torch.equal(got[1][-100:], want[1])
    assert (got[0][:-100] == 0).all() and fw.device_status() == 0


def test_verification_of_many_rows(fw):
    B, T, V = 610, 24, 152000                             # 2.2e9 probabilities
    probs = torch.zeros(B, T, V, device="cuda")
    g = torch.Generator().manual_seed(4)
    row = torch.softmax(2 * torch.randn(2, T, V, generator=g), -1).cuda()
    probs[-2:] = row
    probs[:-2, :, 7] = 1.0
    tokens = torch.full((B, T), 7, dtype=torch.int32, device="cuda")
    tokens[-2:] = torch.randint(0, V, (2, T), generator=g, dtype=torch.int32).cuda()
    parents = (torch.arange(T, dtype=torch.int32, device="cuda") - 1).expand(B, T).contiguous()
    u = torch.full((B, T + 1), 0.37, device="cuda")
    for draft in (None, probs):
        want = fw.verify_drafts(tokens[-2:], parents[-2:], row, u[-2:], draft_probs=None if draft is None else row)
        got = fw.verify_drafts(tokens, parents, probs, u, draft_probs=draft)
        assert all(torch.equal(a[-2:], b) for a, b in zip(got, want))
        assert (got[1][:-2] == T).all() and (got[2][:-2] == 7).all()
    assert fw.device_status() == 0
