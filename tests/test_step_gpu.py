"""The operators of a server's step together: a prompt in two chunks (page tables, norm and
rotation into the cache, chunk attention), then a speculative step (tree masks, page
tables, norm and rotation of the drafts at their depths, tree decode, verification, commit),
in every layer of a packed cache; eagerly and replayed from one CUDA graph."""
import numpy as np
import pytest
import torch

from oracle import spec, step
from tests import test_paged_prefill_gpu as chunk
from tests import test_tree_decode_gpu as tree
from tests.gpu_common import built_library

pytestmark = pytest.mark.gpu

B, T, LAYERS, HQ, HKV, D, PS, PAGES, WIDTH, V = 3, 6, 2, 8, 2, 128, 16, 40, 20, 97
SCALE = D ** -0.5


@pytest.fixture(scope="module")
def fw():
    return built_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Server:
    def __init__(self, kv8, seed):
        g = torch.Generator().manual_seed(seed)
        dt = torch.float8_e4m3fn if kv8 else torch.bfloat16
        self.scales = dict(k_scale=0.05, v_scale=0.02) if kv8 else dict(k_scale=1.0, v_scale=1.0)
        self.g, self.kv8 = g, kv8
        self.k, self.v = (torch.zeros(LAYERS * PAGES, PS, HKV, D, dtype=dt, device="cuda") for _ in range(2))
        self.table, self.held = torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda"), i32([0] * B)
        self.ring, self.range = (torch.randperm(PAGES - 1, generator=g) + 1).to(torch.int32).cuda(), i32([0, PAGES - 1])
        self.freq = (1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
        self.w = [(1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]

    def rand(self, *s):
        return torch.randn(*s, generator=self.g).to(torch.bfloat16).cuda()

    def state(self):
        return [self.k, self.v, self.table, self.held, self.ring, self.range]

    def layer(self, cache, l):
        return cache[l * PAGES:(l + 1) * PAGES]

    def put(self, fw, l, qkv, positions, slots):
        n = qkv.shape[0]
        return fw.qk_norm_rope_append(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], positions, self.freq, slots,
                                      l * PAGES * PS, self.k, self.v, q_weight=self.w[0], k_weight=self.w[1], eps=1e-6,
                                      **self.scales)

    def pages(self, fw, seq, new, slots):
        cu, _, _ = fw.build_page_tables(seq, new, self.held, self.ring, self.range, PS, self.table, slots, held_out=self.held,
                                        range_out=self.range)
        return cu

    def prompt(self, fw, seq, new, positions, qkv):
        """One chunk of every request; the layers' outputs."""
        slots = torch.empty(qkv[0].shape[0], dtype=torch.int32, device="cuda")
        cu = self.pages(fw, seq, new, slots)
        outs = []
        for l in range(LAYERS):
            q = self.put(fw, l, qkv[l], positions, slots)
            outs.append((q, *fw.paged_prefill(q, self.layer(self.k, l), self.layer(self.v, l), self.table, cu, seq, SCALE,
                                              **self.scales)))
        return cu, outs

    def speculate(self, fw, seq, drafts, parents, tokens, qkv, target, draft, uniforms):
        slots = torch.empty(B, T, dtype=torch.int32, device="cuda")
        mask, depths = fw.tree_mask(parents, draft_lens=drafts)
        self.pages(fw, seq, drafts, slots)
        base = seq - drafts
        positions = (base[:, None] + depths.clamp(min=0)).flatten()
        outs = []
        for l in range(LAYERS):
            q = self.put(fw, l, qkv[l], positions, slots)
            q = q.view(B, T, HQ, D)
            outs.append((q, *fw.paged_decode_tree(q, self.layer(self.k, l), self.layer(self.v, l), self.table, seq, mask, SCALE,
                                                  draft_lens=drafts, **self.scales)))
        before = (self.k.clone(), self.v.clone())
        path, n, nxt = fw.verify_drafts(tokens, parents, target, uniforms, draft_probs=draft, draft_lens=drafts)
        lens = fw.kv_commit(path, n, base, self.table, self.k, self.v, num_layers=LAYERS)
        return mask, positions, outs, before, (path, n, nxt, lens)


@pytest.mark.parametrize("kv8", [False, True])
def test_prompt_and_speculative_step(fw, kv8):
    s = Server(kv8, 5)
    full, first = [70, 5, 230], [40, 5, 101]
    done = [0] * B
    for want in (first, full):
        new = [w - x for w, x in zip(want, done)]
        qkv = [s.rand(sum(new), HQ + 2 * HKV, D) for _ in range(LAYERS)]
        pos = i32([x + t for x, n in zip(done, new) for t in range(n)])
        cu, outs = s.prompt(fw, i32(want), i32(new), pos, qkv)
        torch.cuda.synchronize()
        assert fw.device_status() == 0
        for l, (q, out, lse) in enumerate(outs):
            y, size = step.norm_rope(qkv[l][:, :HQ], pos, s.freq, s.w[0])
            assert (np.abs(q.double().cpu().numpy() - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -18 * size).all()
            ref = step.paged_prefill(q.cpu(), s.layer(s.k, l).cpu(), s.layer(s.v, l).cpu(), s.table.cpu(), cu.cpu(), i32(want).cpu(),
                                     SCALE, **s.scales)
            chunk.check(out, lse, ref, D, f"layer {l}")
        done = want

    drafts, seq = [6, 4, 1], [x + d for x, d in zip(full, [6, 4, 1])]
    parents = i32([[-1, 0, 0, 1, 2, 4], [-1, 0, 1, 1, 0, 0], [-1] * T])
    tokens = torch.randint(0, V, (B, T), generator=s.g, dtype=torch.int32).cuda()
    qkv = [s.rand(B * T, HQ + 2 * HKV, D) for _ in range(LAYERS)]
    target, draft = (torch.softmax(torch.randn(B, T, V, generator=s.g), -1).cuda() for _ in range(2))
    target[0, 0, tokens[0, 2]] += 3.0                        # so that request 0 takes drafts 0, 2, 4
    target[0, 2, tokens[0, 4]] += 3.0
    target[0, 0, tokens[0, 1]] = 0.0
    target /= target.sum(-1, keepdim=True)
    uniforms = torch.full((B, T + 1), 0.25, device="cuda")
    args = (i32(seq), i32(drafts), parents, tokens, qkv, target, draft, uniforms)
    saved = [t.clone() for t in s.state()]
    mask, positions, outs, before, (path, n, nxt, lens) = s.speculate(fw, *args)
    torch.cuda.synchronize()
    assert fw.device_status() == 0
    for l, (q, out, lse) in enumerate(outs):
        ref = spec.tree_attention(q.cpu(), s_layer(before[0], l), s_layer(before[1], l), s.table.cpu(), i32(seq).cpu(), mask.cpu(),
                                  SCALE, i32(drafts).cpu(), **s.scales)
        tree.check(out, lse, ref, D, f"tree, layer {l}")
    want = step.verify(tokens.cpu(), parents.cpu(), target.cpu(), uniforms.cpu(), draft.cpu(), draft_lens=drafts)
    assert path.tolist() == want[0] and n.tolist() == want[1] and nxt.tolist() == want[2]
    assert path[0, :3].tolist() == [0, 2, 4]
    assert lens.tolist() == [x + m for x, m in zip(full, n.tolist())]
    table = s.table.cpu()
    raw = lambda c: c.view(torch.uint8).view(LAYERS, PAGES * PS, -1).cpu()
    for now, old in ((s.k, before[0]), (s.v, before[1])):
        now, old = raw(now), raw(old)
        for b in range(B):
            place = lambda x: int(table[b, x // PS]) * PS + x % PS
            for i in range(int(n[b])):
                assert torch.equal(now[:, place(full[b] + i)], old[:, place(full[b] + int(path[b, i]))])

    # The whole step from one graph, on the state as it was.
    eager = [t.clone() for t in s.state()] + [path, n, nxt, lens] + [t for o in outs for t in o]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t, x in zip(s.state(), saved):
            t.copy_(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            _, _, outs, _, result = s.speculate(fw, *args)
        for _ in range(2):
            for t, x in zip(s.state(), saved):
                t.copy_(x)
            graph.replay()
    torch.cuda.synchronize()
    again = s.state() + list(result) + [t for o in outs for t in o]
    view = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
    assert all(torch.equal(view(a), view(b)) for a, b in zip(again, eager)) and fw.device_status() == 0


def s_layer(cache, l):
    return cache[l * PAGES:(l + 1) * PAGES].cpu()
