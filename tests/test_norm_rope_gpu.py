"""Norm and rotation of queries and keys against 64 bits: head dims, partial and
interleaved rotation, several axes, far positions, strided inputs, in place, into
BF16 and FP8 caches, on streams and in graphs.

Tolerance, before the first run.  Relative to the size z = hypot(y_i, y_i') of a
rotated pair, FP32 costs: the norm (13 additions of squares, mean, rsqrt to 2 ulp,
two products) under 2^-20, angles (2^-32 of a turn, a 24-bit half turn: 1e-7 rad)
and the cosine and sine (1 ulp each) under 2^-21, two products and a sum under
2^-22: 2^-18 together with room.  Then one rounding: BF16 half a step, 2^-8 |y|;
E4M3 2^-4 |y| or, among its subnormals, half of 2^-9."""
import numpy as np
import pytest
import torch

from oracle import step
from tests.gpu_common import built_library

pytestmark = pytest.mark.gpu
FP32 = 2.0 ** -18


@pytest.fixture(scope="module")
def fw():
    return built_library()


def make(N, Hq, Hkv, D, rot=None, axes=1, norm=True, far=5000, seed=0, f32_weight=False):
    g = torch.Generator().manual_seed(seed)
    rot = rot or D
    rand = lambda *s: torch.randn(*s, generator=g)
    scale = 0.1 + 4.0 * torch.rand(N, Hq + 2 * Hkv, 1, generator=g)
    qkv = (rand(N, Hq + 2 * Hkv, D) * scale).to(torch.bfloat16).cuda()
    w = [(1 + 0.4 * rand(D)).to(torch.float32 if f32_weight else torch.bfloat16).cuda() for _ in range(2)]
    pos = torch.randint(0, far, (axes, N) if axes > 1 else (N,), generator=g, dtype=torch.int32).cuda()
    freq = (1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    amap = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32).cuda() if axes > 1 else None
    x = dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], positions=pos, inv_freq=freq, axis_map=amap,
             q_weight=w[0] if norm else None, k_weight=w[1] if norm else None, eps=1e-5)
    return x, qkv[:, Hq + Hkv:]


def want(x, which, interleaved=False):
    return step.norm_rope(x[which], x["positions"], x["inv_freq"], x[which + "_weight"], x["eps"], x["axis_map"], interleaved)


def check_bf16(got, ref, what):
    y, size = ref
    err = np.abs(got.double().cpu().numpy() - y)
    bound = 2.0 ** -8 * np.abs(y) + FP32 * size + 2.0 ** -133
    assert (err <= bound).all(), f"{what}: {np.max(err / bound)} of its bound"


def check_e4m3(got, ref, scale, what):
    y, size = ref
    y, size = np.clip(y / scale, -448, 448), size / scale
    err = np.abs(got.double().cpu().numpy() - y)
    bound = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) + 2 * FP32 * size
    assert (err <= bound).all(), f"{what}: {np.max(err / bound)} of its bound"


@pytest.mark.parametrize("N,Hq,Hkv,D,rot", [
    (1, 40, 8, 128, 128), (3, 8, 2, 128, 64), (77, 7, 1, 128, 128), (5, 3, 3, 64, 64), (33, 12, 4, 64, 24), (9, 5, 2, 256, 256),
    (130, 16, 16, 256, 128), (2, 1, 1, 128, 8), (1000, 4, 1, 64, 32), (700, 40, 8, 128, 128),
])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [True, False])
def test_against_64_bits(fw, N, Hq, Hkv, D, rot, interleaved, norm):
    x, _ = make(N, Hq, Hkv, D, rot, norm=norm, seed=N + D)
    q, k = fw.qk_norm_rope(**x, interleaved=interleaved)
    check_bf16(q, want(x, "q", interleaved), "q")
    check_bf16(k, want(x, "k", interleaved), "k")
    assert fw.device_status() == 0


@pytest.mark.parametrize("axes,interleaved", [(2, False), (3, False), (3, True), (4, True)])
def test_several_axes(fw, axes, interleaved):
    x, _ = make(51, 6, 2, 128, 128, axes=axes, seed=axes)
    q, k = fw.qk_norm_rope(**x, interleaved=interleaved)
    check_bf16(q, want(x, "q", interleaved), "q")
    check_bf16(k, want(x, "k", interleaved), "k")


def test_far_and_negative_positions(fw):
    """Angles of millions of turns; every position of 32 bits."""
    x, _ = make(9, 4, 2, 128, seed=5)
    x["positions"] = torch.tensor([0, 1, -1, 131071, 1000003, -70001, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).cuda()
    q, k = fw.qk_norm_rope(**x)
    check_bf16(q, want(x, "q"), "q")


def test_frequencies_of_more_than_a_turn(fw):
    x, _ = make(20, 4, 2, 64, far=300, seed=6)
    x["inv_freq"] = torch.linspace(-9.0, 40.0, 32).cuda()
    q, k = fw.qk_norm_rope(**x)
    check_bf16(q, want(x, "q"), "q")


def test_weights_of_32_bits_and_one_norm_alone(fw):
    x, _ = make(31, 4, 2, 128, seed=7, f32_weight=True)
    x["k_weight"] = None
    q, k = fw.qk_norm_rope(**x)
    check_bf16(q, want(x, "q"), "q")
    check_bf16(k, want(x, "k"), "k")


def test_zero_heads_and_tiny_ones(fw):
    x, _ = make(4, 4, 2, 128, seed=8)
    x["q"][0] = 0
    x["q"][1] *= 2.0 ** -60
    x["eps"] = 0.0
    x["k"][:] = 1.0
    q, k = fw.qk_norm_rope(**x)
    assert torch.isnan(q[0]).all()                    # 0 / 0 of the definition
    x["eps"] = 1e-6
    q, k = fw.qk_norm_rope(**x)
    assert (q[0] == 0).all()
    check_bf16(q, want(x, "q"), "q")


def test_nan_and_infinity_stay_in_their_head_or_pair(fw):
    x, _ = make(3, 4, 2, 128, rot=64, seed=9)
    clean_q, clean_k = fw.qk_norm_rope(**x)
    x["q"][1, 2, 5] = float("nan")
    q, _ = fw.qk_norm_rope(**x)
    assert torch.isnan(q[1, 2]).all()
    rest = torch.ones(3, 4, dtype=torch.bool)
    rest[1, 2] = False
    assert torch.equal(q[rest.cuda()], clean_q[rest.cuda()])
    x["q_weight"] = x["k_weight"] = None              # without the norm only the pair
    x["q"][1, 2, 100] = float("inf")                  # and an element that does not rotate
    q, _ = fw.qk_norm_rope(**x)
    bad = ~torch.isfinite(q[1, 2].float())
    assert bad.nonzero().flatten().tolist() == [5, 37, 100]


@pytest.mark.parametrize("D,rot", [(128, 128), (64, 32), (256, 256)])
def test_in_place_equals_out_of_place(fw, D, rot):
    x, _ = make(300, 10, 2, D, rot, seed=10)
    q, k = fw.qk_norm_rope(**x)
    a, b = fw.qk_norm_rope(**x, q_out=x["q"], k_out=x["k"])
    assert a.data_ptr() == x["q"].data_ptr() and torch.equal(a, q) and torch.equal(b, k)


def caches(P, ps, Hkv, D, dtype, seed=3):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(P, ps, Hkv, D, generator=g).to(dtype).cuda() for _ in range(2)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("N,Hq,Hkv,D,ps,base", [(1, 40, 8, 128, 16, 0), (37, 7, 1, 128, 8, 16), (200, 6, 3, 64, 100, 300),
                                                (50, 4, 2, 256, 64, 64), (3000, 8, 2, 128, 128, 128)])
def test_append(fw, dtype, N, Hq, Hkv, D, ps, base):
    x, v = make(N, Hq, Hkv, D, seed=N)
    P = (base + N) // ps + 3
    kc, vc = caches(P, ps, Hkv, D, dtype)
    k0, v0 = kc.clone(), vc.clone()
    g = torch.Generator().manual_seed(N)
    slots = torch.randperm(P * ps - base, generator=g)[:N].to(torch.int32)
    if N > 3:
        slots[1], slots[N // 2] = -1, -1
    ks, vs = (0.05, 0.03) if dtype == torch.float8_e4m3fn else (1.0, 1.0)
    q = fw.qk_norm_rope_append(v=v, slot_mapping=slots.cuda(), layer_base_rows=base, k_cache=kc, v_cache=vc, k_scale=ks,
                               v_scale=vs, **x)
    check_bf16(q, want(x, "q"), "q")
    live = slots >= 0
    at = (slots[live].long() + base).cuda()
    raw = lambda c: c.view(torch.uint8 if dtype == torch.float8_e4m3fn else torch.int16).view(P * ps, Hkv, -1)
    y, size = want(x, "k")
    y, size = y[live.numpy()], size[live.numpy()]
    got_k, got_v = kc.view(P * ps, Hkv, D)[at], vc.view(P * ps, Hkv, D)[at]
    if dtype == torch.bfloat16:
        check_bf16(got_k, (y, size), "k")
        assert torch.equal(got_v, v[live.cuda()])
    else:
        check_e4m3(got_k, (y, size), ks, "k")
        kk, vv = torch.empty_like(k0), torch.empty_like(v0)                 # values as the append stores them
        fw.kv_append(x["k"][live.cuda()][:, None].contiguous(), v[live.cuda()][:, None].contiguous(),
                     slots[live].cuda()[:, None].contiguous(), base, kk, vv, k_scale=ks, v_scale=vs)
        assert torch.equal(raw(vc)[at], raw(vv)[at])
    rest = torch.ones(P * ps, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(raw(kc)[rest], raw(k0)[rest]) and torch.equal(raw(vc)[rest], raw(v0)[rest])
    assert fw.device_status() == 0


@pytest.mark.parametrize("scale", [1.0, 0.013, 1 / 3, 0.75, 1.9999999, 448.0, 2.0 ** -70, 1e-30, 1e25, 3e38, 0.1, 7e-4])
def test_every_value_is_coded_as_the_append_codes_it(fw, scale):
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(256, 2, 128).cuda()
    x, _ = make(256, 2, 2, 128, norm=False, seed=4)
    slots = torch.arange(256, dtype=torch.int32, device="cuda")
    a, b = (torch.zeros(16, 16, 2, 128, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    k = torch.zeros_like(a)
    x["positions"].zero_()                            # keys by no angle: as they are
    x["k"] = every
    fw.qk_norm_rope_append(v=every, slot_mapping=slots, layer_base_rows=0, k_cache=k, v_cache=a, k_scale=scale, v_scale=scale, **x)
    fw.kv_append(every[:, None], None, slots[:, None].contiguous(), 0, b, None, k_scale=scale)
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # (A turn by nothing adds zeros, which a key whose partner is not finite does not survive.)
    ok = torch.isfinite(every) & torch.isfinite(every.roll(64, 2)) & (every != 0)
    assert torch.equal(k.view(torch.uint8).view(256, 2, 128)[ok], b.view(torch.uint8).view(256, 2, 128)[ok])


def test_append_of_keys_alone_padded_slots_and_strided_cache(fw):
    x, _ = make(12, 4, 2, 128, seed=1)
    big = torch.zeros(4, 2, 16, 2, 128, dtype=torch.bfloat16, device="cuda")   # K and V halves of every page
    slots = torch.tensor([[0, 5, -1, -1], [17, 18, 19, 40], [63, -1, -1, -1]], dtype=torch.int32, device="cuda")
    q = fw.qk_norm_rope_append(v=None, slot_mapping=slots, layer_base_rows=0, k_cache=big[:, 0], v_cache=None, **x)
    y, size = want(x, "k")
    at = slots.flatten().cpu()
    rows = big[:, 0].reshape(64, 2, 128)
    check_bf16(rows[at[at >= 0].long().cuda()], (y[(at >= 0).numpy()], size[(at >= 0).numpy()]), "k")
    assert (big[:, 1] == 0).all() and int((rows.abs().sum((1, 2)) > 0).sum()) == int((at >= 0).sum())
    check_bf16(q, want(x, "q"), "q")


def test_slot_behind_the_cache_is_skipped_and_told(fw):
    x, v = make(3, 4, 2, 128, seed=2)
    kc, vc = caches(2, 16, 2, 128, torch.bfloat16)
    k0 = kc.clone()
    slots = torch.tensor([32, 2 ** 31 - 1, 31], dtype=torch.int32, device="cuda")
    fw.qk_norm_rope_append(v=v, slot_mapping=slots, layer_base_rows=0, k_cache=kc, v_cache=vc, **x)
    assert fw.device_status() == 1 and fw.device_status() == 0
    assert torch.equal(kc.view(32, 2, 128)[:31], k0.view(32, 2, 128)[:31])
    assert not torch.equal(kc.view(32, 2, 128)[31], k0.view(32, 2, 128)[31])


def test_axis_out_of_range_is_told(fw):
    x, _ = make(3, 4, 2, 128, axes=2, seed=2)
    x["axis_map"][7] = 2
    q, _ = fw.qk_norm_rope(**x)
    assert fw.device_status() == 1
    x["axis_map"][7] = 0
    assert torch.equal(q, fw.qk_norm_rope(**x)[0])


def test_no_tokens(fw):
    x, v = make(4, 4, 2, 128)
    for name in ("q", "k"):
        x[name] = x[name][:0]
    x["positions"] = x["positions"][:0]
    before = fw.launch_count()
    q, k = fw.qk_norm_rope(**x)
    assert q.shape == (0, 4, 128) and k.shape == (0, 2, 128) and fw.launch_count() == before


def test_stream_and_graph(fw):
    x, v = make(64, 8, 2, 128, seed=11)
    kc, vc = caches(8, 16, 2, 128, torch.bfloat16)
    slots = torch.randperm(128)[:64].to(torch.int32).cuda()
    call = lambda: fw.qk_norm_rope_append(v=v, slot_mapping=slots, layer_base_rows=0, k_cache=kc, v_cache=vc, **x)
    ref = call()
    kref = kc.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    kc.zero_()
    s.wait_stream(torch.cuda.current_stream())
    q = fw.qk_norm_rope_append(v=v, slot_mapping=slots, layer_base_rows=0, k_cache=kc, v_cache=vc, stream=s, **x)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(q, ref) and torch.equal(kc.view(128, 2, 128)[slots.long()], kref.view(128, 2, 128)[slots.long()])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = call()
    x["q"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q, -ref)
