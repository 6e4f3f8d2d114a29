"""Expert choice (moe_route_from_logits, moe_route_topk) against the rules in
64 bits, written as plain loops.

The choice is exact: values are compared in fp64 on both sides, and the
random inputs leave no two values within 1e-12 of each other unless the
logits are equal (then the rule is the lower index).  Weights are fp32: the
row's sum of exponentials is the largest error, each off by at most
2 + 1.16 |x| ulp of e^x (so at most 2^-18 of the sum, where terms with
|x| > 20 weigh nothing), then under 40 roundings of 2^-24: RTOL.  Over many
weights these errors have both signs: the 2-norm is held to 2^-20.  Ties and
near ties of the projected logits (moe_route_topk) are compared on the logits
that the call returns."""
import ctypes as C
import math

import numpy as np
import pytest

import quantized_expert_ffn_03_b200 as M

SCORES = {"softmax": M.MOE_SCORE_SOFTMAX, "sigmoid": M.MOE_SCORE_SIGMOID}
GROUPS = {"max": M.MOE_GROUP_MAX, "top2": M.MOE_GROUP_TOP2}
RTOL, ATOL = 2.0 ** -18, 2.0 ** -126


def plain(logits, bias, K, score="softmax", groups=1, keep=1, group_score="max", renorm=True, scale=1.0):
    """logits fp64 [T][E] (already the values of their type); bias fp32 [E] or None."""
    T, E = logits.shape
    per = E // groups
    idx, w = np.zeros((T, K), np.int32), np.zeros((T, K))
    for t in range(T):
        l = np.where(np.isnan(logits[t]), -np.inf, np.minimum(logits[t], float(np.finfo(np.float32).max)))
        with np.errstate(over="ignore"):
            if score == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-l))
            else:
                p = np.exp(l - l.max()) if np.isfinite(l.max()) else np.zeros(E)
                s = p / p.sum() if p.sum() > 0 else p
        with np.errstate(invalid="ignore"):
            v = s if bias is None else s + bias.astype(np.float64)
        v = np.where(np.isnan(v), -np.inf, v)
        order_by = l if bias is None else v
        if groups > 1 and keep < groups:
            val = []
            for g in range(groups):
                m = sorted(v[g * per:(g + 1) * per], reverse=True)
                m0 = m[0] if bias is not None or group_score == "top2" else l[g * per:(g + 1) * per].max()
                val.append(m[0] + m[1] if group_score == "top2" and per > 1 else m0)
            kept = sorted(range(groups), key=lambda g: (-val[g], g))[:keep]
        else:
            kept = range(groups)
        cand = [e for g in kept for e in range(g * per, (g + 1) * per)]
        chosen = sorted(cand, key=lambda e: (-order_by[e], e))[:K]
        idx[t] = chosen
        c = s[chosen]
        if renorm:
            c = c / c.sum() if c.sum() > 0 else np.zeros(K)
        w[t] = c * float(np.float32(scale))
    return idx, w


def run(logits, K, bias=None, score="softmax", groups=1, keep=1, group_score="max", renorm=True, scale=1.0):
    import torch
    T, E = logits.shape
    cfg = M.route_config(E, K, SCORES[score], groups, keep, GROUPS[group_score], renorm, scale)
    idx = torch.full((T + 1, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, K), -7.0, device="cuda")
    b = None if bias is None else torch.from_numpy(bias).cuda()
    M.moe_route_from_logits(cfg, logits, idx[:T], w[:T], select_bias=b)
    torch.cuda.synchronize()
    assert (idx[T] == -7).all() and (w[T] == -7).all()
    return idx[:T].cpu().numpy(), w[:T].cpu().numpy().astype(np.float64)


def check(logits, K, bias=None, **kw):
    gi, gw = run(logits, K, bias, **kw)
    wi, ww = plain(logits.double().cpu().numpy(), bias, K, **kw)
    assert np.array_equal(gi, wi)
    assert np.isfinite(gw).all()
    np.testing.assert_allclose(gw, ww, rtol=RTOL, atol=ATOL)
    assert np.linalg.norm(gw - ww) <= 2.0 ** -20 * np.linalg.norm(ww) + ATOL


def draw(T, E, seed, dtype="f32", pad=0, std=1.3):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    return (torch.randn(T, E + pad, generator=g, device="cuda") * std).to(dt)[:, :E]


def bias_of(E, seed, off=0):
    r = np.random.RandomState(seed)
    b = (0.05 * r.standard_normal(E)).astype(np.float32)
    b[r.permutation(E)[:off]] = -np.inf
    return b


CASES = [  # T, E, K, groups, keep
    (1, 1, 1, 1, 1), (1, 8, 8, 1, 1), (1, 512, 4, 1, 1), (3, 33, 5, 1, 1), (5, 512, 10, 16, 4), (7, 60, 6, 4, 2),
    (65, 256, 8, 8, 4), (9, 96, 8, 32, 5), (4, 31, 7, 31, 9), (130, 1000, 16, 1, 1), (17, 1024, 32, 16, 3),
    (6, 2048, 32, 32, 7), (2, 1999, 3, 1, 1), (700, 128, 2, 4, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K,groups,keep", CASES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_matches_rules(T, E, K, groups, keep, score, dtype):
    logits = draw(T, E, T + E + K, dtype, pad=3 if T > 4 else 0)
    for group_score in ("max", "top2") if groups > 1 else ("max",):
        for bias in (None, bias_of(E, E, off=E // 9)):
            check(logits, K, bias, score=score, groups=groups, keep=keep, group_score=group_score)
            check(logits, K, bias, score=score, groups=groups, keep=keep, group_score=group_score, renorm=False,
                  scale=2.5)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 2)])
def test_ties_go_to_the_lower_index(score, groups, keep):
    """Equal logits, zeros of both signs, and two values one fp32 rounding apart (their fp32 sigmoids are equal)."""
    import torch
    l = torch.zeros(5, 64, device="cuda")
    l[1, ::2] = -0.0
    l[2] = draw(1, 64, 1).round()[0]
    l[3, :] = 9.0
    l[3, 63] = float(np.nextafter(np.float32(9.0), np.float32(10.0)))
    l[4, 5:] = -3e38
    for bias in (None, np.zeros(64, np.float32)):
        for gs in ("max", "top2"):
            check(l, 6, bias, score=score, groups=groups, keep=keep, group_score=gs)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,keep", [(30, 1, 1), (64, 16, 5), (512, 16, 4)])
@pytest.mark.parametrize("spread", [2e-6, 1e-4, 1e-2])
def test_near_ties_follow_fp64(score, E, groups, keep, spread):
    """Logits a few fp32 steps apart and biases that nearly make up for them: fp32 scores cannot order these values."""
    import torch
    r = np.random.RandomState(E)
    l = np.float32(2.0) + (spread * r.standard_normal((300, E))).astype(np.float32)
    l = torch.from_numpy(l.astype(np.float32)).cuda()
    for bias in (np.zeros(E, np.float32), (0.1 * spread * r.standard_normal(E)).astype(np.float32)):
        for gs in ("max", "top2"):
            for renorm in (True, False):
                check(l, 6, bias, score=score, groups=groups, keep=keep, group_score=gs, renorm=renorm)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("groups,keep", [(1, 1), (6, 2)])
def test_masked_and_non_finite_rows(score, renorm, groups, keep):
    """A row with nothing left, with one expert left, of lowest values, with NaN, with infinities."""
    import torch
    inf = float("inf")
    l = draw(8, 48, 9)
    l[0] = -inf
    l[1] = -inf
    l[1, 40] = 0.5
    l[2] = torch.finfo(torch.float32).min
    l[3, ::3] = float("nan")
    l[4] = float("nan")
    l[5, 7] = inf
    l[5, 30] = inf
    l[6, 3:] = -inf
    l[7, 0] = 1e30
    off = np.zeros(48, np.float32)
    off[10:44] = -np.inf
    nan = np.zeros(48, np.float32)
    nan[2] = np.nan
    always = bias_of(48, 4)
    always[[3, 20, 41]] = np.inf  # experts that every token takes
    huge = (1e30 * np.arange(48)).astype(np.float32)
    for bias in (None, bias_of(48, 3), off, nan, np.full(48, -np.inf, np.float32), always, huge,
                 np.full(48, np.inf, np.float32)):
        for gs in ("max", "top2"):
            for K in (1, 5):
                check(l, K, bias, score=score, renorm=renorm, groups=groups, keep=keep, group_score=gs, scale=1.5)


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    import torch
    T, ld = 40, 1 << 25
    l = torch.empty((T - 1) * ld + 64, device="cuda").as_strided((T, 64), (ld, 1)).copy_(draw(T, 64, 17))
    check(l, 5, bias_of(64, 17), score="sigmoid")


@pytest.mark.gpu
def test_graph_replay_and_other_stream():
    import torch
    l = draw(40, 256, 11)
    cfg = M.route_config(256, 8, M.MOE_SCORE_SIGMOID, 8, 4, M.MOE_GROUP_TOP2)
    want_i, want_w = torch.empty(40, 8, dtype=torch.int32, device="cuda"), torch.empty(40, 8, device="cuda")
    M.moe_route_from_logits(cfg, l, want_i, want_w)
    torch.cuda.synchronize()
    i, w = torch.zeros_like(want_i), torch.zeros_like(want_w)
    st = torch.cuda.Stream()
    M.moe_route_from_logits(cfg, l, i, w, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(i, want_i) and torch.equal(w, want_w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.moe_route_from_logits(cfg, l, i, w)
    i.zero_(), w.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(i, want_i) and torch.equal(w, want_w)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,E", [(1, 4096, 512), (5, 264, 60), (200, 1024, 256)])
@pytest.mark.parametrize("into", ["logits_out", "workspace"])
def test_projection_and_choice(T, H, E, into):
    """moe_route_topk: logits within the fp32 summation bound, the choice exact on them."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + H)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    wr = (torch.randn(E, H, generator=g, device="cuda") * 0.02).bfloat16()
    rb, sb = torch.randn(E, generator=g, device="cuda") * 0.1, torch.from_numpy(bias_of(E, 5)).cuda()
    cfg = M.route_config(E, 4, M.MOE_SCORE_SIGMOID, 4, 2, M.MOE_GROUP_TOP2, True, 1.5)
    idx, w = torch.empty(T, 4, dtype=torch.int32, device="cuda"), torch.empty(T, 4, device="cuda")
    kw = {}
    buf = torch.empty(M.moe_route_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
    logits = buf[:4 * T * E].view(torch.float32).view(T, E) if into == "workspace" else \
        torch.empty(T, E, device="cuda")
    kw[into] = buf if into == "workspace" else logits
    M.moe_route_topk(cfg, x, wr, idx, w, router_bias=rb, select_bias=sb, **kw)
    torch.cuda.synchronize()
    ref = x.double() @ wr.double().T + rb.double()
    lim = 2 * (H + 1) * 2.0 ** -24 * (x.double().abs() @ wr.double().abs().T + rb.double().abs())
    assert ((logits.double() - ref).abs() <= lim).all()
    wi, ww = plain(logits.double().cpu().numpy(), sb.cpu().numpy(), 4, score="sigmoid", groups=4, keep=2,
                   group_score="top2", scale=1.5)
    assert np.array_equal(idx.cpu().numpy(), wi)
    np.testing.assert_allclose(w.cpu().numpy(), ww, rtol=RTOL)


@pytest.mark.gpu
def test_softmax_choice_is_the_routers():
    """Softmax, no groups, renormalised: the choice of moe_topk_from_logits, its weights to fp32 rounding."""
    import torch
    l = draw(33, 512, 21).contiguous()
    idx, w = torch.empty(33, 4, dtype=torch.int32, device="cuda"), torch.empty(33, 4, device="cuda")
    M.moe_topk_from_logits(M.config(4096, 1024, 512, 4), l, idx, w)
    gi, gw = run(l, 4)
    assert np.array_equal(gi, idx.cpu().numpy())
    np.testing.assert_allclose(gw, w.cpu().numpy().astype(np.float64), rtol=2 * RTOL)


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    import torch
    cfg = M.route_config(64, 4)
    l, idx, w = torch.zeros(3, 64, device="cuda"), torch.zeros(3, 4, dtype=torch.int32, device="cuda"), \
        torch.zeros(3, 4, device="cuda")
    M.moe_route_from_logits(cfg, l, idx, w)
    for a in [(l[:, :60], idx, w), (l.double(), idx, w), (l.cpu(), idx, w), (l, idx.long(), w), (l, idx[:2], w),
              (l, idx, w.half()), (torch.zeros(64, 3, device="cuda").T, idx, w),
              (torch.zeros(1, 64, device="cuda").expand(3, 64), idx, w)]:
        with pytest.raises(M.MoeError) as e:
            M.moe_route_from_logits(cfg, *a)
        assert e.value.status == M.MOE_ERR_INVALID_ARG
    with pytest.raises(M.MoeError):
        M.moe_route_from_logits(cfg, l, idx, w, select_bias=torch.zeros(63, device="cuda"))


def test_refusals_on_the_host():
    lib = M.lib()

    def call(cfg, logits=16, dtype=M.MOE_F32, ldl=64, bias=None, T=2, idx=32, w=48):
        return lib.moe_route_from_logits(C.byref(cfg), logits, dtype, ldl, bias, T, idx, w, None)

    good = M.route_config(64, 4, n_groups=8, topk_groups=2)
    assert call(good, T=0) == 0
    for cfg, status in [(M.route_config(0, 1), 1), (M.route_config(64, 0), 1), (M.route_config(64, 33), 2),
                        (M.route_config(4096, 4), 2), (M.route_config(64, 4, n_groups=64, topk_groups=8), 2),
                        (M.route_config(64, 4, n_groups=7, topk_groups=2), 1),
                        (M.route_config(64, 4, n_groups=8, topk_groups=9), 1),
                        (M.route_config(64, 17, n_groups=8, topk_groups=2), 1), (M.route_config(4, 5), 1),
                        (M.route_config(64, 4, score=2), 1), (M.route_config(64, 4, group_score=5), 1),
                        (M.route_config(64, 4, scale=math.inf), 1), (M.route_config(64, 4, scale=math.nan), 1)]:
        assert call(cfg) == status, (cfg.n_experts, cfg.top_k, cfg.n_groups)
        assert M.last_error()
        if status == 1:
            assert M.moe_route_workspace_bytes(cfg, 4) == 0
    for kw in [dict(T=-1), dict(logits=None), dict(idx=None), dict(w=None), dict(ldl=63), dict(logits=18),
               dict(bias=2), dict(idx=33), dict(w=50)]:
        assert call(good, **kw) == 1, kw
    assert call(good, dtype=7) == 2 and call(good, T=(1 << 30) + 1) == 2
    assert M.moe_route_workspace_bytes(good, 3) == 768

    def topk(cfg, hidden=64, x=1024, wr=2048, T=2, idx=32, w=48, lo=None, ws=4096, nb=1 << 20):
        return lib.moe_route_topk(C.byref(cfg), hidden, x, wr, None, None, T, idx, w, lo, ws, nb, None)

    assert topk(good, T=0) == 0
    assert topk(good, hidden=60) == 2 and topk(good, x=None) == 1 and topk(good, x=1032) == 1
    assert topk(good, ws=None) == M.MOE_ERR_WORKSPACE and topk(good, nb=100) == M.MOE_ERR_WORKSPACE


# ---- values that cancel, and far scores ------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B", [1e3, 1e5, 1e6, 3e38])
@pytest.mark.parametrize("per,rest", [(2, 0.0), (8, -1.0), (8, -4.0), (32, -1.0)])
def test_groups_whose_two_values_cancel(score, B, per, rest):
    """Biases +B and -B in every group (the others at rest * B): the sum of the
    two largest is small, the fp32 roundings of its summands are not.  Logits
    so far apart that these roundings decide most rows."""
    import torch
    G, keep = 8, 4
    bias = np.full((G, per), max(rest * B, -3.4e38), np.float32)
    bias[:, 0], bias[:, 1] = B, -B
    r = np.random.RandomState(per)
    bias = np.stack([r.permutation(b) for b in bias]).reshape(-1)
    spread = min(4.0 * 2.0 ** -24 * B * (2 * G if score == "softmax" else 1), 2.0)
    l = torch.from_numpy((0.1 + spread * r.standard_normal((200, G * per))).astype(np.float32)).cuda()
    for K in (1, 6):
        check(l, K, bias, score=score, groups=G, keep=keep, group_score="top2")


@pytest.mark.gpu
def test_cancelling_groups_by_hand():
    """Sigmoid scores (.50004, .5) and (.500029, .500029) under biases (1000, -1000): the second group's sum is larger."""
    import torch
    s = np.array([[0.50004, 0.5, 0.500029, 0.500029]])
    l = torch.from_numpy(np.log(s / (1 - s)).astype(np.float32)).cuda()
    bias = np.array([1000, -1000, 1000, -1000], np.float32)
    idx, _ = run(l, 1, bias, score="sigmoid", groups=2, keep=1, group_score="top2")
    assert idx[0, 0] == 2
    check(l, 2, bias, score="sigmoid", groups=2, keep=1, group_score="top2")


# Weights against the formula, u = 2^-24.  A chosen exponential is within 2 ulp
# (4 u), a sigmoid by its division and 1 + e within 8 u; the sum of the chosen
# adds 8 + 5 u, division and scale 2 u: 23 u.  Softmax without renormalising
# divides by the sum over all experts instead: its fast exponentials 2 + 1.66 |x|
# ulp, where |x| is 4.9 at most on the average weighted by them (20 u), 15
# additions, reciprocal, product and scale, and the chosen one's own 4 u: 42 u.
WEIGHT_RTOL = {True: 2.0 ** -19, False: 2.0 ** -18}  # by "sum of the chosen, or sigmoid"


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scale", [1.0, 2.5, 1e6, 1e-6])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_weights_hold_their_bound(score, renorm, scale, dtype):
    """Every weight within its bound of the formula (or 2^-126): chosen scores
    from the largest to far below fp32's range, forced by the bias."""
    import torch
    r = np.random.RandomState(5)
    for E, low in ((24, -100.0), (512, -30.0), (1000, -60.0), (2048, -8.0)):
        l = np.where(r.rand(40, E) < 0.5, low * r.rand(40, E), 1.3 * r.standard_normal((40, E)))
        l[0], l[1] = -69.0, -88.8
        l[2, :] = np.linspace(-105.0, -60.0, E)
        l[3, 0], l[3, 1:] = 80.0, -60.0
        l = torch.from_numpy(l.astype(np.float32)).to(
            {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]).cuda()
        for bias in (None, (2.0 * r.rand(E)).astype(np.float32)):
            gi, gw = run(l, 16, bias, score=score, renorm=renorm, scale=scale)
            wi, ww = plain(l.double().cpu().numpy(), bias, 16, score=score, renorm=renorm, scale=scale)
            assert np.array_equal(gi, wi)
            np.testing.assert_allclose(gw, ww, rtol=WEIGHT_RTOL[renorm or score == "sigmoid"], atol=ATOL)


@pytest.mark.gpu
def test_a_weight_whose_score_leaves_the_range_of_fp32():
    """Sigmoid scores of -69 and -88.8 (the second is below fp32's normal range) renormalised: 2.5e-9, not 0."""
    import torch
    l = torch.tensor([[-69.0, -88.8, -200.0, -300.0]], device="cuda")
    _, w = run(l, 2, None, score="sigmoid")
    want = np.exp(-88.8 + 69.0)
    np.testing.assert_allclose(w[0, 1], np.exp(np.float64(np.float32(-88.8)) + 69.0), rtol=WEIGHT_RTOL[True])
    assert abs(w[0, 1] / want - 1) < 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("E", [1280, 1281, 1472, 1473, 1500, 1536, 1537, 1984, 2047])
@pytest.mark.parametrize("bias", [False, True])
def test_numbers_of_experts_around_the_shared_memory_limit(E, bias):
    """A row's fp64 keys take 8 bytes of shared memory per expert and warp, next to some static ones; a row of equal
    logits and one of nothing need them."""
    l = draw(6, E, E)
    l[1], l[2] = 0.5, -float("inf")
    for K in (1, 9):
        check(l, K, bias_of(E, 2) if bias else None, score="sigmoid")
