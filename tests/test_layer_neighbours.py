"""The routing and the dense products together with the expert layer, as a
decoder block runs them: projection into the residual stream, choice of
experts, a shared FFN of its own width, the routed experts; and the batched
path under a given routing."""
from dataclasses import replace

import numpy as np
import pytest

import oracle as O
import synth as S
from layer_setup import (DeviceLayer, assert_outputs_close, from_dev_bits, ocfg, oracle_forward, to_dev_bits)

import quantized_expert_ffn_03_b200 as M


def routed(dl, x, res, idx, w, fn):
    import torch
    T = x.shape[0]
    ws = torch.zeros(max(M.moe_layer_batched_workspace_bytes(dl.cfg, T), M.moe_layer_workspace_bytes(dl.cfg, T)),
                     dtype=torch.uint8, device="cuda")
    h, y = torch.full_like(x, 0x7fc0), torch.full_like(x, 0x7fc0)
    getattr(M, fn)(dl.cfg, dl.wts, x, res, idx, w, h, y, ws)
    torch.cuda.synchronize()
    return h, y, M.moe_device_error(ws)[0]


@pytest.mark.gpu
@pytest.mark.parametrize("T,has_shared", [(1, 1), (33, 1), (150, 0)])
def test_batched_with_given_routing_matches_oracle(T, has_shared):
    import torch
    s = replace(S.TINY, tokens=T, has_shared=has_shared)
    dl = DeviceLayer(s)
    x, res = S.activations(s, step=6)
    r = np.random.RandomState(T)
    idx = np.stack([r.permutation(s.n_experts)[:s.top_k] for _ in range(T)]).astype(np.int32)
    idx[-1] = idx[-1, 0]  # one expert named twice
    w = r.uniform(0.1, 0.9, (T, s.top_k)).astype(np.float32)
    h, y, st = routed(dl, to_dev_bits(x), to_dev_bits(res), torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(),
                      "moe_layer_forward_routed_batched")
    assert st == M.MOE_OK
    _, _, h_ref, y_ref = oracle_forward(s, dl.oracle_blobs(), dl.dense, x, res, idx_in=idx, w_in=w.astype(np.float64))
    assert_outputs_close(from_dev_bits(h), h_ref, "h_out")
    assert_outputs_close(from_dev_bits(y), y_ref, "y_norm")


@pytest.mark.gpu
def test_batched_with_its_own_routing_is_the_batched_call():
    """The routing that moe_layer_forward_batched finds, given back, gives its result bit for bit."""
    import torch
    s = replace(S.TINY, tokens=70)
    dl = DeviceLayer(s)
    x, res = (to_dev_bits(a) for a in S.activations(s, step=7))
    ws = torch.zeros(M.moe_layer_batched_workspace_bytes(dl.cfg, 70), dtype=torch.uint8, device="cuda")
    h, y = torch.empty_like(x), torch.empty_like(x)
    idx = torch.empty((70, s.top_k), dtype=torch.int32, device="cuda")
    w = torch.empty((70, s.top_k), device="cuda")
    M.moe_layer_forward_batched(dl.cfg, dl.wts, x, res, h, y, idx, w, workspace=ws)
    h2, y2, st = routed(dl, x, res, idx, w, "moe_layer_forward_routed_batched")
    assert st == M.MOE_OK and torch.equal(h, h2) and torch.equal(y, y2)


@pytest.mark.gpu
def test_batched_with_a_bad_id_reports_it_and_the_next_call_is_right():
    import torch
    s = replace(S.TINY, tokens=40)
    dl = DeviceLayer(s)
    x, res = (to_dev_bits(a) for a in S.activations(s, step=8))
    idx = torch.zeros((40, s.top_k), dtype=torch.int32, device="cuda")
    idx[:, 1] = 3
    w = torch.full((40, s.top_k), 0.5, device="cuda")
    good = routed(dl, x, res, idx, w, "moe_layer_forward_routed_batched")
    bad = idx.clone()
    bad[5, 0], bad[7, 1], bad[9, 0] = s.n_experts, -1, 2 ** 30
    assert routed(dl, x, res, bad, w, "moe_layer_forward_routed_batched")[2] == M.MOE_ERR_DEVICE
    again = routed(dl, x, res, idx, w, "moe_layer_forward_routed_batched")
    assert good[2] == again[2] == M.MOE_OK and torch.equal(good[0], again[0])


def test_batched_routed_refusals_on_the_host():
    import ctypes as C
    lib, cfg = M.lib(), M.config(256, 128, 16, 2)
    wts = M.MoeLayerWeights()
    args = lambda idx, w: (C.byref(cfg), C.byref(wts), 16, 16, 40, idx, w, 16, 16, 256, 1 << 20, None)  # noqa: E731
    assert lib.moe_layer_forward_routed_batched(*args(None, 16)) == 1
    assert lib.moe_layer_forward_routed_batched(*args(16, None)) == 1
    assert lib.moe_layer_forward_routed_batched(*args(16, 16)) == 1 and "NULL" in M.last_error()
    assert lib.moe_layer_forward_routed_batched(C.byref(cfg), C.byref(wts), 16, 16, 0, None, None, 16, 16, 256, 0,
                                                None) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 6, 90])
def test_a_block_around_the_layer(T):
    """h = h0 + proj(a); experts by sigmoid with a balance bias and groups; a gated shared FFN three times as wide as
    the experts whose sum enters as the layer's residual; the routed experts.  Every step is compared with 64 bits
    on the device's own inputs of that step, the layer with the oracle."""
    import torch
    from test_linear import check, reference
    s = replace(S.TINY, tokens=T, has_shared=0)
    H, wide = s.hidden, 3 * s.inter
    dl = DeviceLayer(s)
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *sh, std=1.0: (torch.randn(*sh, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    a, h = rnd(T, 512), rnd(T, H)
    wo, wr = rnd(H, 512, std=0.02), rnd(s.n_experts, H, std=0.05)
    wg, wu, wd = rnd(wide, H, std=0.02), rnd(wide, H, std=0.02), rnd(H, wide, std=0.02)
    # projection into the residual stream, in place
    ref = reference(a, wo, None, "none", res=h)
    cfg = M.linear_config(512, H)
    M.moe_linear_forward(cfg, M.linear_weights(cfg, wo), a, h, residual=h)
    check(h, *ref)
    x = h
    # choice
    rc = M.route_config(s.n_experts, s.top_k, M.MOE_SCORE_SIGMOID, 4, 2, M.MOE_GROUP_TOP2, True, 1.5)
    idx = torch.empty(T, s.top_k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, s.top_k, device="cuda")
    sb = torch.randn(s.n_experts, generator=g, device="cuda") * 0.05
    logits = torch.empty(T, s.n_experts, device="cuda")
    M.moe_route_topk(rc, x, wr, idx, w, select_bias=sb, logits_out=logits)
    from test_route import plain
    wi, ww = plain(logits.double().cpu().numpy(), sb.cpu().numpy(), s.top_k, score="sigmoid", groups=4, keep=2,
                   group_score="top2", scale=1.5)
    assert np.array_equal(idx.cpu().numpy(), wi)
    # shared FFN of its own width; its sum with h is the layer's residual
    up = M.linear_config(H, wide, act=M.MOE_ACT_SILU, gated=True)
    mid = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")
    M.moe_linear_forward(up, M.linear_weights(up, wg, w_up=wu), x, mid)
    check(mid, *reference(x, wg, None, "silu", wu))
    down = M.linear_config(wide, H)
    res = torch.empty_like(h)
    M.moe_linear_forward(down, M.linear_weights(down, wd), mid, res, residual=h)
    check(res, *reference(mid, wd, None, "none", res=h))
    bits = lambda t: t.view(torch.int16)  # noqa: E731
    fn = "moe_layer_forward_routed_batched" if T >= 32 else "moe_layer_forward_routed"
    ho, yo, st = routed(dl, bits(x), bits(res), idx, w, fn)
    assert st == M.MOE_OK and M.moe_linear_device_error() == (M.MOE_OK, 0)
    _, _, h_ref, y_ref = oracle_forward(s, dl.oracle_blobs(), dl.dense, from_dev_bits(bits(x)),
                                        from_dev_bits(bits(res)), idx_in=idx.cpu().numpy(),
                                        w_in=w.cpu().numpy().astype(np.float64))
    assert_outputs_close(from_dev_bits(ho), h_ref, "h_out")
    assert_outputs_close(from_dev_bits(yo), y_ref, "y_norm")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 12, 60, 700])
@pytest.mark.parametrize("graph", [False, True])
def test_dependent_calls_back_to_back(T, graph):
    """Kernels that start before the one ahead has ended wait for its results: a chain of products, choices and
    torch operations, each reading what the one before wrote, gives the same bits with and without waits between."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    H, E = 1024, 64
    w = [(torch.randn(H, H, generator=g, device="cuda") * 0.01).bfloat16() for _ in range(3)]
    cfg = M.linear_config(H, H, act=M.MOE_ACT_SILU, gated=True)
    wts = [M.linear_weights(cfg, w[i], w_up=w[(i + 1) % 3]) for i in range(3)]
    wr = (torch.randn(E, H, generator=g, device="cuda") * 0.05).bfloat16()
    rc = M.route_config(E, 4, M.MOE_SCORE_SIGMOID, 8, 3, M.MOE_GROUP_TOP2)
    x0 = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    sb = torch.zeros(E, device="cuda")
    bufs = [torch.empty_like(x0) for _ in range(2)]
    idx, wt = torch.empty(T, 4, dtype=torch.int32, device="cuda"), torch.empty(T, 4, device="cuda")
    logits = torch.empty(T, E, device="cuda")
    seen = torch.zeros(24, T, 4, dtype=torch.int32, device="cuda")

    def chain(wait):
        bufs[0].copy_(x0)
        for i in range(24):
            a, b = bufs[i % 2], bufs[(i + 1) % 2]
            M.moe_linear_forward(cfg, wts[i % 3], a, b, residual=a)
            wait()
            if i % 4 == 1:
                b.div_(b.float().abs().amax() + 0.25)  # keeps the stream's size
                wait()
            M.moe_route_topk(rc, b, wr, idx, wt, select_bias=sb, logits_out=logits)
            wait()
            if i % 3 == 0:
                sb.copy_(wt[0].sum() * logits[-1] * 0.01)
                wait()
            seen[i].copy_(idx)
        return bufs[0].clone(), seen.clone(), wt.clone()

    sb.zero_()
    want = chain(torch.cuda.synchronize)
    assert all(torch.isfinite(a.float()).all() for a in want)
    for _ in range(5):
        sb.zero_()
        if graph:
            torch.cuda.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                got = chain(lambda: None)
            sb.zero_()
            gr.replay()
        else:
            got = chain(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert M.moe_linear_device_error() == (M.MOE_OK, 0)


@pytest.mark.parametrize("fn", ["moe_layer_forward_routed", "moe_layer_forward_routed_batched"])
def test_a_given_routing_off_its_elements_is_refused_on_the_host(fn):
    """Kernels read idx and w as 4-byte elements: other addresses never reach them."""
    import ctypes as C
    lib, cfg, wts = M.lib(), M.config(256, 128, 16, 2), M.MoeLayerWeights()
    for idx, w in ((18, 16), (16, 17), (17, 18)):
        assert getattr(lib, fn)(C.byref(cfg), C.byref(wts), 16, 16, 40, idx, w, 16, 16, 256, 1 << 20, None) == 1
        assert "aligned to their elements" in M.last_error(), (idx, w)
    assert getattr(lib, fn)(C.byref(cfg), C.byref(wts), 16, 16, 0, 18, 17, 16, 16, 256, 0, None) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 14, 50, 300, 2200])
def test_biases_that_start_between_16_byte_boundaries(T):
    """Biases cut out of a longer vector: products, and choices with and without groups."""
    import torch
    from test_linear import check, make
    from test_route import draw, plain
    for gated in (False, True):
        d = make(T, 136, 200, "bf16", "bf16", "silu", gated, bias=True, seed=14)
        cut = lambda b: None if b is None else torch.cat([b.new_full((1,), float("nan")), b])[1:]  # noqa: E731
        wts = M.linear_weights(d["cfg"], d["w"], cut(d["bias"]), d["wu"], cut(d["bias_u"]))
        out = torch.empty(T, 200, dtype=torch.bfloat16, device="cuda")
        M.moe_linear_forward(d["cfg"], wts, d["x"], out)
        check(out, *d["ref"])
    l = draw(T, 128, 15)
    sb = torch.randn(131, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")[3:] * 0.1
    for groups, keep in ((1, 1), (8, 3)):
        cfg = M.route_config(128, 6, M.MOE_SCORE_SIGMOID, groups, keep, M.MOE_GROUP_TOP2)
        idx, w = torch.empty(T, 6, dtype=torch.int32, device="cuda"), torch.empty(T, 6, device="cuda")
        M.moe_route_from_logits(cfg, l, idx, w, select_bias=sb)
        wi, _ = plain(l.double().cpu().numpy(), sb.cpu().numpy(), 6, score="sigmoid", groups=groups, keep=keep,
                      group_score="top2")
        assert np.array_equal(idx.cpu().numpy(), wi)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 700])
def test_captured_between_copies_and_forks(T):
    """A graph whose calls stand behind a host copy, a memset, a fork and a join, replayed on new inputs: each call
    waits for all that is ahead of it."""
    import torch
    g = torch.Generator().manual_seed(T)
    H, E = 512, 64
    w = [(torch.randn(H, H, generator=g) * 0.05).bfloat16().cuda() for _ in range(3)]
    wr = (torch.randn(E, H, generator=g) * 0.05).bfloat16().cuda()
    cfg = M.linear_config(H, H)
    wts = [M.linear_weights(cfg, a) for a in w]
    rc = M.route_config(E, 4, M.MOE_SCORE_SIGMOID, 8, 3, M.MOE_GROUP_TOP2)
    host = torch.empty(T, H, dtype=torch.bfloat16, pin_memory=True)
    x, a, b, y = (torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    logits = torch.empty(T, E, device="cuda")
    idx, wt = torch.empty(T, 4, dtype=torch.int32, device="cuda"), torch.empty(T, 4, device="cuda")
    back = torch.empty(T, 4, dtype=torch.int32, pin_memory=True)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        x.copy_(host, non_blocking=True)
        y.zero_()
        M.moe_linear_forward(cfg, wts[0], x, a)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            M.moe_linear_forward(cfg, wts[1], a, b)
        M.moe_linear_forward(cfg, wts[2], a, y, residual=y)
        main.wait_stream(side)
        M.moe_linear_forward(cfg, wts[0], b, y, residual=y)
        M.moe_route_topk(rc, y, wr, idx, wt, logits_out=logits)
        back.copy_(idx, non_blocking=True)

    ins = [torch.randn(T, H, generator=g).bfloat16() for _ in range(6)]
    host.copy_(ins[0])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for v in ins:
        host.copy_(v)
        step()
        torch.cuda.synchronize()
        want = y.clone(), wt.clone(), back.clone()
        for t in (x, a, b, y, logits):
            t.fill_(float("nan"))
        back.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(wt, want[1]) and torch.equal(back, want[2])
    assert M.moe_linear_device_error() == (M.MOE_OK, 0)
