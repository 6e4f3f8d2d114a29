"""Dense product with its epilogue (moe_linear_forward) against the formula in
64 bits.

Tolerance of one output, from the arithmetic: the sums are fp32 sums of K
exact products in some order, off by at most 2 K 2^-24 sum|x w| (twice the
usual bound: a tensor core may truncate where fp32 rounds); an activation
passes an error on with a slope of at most 1.13; the epilogue's own fp32
steps and its exponential are within 2^-20 relative; the final rounding is at
most half a step of the output type."""
import ctypes as C

import numpy as np
import pytest

import quantized_expert_ffn_03_b200 as M

ACTS = {"none": M.MOE_ACT_NONE, "silu": M.MOE_ACT_SILU, "gelu": M.MOE_ACT_GELU, "gelu_tanh": M.MOE_ACT_GELU_TANH,
        "relu": M.MOE_ACT_RELU}
CODES = {"bf16": M.MOE_BF16, "f16": M.MOE_F16, "f32": M.MOE_F32}
SENTINEL = 7.0


def torch_type(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def act64(v, act):
    import torch
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (v + 0.044715 * v ** 3))
    return torch.relu(v) if act == "relu" else v


def reference(x, w, bias, act, wu=None, bias_u=None, res=None):
    """(value, bound before the last rounding), both fp64 [T][N]."""
    x, w = x.double(), w.double()
    K = x.shape[1]

    def product(m, b):
        v, mag = x @ m.T, x.abs() @ m.abs().T
        if b is not None:
            v, mag = v + b.double(), mag + b.double().abs()
        return v, 2 * (K + 1) * 2.0 ** -24 * mag

    g, dg = product(w, bias)
    y = act64(g, act)
    dy = 1.13 * dg + 2.0 ** -20 * y.abs()
    if wu is not None:
        u, du = product(wu.double(), bias_u)
        dy = dy * u.abs() + y.abs() * du + dy * du
        y = y * u
        dy = dy + 2.0 ** -24 * y.abs()
    if res is not None:
        y = y + res.double()
        dy = dy + 2.0 ** -24 * y.abs()
    return y, dy


def check(out, ref, slack):
    """Every output within its bound plus half a step of its type."""
    import torch
    half = torch.finfo(out.dtype).eps / 2
    tiny = torch.finfo(out.dtype).smallest_normal * half * 2
    err = (out.double() - ref).abs()
    lim = slack + half * (ref.abs() + slack) + tiny
    assert torch.isfinite(out).all()
    worst = (err / lim).max().item()
    assert worst <= 1.0, worst


def make(T, K, N, dtype="bf16", out="bf16", act="none", gated=False, bias=False, res=False, pad=0, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + T + 7 * K + 13 * N)
    dt = torch_type(dtype)

    def rows(n, k, extra, std):
        ld = (k + 7) // 8 * 8 + extra
        buf = (torch.randn(n, ld, generator=g, device="cuda") * std).to(dt)
        buf[:, k:] = float("nan")  # columns behind the last are never used
        return buf[:, :k]

    d = dict(x=rows(T, K, pad, 1.0), w=rows(N, K, 8 if pad else 0, 0.05), wu=None, bias=None, bias_u=None, res=None)
    if gated:
        d["wu"] = rows(N, K, 16 if pad else 0, 0.05)
    if bias:
        d["bias"] = torch.randn(N, generator=g, device="cuda") * 0.2
        d["bias_u"] = torch.randn(N, generator=g, device="cuda") * 0.2 if gated else None
    if res:
        d["res"] = torch.randn(T, N, generator=g, device="cuda").to(torch_type(out))
    d["cfg"] = M.linear_config(K, N, act=ACTS[act], gated=gated, dtype=CODES[dtype], out_dtype=CODES[out])
    d["wts"] = M.linear_weights(d["cfg"], d["w"], d["bias"], d["wu"], d["bias_u"])
    d["ref"] = reference(d["x"], d["w"], d["bias"], act, d["wu"], d["bias_u"], d["res"])
    return d


def run_guarded(d, T, N, out, ldo=None):
    """The call on rows in the middle of a larger buffer: nothing around them changes."""
    import torch
    ldo = ldo or N
    buf = torch.full((T + 4, ldo), SENTINEL, dtype=torch_type(out), device="cuda")
    view = buf[2:2 + T, :N]
    M.moe_linear_forward(d["cfg"], d["wts"], d["x"], view, residual=d["res"])
    torch.cuda.synchronize()
    assert M.moe_linear_device_error() == (M.MOE_OK, 0)
    assert (buf[:2] == SENTINEL).all() and (buf[2 + T:] == SENTINEL).all()
    assert (buf[:, N:] == SENTINEL).all()
    return view


# one token to long inputs; sizes below, at and above every tile and unit
SHAPES = [(1, 1, 1), (1, 8, 3), (1, 4096, 512), (2, 64, 16), (3, 100, 17), (5, 4095, 33), (7, 72, 1024),
          (8, 2048, 48), (9, 520, 129), (13, 2040, 1001), (16, 1024, 128), (17, 640, 200), (31, 96, 257),
          (33, 4096, 130), (64, 1024, 512), (65, 1000, 96), (100, 33, 640), (127, 512, 256), (128, 128, 384),
          (129, 768, 383), (200, 72, 520), (256, 2048, 1024), (257, 1000, 1000), (300, 4096, 64), (511, 65, 129),
          (1025, 320, 640), (2048, 256, 2304), (4099, 136, 72)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("form", ["plain", "full", "gated"])
def test_matches_formula(T, K, N, form):
    kw = {"plain": dict(), "full": dict(dtype="f16", out="f16", act="gelu", bias=True, res=True, pad=8),
          "gated": dict(act="silu", gated=True, bias=True, res=True)}[form]
    d = make(T, K, N, **kw)
    check(run_guarded(d, T, N, kw.get("out", "bf16")), *d["ref"])


@pytest.mark.gpu
@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("T,K,N", [(1, 256, 100), (40, 512, 264), (600, 192, 520)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
def test_activations_and_types(act, T, K, N, dtype, out):
    for gated in (False, True):
        d = make(T, K, N, dtype, out, act, gated, bias=True, res=True, pad=24, seed=3)
        check(run_guarded(d, T, N, out, ldo=N + 8), *d["ref"])  # rows on 16-byte boundaries, wider than N
        check(run_guarded(d, T, N, out, ldo=N + 5), *d["ref"])  # rows that start anywhere


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 12, 20, 64, 130, 300, 1500])
@pytest.mark.parametrize("K,N", [(4100, 520), (16384, 200), (16384, 4096), (40000, 264)])
@pytest.mark.parametrize("gated", [False, True])
def test_long_sums_in_fp32(T, K, N, gated):
    """The tensor cores cut each step of 16 columns towards zero, which loses
    2^-24 of the running sum on the average; a sum that is finished every 512
    columns loses at most 32 such steps of it, 2^-19, whatever K (the running
    sum is smaller than the last one on the average, which leaves more than
    the additions of the parts, rounded to nearest, take).  A gated output is
    the product of two such sums.  In the 2-norm over all outputs."""
    d = make(T, K, N, "bf16", "f32", "none", gated, bias=True, res=False, seed=9)
    out = run_guarded(d, T, N, "f32")
    ref = d["ref"][0]
    assert (out.double() - ref).norm() <= (2 if gated else 1) * 2.0 ** -19 * ref.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20, 150, 1300])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_residual_in_place_and_out_of_place_agree(T, out):
    import torch
    d = make(T, 512, 392, out=out, res=True, seed=4)
    apart = torch.empty_like(d["res"])
    M.moe_linear_forward(d["cfg"], d["wts"], d["x"], apart, residual=d["res"])
    M.moe_linear_forward(d["cfg"], d["wts"], d["x"], d["res"], residual=d["res"])
    assert torch.equal(apart, d["res"])
    check(apart, *d["ref"])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 30, 300, 2000])
def test_tokens_do_not_depend_on_each_other_and_runs_repeat(T):
    """A token of NaN and one of infinities leave the others as they were; a second run gives the same bits."""
    import torch
    d = make(T, 768, 520, act="silu", gated=True, seed=5)
    a = torch.empty(T, 520, dtype=torch.bfloat16, device="cuda")
    b = torch.empty_like(a)
    M.moe_linear_forward(d["cfg"], d["wts"], d["x"], a)
    M.moe_linear_forward(d["cfg"], d["wts"], d["x"], b)
    assert torch.equal(a, b)
    bad = sorted({0, T // 2})
    x = d["x"].clone()
    x[bad[0]] = float("nan")
    x[bad[-1], 5] = float("inf")
    M.moe_linear_forward(d["cfg"], d["wts"], x, b)
    rest = [t for t in range(T) if t not in bad]
    assert torch.equal(a[rest], b[rest])
    assert not torch.isfinite(b[bad].float()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,N", [(20, 63), (300, 1001), (513, 510), (40, 33)])
@pytest.mark.parametrize("off", [0, 1])
def test_rows_that_start_anywhere(T, N, off):
    """Odd row lengths, a first row that starts between two 4-byte boundaries, a residual laid out otherwise."""
    import torch
    d = make(T, 200, N, act="relu", bias=True, res=True, seed=8)
    buf = torch.full((T * N + 8,), SENTINEL, dtype=torch.bfloat16, device="cuda")
    view = buf[off:off + T * N].view(T, N)
    wide = torch.zeros(T, N + 3, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:N + 1] = d["res"]
    M.moe_linear_forward(d["cfg"], d["wts"], d["x"], view, residual=wide[:, 1:N + 1])
    check(view, *d["ref"])
    assert (buf[:off] == SENTINEL).all() and (buf[off + T * N:] == SENTINEL).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 20, 300])
def test_offsets_beyond_32_bits(T):
    """Rows of x, residual and out that lie more than 2^32 bytes apart in all."""
    import torch
    d = make(T, 128, 96, res=True, seed=9)
    ld = ((5 << 30) // 2 // (T - 1) + 7) // 8 * 8  # elements of 2 bytes: 5 GB from the first row to the last
    far = lambda a: torch.empty((T - 1) * ld + a.shape[1], dtype=a.dtype, device="cuda").as_strided(  # noqa: E731
        a.shape, (ld, 1)).copy_(a)
    x, res = far(d["x"]), far(d["res"])
    M.moe_linear_forward(d["cfg"], d["wts"], x, res, residual=res)
    check(res, *d["ref"])


@pytest.mark.gpu
def test_zero_tokens_writes_nothing():
    import torch
    cfg = M.linear_config(64, 32)
    wts = M.linear_weights(cfg, torch.ones(32, 64, dtype=torch.bfloat16, device="cuda"))
    M.moe_linear_forward(cfg, wts, torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                         torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 48, 700])
def test_two_streams_and_replayed_graphs(T):
    """Calls on two streams at once, and two captured graphs replayed at once, share nothing."""
    import torch
    ds = [make(T, 1024, 640, act="gelu_tanh", bias=True, seed=s) for s in (6, 7)]
    want = []
    for d in ds:
        o = torch.empty(T, 640, dtype=torch.bfloat16, device="cuda")
        M.moe_linear_forward(d["cfg"], d["wts"], d["x"], o)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [torch.zeros_like(o) for o in want]
    for _ in range(20):
        for d, o, st in zip(ds, got, streams):
            M.moe_linear_forward(d["cfg"], d["wts"], d["x"], o, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for d, o, st in zip(ds, got, streams):
        o.zero_()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            M.moe_linear_forward(d["cfg"], d["wts"], d["x"], o)
        graphs.append(g)
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert M.moe_linear_device_error() == (M.MOE_OK, 0)


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    import torch
    bf = dict(dtype=torch.bfloat16, device="cuda")
    cfg = M.linear_config(64, 32)
    w, x, out = torch.ones(32, 64, **bf), torch.ones(4, 64, **bf), torch.zeros(4, 32, **bf)
    wts = M.linear_weights(cfg, w)
    M.moe_linear_forward(cfg, wts, x, out)
    bad = [dict(x=x.float()), dict(x=x[:, :56]), dict(x=torch.ones(64, 4, **bf).T), dict(x=x.cpu()),
           dict(out=out[:3]), dict(out=out.float()), dict(residual=torch.zeros(4, 31, **bf)),
           dict(x=torch.ones(4, 65, **bf)[:, 1:]), dict(x=torch.ones(4, 68, **bf)[:, :64]),
           dict(out=x[:, :32]), dict(residual=torch.zeros(1, 32, **bf).expand(4, 32)),
           dict(out=torch.zeros(1, 32, **bf).expand(4, 32))]
    for kw in bad:
        args = dict(x=x, out=out, residual=None, **{})
        args.update(kw)
        with pytest.raises(M.MoeError) as e:
            M.moe_linear_forward(cfg, wts, args["x"], args["out"], residual=args["residual"])
        assert e.value.status == M.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(w_up=w), dict(bias=torch.zeros(31, device="cuda")), dict(bias_up=torch.zeros(32, device="cuda"))):
        with pytest.raises(M.MoeError):
            M.linear_weights(cfg, w, **kw)
    with pytest.raises(M.MoeError):  # weights made for another config
        M.moe_linear_forward(M.linear_config(64, 32, gated=True), wts, x, out)


def test_refusals_on_the_host():
    """Every bad argument is refused before any device work."""
    lib = M.lib()

    def call(cfg, w=16, w_up=None, bias=None, ldw=64, ldw_up=0, x=1024, ldx=64, res=None, ldr=0, T=4, out=4096, ldo=32,
             bias_up=None):
        wts = M.MoeLinearWeights(w, w_up, bias, bias_up, ldw, ldw_up)
        return lib.moe_linear_forward(C.byref(cfg), C.byref(wts), x, ldx, res, ldr, T, out, ldo, None)

    good = M.linear_config(64, 32)
    assert call(good, T=0) == 0
    for cfg, status in [(M.linear_config(0, 32), 1), (M.linear_config(64, -1), 1), (M.linear_config(64, 32, act=9), 1),
                        (M.linear_config(64, 32, dtype=M.MOE_F32), 2),
                        (M.linear_config(64, 32, out_dtype=M.MOE_F16), 2), (M.linear_config(64, 1 << 21), 2),
                        (M.linear_config(64, 32, gated=True), 1)]:
        assert call(cfg) == status, (cfg.in_features, cfg.out_features)
    for kw in [dict(T=-1), dict(x=None), dict(w=None), dict(out=None), dict(x=1032), dict(w=8), dict(ldx=60),
               dict(ldx=68), dict(ldw=63), dict(ldw=72 + 4), dict(ldo=31), dict(out=4097), dict(res=4096, ldr=31),
               dict(res=4096, ldr=40), dict(res=4099, ldr=32), dict(bias=18), dict(out=1024)]:
        assert call(good, **kw) == 1, kw
        assert M.last_error()
    assert call(good, ldx=1 << 40) == 2 and call(good, T=(1 << 30) + 1) == 2
    gated = M.linear_config(64, 32, gated=True)
    assert call(gated, w_up=24, ldw_up=64) == 1 and call(gated, w_up=32, ldw_up=60) == 1
    assert lib.moe_linear_forward(None, None, None, 0, None, 0, 0, None, 0, None) == 1


# ---- the activation alone -------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,N", [(1, 5), (12, 33), (60, 64), (300, 96), (2500, 512)])
@pytest.mark.parametrize("gated", [False, True])
def test_activations_alone_in_fp32(act, T, N, gated):
    """K = 1 and x = 1: the sum is the weight itself, so the output is the
    activation of it.  With u = 2^-24: SiLU's e^-v is off by 1.3 |v| u (the
    rounded v log2 e, about what half a step of v makes of it) and 6 u, the rest
    by 5 u.  GELU: the normal CDF (5 ulp: 10 u) and the product.  The tanh
    form's exponent z = 2 sqrt(2/pi) (v + 0.044715 v^3) is off by 6 u of it more
    (two constants and four steps).  So 2^-20 of the value, for SiLU
    2^-20 (1 + |v| / 8), for the tanh form 2^-20 (1 + |z| / 2), or 2^-126; a gate's
    product rounds once more."""
    import torch
    v = torch.cat([torch.linspace(-130, 130, 257), torch.linspace(-12, 12, 129), -torch.logspace(-30, 2, 65),
                   torch.linspace(-89, -87, 17)])
    v = v.repeat((N + len(v) - 1) // len(v) + 1)[:N + 468]
    worst = 0.0
    for first in range(0, 468, max(1, min(N, 64))):
        w = v[first:first + N].bfloat16().cuda().view(N, 1)
        x = torch.ones(T, 1, dtype=torch.bfloat16, device="cuda")
        x = torch.cat([x, torch.zeros(T, 7, dtype=torch.bfloat16, device="cuda")], 1)[:, :1]
        wpad = torch.zeros(N, 8, dtype=torch.bfloat16, device="cuda")
        wpad[:, :1] = w
        up = torch.zeros(N, 8, dtype=torch.bfloat16, device="cuda")
        up[:, :1] = 3.0
        cfg = M.linear_config(1, N, act=ACTS[act], gated=gated, out_dtype=M.MOE_F32)
        wts = M.linear_weights(cfg, wpad[:, :1], w_up=up[:, :1] if gated else None)
        out = torch.empty(T, N, device="cuda")
        M.moe_linear_forward(cfg, wts, x, out)
        d = w.double().view(1, N)
        # (the normal CDF of large negative v by erfc: 1 + erf cancels there)
        ref = (d * 0.5 * torch.special.erfc(-d * 0.5 ** 0.5) if act == "gelu" else act64(d, act)) * (3.0 if gated else 1.0)
        far = {"silu": d.abs() / 8, "gelu": 0.0,
               "gelu_tanh": (2 / np.pi) ** 0.5 * (d + 0.044715 * d ** 3).abs()}[act]
        lim = (2.0 ** -20 * (1 + far) + 2.0 ** -24) * ref.abs() + 2.0 ** -126
        worst = max(worst, ((out.double() - ref).abs() / lim).max().item())
    assert worst <= 1.0, worst


@pytest.mark.gpu
@pytest.mark.parametrize("T,N", [(12, 72), (40, 64), (200, 96), (600, 512), (1500, 2048)])
@pytest.mark.parametrize("dtype,K", [("f16", 8192), ("f16", 16384), ("f16", 16448), ("f16", 1 << 18),
                                     ("f16", 1 << 20), ("bf16", 1 << 15), ("bf16", 1 << 17), ("bf16", 1 << 20)])
@pytest.mark.parametrize("gated", [False, True])
def test_long_sums_in_16_bits(T, N, dtype, K, gated):
    """Operands of one sign: what the tensor cores cut off adds up over K.  A
    16-bit output is within half a step of its type of the sum, and 1/16 of
    that half step for the sum's own error (twice for the product of two)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(K + T)
    dt = torch_type(dtype)
    x = (0.5 + torch.rand(T, K, generator=g, device="cuda")).to(dt)
    w = ((0.5 + torch.rand(N, K, generator=g, device="cuda")) * (100.0 / K)).to(dt)
    wu = ((0.5 + torch.rand(N, K, generator=g, device="cuda")) * (100.0 / K)).to(dt) if gated else None
    cfg = M.linear_config(K, N, gated=gated, dtype=CODES[dtype])
    out = torch.empty(T, N, dtype=dt, device="cuda")
    M.moe_linear_forward(cfg, M.linear_weights(cfg, w, w_up=wu), x, out)

    def product(m):  # in fp64, a slice of K at a time
        return sum(x[:, k:k + 65536].double() @ m[:, k:k + 65536].double().T for k in range(0, K, 65536))

    ref = product(w) * (product(wu) if gated else 1.0)
    half = torch.finfo(dt).eps / 2
    assert ((out.double() - ref).abs() <= (1 + (2 if gated else 1) / 16) * half * ref.abs()).all()


@pytest.mark.gpu
def test_an_expired_wait_is_reported_to_its_stream_alone():
    """A wait that runs out on one stream: reads on other streams neither show nor clear it, its own does both once."""
    import torch
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    M.moe_linear_selftest_bounded_wait(2_000_000, stream=a)
    torch.cuda.synchronize()
    assert M.moe_linear_device_error(b) == (M.MOE_OK, 0)
    assert M.moe_linear_device_error() == (M.MOE_OK, 0)
    assert M.moe_linear_device_error(a) == (6, 1)  # MOE_ERR_TIMEOUT
    assert M.moe_linear_device_error(a) == (M.MOE_OK, 0)
    M.moe_linear_selftest_bounded_wait(2_000_000)  # the default stream's own
    assert M.moe_linear_device_error(a) == (M.MOE_OK, 0)
    assert M.moe_linear_device_error() == (6, 1)
    d = make(40, 256, 64)
    for st in (a, b, None):  # and products run as before
        out = torch.empty(40, 64, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        M.moe_linear_forward(d["cfg"], d["wts"], d["x"], out, stream=st)
        assert M.moe_linear_device_error(st) == (M.MOE_OK, 0)
        check(out, *d["ref"])


def test_selftest_limit_is_refused_on_the_host():
    assert M.lib().moe_linear_selftest_bounded_wait(1 << 40, None) == M.MOE_ERR_INVALID_ARG


@pytest.mark.gpu
def test_first_calls_from_many_host_threads():
    """Eight host threads whose first calls of every kernel meet, each on its own stream, in a fresh process."""
    import subprocess
    import sys
    code = """
import sys, threading
sys.path[:0] = %r
import torch
import quantized_expert_ffn_03_b200 as M
torch.cuda.init()
sizes = [(1, 512, 200), (12, 512, 200), (20, 512, 96), (64, 1024, 256), (300, 512, 512), (2100, 256, 1024)]
data = []
for i in range(8):
    for T, K, N in sizes:
        x, w = (torch.randn(n, K, device="cuda").bfloat16() for n in (T, N))
        data.append((i, x, w, torch.zeros(T, N, device="cuda"), x.double() @ w.double().T))
torch.cuda.synchronize()
meet, bad = threading.Barrier(8), []
def work(i):
    try:
        st = torch.cuda.Stream()
        meet.wait()
        for j, x, w, out, _ in data:
            if j == i:
                cfg = M.linear_config(x.shape[1], w.shape[0], out_dtype=M.MOE_F32)
                M.moe_linear_forward(cfg, M.linear_weights(cfg, w), x, out, stream=st)
        if M.moe_linear_device_error(st) != (M.MOE_OK, 0):
            bad.append("device error")
    except Exception as e:
        bad.append(repr(e))
ts = [threading.Thread(target=work, args=(i,)) for i in range(8)]
[t.start() for t in ts]
[t.join() for t in ts]
torch.cuda.synchronize()
# a sum of K products of 8-bit significands in fp32: 2 K 2^-24 of their magnitudes
for _, x, w, out, ref in data:
    lim = 2 * x.shape[1] * 2.0 ** -24 * (x.double().abs() @ w.double().abs().T)
    if not ((out.double() - ref).abs() <= lim).all():
        bad.append(tuple(out.shape))
print(bad)
sys.exit(1 if bad else 0)
""" % ([p for p in sys.path if p],)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 12, 17, 70, 200, 2600])
@pytest.mark.parametrize("N", [1, 33, 50, 129, 250, 1003])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("gated", [False, True])
def test_ragged_features_in_rows_on_16_byte_boundaries(T, N, dtype, out, gated):
    """N features that end inside 16 bytes of rows that start on them: what lies behind N in the row stays as it was,
    whether the residual is laid out alike, otherwise, or is the output itself."""
    import torch
    ldo = (N + 7) // 8 * 8 + 8
    d = make(T, 200, N, dtype, out, "silu", gated, bias=True, res=True, seed=12)
    ref, apart = d["ref"], d["res"]
    check(run_guarded(d, T, N, out, ldo=ldo), *ref)
    alike = torch.full((T, ldo), float("nan"), dtype=apart.dtype, device="cuda")
    alike[:, :N] = apart
    d["res"] = alike[:, :N]
    check(run_guarded(d, T, N, out, ldo=ldo), *ref)
    place = torch.full((T, ldo), SENTINEL, dtype=apart.dtype, device="cuda")
    place[:, :N] = apart
    M.moe_linear_forward(d["cfg"], d["wts"], d["x"], place[:, :N], residual=place[:, :N])
    check(place[:, :N], *ref)
    assert (place[:, N:] == SENTINEL).all()
    d["res"] = None
    y = reference(d["x"], d["w"], d["bias"], "silu", d["wu"], d["bias_u"])
    check(run_guarded(d, T, N, out, ldo=ldo), *y)


# ---- every kernel and tile that the sizes can choose --------------------------------------

# T, K, N, gated, 16-bit type, output type; tokens and width of a tile, CTAs that
# split its K, sums of parts: linear_way's choice on 148 SMs.  Ragged ends in
# every dimension; pairs beyond 2048 tokens number their tiles in groups of 8,
# the last one shorter.
WAYS = [
    (5, 1100, 90, 0, "bf16", "bf16", (8, 8, 1, 0)), (11, 1100, 90, 1, "f16", "f32", (16, 8, 1, 0)),
    (17, 90, 50, 0, "bf16", "f32", (32, 32, 1, 0)), (19, 300, 90, 1, "bf16", "bf16", (32, 32, 1, 0)),
    (12, 11000, 2050, 0, "f16", "f16", (32, 32, 2, 1)), (18, 2100, 100, 0, "bf16", "bf16", (32, 32, 4, 0)),
    (20, 2200, 70, 1, "f16", "f32", (32, 32, 4, 1)), (17, 1150, 2080, 0, "f16", "f32", (32, 32, 2, 1)),
    (17, 2327, 2080, 1, "bf16", "bf16", (32, 32, 2, 0)), (17, 40, 4850, 0, "bf16", "bf16", (32, 64, 1, 0)),
    (18, 1133, 2478, 0, "f16", "f32", (32, 64, 2, 1)), (17, 2242, 2531, 1, "f16", "f16", (32, 64, 2, 0)),
    (17, 2116, 1075, 1, "bf16", "f32", (32, 64, 4, 1)), (19, 1123, 4757, 0, "bf16", "bf16", (32, 128, 2, 0)),
    (17, 1100, 2135, 0, "f16", "f16", (32, 128, 4, 0)),
    (44, 5400, 5430, 0, "bf16", "bf16", (64, 128, 2, 0)), (57, 1690, 2105, 0, "f16", "f16", (64, 128, 4, 0)),
    (33, 1089, 2122, 0, "f16", "f16", (64, 32, 2, 0)), (36, 2454, 1061, 1, "f16", "f32", (64, 64, 4, 1)),
    (40, 100, 4817, 1, "bf16", "bf16", (64, 64, 1, 0)), (33, 531, 4959, 0, "f16", "f32", (64, 64, 1, 1)),
    (67, 100, 90, 0, "bf16", "bf16", (128, 32, 1, 0)), (70, 1900, 90, 1, "f16", "f32", (128, 32, 2, 1)),
    (69, 2400, 70, 0, "bf16", "f32", (128, 32, 4, 1)), (70, 4000, 70, 1, "f16", "f16", (128, 32, 4, 0)),
    (135, 1261, 1223, 0, "f16", "f32", (128, 64, 2, 1)), (131, 40, 2421, 1, "f16", "f32", (128, 64, 1, 0)),
    (69, 2650, 2391, 1, "bf16", "bf16", (128, 64, 2, 0)), (70, 2850, 1071, 0, "f16", "f32", (128, 64, 4, 1)),
    (132, 36, 4764, 0, "bf16", "bf16", (128, 128, 1, 0)), (67, 1247, 4894, 0, "f16", "f16", (128, 128, 2, 0)),
    (820, 2740, 402, 0, "bf16", "bf16", (128, 128, 4, 0)), (131, 2740, 1269, 0, "bf16", "bf16", (128, 128, 4, 0)),
    (262, 40, 6476, 0, "bf16", "bf16", (256, 128, 1, 0)), (6406, 40, 257, 0, "f16", "f32", (256, 128, 1, 0)),
    (6328, 40, 132, 1, "bf16", "bf16", (256, 128, 1, 0)), (130, 100, 4780, 1, "f16", "f32", (256, 128, 1, 0)),
    (6385, 1030, 133, 0, "f16", "f32", (256, 128, 1, 1)), (6824, 1090, 65, 1, "bf16", "f32", (256, 128, 1, 1)),
    (6407, 620, 257, 0, "f16", "f16", (256, 256, 1, 0)), (2500, 700, 1301, 0, "bf16", "bf16", (256, 256, 1, 0)),
    (4000, 500, 2000, 0, "bf16", "f32", (256, 256, 1, 0)), (6285, 623, 135, 1, "bf16", "bf16", (256, 256, 1, 0)),
    (2300, 700, 1000, 1, "f16", "f16", (256, 256, 1, 0)), (2300, 510, 2001, 1, "f16", "f32", (256, 256, 1, 0)),
    (14, 9000, 4400, 0, "f16", "f16", (32, 64, 2, 1))]
WAY_DRIVER = """
#include <cstdio>
#include "moe_linear_way.h"
int main() {
  int T, K, N, gated, f16, f32;
  while (scanf("%d %d %d %d %d %d", &T, &K, &N, &gated, &f16, &f32) == 6) {
    const moe::LinearWay w = moe::linear_way(T, K, N, gated, f16, f32, 148);
    printf("%d %d %d %d\\n", w.tokens, w.width, w.split, (int)w.sums);
  }
}
"""


def test_ways_that_the_sizes_choose(tmp_path):
    """The table below is what linear_way chooses, so that the GPU test reaches every kernel and tile."""
    import os
    import subprocess
    src, exe = tmp_path / "ways.cpp", tmp_path / "ways"
    src.write_text(WAY_DRIVER)
    csrc = os.path.join(os.path.dirname(M.LIB_PATH), "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", csrc, str(src), "-o", str(exe)])
    text = "".join("%d %d %d %d %d %d\n" % (*c[:4], c[4] == "f16", c[5] == "f32") for c in WAYS)
    out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    got = [tuple(int(v) for v in line.split()) for line in out]
    assert [(c[:6], w) for c, w in zip(WAYS, got) if w != c[6]] == []
    tiles = {(w[0], w[1]) for w in got}
    assert tiles == {(8, 8), (16, 8), (256, 128), (256, 256)} | {(t, f) for t in (32, 64, 128) for f in (32, 64, 128)}


@pytest.mark.gpu
@pytest.mark.parametrize("case", WAYS, ids=lambda c: "x".join(map(str, c[:3])) + "-" + "-".join(map(str, c[6])))
def test_every_way_matches_formula(case):
    """Against 64 bits with bias, activation and residual, rows of the output on 16-byte boundaries and anywhere; a
    second run gives the same bits."""
    T, K, N, gated, dtype, out, _ = case
    d = make(T, K, N, dtype, out, "silu" if gated else "gelu", bool(gated), bias=True, res=True, pad=8, seed=11)
    wide = (N + 7) // 8 * 8 + 8
    a = run_guarded(d, T, N, out, ldo=wide)
    check(a, *d["ref"])
    assert (run_guarded(d, T, N, out, ldo=wide) == a).all()
    check(run_guarded(d, T, N, out, ldo=wide + 1), *d["ref"])
    import torch
    far = torch.zeros(T, wide, dtype=d["res"].dtype, device="cuda")  # the residual on such boundaries as well
    far[:, :N] = d["res"]
    d["res"] = far[:, :N]
    assert (run_guarded(d, T, N, out, ldo=wide) == a).all()
