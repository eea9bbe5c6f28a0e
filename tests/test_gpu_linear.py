"""moe_linear and moe_linear_backward against 64-bit references on the same 16-bit inputs.

Tolerances, from the arithmetic.  A matrix instruction adds 32 products to its fp32 accumulator, so
a sum of n products is n / 32 roundings in sequence, at most 32 inside an instruction, and at most
one per split: (n / 32 + 48) 2^-23 sum |x y| bounds its error (2^-23, a whole step, in case the
instruction truncates).  The activation's slope is below 1.13; its own fp32 evaluation is off by a
few steps, 2^-20 (1 + |z|) at most.  The result is then rounded once: half a step of its type.
"""
import math

import pytest

import quantized_expert_layer_amd as q
from tests.gpu_util import case

pytestmark = pytest.mark.gpu

DTYPES = ("fp16", "bf16")


def _t(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _rand(g, shape, scale, dtype):
    import torch
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _strided(t, pad):
    """The same matrix with `pad` NaN columns behind each row."""
    import torch
    if not pad:
        return t
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


def _act64(z, act):
    import torch
    if act == "relu":
        return torch.relu(z)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    return z


def _slope64(z, act):
    import torch
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _half_step(ref, dtype):
    import torch
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def _close(got, ref, tol, what):
    import torch
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    bad = err > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {err.numel()} beyond the bound, worst "
                           f"{float((err / tol).max()):.2f} times it")


def _sum_bound(n):
    return (n / 32 + 48) * 2.0 ** -23


def _check_forward(M, K, N, dtype, out="same", act="none", bias=True, residual=True, preact=True,
                   pads=(0, 0, 0, 0, 0), seed=0, inplace=False):
    import torch
    dt = _t(dtype)
    ot = dt if out == "same" else _t(out)
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = _strided(_rand(g, (M, K), 1.0, dt), pads[0])
    w = _strided(_rand(g, (N, K), K ** -0.5, dt), pads[1])
    b = _rand(g, (N,), 0.5, dt) if bias else None
    r = _strided(_rand(g, (M, N), 1.0, dt), pads[2]) if residual else None
    z64 = a.double() @ w.double().t().contiguous()
    mag = a.double().abs() @ w.double().abs().t().contiguous()
    if bias:
        z64, mag = z64 + b.double(), mag + b.double().abs()
    tol = _sum_bound(K) * mag
    ref = _act64(z64, act)
    if residual:
        ref = ref + r.double()
    o = r if inplace else _strided(torch.full((M, N), float("nan"), dtype=ot, device="cuda"), pads[3])
    z = _strided(torch.full((M, N), float("nan"), dtype=dt, device="cuda"), pads[4]) if preact else None
    got = q.moe_linear(a, w, bias=b, act=act, residual=r, out=o, preact=z)
    torch.cuda.synchronize()
    assert got is o
    own = (1 + z64.abs()) * 2.0 ** -20 if act in ("silu", "gelu") else 0.0
    what = f"linear {M}x{K}x{N} {dtype}->{out} {act}"
    _close(got, ref, 1.13 * tol + own + _half_step(ref.abs() + tol, ot) + 2.0 ** -23 * ref.abs(), what)
    if preact:
        _close(z, z64, tol + _half_step(z64.abs() + tol, dt), what + " preact")
    if pads[3] and not inplace:                     # columns behind the rows stay as they were
        assert torch.isnan(o._base[:, N:].float()).all()


SIZES = [(1, 64, 16), (1, 4096, 16), (17, 2048, 2048), (3, 8, 1), (5, 7, 9), (64, 72, 65),
         (130, 1000, 257), (257, 129, 131), (300, 64, 300), (16, 6400, 48), (33, 640, 4096),
         (1900, 200, 1808), (4000, 72, 3402), (70, 6400, 520), (31, 1024, 2050), (4352, 72, 4120)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", SIZES)
def test_linear_sizes(M, K, N, dtype):
    case(f"linear {M}x{K}x{N} {dtype}")
    _check_forward(M, K, N, dtype)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("dtype,out", [("fp16", "same"), ("bf16", "fp32")])
def test_linear_activations_and_fp32_output(act, dtype, out):
    for M, K, N in ((9, 256, 40), (200, 136, 264)):
        case(f"linear {act} {dtype}->{out} {M}x{K}x{N}")
        _check_forward(M, K, N, dtype, out=out, act=act)
        _check_forward(M, K, N, dtype, out=out, act=act, bias=False, residual=False, preact=False)


@pytest.mark.parametrize("pads", [(8, 16, 8, 8, 8), (3, 5, 1, 7, 2), (64, 0, 2, 0, 0)])
def test_linear_strided_rows_with_nan_behind_them(pads):
    for M, K, N in ((6, 64, 24), (70, 200, 136), (65, 131, 33)):
        case(f"linear strided {pads} {M}x{K}x{N}")
        _check_forward(M, K, N, "bf16", act="relu", pads=pads)


@pytest.mark.parametrize("dtype,out", [("fp16", "same"), ("bf16", "same"), ("bf16", "fp32")])
def test_linear_rows_of_any_length(dtype, out):
    """Rows that start on 2 (fp32: on 4) bytes, in place too, and nothing written behind them."""
    import torch
    for M, K, N in ((20, 96, 61), (130, 200, 259), (300, 64, 1021), (700, 2056, 45)):
        case(f"linear odd rows {M}x{K}x{N} {dtype}->{out}")
        _check_forward(M, K, N, dtype, out=out, act="silu", pads=(1, 3, 5, 7, 9))
        _check_forward(M, K, N, dtype, out=out, act="none", bias=False)
        if out == "same":
            _check_forward(M, K, N, dtype, act="relu", inplace=True, pads=(0, 0, 3, 0, 0))
        g = torch.Generator(device="cuda").manual_seed(N)
        dt, ot = _t(dtype), _t(dtype if out == "same" else out)
        x, w = _rand(g, (M, K), 1.0, dt), _rand(g, (N, K), K ** -0.5, dt)
        buf = torch.full((M, N + 3), 7.0, dtype=ot, device="cuda")
        kept = torch.full((M, N + 6), 7.0, dtype=dt, device="cuda")
        q.moe_linear(x, w, act="relu", out=buf[:, :N], preact=kept[:, :N])
        assert (buf[:, N:] == 7).all() and (kept[:, N:] == 7).all()
        assert torch.equal(buf[:, :N], q.moe_linear(x, w, act="relu", out_dtype=ot))


def test_linear_residual_updated_in_place():
    for M, K, N in ((5, 512, 96), (400, 192, 520)):
        case(f"linear in place {M}x{K}x{N}")
        _check_forward(M, K, N, "fp16", act="gelu", inplace=True, pads=(0, 0, 8, 0, 0))


def test_linear_special_values():
    """A NaN or infinite input reaches exactly the outputs its row or column feeds; extremes of the
    activations stay what the definition gives."""
    import torch
    a = torch.zeros((40, 128), dtype=torch.float16, device="cuda")
    w = torch.zeros((24, 128), dtype=torch.float16, device="cuda")
    w[:, 0] = 1.0
    a[:, 0] = torch.linspace(-30, 30, 40).half()
    a[3, 0], a[7, 0], a[9, 0] = float("nan"), float("inf"), float("-inf")
    case("linear special values")
    for act in ("none", "relu", "silu", "gelu"):
        out = q.moe_linear(a, w, act=act, out_dtype=torch.float32)
        x = a[:, :1].double().expand(-1, 24)
        ref = _act64(x, act)
        if act in ("silu", "gelu"):
            ref[9] = float("nan")                     # -inf times 0
        fin = torch.isfinite(ref)
        assert torch.equal(torch.isnan(out), torch.isnan(ref)), act
        assert torch.equal(out[7], torch.full_like(out[7], float("inf"))), act
        err = (out.double() - ref).abs()[fin]
        assert (err <= 2.0 ** -20 * (1 + x.abs()[fin])).all(), act


def test_linear_empty_and_refusals():
    import torch
    f16, bf16 = torch.float16, torch.bfloat16
    z = lambda *s, dt=f16: torch.zeros(s, dtype=dt, device="cuda")
    assert q.moe_linear(z(0, 64), z(8, 64)).shape == (0, 8)
    assert q.moe_linear(z(4, 64), z(0, 64)).shape == (4, 0)
    bad = [
        (TypeError, lambda: q.moe_linear(z(4, 64, dt=torch.float32), z(8, 64, dt=torch.float32))),
        (TypeError, lambda: q.moe_linear(z(4, 64), z(8, 64, dt=bf16))),
        (TypeError, lambda: q.moe_linear(z(4, 64).cpu(), z(8, 64).cpu())),
        (ValueError, lambda: q.moe_linear(z(4, 64), z(8, 64).cpu())),
        (ValueError, lambda: q.moe_linear(z(4, 64), z(8, 72))),
        (ValueError, lambda: q.moe_linear(z(4, 64), z(64, 8).t())),
        (ValueError, lambda: q.moe_linear(z(4, 64), z(1, 64).expand(8, 64))),
        (ValueError, lambda: q.moe_linear(z(4, 64), z(8, 64), act="swiglu")),
        (ValueError, lambda: q.moe_linear(z(4, 64), z(8, 64), bias=z(9))),
        (ValueError, lambda: q.moe_linear(z(4, 64), z(8, 64), residual=z(4, 9))),
        (TypeError, lambda: q.moe_linear(z(4, 64), z(8, 64), out_dtype=torch.float64)),
        (q.MoEError, lambda: q.moe_linear(z(4, 64), z(8, 64), out_dtype=bf16)),
        (q.MoEError, lambda: q.moe_linear(z(4, 0), z(8, 0))),
        (q.MoEError, lambda: q.moe_linear(z(4, 72)[:, 1:65], z(8, 64))),     # starts off 16 bytes
        (ValueError, lambda: q.moe_linear_backward(z(4, 9), z(4, 64), z(8, 64))),
        (q.MoEError, lambda: q.moe_linear_backward(z(4, 8), z(4, 64), z(8, 64), act="relu")),
        (q.MoEError, lambda: q.moe_linear_backward(z(4, 8), z(4, 64), z(8, 64), need_a=False,
                                                   need_w=False, need_bias=False)),
    ]
    for i, (exc, call) in enumerate(bad):
        with pytest.raises(exc):
            call()
            pytest.fail(f"call {i} was accepted")
    # a workspace that is too short is refused, one of the asked size is taken
    a, w = z(5, 7), z(9, 7)
    need = q.moe_linear_workspace_size(5, 9, 7)
    assert need > 0
    with pytest.raises(q.MoEError):
        q.moe_linear(a, w, ws=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    q.moe_linear(a, w, ws=torch.empty(need, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()


def _check_backward(M, K, N, dtype, grad="same", act="none", pads=(0, 0, 0, 0), seed=0, only=None):
    import torch
    dt = _t(dtype)
    gt = dt if grad == "same" else _t(grad)
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = _strided(_rand(g, (M, K), 1.0, dt), pads[0])
    w = _strided(_rand(g, (N, K), K ** -0.5, dt), pads[1])
    go = _strided(_rand(g, (M, N), 0.1, gt), pads[2])
    z = _strided(_rand(g, (M, N), 1.5, dt), pads[3]) if act != "none" else None
    dz = go.double()
    rel = 0.0                                         # rounding of dz as the products read it
    if act != "none":
        dz = dz * _slope64(z.double(), act)
    absolute = 0.0
    if gt == torch.float32 or (act in ("silu", "gelu") and M < 256):     # two 16-bit parts
        rel = 2.0 ** -17 if dtype == "bf16" else 2.0 ** -21
        absolute = 2.0 ** -25 if dtype == "fp16" else 0.0        # half of fp16's smallest step
    elif act in ("silu", "gelu"):
        rel = torch.finfo(dt).eps / 2
        absolute = 2.0 ** -25 if dtype == "fp16" else 0.0
    if act in ("silu", "gelu"):
        rel += 2.0 ** -20
        absolute += 2.0 ** -20 * 4 * 0.6              # slope off by 2^-20 (1 + |z|), |grad| < 0.6
    need = only or ("a", "w", "bias")
    what = f"linear backward {M}x{K}x{N} {dtype} grad {grad} {act}"
    ga, gw, gb = q.moe_linear_backward(go, a, w, act=act, preact=z, need_a="a" in need,
                                       need_w="w" in need, need_bias="bias" in need)
    torch.cuda.synchronize()
    parts = 2 if gt == torch.float32 or (act in ("silu", "gelu") and M < 256) else 1
    bound = dz.abs() * rel + absolute
    if "a" in need:
        ref = dz @ w.double().contiguous()
        wa = w.double().abs().contiguous()
        tol = _sum_bound(N * parts) * ((dz.abs() + bound) @ wa) + bound @ wa
        _close(ga, ref, tol + _half_step(ref.abs() + tol, dt), what + " grad_a")
    else:
        assert ga is None
    if "w" in need:
        ref = dz.t().contiguous() @ a.double().contiguous()
        aa = a.double().abs().contiguous()
        tol = _sum_bound(M * parts) * ((dz.abs() + bound).t().contiguous() @ aa) \
            + bound.t().contiguous() @ aa
        _close(gw, ref, tol + _half_step(ref.abs() + tol, dt), what + " grad_w")
    else:
        assert gw is None
    if "bias" in need:
        ref = dz.sum(dim=0)
        tol = (M + 8) * 2.0 ** -24 * dz.abs().sum(dim=0) + \
            (2.0 ** -20 * 2.4 * M if act in ("silu", "gelu") else 0.0)
        _close(gb, ref, tol + _half_step(ref.abs() + tol, dt), what + " grad_bias")
    else:
        assert gb is None


BACK_SIZES = [(1, 64, 16), (17, 2048, 64), (5, 7, 9), (544, 256, 60), (3, 8, 1), (130, 1000, 257),
              (257, 129, 131), (1000, 1808, 72), (3000, 136, 24), (1900, 1808, 72), (700, 520, 648),
              (4100, 2056, 136), (4100, 1032, 16), (2100, 2053, 60), (70000, 72, 64), (300, 72, 6400)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", BACK_SIZES)
def test_linear_backward_sizes(M, K, N, dtype):
    case(f"linear backward {M}x{K}x{N} {dtype}")
    _check_backward(M, K, N, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("grad", ["same", "fp32"])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_linear_backward_activations_and_fp32_gradients(act, grad, dtype):
    for M, K, N in ((40, 136, 60), (300, 72, 264), (4111, 1048, 24)):
        case(f"linear backward {act} grad {grad} {dtype} {M}x{K}x{N}")
        _check_backward(M, K, N, dtype, grad=grad, act=act)


@pytest.mark.parametrize("pads", [(8, 16, 8, 8), (3, 5, 1, 7)])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_linear_backward_strided_rows(pads, act):
    for M, K, N in ((6, 64, 24), (70, 200, 136), (65, 131, 33)):
        case(f"linear backward strided {pads} {act} {M}x{K}x{N}")
        _check_backward(M, K, N, "fp16", act=act, pads=pads)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", [(64, 140000, 1), (65, 262144, 33), (150, 70001, 32), (66000, 128, 31),
                                   (17001, 1000, 64), (4229, 1000, 64)])
def test_linear_backward_narrow(M, K, N, dtype):
    """Layers of up to 64 outputs, both gradients in one pass over the rows and the input's alone:
    shares of one stage, rows and columns that end inside one, strides, two parts, the same bits twice."""
    import torch
    for grad, act, pads in (("same", "none", (0, 0, 0, 0)), ("fp32", "relu", (5, 3, 1, 2)),
                            ("same", "silu", (8, 16, 8, 8))):
        case(f"linear backward narrow {M}x{K}x{N} {dtype} {grad} {act} {pads}")
        _check_backward(M, K, N, dtype, grad=grad, act=act, pads=pads)
        _check_backward(M, K, N, dtype, grad=grad, act=act, pads=pads, only=("a",))
    g = torch.Generator(device="cuda").manual_seed(0)
    dt = _t(dtype)
    go, a, w = (_rand(g, s, 1.0, dt) for s in ((M, N), (M, K), (N, K)))
    first = q.moe_linear_backward(go, a, w)
    assert all(torch.equal(x, y) for x, y in zip(first, q.moe_linear_backward(go, a, w)))
    # a row that is not a number reaches its own row of grad_a and all of grad_w, nothing else
    go[M // 2] = float("nan")
    ga, gw, gb = q.moe_linear_backward(go, a, w)
    assert torch.isnan(ga[M // 2]).all() and torch.isnan(gw).all() and torch.isnan(gb).all()
    ga[M // 2] = first[0][M // 2]
    assert torch.equal(ga, first[0])


@pytest.mark.parametrize("only", [("a",), ("w",), ("bias",), ("a", "bias")])
def test_linear_backward_wanted_gradients_only(only):
    case(f"linear backward only {only}")
    _check_backward(70, 200, 136, "bf16", only=only)
    _check_backward(70, 200, 136, "bf16", only=only, act="silu", grad="fp32")


def test_linear_backward_empty_batch_gives_zero_gradients():
    import torch
    z = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")
    case("linear backward empty")
    for act, pre in (("none", None), ("relu", z(0, 24))):
        ga, gw, gb = q.moe_linear_backward(z(0, 24), z(0, 64), z(24, 64), act=act, preact=pre)
        assert ga.shape == (0, 64) and not gw.any() and not gb.any()
    ga, gw, gb = q.moe_linear_backward(z(5, 0), z(5, 64), z(0, 64))
    assert ga.shape == (5, 64) and not ga.any() and gw.shape == (0, 64)
    torch.cuda.synchronize()


def test_linear_backward_against_differences():
    """Central differences of the kernel's own fp32 forward, one input element at a time: the step
    h moves the sum by a known amount, so (f(x + h) - f(x - h)) / 2h is the gradient up to the
    activation's third derivative (below 2) times h^2 / 6 and the sums' rounding over h."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    M, K, N, h = 6, 64, 24, 2.0 ** -4
    a = (torch.randint(-8, 9, (M, K), generator=g, device="cuda") / 16).half()
    w = (torch.randint(-8, 9, (N, K), generator=g, device="cuda") / 64).half()
    up = torch.randn((M, N), generator=g, device="cuda")
    case("linear backward against differences")
    for act in ("silu", "gelu"):
        z = torch.empty((M, N), dtype=torch.float16, device="cuda")
        f = lambda x, y: float((q.moe_linear(x, y, act=act, out_dtype=torch.float32).double()
                                * up.double()).sum())
        q.moe_linear(a, w, act=act, preact=z)
        ga, gw, _ = q.moe_linear_backward(up, a, w, act=act, preact=z)
        for i, j in ((0, 0), (2, 33), (5, 63)):
            d = torch.zeros_like(a)
            d[i, j] = h
            num = (f(a + d, w) - f(a - d, w)) / (2 * h)
            # third derivative, stored argument (half an fp16 step of |z| <= 2 on a slope that
            # changes by at most 1), output rounding, fp32 sums over h
            wmax, wsum = float(w.abs().max()), float((up[i].abs() * w[:, j].abs().float()).sum())
            tol = wsum * (2 * (wmax * h) ** 2 / 6 + 2.0 ** -10) + abs(num) * 2.0 ** -10 + 2.0 ** -10
            assert abs(float(ga[i, j]) - num) <= tol, (act, i, j, float(ga[i, j]), num, tol)
        for n, j in ((0, 0), (11, 40), (23, 63)):
            d = torch.zeros_like(w)
            d[n, j] = h / 4
            num = (f(a, w + d) - f(a, w - d)) / (h / 2)
            amax, asum = float(a.abs().max()), float((up[:, n].abs() * a[:, j].abs().float()).sum())
            tol = asum * (2 * (amax * h / 4) ** 2 / 6 + 2.0 ** -10) + abs(num) * 2.0 ** -10 + 2.0 ** -9
            assert abs(float(gw[n, j]) - num) <= tol, (act, n, j, float(gw[n, j]), num, tol)


def test_linear_on_a_side_stream_and_twice_the_same_bits():
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    a, w = _rand(g, (130, 1000), 1.0, torch.bfloat16), _rand(g, (96, 1000), 0.03, torch.bfloat16)
    go = _rand(g, (130, 96), 0.1, torch.float32)
    case("linear on a side stream")
    want = (q.moe_linear(a, w),) + q.moe_linear_backward(go, a, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = (q.moe_linear(a, w, stream=s),) + q.moe_linear_backward(go, a, w, stream=s)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_linear_in_a_captured_graph():
    """Forward and backward captured with odd sizes (packed copies, splits), replayed on new inputs
    with eager work in between."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(4)
    M, K, N = 77, 1003, 61
    a, w = _rand(g, (M, K), 1.0, torch.float16), _rand(g, (N, K), 0.03, torch.float16)
    go = _rand(g, (M, N), 0.1, torch.float16)

    def step():
        z = torch.empty((M, N), dtype=torch.float16, device="cuda")
        y = q.moe_linear(a, w, act="silu", preact=z)
        return (y, z) + q.moe_linear_backward(go, a, w, act="silu", preact=z)

    case("linear graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        a.copy_(_rand(g, (M, K), 1.0, torch.float16))
        go.copy_(_rand(g, (M, N), 0.1, torch.float16))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want)), i


def test_linear_offsets_past_32_bits():
    """A batch of 2.4e9 elements: rows at both ends against the reference, and a weight gradient that
    only the last rows feed (every other row's gradient is zero)."""
    import torch
    M, K, N = 590001, 4096, 24
    case(f"linear {M}x{K}x{N}")
    g = torch.Generator(device="cuda").manual_seed(11)
    a = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, M // 2, M - 130, M - 2, M - 1], device="cuda")
    a[rows] = _rand(g, (len(rows), K), 1.0, torch.bfloat16)
    w = _rand(g, (N, K), K ** -0.5, torch.bfloat16)
    out = q.moe_linear(a, w, out_dtype=torch.float32)
    ref = a[rows].double() @ w.double().t().contiguous()
    tol = _sum_bound(K) * (a[rows].double().abs() @ w.double().abs().t().contiguous())
    _close(out[rows], ref, tol + 2.0 ** -23 * ref.abs(), "last rows")
    live = torch.ones(M, dtype=torch.bool, device="cuda")
    live[rows] = False
    assert not out[live].any()
    go = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    go[rows] = _rand(g, (len(rows), N), 1.0, torch.bfloat16)
    ga, gw, gb = q.moe_linear_backward(go, a, w)
    r64 = go[rows].double()
    ref = r64.t().contiguous() @ a[rows].double()
    mag = r64.abs().t().contiguous() @ a[rows].double().abs()
    _close(gw, ref, _sum_bound(M) * mag + _half_step(ref.abs(), torch.bfloat16) * 1.01, "weight gradient")
    ref = r64 @ w.double().contiguous()
    mag = r64.abs() @ w.double().abs()
    _close(ga[rows], ref, _sum_bound(N) * mag + _half_step(ref.abs(), torch.bfloat16) * 1.01, "input gradient")
    assert not ga[live].any()


def test_linear_two_streams_at_once():
    """Calls that overlap on two streams, each with the workspace the binding gives it."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(12)
    a = [_rand(g, (300, 1001), 1.0, torch.float16) for _ in range(2)]
    w = [_rand(g, (200, 1001), 0.03, torch.float16) for _ in range(2)]
    go = [_rand(g, (300, 200), 0.1, torch.float16) for _ in range(2)]
    call = lambda i, s=None: (q.moe_linear(a[i], w[i], act="gelu", stream=s),) \
        + q.moe_linear_backward(go[i], a[i], w[i], stream=s)
    case("linear on two streams")
    want = [call(0), call(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            got[i].append(call(i, streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(outs, want[i]))
