"""Host-side checks of the dense products and the router gradients (no GPU needed): argument
validation of the C entry points with their documented status codes, and the workspace sizes."""
import pytest

import quantized_expert_layer_amd as q
from tests.conftest import gpu_available

FAKE, MIS, BIG = 0x10000, 0x10002, 1 << 40

# moe_linear(a, lda, w, ldw, bias, residual, ldr, M, N, K, dtype, act, out, ldo, out_dtype, preact,
#            ldp, ws, ws_bytes, stream)
LINEAR = dict(a=FAKE, lda=64, w=FAKE, ldw=64, bias=None, residual=None, ldr=0, M=4, N=8, K=64,
              dtype=0, act=0, out=FAKE, ldo=8, out_dtype=0, preact=None, ldp=0, ws=FAKE, n=BIG,
              stream=None)
BACK = dict(grad=FAKE, ldg=8, gdt=0, preact=None, ldp=0, a=FAKE, lda=64, w=FAKE, ldw=64, M=4, N=8,
            K=64, dtype=0, act=0, ga=FAKE, gw=FAKE, gb=FAKE, ws=FAKE, n=BIG, stream=None)
BALANCE = dict(logits=FAKE, ids=FAKE, active=None, off=None, S=1, T=4, E=8, k=2, coef=1.0, loss=FAKE,
               counts=FAKE, probs=FAKE, tokens=FAKE, ws=FAKE, n=BIG, stream=None)
ROUTE = dict(logits=FAKE, ids=FAKE, w=FAKE, gw=FAKE, active=None, off=None, S=1, T=4, E=8, k=2, gate=0,
             counts=FAKE, tokens=FAKE, coef=1.0, gl=None, grad=FAKE, stream=None)
COMBINE = dict(go=FAKE, y=FAKE, inv=FAKE, w=FAKE, T=4, k=2, d=16, gw=FAKE, gy=FAKE, stream=None)

INVALID, UNSUPPORTED, WORKSPACE = q.MOE_ERR_INVALID, q.MOE_ERR_UNSUPPORTED, q.MOE_ERR_WORKSPACE

REFUSALS = [
    ("moe_linear", LINEAR, [
        (INVALID, dict(M=-1)), (INVALID, dict(N=-1)), (INVALID, dict(K=0)), (INVALID, dict(dtype=2)),
        (INVALID, dict(dtype=-1)), (INVALID, dict(act=5)), (INVALID, dict(act=-1)),
        (UNSUPPORTED, dict(act=2)), (INVALID, dict(out_dtype=3)), (UNSUPPORTED, dict(out_dtype=1)),
        (INVALID, dict(lda=63)), (INVALID, dict(ldw=0)), (INVALID, dict(ldo=7)),
        (INVALID, dict(residual=FAKE, ldr=7)), (INVALID, dict(preact=FAKE + 64, ldp=7)),
        (UNSUPPORTED, dict(lda=1 << 23)), (UNSUPPORTED, dict(ldo=1 << 23)),
        (UNSUPPORTED, dict(M=(1 << 28) + 1)), (UNSUPPORTED, dict(N=1 << 23, ldo=1 << 23)),
        (UNSUPPORTED, dict(M=1 << 28, N=1 << 10, ldo=1 << 10)),
        (INVALID, dict(a=None)), (INVALID, dict(w=None)), (INVALID, dict(out=None)),
        (INVALID, dict(a=MIS)), (INVALID, dict(w=MIS)), (INVALID, dict(out=MIS)),
        (INVALID, dict(residual=MIS, ldr=8)), (INVALID, dict(preact=MIS, ldp=8)),
        (INVALID, dict(bias=FAKE + 1)), (INVALID, dict(preact=FAKE, ldp=8)),
        (INVALID, dict(residual=FAKE, ldr=16)), (INVALID, dict(residual=FAKE, ldr=8, out_dtype=2)),
        (WORKSPACE, dict(K=63, ws=None)), (WORKSPACE, dict(K=63, n=100)),
        (WORKSPACE, dict(K=63, ws=MIS))]),
    ("moe_linear_backward", BACK, [
        (INVALID, dict(M=-1)), (INVALID, dict(K=0)), (INVALID, dict(dtype=2)), (INVALID, dict(gdt=3)),
        (UNSUPPORTED, dict(gdt=1)), (UNSUPPORTED, dict(act=2)), (INVALID, dict(act=9)),
        (INVALID, dict(ga=None, gw=None, gb=None)), (INVALID, dict(ldg=7)), (INVALID, dict(lda=1)),
        (INVALID, dict(ldw=1)), (INVALID, dict(act=1, ldp=8)), (INVALID, dict(act=1, preact=FAKE, ldp=7)),
        (INVALID, dict(grad=None)), (INVALID, dict(w=None)), (INVALID, dict(a=None)),
        (INVALID, dict(grad=MIS)), (INVALID, dict(a=MIS)), (INVALID, dict(w=MIS)),
        (INVALID, dict(ga=MIS)), (INVALID, dict(gw=MIS)), (INVALID, dict(gb=FAKE + 1)),
        (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(n=0)), (WORKSPACE, dict(M=0, n=0))]),
    ("moe_balance_loss", BALANCE, [
        (INVALID, dict(T=-1)), (INVALID, dict(E=0)), (INVALID, dict(E=257)), (INVALID, dict(k=0)),
        (INVALID, dict(k=9)), (INVALID, dict(S=0)), (INVALID, dict(S=2)), (INVALID, dict(off=MIS - 1)),
        (UNSUPPORTED, dict(S=(1 << 20) + 1, off=FAKE)), (UNSUPPORTED, dict(T=1 << 28, E=1)),
        (UNSUPPORTED, dict(T=1 << 24, E=128)), (INVALID, dict(logits=None)), (INVALID, dict(ids=None)),
        (INVALID, dict(loss=None)), (INVALID, dict(counts=None)), (INVALID, dict(probs=None)),
        (INVALID, dict(tokens=None)), (INVALID, dict(logits=MIS)), (INVALID, dict(loss=MIS)),
        (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(n=64)), (WORKSPACE, dict(ws=MIS))]),
    ("moe_route_backward", ROUTE, [
        (INVALID, dict(T=-1)), (INVALID, dict(E=300)), (INVALID, dict(k=9)), (INVALID, dict(gate=2)),
        (INVALID, dict(S=3)), (INVALID, dict(gw=None, counts=None, tokens=None)),
        (INVALID, dict(tokens=None)), (INVALID, dict(counts=None)), (INVALID, dict(w=None)),
        (INVALID, dict(ids=None)), (INVALID, dict(logits=None)), (INVALID, dict(grad=None)),
        (INVALID, dict(grad=MIS)), (INVALID, dict(gl=MIS))]),
    ("moe_combine_backward", COMBINE, [
        (INVALID, dict(T=-1)), (INVALID, dict(k=0)), (INVALID, dict(k=9)), (INVALID, dict(d=0)),
        (UNSUPPORTED, dict(d=12)), (UNSUPPORTED, dict(T=1 << 24)), (INVALID, dict(gw=None, gy=None)),
        (INVALID, dict(go=None)), (INVALID, dict(y=None)), (INVALID, dict(inv=None)),
        (INVALID, dict(w=None)), (INVALID, dict(go=MIS)), (INVALID, dict(y=MIS)),
        (INVALID, dict(gy=MIS))]),
]


@pytest.mark.parametrize("name,good,bad", REFUSALS, ids=[r[0] for r in REFUSALS])
def test_refusals_come_before_the_device(name, good, bad):
    f = getattr(q.lib(), name)
    for status, change in bad:
        args = dict(good, **change)
        assert list(args) == list(good)
        assert f(*args.values()) == status, (name, change)
    if not gpu_available():
        assert f(*good.values()) == q.MOE_ERR_NO_DEVICE


def test_nothing_to_do_is_accepted_without_pointers():
    L = q.lib()
    none = dict(a=None, w=None, out=None, ws=None, n=0)
    assert L.moe_linear(*dict(LINEAR, M=0, **none).values()) == q.MOE_OK
    assert L.moe_linear(*dict(LINEAR, N=0, ldo=0, **none).values()) == q.MOE_OK
    nog = dict(grad=None, a=None, w=None, gw=None, gb=None, ws=None, n=0)
    assert L.moe_linear_backward(*dict(BACK, M=0, **nog).values()) == q.MOE_OK
    nog = dict(grad=None, a=None, w=None, ga=None, ws=None, n=0)
    assert L.moe_linear_backward(*dict(BACK, N=0, ldg=0, **nog).values()) == q.MOE_OK
    assert L.moe_route_backward(*dict(ROUTE, T=0, logits=None, grad=None).values()) == q.MOE_OK
    assert L.moe_combine_backward(*dict(COMBINE, T=0, go=None).values()) == q.MOE_OK


def test_sizes_past_32_bits_are_refused_and_not_cut_off():
    import torch
    n = (1 << 32) + 4                                  # 4 in 32 bits
    like = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="meta")
    f32, i32 = torch.float32, torch.int32
    for call in (lambda: q.moe_linear(like(n, 8), like(8, 8)),
                 lambda: q.moe_linear(like(8, 8), like(n, 8)),
                 lambda: q.moe_linear_backward(like(n, 8), like(n, 8), like(8, 8)),
                 lambda: q.moe_balance_loss(like(n, 2, dtype=f32), like(n, 1, dtype=i32), 1.0),
                 lambda: q.moe_route_backward(like(n, 2, dtype=f32), like(n, 1, dtype=i32)),
                 lambda: q.moe_combine_backward(like(n, 8), like(n, 8), like(n, dtype=i32),
                                                like(n, 1, dtype=f32))):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_workspace_sizes():
    size = q.moe_linear_workspace_size
    assert size(0, 8, 64) == 0 and size(4, 0, 64) == 0 and size(-1, 8, 64) == 0
    # rows that cannot be read in 16-byte pieces are copied, rounded up to 8 columns
    assert size(5, 9, 63) >= 2 * 64 * (5 + 9)
    assert size(5, 9, 64, lda=65, ldw=64) >= 2 * 64 * 5
    back = q.moe_linear_backward_workspace_size
    assert back(100, 64, 64, grad_f32=True) >= 2 * 2 * 100 * 64       # two 16-bit parts
    assert back(100, 60, 64) >= 2 * 100 * 64                          # gradient rows rounded up
    assert back(100, 64, 64, act="relu") >= 2 * 100 * 64
    assert q.moe_balance_workspace_size(544, 60) >= 4 * 2 * 60 * (544 // 512)
    assert q.moe_balance_workspace_size(-1, 60) == 0 and q.moe_balance_workspace_size(4, 257) == 0
