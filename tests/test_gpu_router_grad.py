"""moe_balance_loss, moe_route_backward and moe_combine_backward against 64-bit references, and a
router tuning step run as a user would: product, gate, layer, loss and the gradients back.

Tolerances: a probability is one exp, a sum of E terms and a product, (E + 8) 2^-24 relative, as the
gate weights'; a mean of n of them adds n 2^-24 at most; every other quantity is a few products of
these and inherits their relative error times the sum of its terms' magnitudes."""
import numpy as np
import pytest

import quantized_expert_layer_amd as q
import synth
from tests.gpu_util import case

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _inputs(T, E, k, seed, masked=0.0, drop=0.0):
    """Logits with some experts masked (-inf or the type's lowest value), routed ids, active flags."""
    import torch
    r = np.random.default_rng(seed)
    logits = r.standard_normal((T, E)).astype(np.float32) * 2
    if masked:
        m = r.random((T, E)) < masked
        logits[m] = np.where(r.random(int(m.sum())) < 0.5, -np.inf, np.finfo(np.float32).min)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    if drop:
        ids[r.random((T, k)) < drop] = -1
    active = (r.random(T) < 0.8).astype(np.uint8)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return dev(logits), dev(ids), dev(active)


def _softmax64(logits):
    import torch
    x = logits.double()
    x = torch.where(torch.isnan(x), torch.full_like(x, float("-inf")), x)
    m = x.amax(dim=1, keepdim=True)
    e = torch.where(x == float("-inf"), torch.zeros_like(x), torch.exp(x - m))
    s = e.sum(dim=1, keepdim=True)
    return torch.where(s > 0, e / s, torch.zeros_like(e))


def _ref_balance(logits, ids, active, offsets, coef, grad_loss=1.0):
    """(loss, counts, probs, tokens, gradient) by the definition, segment by segment."""
    import torch
    T, E = logits.shape
    k = ids.shape[1]
    cuts = [0, T] if offsets is None else offsets.tolist()
    S = len(cuts) - 1
    live = torch.ones(T, dtype=torch.bool) if active is None else active.cpu().bool()
    p = _softmax64(logits).cpu()
    idc = ids.cpu()
    counts = torch.zeros((S, E), dtype=torch.int32)
    probs = torch.zeros((S, E), dtype=torch.float64)
    tokens = torch.zeros(S, dtype=torch.int32)
    grad = torch.zeros((T, E), dtype=torch.float64)
    terms, rows_of = [], []
    for s in range(S):
        rows = [t for t in range(cuts[s], cuts[s + 1]) if live[t]]
        tokens[s] = len(rows)
        if not rows:
            continue
        for i in idc[rows].flatten().tolist():
            if 0 <= i < E:
                counts[s, i] += 1
        probs[s] = p[rows].mean(dim=0)
        f = counts[s].double() * E / (k * len(rows))
        terms.append(float((f * probs[s]).sum()))
        rows_of.append((rows, f))
    for rows, f in rows_of:
        pr = p[rows]
        grad[rows] = grad_loss * coef / (len(terms) * len(rows)) * pr * (f - (pr @ f)[:, None])
    loss = coef * sum(terms) / len(terms) if terms else 0.0
    return loss, counts, probs, tokens, grad


def _check_balance(T, E, k, offsets, use_active, seed=0, masked=0.1, drop=0.1, what=""):
    import torch
    logits, ids, active = _inputs(T, E, k, seed, masked, drop)
    active = active if use_active else None
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    coef, gl = 0.01, torch.tensor([3.0], device="cuda")
    case(f"balance T={T} E={E} k={k} {what}")
    loss, counts, probs, tokens = q.moe_balance_loss(logits, ids, coef, active=active, seq_offsets=off)
    grad = q.moe_route_backward(logits, ids, active=active, counts=counts, tokens=tokens, coef=coef,
                                grad_loss=gl, seq_offsets=off)
    torch.cuda.synchronize()
    wl, wc, wp, wt, wg = _ref_balance(logits, ids, active, off, coef, 3.0)
    assert torch.equal(counts.cpu(), wc) and torch.equal(tokens.cpu(), wt)
    n = wt.double().clamp(min=1)[:, None]
    assert ((probs.cpu().double() - wp).abs() <= (E + 8 + n) * U * wp + 1e-45).all()
    assert abs(float(loss) - wl) <= (E + 16 + float(n.max()) + len(wt)) * U * abs(wl)
    # the gradient is p (f - f p): both terms' magnitudes carry the relative error
    cuts = [0, T] if off is None else off.tolist()
    scale = torch.zeros_like(wg)
    p = _softmax64(logits).cpu()
    used = int((wt > 0).sum())
    for s in range(len(wt)):
        a, b = cuts[s], cuts[s + 1]
        if int(wt[s]):
            f = wc[s].double() * E / (k * int(wt[s]))
            scale[a:b] = 3.0 * coef / (used * int(wt[s])) * p[a:b] * (f + (p[a:b] @ f)[:, None])
    assert ((grad.cpu().double() - wg).abs() <= 3 * (E + 16) * U * scale + 1e-45).all()


@pytest.mark.parametrize("E", [1, 8, 16, 17, 60, 64, 65, 128, 200, 256])
def test_balance_expert_counts(E):
    _check_balance(37, E, min(E, 6), None, True, seed=E)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 544, 9000])
def test_balance_token_counts(T):
    _check_balance(T, 60, 4, None, T % 2 == 0, seed=T)


@pytest.mark.parametrize("offsets", [[0, 0, 0, 5, 5, 40, 41, 200, 200],    # empty ones, one token
                                     [3, 17, 33, 180],                      # tokens outside all
                                     [0, 200], [0, 0], [200, 200, 200],
                                     list(range(0, 201, 1)),                # a segment per token
                                     [0] * 70 + [100] * 70 + [200] * 70])   # long runs of empty ones
def test_balance_segments(offsets):
    for use_active in (False, True):
        _check_balance(200, 24, 2, offsets, use_active, seed=len(offsets),
                       what=f"S={len(offsets) - 1}")


def test_balance_packed_batch():
    r = np.random.default_rng(0)
    cuts = np.sort(r.integers(0, 9001, 299)).tolist()
    _check_balance(9000, 64, 6, [0] + cuts + [9000], True, seed=1, what="S=300")


@pytest.mark.parametrize("T,E,k,S", [(40000, 16, 2, 600), (300, 24, 2, 5000), (40000, 60, 4, 5000),
                                     (3000, 130, 3, 129), (3000, 200, 3, 1025)])
def test_balance_many_segments(T, E, k, S):
    """Counts of segments beyond what a wave, a block and one launch deal with, and both terms of the
    gradient in one pass over them."""
    import torch
    cuts = np.sort(np.random.default_rng(S).integers(0, T + 1, S - 1)).tolist()
    offsets = [0] + cuts + [T]
    _check_balance(T, E, k, offsets, True, seed=S, what=f"S={S}")
    logits, ids, active = _inputs(T, E, k, 1)
    g = torch.Generator(device="cuda").manual_seed(S)
    w, gw = (torch.rand((T, k), generator=g, device="cuda") for _ in range(2))
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    _, counts, _, tokens = q.moe_balance_loss(logits, ids, 1.0, active=active, seq_offsets=off)
    part = dict(counts=counts, tokens=tokens, coef=1.0, seq_offsets=off)
    for mode in ("topk", "all"):
        gate = dict(gate_mode=mode, topk_w=w, grad_w=gw)
        both = q.moe_route_backward(logits, ids, active=active, **gate, **part)
        a = q.moe_route_backward(logits, ids, active=active, **gate)
        b = q.moe_route_backward(logits, ids, active=active, **part)
        # "all" adds a slot's term and the row's: three roundings of no more than the terms' sum,
        # which is below k + 1 here
        tol = 2 * U * (a.abs() + b.abs()) if mode == "topk" else 3 * U * (b.abs() + 2 * (k + 1))
        assert ((both - (a + b)).abs() <= tol).all()


def test_balance_all_padding_masked_rows_and_empty_batch():
    import torch
    logits, ids, _ = _inputs(20, 12, 2, 0)
    none = torch.zeros(20, dtype=torch.uint8, device="cuda")
    case("balance without live tokens")
    loss, counts, probs, tokens = q.moe_balance_loss(logits, ids, 0.5, active=none)
    g = q.moe_route_backward(logits, ids, active=none, counts=counts, tokens=tokens, coef=0.5)
    assert float(loss) == 0 and not counts.any() and not probs.any() and not tokens.any() and not g.any()
    # a row with no finite logit counts as a token but has no probability and no gradient
    logits[3] = float("-inf")
    logits[4] = float("nan")
    logits[5, 2] = float("nan")
    ids[3] = -1
    ids[4] = 7                                         # the same expert twice: counted twice
    loss, counts, probs, tokens = q.moe_balance_loss(logits, ids, 0.5)
    g = q.moe_route_backward(logits, ids, counts=counts, tokens=tokens, coef=0.5)
    wl, wc, wp, wt, wg = _ref_balance(logits, ids, None, None, 0.5)
    assert torch.equal(counts.cpu(), wc) and int(tokens) == 20
    assert abs(float(loss) - wl) <= 64 * U * wl and not g[3:5].any() and float(g[5, 2]) == 0
    assert ((probs.cpu().double() - wp).abs() <= 40 * U * wp).all()
    logits[0, 1] = float("inf")                        # no softmax: NaN, not a plausible number
    loss, _, probs, _ = q.moe_balance_loss(logits, ids, 0.5)
    assert torch.isnan(loss).all() and torch.isnan(probs[0, 1])
    for S, off in ((1, None), (3, torch.zeros(4, dtype=torch.int32, device="cuda"))):
        e = torch.empty((0, 12), device="cuda")
        ei = torch.empty((0, 2), dtype=torch.int32, device="cuda")
        loss, counts, probs, tokens = q.moe_balance_loss(e, ei, 0.5, seq_offsets=off)
        assert float(loss) == 0 and counts.shape == (S, 12) and not counts.any() and not tokens.any()
        assert q.moe_route_backward(e, ei, counts=counts, tokens=tokens, coef=0.5,
                                    seq_offsets=off).shape == (0, 12)
    torch.cuda.synchronize()


def _ref_gate(logits, ids, w, gw, mode):
    """Gradient through the gate weights, by the definition in 64 bits, and its terms' magnitudes."""
    import torch
    T, E = logits.shape
    k = ids.shape[1]
    p = _softmax64(logits).cpu()
    grad, mag = torch.zeros((T, E), dtype=torch.float64), torch.zeros((T, E), dtype=torch.float64)
    for t in range(T):
        slots = [(int(ids[t, j]), float(w[t, j]), float(gw[t, j])) for j in range(k)
                 if 0 <= int(ids[t, j]) < E]
        u, um = sum(a * b for _, a, b in slots), sum(abs(a * b) for _, a, b in slots)
        for e, a, b in slots:
            grad[t, e] += a * (b - u) if mode == "topk" else a * b
            mag[t, e] += abs(a) * (abs(b) + um) if mode == "topk" else abs(a * b)
        if mode == "all":
            grad[t] -= p[t] * u
            mag[t] += p[t] * um
    return grad, mag


@pytest.mark.parametrize("mode", ["topk", "all"])
@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (37, 16, 2), (50, 60, 4), (33, 64, 6), (20, 256, 8)])
def test_gate_gradient(T, E, k, mode):
    import torch
    logits, ids, active = _inputs(T, E, k, T)
    ids, w = q.moe_route_topk(logits, k, mode, active=active)
    gw = torch.randn((T, k), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    case(f"gate gradient T={T} E={E} k={k} {mode}")
    grad = q.moe_route_backward(logits, ids, gate_mode=mode, topk_w=w, grad_w=gw, active=active)
    ref, mag = _ref_gate(logits, ids.cpu(), w.cpu(), gw.cpu(), mode)
    assert ((grad.cpu().double() - ref).abs() <= (E + 24) * U * mag + 1e-45).all()
    assert not grad[active == 0].any()
    # both terms in one pass are the sum of each alone
    loss, counts, probs, tokens = q.moe_balance_loss(logits, ids, 0.1, active=active)
    bal = q.moe_route_backward(logits, ids, active=active, counts=counts, tokens=tokens, coef=0.1)
    both = q.moe_route_backward(logits, ids, gate_mode=mode, topk_w=w, grad_w=gw, active=active,
                                counts=counts, tokens=tokens, coef=0.1)
    assert ((both - (grad + bal)).abs().cpu().double()
            <= 8 * U * (mag + bal.abs().cpu().double()) + 1e-45).all()


@pytest.mark.parametrize("mode", ["topk", "all"])
def test_gate_and_balance_gradients_against_differences(mode):
    """Central differences in 64 bits of the definitions themselves (weights of the chosen experts;
    the balance loss with its counts held fixed, as they have no gradient).  With |g| < 4 and smooth
    terms of order one the h^2 error is below 1e-8 and the rounding over h below 1e-9."""
    import torch
    T, E, k, h, coef = 5, 12, 3, 1e-4, 0.7
    logits, ids, _ = _inputs(T, E, k, 9)
    ids, w = q.moe_route_topk(logits, k, mode)
    gw = torch.randn((T, k), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    _, counts, _, tokens = q.moe_balance_loss(logits, ids, coef)
    case(f"router gradients against differences {mode}")
    grad = q.moe_route_backward(logits, ids, gate_mode=mode, topk_w=w, grad_w=gw, counts=counts,
                                tokens=tokens, coef=coef).cpu().double()
    x0, idc, g64 = logits.cpu().double(), ids.cpu().long(), gw.cpu().double()
    f = counts.cpu().double()[0] * E / (k * T)

    def value(x):
        p = torch.softmax(x, dim=1)
        c = p.gather(1, idc)
        weights = c / c.sum(dim=1, keepdim=True) if mode == "topk" else c
        return float((weights * g64).sum() + coef * (f * p.mean(dim=0)).sum())

    for t in range(T):
        for e in range(E):
            d = torch.zeros_like(x0)
            d[t, e] = h
            num = (value(x0 + d) - value(x0 - d)) / (2 * h)
            assert abs(float(grad[t, e]) - num) <= 1e-7 + 2e-6 * 4, (t, e, float(grad[t, e]), num)


@pytest.mark.parametrize("T,d,k,E", [(1, 8, 1, 4), (17, 2048, 4, 60), (40, 1024, 1, 32),
                                     (9, 4096, 8, 16), (33, 2056, 6, 64), (200, 136, 2, 8)])
def test_combine_gradients(T, d, k, E):
    import torch
    r = np.random.default_rng(T)
    ids = np.stack([r.choice(E, k, replace=False) if k <= E else r.integers(0, E, k)
                    for _ in range(T)]).astype(np.int32)
    ids[r.random((T, k)) < 0.1] = -1                      # dropped slots
    idd = torch.from_numpy(ids).cuda()
    g = torch.Generator(device="cuda").manual_seed(T)
    R = T * k + 3                                         # rows behind the last expert's
    y = torch.randn((R, d), generator=g, device="cuda").half()
    go = torch.randn((T, d), generator=g, device="cuda").half()
    w = torch.rand((T, k), generator=g, device="cuda")
    case(f"combine gradients T={T} d={d} k={k}")
    _, inv, off, _, _ = q.moe_permute(idd, w, go, E, want_x_perm=False)
    mark = torch.full((R, d), 7.0, dtype=torch.float16, device="cuda")
    gw, gy = q.moe_combine_backward(go, y, inv, w, grad_y=mark.clone())
    torch.cuda.synchronize()
    pos = inv.long().reshape(T, k)
    ok = pos >= 0
    assert torch.equal(ok.cpu(), torch.from_numpy(ids >= 0))
    rows = y.double()[pos.clamp(min=0)]
    ref = (rows * go.double()[:, None, :]).sum(dim=2) * ok
    mag = (rows * go.double()[:, None, :]).abs().sum(dim=2)
    assert ((gw.double() - ref).abs() <= (d / 64 + 16) * U * mag).all() and not gw[~ok].any()
    want = mark.clone()
    want[pos[ok]] = (w[:, :, None] * go.float()[:, None, :]).half()[ok]
    assert torch.equal(gy, want)                          # one product, rounded once: exact
    a, b = q.moe_combine_backward(go, y, inv, w, need_y=False)
    assert b is None and torch.equal(a, gw)
    a, b = q.moe_combine_backward(go, y, inv, w, need_w=False, grad_y=mark.clone())
    assert a is None and torch.equal(b, gy)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -130])             # 2^-130: subnormal terms
def test_gate_gradient_of_one_expert_in_every_slot(scale):
    """Eight slots of a token that name one expert, or two: their terms add up, the same bits each time."""
    import torch
    T, E, k = 100, 24, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn((T, E), generator=g, device="cuda")
    w = torch.rand((T, k), generator=g, device="cuda") * scale
    gw = torch.randn((T, k), generator=g, device="cuda")
    ids = torch.full((T, k), 5, dtype=torch.int32, device="cuda")
    ids[50:, ::3] = 19
    case(f"gate gradient of repeated ids, scale {scale}")
    for mode in ("topk", "all"):
        first = q.moe_route_backward(logits, ids, gate_mode=mode, topk_w=w, grad_w=gw)
        for _ in range(20):
            assert torch.equal(first, q.moe_route_backward(logits, ids, gate_mode=mode, topk_w=w, grad_w=gw))
        w64, gw64 = w.double().cpu(), gw.double().cpu()
        u = (w64 * gw64).sum(dim=1, keepdim=True)
        ref = torch.zeros((T, E), dtype=torch.float64)
        # magnitude of all terms, on every expert: a slot's product, the row's sum and its share
        mag = (w64 * gw64).abs().sum(dim=1, keepdim=True) * (1 + w64.sum(dim=1, keepdim=True)) + u.abs()
        if mode == "topk":
            ref.scatter_add_(1, ids.cpu().long(), w64 * (gw64 - u))
        else:
            ref.scatter_add_(1, ids.cpu().long(), w64 * gw64)
            ref -= _softmax64(logits).cpu() * u
        # about 40 roundings of at most 2^-24 of that, each of a subnormal of at most 2^-150
        assert ((first.cpu().double() - ref).abs() <= 40 * (U * mag + 2.0 ** -150)).all(), mode


def test_router_refusals():
    import torch
    logits, ids, active = _inputs(6, 8, 2, 0)
    w = torch.rand((6, 2), device="cuda")
    y = torch.zeros((12, 16), dtype=torch.float16, device="cuda")
    go = torch.zeros((6, 16), dtype=torch.float16, device="cuda")
    inv = torch.arange(12, dtype=torch.int32, device="cuda")
    counts = torch.zeros((1, 8), dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    bad = [
        (TypeError, lambda: q.moe_balance_loss(logits.half(), ids, 1.0)),
        (TypeError, lambda: q.moe_balance_loss(logits.cpu(), ids, 1.0)),
        (TypeError, lambda: q.moe_balance_loss(logits, ids.long(), 1.0)),
        (ValueError, lambda: q.moe_balance_loss(logits, ids[:3], 1.0)),
        (ValueError, lambda: q.moe_balance_loss(logits, ids, 1.0, active=active[:3])),
        (ValueError, lambda: q.moe_balance_loss(logits, ids, 1.0, seq_offsets=off[:1])),
        (ValueError, lambda: q.moe_balance_loss(logits, ids, 1.0, counts=counts, seq_offsets=off)),
        (q.MoEError, lambda: q.moe_balance_loss(logits, ids.repeat(1, 5), 1.0)),          # k = 10
        (q.MoEError, lambda: q.moe_balance_loss(
            logits, ids, 1.0, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))),
        (q.MoEError, lambda: q.moe_route_backward(logits, ids)),                           # no gradient
        (q.MoEError, lambda: q.moe_route_backward(logits, ids, grad_w=w)),                 # no weights
        (q.MoEError, lambda: q.moe_route_backward(logits, ids, counts=counts)),            # no tokens
        (ValueError, lambda: q.moe_route_backward(logits, ids, topk_w=w, grad_w=w[:3])),
        (q.MoEError, lambda: q.moe_combine_backward(go, y, inv, w, need_w=False, need_y=False)),
        (ValueError, lambda: q.moe_combine_backward(go, y[:11], inv, w)),
        (ValueError, lambda: q.moe_combine_backward(go, y, inv[:11], w)),
        (q.MoEError, lambda: q.moe_combine_backward(go[:, :12].contiguous(), y[:, :12].contiguous(),
                                                    inv, w)),
    ]
    for i, (exc, call) in enumerate(bad):
        with pytest.raises(exc):
            call()
            pytest.fail(f"call {i} was accepted")


def _tune_step(layer, wr, x, active, target, offsets, ws):
    """One router tuning step over frozen experts: returns everything a program would look at."""
    import torch
    logits = q.moe_linear(x, wr, out_dtype=torch.float32)
    out = layer.forward(x, logits, ws=ws, gate_in_gemm=False, active=active)
    grad_out = (out.float() - target).half()
    loss, counts, probs, tokens = q.moe_balance_loss(logits, ws.bufs["ids"], 0.05, active=active,
                                                     seq_offsets=offsets)
    grad_logits = layer.router_backward(grad_out, logits, ws, active=active, counts=counts,
                                        tokens=tokens, coef=0.05, seq_offsets=offsets)
    gx, gwr, _ = q.moe_linear_backward(grad_logits, x, wr, need_bias=False)
    return out, loss, counts, grad_logits, gx, gwr


@pytest.mark.parametrize("name,T", [("tiny", 24), ("dsv2_lite", 40)])
def test_router_tuning_step(name, T):
    """The chain's gradients against the chain rule in 64 bits, from the layer's own expert rows,
    and replays of a captured step against the eager one."""
    import torch
    cfg = synth.get_config(name)
    inp = synth.make_inputs(cfg, T)
    layer = q.DeviceLayer.from_inputs(inp)
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.from_numpy(inp.x).cuda()
    wr = (torch.randn((cfg.E, cfg.d), generator=g, device="cuda") * cfg.d ** -0.5).half()
    target = torch.randn((T, cfg.d), generator=g, device="cuda") * 0.1
    active = torch.ones(T, dtype=torch.uint8, device="cuda")
    active[5] = 0
    offsets = torch.tensor([0, 7, 7, T], dtype=torch.int32, device="cuda")
    case(f"router tuning {name} T={T}")
    ws = layer.workspace(T)
    out, loss, counts, gl, gx, gwr = _tune_step(layer, wr, x, active, target, offsets, ws)
    torch.cuda.synchronize()
    b = ws.bufs
    logits64 = x.double() @ wr.double().t().contiguous()
    go = (out.float() - target).half().double()
    pos = b["inv"].long().reshape(T, cfg.k).clamp(min=0)
    gw = (b["y"].double()[pos] * go[:, None, :]).sum(dim=2).float()
    lg = logits64.float()
    gate, mag = _ref_gate(lg, b["ids"].cpu(), b["w"].cpu(), gw.cpu(), cfg.gate_mode)
    _, wc, _, _, bal = _ref_balance(lg, b["ids"], active, offsets, 0.05)
    assert torch.equal(counts.cpu(), wc)
    ref = gate + bal
    # fp32 logits off by their sum's rounding (below 2^-14 here) move a probability by as much
    tol = (mag + 0.05 * cfg.E) * 2.0 ** -13
    assert ((gl.cpu().double() - ref).abs() <= tol).all()
    ref_w = gl.double().t().contiguous() @ x.double()
    err = (gwr.double() - ref_w).abs()
    assert (err <= 2.0 ** -10 * ref_w.abs()
            + 2.0 ** -14 * (gl.double().abs().t().contiguous() @ x.double().abs())).all()
    ref_x = gl.double() @ wr.double()
    assert ((gx.double() - ref_x).abs() <= 2.0 ** -10 * ref_x.abs()
            + 2.0 ** -14 * (gl.double().abs() @ wr.double().abs()) + 2.0 ** -24).all()

    ws2 = layer.workspace(T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _tune_step(layer, wr, x, active, target, offsets, ws2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = _tune_step(layer, wr, x, active, target, offsets, ws2)
    for i in range(3):
        x.copy_((torch.randn(x.shape, generator=g, device="cuda")).half())
        graph.replay()
        torch.cuda.synchronize()
        now = _tune_step(layer, wr, x, active, target, offsets, ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(cap, now)), i
    with pytest.raises(ValueError):                  # a layer that only makes the decode call
        only = q.DeviceLayer.from_inputs(inp, decode=True)
        only.router_backward(out, lg, ws)
    # a workspace that holds no unscaled expert rows: none yet, or of a forward() or a plan with the
    # gate weight in the GEMM
    fresh = layer.workspace(T)
    with pytest.raises(ValueError):
        layer.router_backward(out, lg, fresh)
    for fill in (lambda: layer.forward(x, lg, ws=fresh), lambda: layer.plan(fresh, x, lg)):
        layer.forward(x, lg, ws=fresh, gate_in_gemm=False)
        layer.router_backward(out, lg, fresh)
        fill()
        with pytest.raises(ValueError):
            layer.router_backward(out, lg, fresh)
    torch.cuda.synchronize()


def test_router_offsets_past_32_bits():
    """Logits of 4.6 GB: counts in all, and the gradient of tokens at both ends."""
    import torch
    T, E, k = 4_500_001, 256, 2
    case(f"balance T={T} E={E}")
    logits = torch.zeros((T, E), device="cuda")
    ends = torch.tensor([0, 1, T // 2, T - 3, T - 1], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    logits[ends] = torch.randn((len(ends), E), generator=g, device="cuda")
    ids = (torch.arange(T * k, device="cuda") % E).to(torch.int32).reshape(T, k)
    loss, counts, probs, tokens = q.moe_balance_loss(logits, ids, 1.0)
    assert torch.equal(counts[0].long(), torch.bincount(ids.flatten().long(), minlength=E))
    assert int(tokens) == T
    # nearly uniform probabilities and counts: the loss is 1 up to the five rows' part and rounding
    assert abs(float(loss) - 1) <= 1e-5
    w = torch.rand((T, k), generator=g, device="cuda")
    gw = torch.randn((T, k), generator=g, device="cuda")
    grad = q.moe_route_backward(logits, ids, topk_w=w, grad_w=gw, counts=counts, tokens=tokens, coef=1.0)
    ref, mag = _ref_gate(logits[ends], ids[ends].cpu(), w[ends].cpu(), gw[ends].cpu(), "topk")
    f = counts[0].cpu().double() * E / (k * T)
    p = _softmax64(logits[ends]).cpu()
    ref += p * (f - (p @ f)[:, None]) / T
    assert ((grad[ends].cpu().double() - ref).abs() <= (E + 24) * U * (mag + 2 * p / T) + 1e-45).all()


def test_combine_offsets_past_32_bits():
    import torch
    T, k, d = 66000, 8, 4096
    case(f"combine gradients T={T} k={k} d={d}")
    g = torch.Generator(device="cuda").manual_seed(4)
    y = torch.zeros((T * k, d), dtype=torch.float16, device="cuda")
    inv = torch.arange(T * k - 1, -1, -1, dtype=torch.int32, device="cuda")
    go = torch.zeros((T, d), dtype=torch.float16, device="cuda")
    for t in (0, T - 1):
        go[t] = torch.randn(d, generator=g, device="cuda").half()
        for j in range(k):
            y[int(inv[t * k + j])] = torch.randn(d, generator=g, device="cuda").half()
    w = torch.rand((T, k), generator=g, device="cuda")
    gw, gy = q.moe_combine_backward(go, y, inv, w)
    for t in (0, T - 1):
        rows = y[inv[t * k:(t + 1) * k].long()].double()
        ref, mag = (rows * go[t].double()).sum(dim=1), (rows * go[t].double()).abs().sum(dim=1)
        assert ((gw[t].double() - ref).abs() <= (d / 64 + 16) * U * mag).all()
        want = (w[t][:, None] * go[t].float()[None, :]).half()
        assert torch.equal(gy[inv[t * k:(t + 1) * k].long()], want)
    assert not gw[1:T - 1].any()


def test_router_calls_on_a_side_stream_give_the_same_bits():
    import torch
    logits, ids, active = _inputs(700, 60, 4, 5, masked=0.05)
    ids, w = q.moe_route_topk(logits, 4, "all", active=active)
    gw = torch.randn((700, 4), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    off = torch.tensor([0, 3, 300, 300, 690], dtype=torch.int32, device="cuda")

    def step(s=None):
        loss, counts, probs, tokens = q.moe_balance_loss(logits, ids, 0.3, active=active,
                                                         seq_offsets=off, stream=s)
        g = q.moe_route_backward(logits, ids, gate_mode="all", topk_w=w, grad_w=gw, active=active,
                                 counts=counts, tokens=tokens, coef=0.3, seq_offsets=off, stream=s)
        return loss, counts, probs, tokens, g

    case("router calls on a side stream")
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = step(s)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
