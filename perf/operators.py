"""The operators around the MoE layer, case by case: what each computes in plain torch operations,
the calls that a program makes of this framework for the same result, and what each has to move
and compute.

  linear            out = act(a w^T + bias) + residual       the products beside the experts
  linear_backward   gradients of a, w and bias
  balance           the router's balance loss, its counts and mean probabilities, and the loss's
                    gradient with respect to the router logits
  route_backward    gradient of the router logits through the gate weights and the balance loss
  combine_backward  gradients of the gate weights and of the expert rows
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
LAYOUT = {"linear": 1, "linear_backward": 2, "balance": 3, "route_backward": 4,
          "combine_backward": 5}


def listed():
    return [
        # one decode token's router logits (hidden 4096, 16 experts), fp32 for the gating
        _linear("router_token", M=1, K=4096, N=16, dtype="fp16", out="fp32"),
        # a verify step's output projection (16 drafted tokens and one) added to the residual
        _linear("verify_projection", M=17, K=2048, N=2048, dtype="bf16", residual=True),
        # the dense FFN layer between two MoE layers of the MT encoder: 96 sentences x 40 tokens
        _linear("mt_ffn_up", M=3840, K=1024, N=4096, dtype="fp16", act="relu", bias=True),
        # a training forward that keeps the activation's argument, at the widest expert's size
        _linear("wide_ffn_train", M=8192, K=4096, N=6400, dtype="bf16", act="gelu", bias=True,
                residual=True, preact=True),
        # the router's own gradient: fp32 logit gradients, a long and narrow product
        _linear_backward("router_back", M=8192, K=4096, N=16, dtype="bf16", grad="fp32"),
        # the MT encoder's FFN layer backwards, with a ragged number of tokens
        _linear_backward("mt_ffn_up_back", M=3777, K=1024, N=4096, dtype="fp16", act="relu"),
        # one prompt batch of the 60-expert layer
        _balance("balance_prompts", T=544, E=60, k=4, S=1),
        # a training batch of packed sequences, some of their tokens padding
        _balance("balance_packed", T=65531, E=64, k=6, S=48, padded=True),
        _route_backward("gate_prompts", T=544, E=60, k=4, S=1, gate="topk"),
        _route_backward("gate_packed", T=65531, E=64, k=6, S=48, gate="all", padded=True),
        # a verify step's gate weights
        _combine_backward("combine_verify", T=17, d=2048, k=4, E=60),
        # a long batch of the widest layer, its gate weights and its expert rows
        _combine_backward("combine_long", T=8192, d=4096, k=2, E=16),
    ]


def _linear(name, M, K, N, dtype, out=None, act="none", bias=False, residual=False, preact=False):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "dtype": dtype,
            "out": out or dtype, "act": act, "bias": bias, "residual": residual, "preact": preact}


def _linear_backward(name, M, K, N, dtype, grad=None, act="none"):
    return {"name": name, "op": "linear_backward", "M": M, "K": K, "N": N, "dtype": dtype,
            "grad": grad or dtype, "act": act}


def _balance(name, T, E, k, S, padded=False):
    return {"name": name, "op": "balance", "T": T, "E": E, "k": k, "S": S, "padded": padded}


def _route_backward(name, T, E, k, S, gate, padded=False):
    return {"name": name, "op": "route_backward", "T": T, "E": E, "k": k, "S": S, "gate": gate,
            "padded": padded}


def _combine_backward(name, T, d, k, E):
    return {"name": name, "op": "combine_backward", "T": T, "d": d, "k": k, "E": E}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(sorted(LAYOUT))
    if op in ("linear", "linear_backward"):
        # widths are mostly multiples of 8, now and then of nothing; a product that costs no
        # more than the widest listed one (its gradients are two products)
        limit = 2.0 * 8192 * 4096 * 6400 / (1 if op == "linear" else 2)
        M = _log_int(rng, 1, 8192)
        step = rng.choice((8, 8, 8, 1))
        K = step * _log_int(rng, 64 // step, 6400 // step)
        N = step * _log_int(rng, 16 // step, 6400 // step)
        while 2.0 * M * K * N > limit:
            M = max(1, M // 2)
        dtype = rng.choice(("fp16", "bf16"))
        act = rng.choice(("none", "relu", "silu", "gelu"))
        if op == "linear":
            return _drop_name(_linear("", M, K, N, dtype, out=rng.choice((dtype, dtype, "fp32")),
                                      act=act, bias=rng.random() < 0.5,
                                      residual=rng.random() < 0.5, preact=rng.random() < 0.3))
        return _drop_name(_linear_backward("", M, K, N, dtype, act=act,
                                           grad=rng.choice((dtype, dtype, "fp32"))))
    if op == "combine_backward":
        E = rng.randint(8, 256)
        return _drop_name(_combine_backward("", T=_log_int(rng, 1, 8192), E=E, k=rng.randint(1, 2),
                                            d=8 * _log_int(rng, 16, 512)))
    T, E, k = _log_int(rng, 1, 65536), rng.randint(8, 64), rng.randint(1, 6)
    S = rng.choice((1, _log_int(rng, 1, 48)))
    padded = rng.random() < 0.5
    if op == "balance":
        return _drop_name(_balance("", T, E, k, S, padded))
    return _drop_name(_route_backward("", T, E, k, S, rng.choice(("topk", "all")), padded))


def _drop_name(case):
    del case["name"]
    return case


# ------------------------------------------------------------------------------ inputs
def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + LAYOUT[case["op"]])
    return g


def _normal(g, shape, scale, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _routing(case, g):
    """Router logits with a per-expert popularity, the chosen experts and their gate weights."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = _normal(g, (T, E), 1.0, torch.float32) + _normal(g, (1, E), 0.7, torch.float32)
    ids = logits.topk(k, dim=1).indices.to(torch.int32)
    return logits, ids


def _segments(case, g, state):
    """Ragged sequences that tile the batch (some may be empty), and the tokens that are padding."""
    T, S = case["T"], case["S"]
    state["offsets"] = None
    if S > 1:
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
        ends = torch.tensor([0, T], device="cuda")
        state["offsets"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
    state["active"] = None
    if case["padded"]:
        state["active"] = (torch.rand(T, generator=g, device="cuda") < 0.9).to(torch.uint8)
        state["ids"][state["active"] == 0] = -1


def prepare(case, seed):
    g, op = _generator(case, seed), case["op"]
    s = {"case": case}
    if op in ("linear", "linear_backward"):
        M, K, N, dt = case["M"], case["K"], case["N"], DTYPES[case["dtype"]]
        s["a"] = _normal(g, (M, K), 1.0, dt)
        s["w"] = _normal(g, (N, K), K ** -0.5, dt)
        if op == "linear":
            s["bias"] = _normal(g, (N,), 0.2, dt) if case["bias"] else None
            s["residual"] = _normal(g, (M, N), 1.0, dt) if case["residual"] else None
        else:
            s["grad"] = _normal(g, (M, N), 0.05, DTYPES[case["grad"]])
            s["preact"] = _normal(g, (M, N), 1.0, dt) if case["act"] != "none" else None
    elif op == "balance":
        s["logits"], s["ids"] = _routing(case, g)
        _segments(case, g, s)
        s["coef"] = 0.01
        s["grad_loss"] = torch.full((1,), 100.0, device="cuda")
    elif op == "route_backward":
        s["logits"], s["ids"] = _routing(case, g)
        logits, ids = s["logits"], s["ids"].long()
        p = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        chosen = p.gather(1, ids)
        s["w"] = chosen / (chosen if case["gate"] == "topk" else p).sum(dim=1, keepdim=True)
        _segments(case, g, s)
        if s["active"] is not None:
            s["w"] = torch.where(s["active"][:, None] != 0, s["w"], torch.zeros_like(s["w"]))
        s["grad_w"] = _normal(g, s["w"].shape, 1.0, torch.float32)
        s["coef"] = 0.01
        s["counts"], s["tokens"] = _counted(s, case)
        s["grad_loss"] = torch.full((1,), 100.0, device="cuda")
    else:
        T, d, k, E = case["T"], case["d"], case["k"], case["E"]
        ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.reshape(-1)
        order = ids.sort(stable=True).indices          # rows sorted by expert, as the GEMM's are
        inv = torch.empty(T * k, dtype=torch.int32, device="cuda")
        inv[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
        s["inv"] = inv
        s["y"] = _normal(g, (T * k, d), 0.5, torch.float16)
        s["w"] = torch.rand((T, k), generator=g, device="cuda") + 0.05
        s["w"] /= s["w"].sum(dim=1, keepdim=True)
        s["grad"] = _normal(g, (T, d), 0.05, torch.float16)
    return s


# ------------------------------------------------------------------------------ plain forms
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    phi = torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * phi


def _segment_of(s, case):
    """(sequence of every token, or S where it takes no part; number of sequences)."""
    T, S = case["T"], case["S"]
    at = torch.arange(T, device="cuda")
    if s["offsets"] is None:
        seg = torch.zeros_like(at)
    else:
        seg = (torch.searchsorted(s["offsets"].long(), at, right=True) - 1)
    if s["active"] is not None:
        seg = torch.where(s["active"] != 0, seg, torch.full_like(seg, S))
    return seg, S


def _counted(s, case):
    """Routed slots per sequence and expert, and active tokens per sequence (int32)."""
    seg, S = _segment_of(s, case)
    E, k = case["E"], case["k"]
    ids = s["ids"].long()
    slot = torch.where(ids >= 0, seg[:, None] * E + ids, torch.full_like(ids, S * E)).reshape(-1)
    counts = torch.bincount(slot.clamp(max=S * E), minlength=S * E + 1)[:S * E].reshape(S, E)
    tokens = torch.bincount(seg, minlength=S + 1)[:S]
    return counts.to(torch.int32), tokens.to(torch.int32)


def _probabilities(logits):
    e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _balance_slope(s, case, p, counts, tokens):
    """Gradient of the balance loss with respect to the router logits."""
    E, k = case["E"], case["k"]
    seg, S = _segment_of(s, case)
    n = torch.cat([tokens, tokens.new_ones(1)]).clamp(min=1).float()[seg][:, None]
    f = torch.cat([counts, counts.new_zeros(1, E)]).float()[seg] * E / (k * n)
    used = (tokens > 0).sum().clamp(min=1)
    grad = (s["grad_loss"] * s["coef"] / used / n) * p * (f - (f * p).sum(dim=1, keepdim=True))
    return torch.where((seg < S)[:, None], grad, torch.zeros_like(grad))


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "linear":
        dt = DTYPES[case["dtype"]]
        z = s["a"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        out = _act(z, case["act"])
        if s["residual"] is not None:
            out = out + s["residual"].float()
        out = out.to(DTYPES[case["out"]])
        return (out, z.to(dt)) if case["preact"] else out
    if op == "linear_backward":
        dt = DTYPES[case["dtype"]]
        dz = s["grad"].float()
        if s["preact"] is not None:
            dz = dz * _act_slope(s["preact"].float(), case["act"])
        return ((dz @ s["w"].float()).to(dt), (dz.t() @ s["a"].float()).to(dt),
                dz.sum(dim=0).to(dt))
    if op == "balance":
        E, k = case["E"], case["k"]
        counts, tokens = _counted(s, case)
        seg, S = _segment_of(s, case)
        p = _probabilities(s["logits"])
        probs = torch.zeros((S + 1, E), device="cuda").index_add_(0, seg, p)[:S]
        n = tokens.clamp(min=1).float()[:, None]
        probs = probs / n
        f = counts.float() * E / (k * n)
        used = (tokens > 0).sum().clamp(min=1)
        loss = s["coef"] * (f * probs).sum() / used
        return loss.reshape(1), counts, probs, tokens, _balance_slope(s, case, p, counts, tokens)
    if op == "route_backward":
        p = _probabilities(s["logits"])
        ids = s["ids"].long()
        routed = ids >= 0
        gw = torch.where(routed, s["grad_w"] * s["w"], torch.zeros_like(s["w"]))
        total = gw.sum(dim=1, keepdim=True)
        away = gw - s["w"] * total if case["gate"] == "topk" else gw
        grad = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0), away * routed)
        if case["gate"] == "all":
            grad = grad - p * total
        return grad + _balance_slope(s, case, p, s["counts"], s["tokens"])
    T, k = s["w"].shape
    g, inv = s["grad"].float(), s["inv"].long()
    rows = s["y"].float()[inv].reshape(T, k, -1)
    grad_w = (rows * g[:, None, :]).sum(dim=2)
    grad_y = torch.empty_like(s["y"])
    grad_y[inv] = (s["w"][:, :, None] * g[:, None, :]).reshape(T * k, -1).to(torch.float16)
    return grad_w, grad_y


# ------------------------------------------------------------------------------ the calls
def _run_own(s):
    import quantized_expert_layer_amd as q

    case = s["case"]
    op = case["op"]
    if op == "linear":
        z = torch.empty((case["M"], case["N"]), dtype=s["a"].dtype, device="cuda") \
            if case["preact"] else None
        out = q.moe_linear(s["a"], s["w"], bias=s["bias"], act=case["act"],
                           residual=s["residual"], out_dtype=DTYPES[case["out"]], preact=z)
        return (out, z) if case["preact"] else out
    if op == "linear_backward":
        return q.moe_linear_backward(s["grad"], s["a"], s["w"], act=case["act"],
                                     preact=s["preact"])
    if op == "balance":
        loss, counts, probs, tokens = q.moe_balance_loss(
            s["logits"], s["ids"], s["coef"], active=s["active"], seq_offsets=s["offsets"])
        grad = q.moe_route_backward(s["logits"], s["ids"], active=s["active"], counts=counts,
                                    tokens=tokens, coef=s["coef"], grad_loss=s["grad_loss"],
                                    seq_offsets=s["offsets"])
        return loss, counts, probs, tokens, grad
    if op == "route_backward":
        return q.moe_route_backward(s["logits"], s["ids"], gate_mode=case["gate"],
                                    topk_w=s["w"], grad_w=s["grad_w"], active=s["active"],
                                    counts=s["counts"], tokens=s["tokens"], coef=s["coef"],
                                    grad_loss=s["grad_loss"], seq_offsets=s["offsets"])
    return q.moe_combine_backward(s["grad"], s["y"], s["inv"], s["w"])


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------------------------------ what it takes
def work(case):
    op = case["op"]
    if op in ("linear", "linear_backward"):
        M, K, N = case["M"], case["K"], case["N"]
        if op == "linear":
            size = 4 if case["out"] == "fp32" else 2
            moved = 2 * (M * K + N * K) + size * M * N
            moved += 2 * N * case["bias"] + 2 * M * N * (case["residual"] + case["preact"])
            return {"bytes": moved, "flops": 2 * M * N * K}
        size = 4 if case["grad"] == "fp32" else 2
        moved = 2 * (2 * M * K + 2 * N * K + N) + M * N * (size + 2 * (case["act"] != "none"))
        return {"bytes": moved, "flops": 4 * M * N * K}
    if op == "combine_backward":
        T, d, k = case["T"], case["d"], case["k"]
        return {"bytes": 2 * T * d * (1 + 2 * k) + 12 * T * k, "flops": 3 * T * d * k}
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    if op == "balance":
        return {"bytes": 4 * T * (2 * E + k) + T * case["padded"] + 8 * S * E,
                "flops": 10 * T * E}
    return {"bytes": 4 * T * (2 * E + 3 * k) + T * case["padded"] + 4 * S * E, "flops": 10 * T * E}


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        z = torch.mm(s["a"].double(), s["w"].double().transpose(0, 1).contiguous())
        if s["bias"] is not None:
            z += s["bias"].double()
        h = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0),
             "silu": lambda v: v * torch.sigmoid(v),
             "gelu": lambda v: v * torch.special.ndtr(v)}[case["act"]](z)
        if s["residual"] is not None:
            h = h + s["residual"].double()
        return (h, z) if case["preact"] else h
    if op == "linear_backward":
        dz = s["grad"].double()
        if s["preact"] is not None:
            v = s["preact"].double()
            if case["act"] == "relu":
                dz = dz.masked_fill(v <= 0, 0.0)
            elif case["act"] == "silu":
                dz = dz * (torch.sigmoid(v) + v * torch.sigmoid(v) * torch.sigmoid(-v))
            else:
                dz = dz * (torch.special.ndtr(v)
                           + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi))
        return (torch.mm(dz, s["w"].double()), torch.mm(dz.t().contiguous(), s["a"].double()),
                dz.sum(dim=0))
    if op == "combine_backward":
        T, k = s["w"].shape
        g = s["grad"].double().repeat_interleave(k, dim=0)
        at = s["inv"].long()
        grad_w = torch.mul(s["y"].double()[at], g).sum(dim=1).view(T, k)
        back = torch.argsort(at)
        grad_y = (g * s["w"].double().view(-1, 1))[back]
        return grad_w, grad_y
    # sequences one after the other, straight from the definition
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    cuts = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    live = torch.ones(T, dtype=torch.bool, device="cuda") if s["active"] is None \
        else s["active"].bool()
    soft = torch.softmax(s["logits"].double(), dim=1)
    counts = torch.zeros((S, E), dtype=torch.int32, device="cuda")
    tokens = torch.zeros(S, dtype=torch.int32, device="cuda")
    probs = torch.zeros((S, E), dtype=torch.float64, device="cuda")
    grad = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    terms = []
    for i, (lo, hi) in enumerate(zip(cuts[:-1], cuts[1:])):
        rows = torch.arange(lo, hi, device="cuda")[live[lo:hi]]
        if not len(rows):
            continue
        tokens[i] = len(rows)
        chosen = s["ids"][rows].flatten()
        counts[i] = torch.bincount(chosen[chosen >= 0].long(), minlength=E).to(torch.int32)
        probs[i] = soft[rows].mean(dim=0)
        share = counts[i].double() * E / (k * len(rows))
        terms.append((share * probs[i]).sum())
        p = soft[rows]
        pull = share[None, :] - (p @ share)[:, None]
        grad[rows] = p * pull * (float(s["grad_loss"]) * s["coef"] / len(rows))
    grad /= max(1, len(terms))
    if op == "balance":
        loss = s["coef"] * torch.stack(terms).mean() if terms else torch.zeros((), device="cuda",
                                                                               dtype=torch.float64)
        return loss.reshape(1), counts, probs, tokens, grad
    rows = torch.nonzero(live).flatten()
    ids, w, gw = s["ids"][rows].long(), s["w"][rows].double(), s["grad_w"][rows].double()
    mean = (w * gw).sum(dim=1, keepdim=True)
    if case["gate"] == "topk":
        gate = torch.zeros((len(rows), E), dtype=torch.float64, device="cuda")
        gate.scatter_(1, ids, w * (gw - mean))
    else:
        gate = torch.zeros((len(rows), E), dtype=torch.float64, device="cuda")
        gate.scatter_(1, ids, w * gw)
        gate -= soft[rows] * mean
    grad[rows] += gate
    return grad
