"""Cases of libq4's fused linear layer, expert routing, expert products and expert layer.

`run` computes an operator in its plain form (elementary torch operations in
32 bits, selection in 64) or, where `own` is set, through libq4's entry points
`q4_linear`, `q4_route`, `q4_route_plan`, `q4_experts` and `q4_moe`.

Formulas (w = (q - 8) d is the decoded Q4_0 weight, act one of none, relu,
gelu (tanh form) and silu):

  linear   z = x W^T + b;  y = act(z) + r, or with a gate y = act(z[:, :n/2]) z[:, n/2:] + r
  route    s = softmax(l) or sigmoid(l); the experts of the largest s + b (in the
           best groups) are chosen, ties to the lowest index; their weights are s,
           renormalised over the chosen ones and scaled
  experts  row (i, j) of token i's j-th expert e: z = x W_e^T + b_e, then as linear;
           combined: y[i] = sum_j weight[i, j] row(i, j) + r[i]
  moe      route, experts with a gate, experts combined
"""
import math

import torch

own = False

QK, BLOCK = 32, 18
_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _linear(m, n, k, dtype, act="none", gated=False, bias=False, residual=False):
    return {"op": "linear", "m": m, "n": n, "k": k, "dtype": dtype, "act": act, "gated": gated,
            "bias": bias, "residual": residual}


def _route(m, experts, topk, dtype, score="softmax", bias=False, groups=1, group_topk=1,
           group_score="max", renormalise=True, scale=1.0, masked=0.0):
    return {"op": "route", "m": m, "experts": experts, "topk": topk, "dtype": dtype, "score": score,
            "bias": bias, "groups": groups, "group_topk": group_topk, "group_score": group_score,
            "renormalise": renormalise, "scale": scale, "masked": masked}


def _experts(m, experts, topk, n, k, dtype, act="none", gated=False, bias=False, combine=False,
             residual=False):
    return {"op": "experts", "m": m, "experts": experts, "topk": topk, "n": n, "k": k,
            "dtype": dtype, "act": act, "gated": gated, "bias": bias, "combine": combine,
            "residual": residual}


def _moe(m, experts, topk, hidden, inter, dtype, score="softmax", bias=False, residual=True):
    return {"op": "moe", "m": m, "experts": experts, "topk": topk, "hidden": hidden, "inter": inter,
            "dtype": dtype, "score": score, "bias": bias, "residual": residual}


def listed():
    return [
        # One small fp32 linear, one row, with its bias: the latency of a call.
        dict(_linear(1, 512, 512, "f32", bias=True), name="linear_512_f32_m1"),
        # The fused q/k/v projection of a decoder layer, one token, with its biases.
        dict(_linear(1, 7168, 5120, "f16", bias=True), name="linear_qkv_f16_m1"),
        # The fused gate/up projection in batched decode (ten sessions), SiLU-gated.
        dict(_linear(10, 34816, 5120, "f16", act="silu", gated=True), name="linear_gate_up_f16_m10"),
        # The down projection of a 256-row prefill chunk, added to the residual stream.
        dict(_linear(256, 5120, 17408, "f16", residual=True), name="linear_down_f16_m256"),
        # The gate/up projection of a long bfloat16 prompt, SiLU-gated.
        dict(_linear(2048, 34816, 5120, "bf16", act="silu", gated=True), name="linear_gate_up_bf16_m2048"),
        # Routing of one decode step: 16 tokens, softmax scores, the chosen renormalised.
        dict(_route(16, 128, 8, "f32"), name="route_softmax_m16"),
        # Routing of a prompt: sigmoid scores, balance bias, four of eight groups.
        dict(_route(4096, 256, 8, "bf16", score="sigmoid", bias=True, groups=8, group_topk=4,
                    group_score="top2", scale=2.5), name="route_groups_m4096"),
        # The experts' gate/up products of a batched decode step.
        dict(_experts(10, 64, 6, 2816, 2048, "f16", act="silu", gated=True), name="experts_gate_up_f16_m10"),
        # The experts' down products of a prompt, combined by the routing weights.
        dict(_experts(1024, 64, 6, 2048, 1408, "bf16", combine=True, residual=True),
             name="experts_down_bf16_m1024"),
        # A whole expert layer: one token, a decode batch, a prompt.
        dict(_moe(1, 128, 8, 2048, 768, "f16"), name="moe_f16_m1"),
        dict(_moe(64, 128, 8, 2048, 768, "bf16", score="sigmoid", bias=True), name="moe_bf16_m64"),
        dict(_moe(2048, 128, 8, 2048, 1024, "bf16"), name="moe_bf16_m2048"),
    ]


def _span(rng, lo, hi):
    """An integer of lo .. hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _blocks(rng, lo, hi):
    """An input width: mostly whole pairs of 256 as model widths are, else any count of Q4_0 blocks."""
    k = _span(rng, lo, hi)
    step = rng.choice((512, 256, 256, 128, 64, 32))
    return max(step, k // step * step)


def draw(rng):
    op = rng.choice(("linear", "linear", "route", "experts", "moe"))
    half = rng.choice(("f16", "bf16"))
    if op == "linear":
        gated = rng.random() < 0.4
        m = _span(rng, 1, 2048)
        n, k = _span(rng, 256, 34816), _blocks(rng, 512, 17408)
        dtype = "f32" if rng.random() < 0.15 else half
        if dtype == "f32":
            m, n = min(m, 32), min(n, 4096)
        while m * n * k > 2048 * 34816 * 5120:
            n = n // 2 + 1
        return _linear(m, n // 2 * 2 if gated else n, k, dtype,
                       act=rng.choice(("silu", "gelu", "relu") if gated else ("none", "none", "gelu", "silu", "relu")),
                       gated=gated, bias=rng.random() < 0.5, residual=rng.random() < 0.5)
    experts = rng.choice((8, 16, 32, 60, 64, 128, 256))
    topk = min(rng.choice((1, 2, 4, 6, 8)), experts)
    if op == "route":
        groups = rng.choice((1, 1, 4))
        sigmoid = rng.random() < 0.5
        return _route(_span(rng, 1, 8192), experts, topk, rng.choice(("f32", "f16", "bf16")),
                      score="sigmoid" if sigmoid else "softmax", bias=sigmoid and rng.random() < 0.7,
                      groups=groups, group_topk=2 if groups > 1 else 1,
                      group_score="top2" if sigmoid else "max", renormalise=rng.random() < 0.7,
                      scale=rng.choice((1.0, 1.0, 2.5)), masked=rng.choice((0.0, 0.0, 0.1)))
    m = _span(rng, 1, 2048)
    if op == "experts":
        gated = rng.random() < 0.5
        n, k = _span(rng, 256, 4096), _blocks(rng, 512, 4096)
        while experts * n * k > 128 * 2048 * 2048 or m * topk * n * k > 2048 * 8 * 4096 * 1024:
            n = n // 2 + 1
        return _experts(m, experts, topk, n // 2 * 2 if gated else n, k, half,
                        act=rng.choice(("silu", "gelu")) if gated else "none", gated=gated,
                        bias=rng.random() < 0.3, combine=not gated and rng.random() < 0.7,
                        residual=rng.random() < 0.3)
    hidden, inter = _blocks(rng, 512, 4096), _blocks(rng, 256, 2048)
    while experts * hidden * inter > 128 * 2048 * 1024 or m * topk * hidden * inter > 2048 * 8 * 2048 * 1024:
        experts, m = max(8, experts // 2), m // 2 + 1
    sigmoid = rng.random() < 0.4
    return _moe(m, experts, min(topk, experts), hidden, inter, half, score="sigmoid" if sigmoid else "softmax",
                bias=sigmoid, residual=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _pack(w):
    """Q4_0 bytes of w [..., k] (fp32): [..., k / 32 * 18] uint8."""
    b = w.unflatten(-1, (-1, QK))
    at = b.abs().argmax(-1, keepdim=True)
    d = (b.gather(-1, at) / -8).half()
    q = torch.where(d == 0, torch.full_like(b, 8), b / d.float() + 8.5).trunc().clamp(0, 15).to(torch.uint8)
    codes = q[..., :16] | (q[..., 16:] << 4)
    return torch.cat((d.view(torch.uint8), codes), -1).flatten(-2)


def _weight(g, *shape):
    return _pack(torch.randn(shape, generator=g, device="cuda") * 0.02)


def _rows(g, dtype, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(_TYPES[dtype])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    m, t = c["m"], c["dtype"]
    if c["op"] == "linear":
        n, k = c["n"], c["k"]
        out = n // 2 if c["gated"] else n
        s["packed"] = _weight(g, n, k)
        s["x"] = _rows(g, t, m, k)
        s["bias"] = _rows(g, t, n, scale=0.1) if c["bias"] else None
        s["residual"] = _rows(g, t, m, out) if c["residual"] else None
        return s
    e = c["experts"]
    if c["op"] in ("route", "moe"):
        # Router logits as a trained router gives them: a spread of a few units.
        s["logits"] = _rows(g, t if c["op"] == "route" else "f32", m, e, scale=1.5)
        if c.get("masked"):
            s["logits"][torch.rand((m, e), generator=g, device="cuda") < c["masked"]] = -math.inf
        s["balance"] = torch.randn(e, generator=g, device="cuda") * 0.02 if c["bias"] else None
        if c["op"] == "route":
            return s
        s["x"] = _rows(g, t, m, c["hidden"])
        s["gate_up"] = _weight(g, e, 2 * c["inter"], c["hidden"])
        s["down"] = _weight(g, e, c["hidden"], c["inter"])
        s["residual"] = _rows(g, t, m, c["hidden"]) if c["residual"] else None
        return s
    n, k, topk = c["n"], c["k"], c["topk"]
    scores = torch.randn((m, e), generator=g, device="cuda").topk(topk, -1)
    s["ids"] = scores.indices.int()
    s["weights"] = torch.softmax(scores.values, -1) if c["combine"] else None
    s["packed"] = _weight(g, e, n, k)
    s["x"] = _rows(g, t, m * topk if c["combine"] else m, k)
    s["bias"] = _rows(g, t, e, n, scale=0.1) if c["bias"] else None
    out = n // 2 if c["gated"] else n
    s["residual"] = _rows(g, t, m if c["combine"] else m * topk, out) if c["residual"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _decode(packed):
    """fp32 weights of Q4_0 bytes [..., k / 32 * 18]."""
    b = packed.unflatten(-1, (-1, BLOCK))
    d = b[..., :2].contiguous().view(torch.float16).float()
    codes = b[..., 2:]
    q = torch.cat((codes & 15, codes >> 4), -1).float()
    return ((q - 8) * d).flatten(-2)


def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _finish(z, act, gated):
    if not gated:
        return _act(z, act)
    gate, up = z.chunk(2, -1)
    return _act(gate, act) * up


def _plain_linear(x, packed, bias, act, gated, residual):
    z = x.float() @ _decode(packed).t()
    if bias is not None:
        z = z + bias.float()
    y = _finish(z, act, gated)
    if residual is not None:
        y = y + residual.float()
    return y


def _plain_route(logits, c, balance):
    """ids (-1 where nothing is left to choose) and weights."""
    live = logits > -math.inf
    l = logits.double()
    if c["score"] == "softmax":
        p = torch.exp(l - l.masked_fill(~live, -1e300).amax(-1, keepdim=True)) * live
        score = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
    else:
        score = 1 / (1 + torch.exp(-l)) * live
    additive = balance is not None or c.get("group_score", "max") == "top2"
    key = score + (0 if balance is None else balance.double()) if additive else l
    key = key.masked_fill(~live, -math.inf)
    groups = c.get("groups", 1)
    if groups > 1:
        by = key.unflatten(-1, (groups, -1))
        if c["group_score"] == "top2":
            two = by.sort(dim=-1, descending=True).values[..., :2]
            of = (two.masked_fill(two == -math.inf, 0)).sum(-1).masked_fill(two[..., 0] == -math.inf, -math.inf)
        else:
            of = by.amax(-1)
        first = of.sort(dim=-1, descending=True, stable=True).indices[..., :c["group_topk"]]
        chosen = torch.zeros_like(of, dtype=torch.bool).scatter(-1, first, True)
        key = key.masked_fill(~chosen.repeat_interleave(key.shape[-1] // groups, -1), -math.inf)
    best = key.sort(dim=-1, descending=True, stable=True)
    ids, top = best.indices[..., :c["topk"]], best.values[..., :c["topk"]]
    w = score.gather(-1, ids).masked_fill(top == -math.inf, 0)
    if c.get("renormalise", True):
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    return ids.masked_fill(top == -math.inf, -1).int(), (w * c.get("scale", 1.0)).float()


def _plain_plan(ids, experts):
    """First place of each expert's pairs in the order by expert, and that order (-1 behind the last)."""
    flat = ids.flatten().long()
    at = torch.where(flat < 0, torch.full_like(flat, experts), flat)
    counts = torch.bincount(at, minlength=experts + 1)
    offsets = torch.cat((counts.new_zeros(1), counts[:experts].cumsum(0)))
    order = at.sort(dim=0, stable=True).indices
    live = torch.arange(order.numel(), device=order.device) < offsets[-1]
    return offsets.int(), torch.where(live, order, torch.full_like(order, -1)).int()


def _plain_experts(rows, ids, packed, bias, act, gated):
    """Row p of the result is row p of `rows` [m topk, k] through the expert ids.flatten()[p]; the reached experts alone are decoded."""
    reached, at = ids.flatten().unique(return_inverse=True)
    counts = torch.bincount(at)
    order = at.sort(dim=0, stable=True).indices
    first = counts.cumsum(0) - counts
    place = torch.arange(at.numel(), device=at.device) - first[at[order]]
    batch = rows.new_zeros((reached.numel(), int(counts.max()), rows.shape[1]))
    batch[at[order], place] = rows[order]
    reached = reached.long()
    z = torch.bmm(batch, _decode(packed[reached]).transpose(1, 2).contiguous())
    if bias is not None:
        z = z + bias[reached].float()[:, None]
    z = _finish(z, act, gated)
    out = z.new_empty((at.numel(), z.shape[-1]))
    out[order] = z[at[order], place]
    return out


def _plain(s):
    c = s["case"]
    t = _TYPES[c["dtype"]]
    if c["op"] == "linear":
        return _plain_linear(s["x"], s["packed"], s["bias"], c["act"], c["gated"], s["residual"]).to(t)
    if c["op"] == "route":
        ids, weights = _plain_route(s["logits"], c, s["balance"])
        offsets, order = _plain_plan(ids, c["experts"])
        return {"ids": ids, "weights": weights, "offsets": offsets, "order": order}
    topk = c["topk"]
    if c["op"] == "experts":
        x = s["x"].float()
        rows = x if c["combine"] else x.repeat_interleave(topk, 0)
        y = _plain_experts(rows, s["ids"], s["packed"], s["bias"], c["act"], c["gated"])
        if c["combine"]:
            y = (y.unflatten(0, (-1, topk)) * s["weights"][..., None]).sum(1)
    else:
        ids, weights = _plain_route(s["logits"], c, s["balance"])
        h = _plain_experts(s["x"].float().repeat_interleave(topk, 0), ids, s["gate_up"], None, "silu", True)
        y = _plain_experts(h, ids, s["down"], None, "none", False)
        y = (y.unflatten(0, (-1, topk)) * weights[..., None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(t)


def _own(s):
    import bit_block_quantized_q4_amd as q4
    c = s["case"]
    if c["op"] == "linear":
        return q4.q4_linear(s["x"], s["packed"], bias=s["bias"], activation=c["act"], gated=c["gated"],
                            residual=s["residual"])
    if c["op"] == "route":
        ids, weights, plan = q4.q4_route(s["logits"], c["topk"], score=c["score"], bias=s["balance"],
                                         groups=c["groups"], group_topk=c["group_topk"],
                                         group_score=c["group_score"], renormalise=c["renormalise"],
                                         scale=c["scale"])
        return {"ids": ids, "weights": weights, "offsets": plan.offsets, "order": plan.order}
    if c["op"] == "experts":
        plan = q4.q4_route_plan(s["ids"], c["experts"])
        return q4.q4_experts(s["x"], s["packed"], plan, bias=s["bias"], activation=c["act"],
                             gated=c["gated"], weights=s["weights"], residual=s["residual"])
    return q4.q4_moe(s["x"], s["logits"], s["gate_up"], s["down"], c["topk"], activation="silu",
                     score=c["score"], route_bias=s["balance"], residual=s["residual"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work

def _active(experts, pairs, topk):
    """Experts that a step's tokens reach, on average."""
    return experts * (1 - (1 - topk / experts) ** (pairs / topk))


def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    m = c["m"]
    if c["op"] == "linear":
        n, k = c["n"], c["k"]
        out = n // 2 if c["gated"] else n
        b = n * k // QK * BLOCK + size * (m * k + m * out + (n if c["bias"] else 0) + (m * out if c["residual"] else 0))
        return {"bytes": b, "flops": 2 * m * n * k}
    e, topk = c["experts"], c["topk"]
    pairs = m * topk
    if c["op"] == "route":
        return {"bytes": size * m * e + 12 * pairs + 4 * e + (4 * e if c["bias"] else 0), "flops": 10 * m * e}
    if c["op"] == "experts":
        n, k = c["n"], c["k"]
        out = n // 2 if c["gated"] else n
        rows_in, rows_out = (pairs, m) if c["combine"] else (m, pairs)
        b = _active(e, pairs, topk) * n * (k // QK * BLOCK + (size if c["bias"] else 0)) + 4 * pairs
        b += size * (rows_in * k + rows_out * out * (2 if c["residual"] else 1)) + (4 * pairs if c["combine"] else 0)
        return {"bytes": b, "flops": 2 * pairs * n * k}
    hidden, inter = c["hidden"], c["inter"]
    weights = _active(e, pairs, topk) * 3 * hidden * inter // QK * BLOCK
    return {"bytes": weights + size * m * hidden * (3 if c["residual"] else 2) + 4 * m * e,
            "flops": 6 * pairs * hidden * inter}


# ------------------------------------------------------------------ 64 bits

def _weights64(packed):
    """Decoded weights in 64 bits: element i of a block is the low nibble of byte i, element i + 16 its high nibble."""
    rows = packed.reshape(-1, BLOCK)
    d = rows[:, 0].to(torch.int32) + 256 * rows[:, 1].to(torch.int32)
    d = d.to(torch.int16).view(torch.float16).double()
    w = torch.empty((rows.shape[0], QK), dtype=torch.float64, device=packed.device)
    w[:, :16] = (rows[:, 2:] % 16).double() - 8
    w[:, 16:] = (rows[:, 2:] // 16).double() - 8
    w *= d[:, None]
    return w.view(*packed.shape[:-1], -1)


def _layer64(x, w, bias, act, gated):
    z = torch.matmul(x, w.mT)
    if bias is not None:
        z += bias.double()
    n = z.shape[-1]
    a = z[..., :n // 2] if gated else z
    if act == "silu":
        a = a * torch.sigmoid(a)
    elif act == "gelu":
        a = a / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
    elif act == "relu":
        a = a.clamp_min(0)
    return a * z[..., n // 2:] if gated else a


def _choose64(logits, c, balance):
    l = logits.double()
    s = torch.softmax(l, -1) if c["score"] == "softmax" else torch.sigmoid(l)
    s = torch.nan_to_num(s, nan=0.0)
    dead = l == -math.inf
    plain_order = balance is None and c.get("group_score", "max") == "max"
    key = l.clone() if plain_order else s + (balance.double() if balance is not None else 0.0)
    key[dead] = -math.inf
    groups = c.get("groups", 1)
    if groups > 1:
        g = key.view(key.shape[0], groups, -1)
        if c["group_score"] == "max":
            value = g.max(-1).values
        else:
            top = g.topk(min(2, g.shape[-1]), -1).values
            value = torch.where(torch.isinf(top), torch.zeros_like(top), top).sum(-1)
            value[torch.isinf(top[..., 0])] = -math.inf
        rank = torch.argsort(torch.argsort(-value, dim=-1, stable=True), dim=-1, stable=True)
        g[rank >= c["group_topk"]] = -math.inf
        key = g.reshape(key.shape)
    ids = torch.argsort(-key, dim=-1, stable=True)[:, :c["topk"]]
    none = torch.isinf(torch.gather(key, 1, ids))
    w = torch.where(none, torch.zeros_like(s[:, :1]), torch.gather(s, 1, ids))
    if c.get("renormalise", True):
        w = w / w.sum(-1, keepdim=True).clamp_min(1e-300)
    return torch.where(none, torch.full_like(ids, -1), ids), w * c.get("scale", 1.0)


def _through64(x, per_token, ids, packed, bias, act, gated):
    """Every pair's row, expert by expert."""
    flat = ids.flatten()
    out = None
    for e in flat.unique().tolist():
        if e < 0:
            continue
        at = (flat == e).nonzero().flatten()
        z = _layer64(x[at // per_token].double(), _weights64(packed[e]), None if bias is None else bias[e], act, gated)
        if out is None:
            out = z.new_zeros((flat.numel(), z.shape[-1]))
        out[at] = z
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "linear":
        y = _layer64(s["x"].double(), _weights64(s["packed"]), s["bias"], c["act"], c["gated"])
        return y if s["residual"] is None else y + s["residual"].double()
    if c["op"] == "route":
        ids, w = _choose64(s["logits"], c, s["balance"])
        return {"ids": None, "weights": w, "offsets": None, "order": None}
    topk = c["topk"]
    if c["op"] == "experts":
        y = _through64(s["x"], 1 if c["combine"] else topk, s["ids"], s["packed"], s["bias"], c["act"], c["gated"])
        w = s["weights"]
    else:
        ids, w = _choose64(s["logits"], c, s["balance"])
        h = _through64(s["x"], topk, ids, s["gate_up"], None, "silu", True)
        y = _through64(h, 1, ids, s["down"], None, "none", False)
    if w is not None:
        y = torch.einsum("mjn,mj->mn", y.view(-1, topk, y.shape[-1]), w.double())
    return y if s["residual"] is None else y + s["residual"].double()
