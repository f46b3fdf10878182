"""The experts' feed-forward network: cases, plain forms and exact results.

Between hc_mix_expert_dispatch and hc_mix_expert_combine the rows xs[R, K], sorted by expert, pass
through their experts' weights.  Expert e has rows offsets[e] .. offsets[e + 1] - 1:

    product        ys[r] = W[e(r)] xs[r]                               W[E, N, K]
    gated          h[r] = silu(g) * u with (g, u) = W[e(r)] xs[r]      W[E, 2 F, K], g the first F
    product back   dxs[r] = W[e(r)]^T dys[r], dW[e] = sum over its rows of dys[r] xs[r]^T
    gate back      (dg, du) for dh and the (g, u) that the forward pass keeps
    product q4     both products with weights of 4 bits: W = (code - 8) * scale of its group

Rows behind the last expert's (pairs that no expert took) are zero in every result.  `across`:
the weights lie as W[E, K, N], as a model that writes xs @ W keeps them.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------------------- cases


def product(tokens, top, of, width, out, dtype, gated=False, saved=False, back=False, drop=False, across=False):
    """`out` features of each row of `width`, F for a gated product; `saved`: (g, u) too, as a training step keeps it;
    `drop`: some pairs are over their expert's capacity."""
    return {"op": "product", "tokens": tokens, "top": top, "of": of, "width": width, "out": out, "type": dtype, "gated": gated, "saved": saved,
            "back": back, "drop": drop, "across": across}


def gate(rows, width, dtype):
    return {"op": "gate", "rows": rows, "width": width, "type": dtype, "back": True}


def product_q4(tokens, top, of, width, out, group, dtype, gated=False, drop=False):
    return {"op": "q4", "tokens": tokens, "top": top, "of": of, "width": width, "out": out, "group": group, "type": dtype, "gated": gated, "drop": drop}


def listed():
    named = {
        # one sequence, one new token, back from its 8 experts' inner width: a call's latency
        "product one token": product(1, 8, 128, 2048, 5120, "bf16"),
        # 16 sequences, one new token each, into the experts: bound by the weights that they name
        "gated decode": product(16, 8, 128, 5120, 2048, "bf16", gated=True),
        # a prefill chunk's rows back from the inner width
        "product prefill": product(4096, 8, 128, 2048, 5120, "bf16"),
        # the largest: the rows of a 16384-token prefill into the experts
        "gated prefill": product(16384, 8, 128, 5120, 2048, "bf16", gated=True),
        # a small fp16 mixture of odd widths, its weights written for xs @ W, with capacity drops
        "product ragged": product(1531, 3, 61, 1023, 1001, "f16", drop=True, across=True),
        # a training step's gradients of the rows and of the weights of both inner projections
        "product backward": product(4096, 4, 32, 5120, 4096, "bf16", back=True),
        # and of a small fp16 mixture of odd widths
        "product backward ragged": product(777, 2, 8, 515, 391, "f16", back=True, drop=True),
        # the gate's gradient for a training step's rows
        "gate backward": gate(32768, 2048, "bf16"),
        # an fp32 gate of an odd width
        "gate backward ragged": gate(3001, 1001, "f32"),
        # 16 new tokens into experts served with weights of 4 bits
        "q4 gated decode": product_q4(16, 8, 128, 5120, 2048, 128, "bf16", gated=True),
        # one token back from them
        "q4 one token": product_q4(1, 8, 128, 2048, 5120, 64, "f16"),
        # a dense projection (one expert) of a few tokens, an odd number of features, small groups
        "q4 dense ragged": product_q4(7, 1, 1, 5120, 20477, 32, "bf16"),
    }
    return [dict(c, name=n) for n, c in named.items()]


def _spread(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 200)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("product", "product", "gated", "back", "back", "gate", "q4", "q4"))
        dtype = rng.choice(("bf16", "bf16", "f16"))
        width, out = _spread(rng, 64, 8192), _spread(rng, 64, 8192)
        if rng.random() < 0.6:
            width, out = -(-width // 64) * 64, -(-out // 64) * 64
        of = _spread(rng, 1, 128)
        top, drop, across = rng.randint(1, min(8, of)), rng.random() < 0.3, rng.random() < 0.3
        if op == "gate":
            c = gate(_spread(rng, 1, 65536), width, rng.choice(("bf16", "f16", "f32")))
        elif op == "q4":
            group = rng.choice((32, 64, 128))
            c = product_q4(_spread(rng, 1, 64), top, of, -(-width // group) * group, out, group, dtype, rng.random() < 0.5, drop)
        else:
            gated = op == "gated"
            c = product(_spread(rng, 1, 16384), top, of, width, out, dtype, gated, gated and rng.random() < 0.5, op == "back", drop, across)
        # weights and rows no larger than the listed cases'
        if c["op"] == "gate" or (of * width * _features(c) <= 128 * 5120 * 4096 and c["tokens"] * top * max(width, out) <= 16384 * 8 * 5120):
            if _cost(c) <= most:
                return c


def _features(c):
    """Rows of one expert's weights."""
    return c["out"] * (2 if c["gated"] else 1)


# ------------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    c = dict(case, type=TYPES[case["type"]])
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T = c["type"]

    def normal(*shape, std=1.0, dtype=T):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype) * std).to(dtype)

    s = {"case": c}
    if c["op"] == "gate":
        s["dh"], s["gu"] = normal(c["rows"], c["width"], std=0.02), normal(c["rows"], 2 * c["width"])
        return s
    M, E, k, K, N = c["tokens"], c["of"], c["top"], c["width"], _features(c)
    # which experts a token takes: a few tokens' are spread evenly, among many some experts are more popular than others
    score = normal(M, E, dtype=torch.float32)
    if M * k > 4 * E:
        score = score + 0.7 * normal(E, dtype=torch.float32)
    ids = torch.topk(score, k, dim=1).indices
    if c["drop"]:
        ids = torch.where(torch.rand(M, k, generator=g, device="cuda") < 0.05, E, ids)
    counts = torch.bincount(ids.reshape(-1), minlength=E + 1)[:E]
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["most"] = int(counts.max())  # rows of one expert: the plain form pads all to this
    held = torch.arange(M * k, device="cuda") < s["offsets"][E]
    if c["op"] == "q4":
        s["xs"] = torch.where(held[:, None], normal(M * k, K), 0)
        s["codes"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = (torch.rand(E, N, K // c["group"], generator=g, device="cuda") * 0.5 + 0.75).mul_(0.2 * K ** -0.5).to(T)
        return s
    s["xs"] = torch.where(held[:, None], normal(M * k, K), 0)
    s["weight"] = normal(*((E, K, N) if c["across"] else (E, N, K)), std=K ** -0.5)
    if c["back"]:
        s["dys"] = torch.where(held[:, None], normal(M * k, N, std=0.02), 0)
    return s


# ------------------------------------------------------------------------------- one pass


def run(s):
    return _own(s, s["case"]) if own else _plain(s, s["case"])


def _own(s, c):
    from hyper_connection_mix_gb300 import experts

    if c["op"] == "gate":
        return experts.hc_mix_expert_gate_backward(s["dh"], s["gu"])
    if c["op"] == "q4":
        return experts.hc_mix_expert_product_q4(s["xs"], s["codes"], s["scales"], s["offsets"], gated=c["gated"])
    if c["back"]:
        return experts.hc_mix_expert_product_backward(s["dys"], s["xs"], s["weight"], s["offsets"], transposed=c["across"])
    if c["gated"]:
        return experts.hc_mix_expert_product_gated(s["xs"], s["weight"], s["offsets"], transposed=c["across"], want_saved=c["saved"])
    return experts.hc_mix_expert_product(s["xs"], s["weight"], s["offsets"], transposed=c["across"])


def _gated(gu):
    g, u = gu.chunk(2, -1)
    return g * torch.sigmoid(g) * u


def _places(s, R):
    """Each row's expert and its place among the expert's rows; a row behind the last has expert E."""
    at = torch.arange(R, device=s["offsets"].device, dtype=torch.int32)
    expert = torch.searchsorted(s["offsets"][1:], at, right=True)
    first = torch.where(expert < s["offsets"].numel() - 1, s["offsets"][expert], at)
    return expert, at - first


def _padded(x, s, places):
    """The rows of x as [E, most, width], zeros behind each expert's."""
    E = s["offsets"].numel() - 1
    p = torch.zeros(E + 1, max(s["most"], 1), x.shape[1], device=x.device)
    p[places] = x.float()
    return p[:E]


def _rows(p, places):
    """The padded [E, most, width] as rows again, zeros where no expert is."""
    expert, place = places
    rows = p[expert.clamp(max=p.shape[0] - 1), place]
    return torch.where(expert[:, None] < p.shape[0], rows, 0)


def _plain(s, c):
    T = c["type"]
    if c["op"] == "gate":
        dh = s["dh"].float()
        g, u = s["gu"].float().chunk(2, 1)
        q = torch.sigmoid(g)
        return torch.cat([dh * u * q * (1 + g * (1 - q)), dh * g * q], 1).to(T)
    xs = s["xs"]
    places = _places(s, xs.shape[0])
    if c["op"] == "q4":
        q = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).flatten(2)
        w = (q.float() - 8).unflatten(2, (-1, c["group"])) * s["scales"].float()[..., None]
        gu = _rows(torch.bmm(_padded(xs, s, places), w.flatten(2).mT), places)
        return (_gated(gu) if c["gated"] else gu).to(T)
    w = s["weight"].float()
    w = w.mT if c["across"] else w  # [E, N, K]
    if c["back"]:
        dys = _padded(s["dys"], s, places)
        dw = torch.bmm(dys.mT, _padded(xs, s, places)).to(T)
        return _rows(torch.bmm(dys, w), places).to(T), dw.mT.contiguous() if c["across"] else dw
    ys = _rows(torch.bmm(_padded(xs, s, places), w.mT), places)
    if c["gated"]:
        return (_gated(ys).to(T), ys.to(T)) if c["saved"] else _gated(ys).to(T)
    return ys.to(T)


# ------------------------------------------------------------------------------------- work


def work(case):
    c = case
    n = BYTES[c["type"]]
    if c["op"] == "gate":  # dh, g, u -> dg, du
        return {"bytes": 5 * c["rows"] * c["width"] * n, "flops": 12 * c["rows"] * c["width"]}
    M, E, k, K, N = c["tokens"], c["of"], c["top"], c["width"], _features(c)
    rows = M * k * (0.95 if c["drop"] else 1)
    used = E * (1 - (1 - k / E) ** M)  # experts that have a row, on average
    flops = 2 * rows * N * K
    if c["op"] == "q4":
        weights = used * N * (K / 2 + K / c["group"] * n)
        return {"bytes": round(weights + M * k * (K + c["out"]) * n), "flops": round(flops)}
    if c["back"]:  # dys, xs, W -> dxs, dW, which has all experts' places
        return {"bytes": round((used + E) * N * K * n + M * k * (2 * K + N) * n), "flops": round(2 * flops)}
    return {"bytes": round(used * N * K * n + M * k * (K + c["out"] + (N if c["saved"] else 0)) * n), "flops": round(flops)}


# ------------------------------------------------------------------------------------ exact


def exact(case, seed):
    """The same results in 64 bits, expert by expert; gradients by differentiating the forward definition."""
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "gate":
        gu = s["gu"].double().requires_grad_()
        F = c["width"]
        h = gu[:, :F] / (1 + torch.exp(-gu[:, :F])) * gu[:, F:]
        return torch.autograd.grad(h, gu, s["dh"].double())[0]
    at = s["offsets"].tolist()
    R, E, N = s["xs"].shape[0], c["of"], _features(c)

    def zeros(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device="cuda")

    if c.get("back"):
        dxs = zeros(R, c["width"])
        dw = torch.zeros_like(s["weight"], dtype=torch.float64)
        for e in range(E):
            r = slice(at[e], at[e + 1])
            x, w = s["xs"][r].double().requires_grad_(), s["weight"][e].double().requires_grad_()
            y = x @ w if c["across"] else x @ w.t()
            dxs[r], dw[e] = torch.autograd.grad(y, (x, w), s["dys"][r].double())
        return dxs, dw
    ys = zeros(R, N)
    for e in range(E):
        r = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        if c["op"] == "q4":
            b = s["codes"][e].long()
            w = zeros(N, c["width"])
            w[:, 0::2], w[:, 1::2] = (b % 16 - 8).double(), (b // 16 - 8).double()
            w = w * s["scales"][e].double().repeat_interleave(c["group"], 1)
        else:
            w = s["weight"][e].double()
            w = w.t() if c["across"] else w
        ys[r] = s["xs"][r].double() @ w.t()
    if not c["gated"]:
        return ys
    F = c["out"]
    h = ys[:, :F] / (1 + torch.exp(-ys[:, :F])) * ys[:, F:]
    return (h, ys) if c.get("saved") else h
