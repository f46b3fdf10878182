"""Operators around a hyper-connection sublayer: cases, plain forms and exact results.

A layer of the hyper-connection forward keeps four residual streams x[M, 4 * D].  Around each
sublayer (attention, or a mixture of experts) it runs

    collapse   h = sum_i pre[i] * x_i, then y = layer norm of h           (the sublayer's input)
    dispatch   the tokens' rows sorted by expert                          (experts only)
    combine    the experts' rows back at their tokens, weighted and added (experts only)
    expand     x'_i = post[i] * y + sum_j comb[i][j] * x_j                (the sublayer's output)

with pre, post and comb as hc_mix_fused gives them, and `norm`, the layer norm on its own, where
there are no streams.  Each is measured forward and backward.  The backward cases start from what
the forward pass leaves (statistics, slots), as a training step's do.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
HC = 4
EPS = 1e-5


# ------------------------------------------------------------------------------------- cases


def norm(rows, width, dtype, back=False, wide=True):
    """`wide`: fp32 weight and bias; else of x's type."""
    return {"op": "norm", "rows": rows, "width": width, "type": dtype, "back": back, "wide": wide}


def collapse(rows, width, dtype, back=False, saved=False):
    """`saved`: also what a training step keeps (h, mean, rstd).  `width` is one stream's."""
    return {"op": "collapse", "rows": rows, "width": width, "type": dtype, "back": back, "saved": saved}


def expand(rows, width, dtype, back=False):
    return {"op": "expand", "rows": rows, "width": width, "type": dtype, "back": back}


def experts(op, tokens, top, of, width, dtype, back=False, drop=False, ids="int64"):
    """`top` experts of `of` for each token; `drop`: some pairs are over their expert's capacity (id -1)."""
    return {"op": op, "rows": tokens, "top": top, "of": of, "width": width, "type": dtype, "back": back, "drop": drop, "ids": ids}


def listed():
    named = {
        # 16 sequences, one new token each: a call's latency
        "norm decode": norm(16, 5120, "bf16"),
        # a training step of 4096 rows: dx, and the weight's and bias's gradient over all rows
        "norm backward": norm(4096, 5120, "bf16", back=True),
        # an fp32 model of an odd width, whose rows start at every alignment
        "norm ragged": norm(3001, 2051, "f32"),
        # the input side of one sublayer of the 43-layer forward at 16384 rows
        "collapse prefill": collapse(16384, 5120, "bf16"),
        # its gradient in a training step, added to the one that came through the streams
        "collapse backward": collapse(4096, 5120, "bf16", back=True),
        # the output side for one new token of 16 sequences
        "expand decode": expand(16, 5120, "bf16"),
        # the output side of one sublayer of the 43-layer forward: the largest call
        "expand prefill": expand(16384, 5120, "bf16"),
        # its gradient in a training step: dx, dy, dpost, dcomb
        "expand backward": expand(4096, 5120, "bf16", back=True),
        # 16 tokens to 8 of 128 experts each: sort and copy, latency
        "dispatch decode": experts("dispatch", 16, 8, 128, 5120, "bf16"),
        # a prefill chunk's tokens to their experts
        "dispatch prefill": experts("dispatch", 4096, 8, 128, 5120, "bf16"),
        # and back
        "combine prefill": experts("combine", 4096, 8, 128, 5120, "bf16"),
        # a small fp16 mixture in training: odd everywhere, capacity drops
        "combine backward ragged": experts("combine", 1531, 3, 61, 1023, "f16", back=True, drop=True, ids="int32"),
    }
    return [dict(c, name=n) for n, c in named.items()]


def _spread(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(("norm", "collapse", "expand", "dispatch", "combine"))
        rows, width = _spread(rng, 1, 16384), _spread(rng, 64, 20480 if op == "norm" else 8192)
        if rng.random() < 0.6:
            width = -(-width // 64) * 64
        dtype, back = rng.choice(("bf16", "bf16", "f16", "f32")), rng.random() < 0.5
        if op == "norm":
            c = norm(rows, width, dtype, back, wide=rng.random() < 0.5)
        elif op == "collapse":
            c = collapse(rows, width, dtype, back, saved=not back and rng.random() < 0.5)
        elif op == "expand":
            c = expand(rows, width, dtype, back)
        else:
            of = _spread(rng, 8, 512)
            c = experts(op, rows, rng.randint(1, 8), of, width, dtype, back, rng.random() < 0.3, rng.choice(("int32", "int64")))
        if work(c)["bytes"] <= most:
            return c


# ------------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    c = dict(case, type=TYPES[case["type"]])
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    M, D, T = c["rows"], c["width"], c["type"]

    def normal(*shape, std=1.0, mean=0.0, dtype=T):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": c}
    if c["op"] == "norm" or (c["op"] == "collapse" and not c["back"]):
        at = torch.float32 if c.get("wide", True) else T
        s["weight"], s["bias"] = normal(D, std=0.2, mean=1.0, dtype=at), normal(D, std=0.1, dtype=at)
    if c["op"] == "norm":
        s["x"] = normal(M, D, mean=0.1)
        s["x"][:, :: 97] *= 20  # outlier channels
        if c["back"]:
            s["dy"] = normal(M, D, std=0.02)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt(x.sub_(s["mean"][:, None]).square_().mean(1) + EPS)
    elif c["op"] in ("collapse", "expand"):
        s["x"] = normal(M, HC * D)
        s["x"][:, :: 97] *= 20
        if c["op"] == "collapse":
            s["pre"] = torch.sigmoid(normal(M, HC, dtype=torch.float32))
            if c["back"]:
                s["dh"], s["dx_add"] = normal(M, D, std=0.02), normal(M, HC * D, std=0.02)
        else:
            s["y"] = normal(M, D)
            s["post"] = 2 * torch.sigmoid(normal(M, HC, dtype=torch.float32))
            comb = torch.exp(normal(M, HC, HC, dtype=torch.float32))
            for _ in range(20):
                comb = comb / comb.sum(2, keepdim=True)
                comb = comb / comb.sum(1, keepdim=True)
            s["comb"] = comb
            if c["back"]:
                s["dout"] = normal(M, HC * D, std=0.02)
    else:
        E, k = c["of"], min(c["top"], c["of"])
        # some experts are more popular than others
        score = normal(M, E, dtype=torch.float32) + 0.7 * normal(E, dtype=torch.float32)
        best = torch.topk(score, k, dim=1)
        s["weights"] = torch.softmax(best.values, 1)
        s["ids"] = best.indices.to(torch.int32 if c["ids"] == "int32" else torch.int64)
        if c["drop"]:
            s["ids"][uniform(M, k) < 0.05] = -1
        if c["op"] == "dispatch" and not c["back"]:
            s["x"] = normal(M, D)
        else:
            s["offsets"], s["slots"], _ = _sort(s["ids"], E)
            if c["op"] == "dispatch":
                s["dxs"] = normal(M * k, D, std=0.02)
            else:
                s["ys"] = normal(M * k, D)
                if c["back"]:
                    s["dy"] = normal(M, D, std=0.02)
    return s


# ------------------------------------------------------------------------------- one pass


def run(s):
    c = s["case"]
    kind = c["op"] + (" back" if c["back"] else "")
    return _own(kind, s, c) if own else _plain(kind, s, c)


def _own(kind, s, c):
    from hyper_connection_mix_gb300 import sublayer as sub

    if kind == "norm":
        return sub.hc_mix_layer_norm(s["x"], s["weight"], s["bias"], EPS, want_stats=True)
    if kind == "norm back":
        return sub.hc_mix_layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
    if kind == "collapse":
        return sub.hc_mix_collapse_norm(s["x"], s["pre"], s["weight"], s["bias"], EPS, want_saved=c["saved"])
    if kind == "collapse back":
        return sub.hc_mix_collapse_backward(s["dh"], s["x"], s["pre"], dx_add=s["dx_add"])
    if kind == "expand":
        return sub.hc_mix_expand(s["x"], s["y"], s["post"], s["comb"])
    if kind == "expand back":
        return sub.hc_mix_expand_backward(s["dout"], s["x"], s["y"], s["post"], s["comb"])
    if kind == "dispatch":
        offsets, slots, source = sub.hc_mix_expert_sort(s["ids"], c["of"])
        return offsets, slots, source, sub.hc_mix_expert_dispatch(s["x"], slots, offsets)
    if kind == "dispatch back":
        return sub.hc_mix_expert_combine(s["dxs"], s["slots"])
    if kind == "combine":
        return sub.hc_mix_expert_combine(s["ys"], s["slots"], s["weights"])
    return sub.hc_mix_expert_combine_backward(s["dy"], s["ys"], s["slots"], s["offsets"], s["weights"])


def _streams(t):
    return t.float().view(t.shape[0], HC, -1)


def _normed(h, weight, bias):
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(1) + EPS)
    return d * rstd[:, None] * weight.float() + bias.float(), mean, rstd


def _sort(ids, E):
    """offsets[E + 1]; slots: each (token, choice) pair's row, -1 where it has no expert; source: each row's pair."""
    k, flat = ids.shape[1], ids.reshape(-1)
    valid = (flat >= 0) & (flat < E)
    ordered, order = torch.sort(torch.where(valid, flat, E), stable=True)
    offsets = torch.searchsorted(ordered, torch.arange(E + 1, device=ids.device, dtype=ids.dtype)).to(torch.int32)
    place = torch.arange(flat.numel(), device=ids.device, dtype=torch.int32)
    slots = torch.empty_like(place)
    slots[order] = place
    source = torch.where(place < offsets[E], order.to(torch.int32), -1)
    return offsets, torch.where(valid, slots, -1).view(-1, k), source


def _plain(kind, s, c):
    T = c["type"]
    if kind == "norm":
        y, mean, rstd = _normed(s["x"].float(), s["weight"], s["bias"])
        return y.to(T), mean, rstd
    if kind == "norm back":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        dyw = dy * s["weight"].float()
        dx = rstd * (dyw - dyw.mean(1, keepdim=True) - xhat * (dyw * xhat).mean(1, keepdim=True))
        return dx.to(T), (dy * xhat).sum(0), dy.sum(0)
    if kind == "collapse":
        h = (s["pre"][:, :, None] * _streams(s["x"])).sum(1)
        y, mean, rstd = _normed(h, s["weight"], s["bias"])
        return (y.to(T), h.to(T), mean, rstd) if c["saved"] else y.to(T)
    if kind == "collapse back":
        dh = s["dh"].float()[:, None, :]
        dx = s["pre"][:, :, None] * dh + _streams(s["dx_add"])
        return dx.to(T).view_as(s["x"]), (dh * _streams(s["x"])).sum(2)
    if kind == "expand":
        out = torch.matmul(s["comb"], _streams(s["x"])) + s["post"][:, :, None] * s["y"].float()[:, None, :]
        return out.to(T).view_as(s["x"])
    if kind == "expand back":
        dout, x, y = _streams(s["dout"]), _streams(s["x"]), s["y"].float()[:, None, :]
        dx = torch.matmul(s["comb"].transpose(1, 2), dout)
        dy = (s["post"][:, :, None] * dout).sum(1)
        return dx.to(T).view_as(s["x"]), dy.to(T), (dout * y).sum(2), torch.matmul(dout, x.transpose(1, 2))
    if kind == "dispatch":
        offsets, slots, source = _sort(s["ids"], c["of"])
        rows = s["x"][source.clamp(min=0) // slots.shape[1]]
        return offsets, slots, source, torch.where(source[:, None] >= 0, rows, 0)
    held = s["slots"] >= 0
    at = s["slots"].clamp(min=0)
    if kind == "dispatch back":
        return (s["dxs"].float()[at] * held[:, :, None]).sum(1).to(T)
    weights = torch.where(held, s["weights"], 0)[:, :, None]
    if kind == "combine":
        return (s["ys"].float()[at] * weights).sum(1).to(T)
    dy = s["dy"].float()[:, None, :]
    dys = torch.zeros_like(s["ys"])
    dys[at[held]] = (weights * dy)[held].to(T)
    return dys, torch.where(held, (s["ys"].float()[at] * dy).sum(2), 0)


# ------------------------------------------------------------------------------------- work


def work(case):
    c = case
    M, D, n = c["rows"], c["width"], BYTES[c["type"]]
    e = M * D  # elements of one stream
    if c["op"] == "norm":
        par = D * (4 if c["wide"] else n)
        return {"bytes": 3 * e * n + 8 * M + par + 8 * D, "flops": 14 * e} if c["back"] else {"bytes": 2 * e * n + 8 * M + 2 * par, "flops": 8 * e}
    if c["op"] == "collapse":
        if c["back"]:  # dh, x, dx_add, pre -> dx, dpre
            return {"bytes": (1 + 3 * HC) * e * n + 8 * HC * M, "flops": 4 * HC * e}
        return {"bytes": (HC + 1 + c["saved"]) * e * n + 4 * HC * M + 8 * D + 8 * M * c["saved"], "flops": (2 * HC + 8) * e}
    if c["op"] == "expand":
        coef = 4 * M * (HC + HC * HC)
        if c["back"]:  # dout, x, y, post, comb -> dx, dy, dpost, dcomb
            return {"bytes": (3 * HC + 2) * e * n + 2 * coef, "flops": (4 * HC * HC + 4 * HC) * e}
        return {"bytes": (2 * HC + 1) * e * n + coef, "flops": (2 * HC * HC + 2 * HC) * e}
    k = min(c["top"], c["of"])
    pairs = M * k
    if c["op"] == "dispatch" and not c["back"]:
        return {"bytes": e * n + pairs * D * n + pairs * (4 if c["ids"] == "int32" else 8) + 8 * pairs + 4 * c["of"] + 4, "flops": 0}
    if c["op"] == "combine" and c["back"]:  # dy, ys, slots, weights -> dys, dweights
        return {"bytes": e * n + 2 * pairs * D * n + 12 * pairs, "flops": 3 * pairs * D}
    return {"bytes": pairs * D * n + e * n + (8 if c["op"] == "combine" else 4) * pairs, "flops": 2 * pairs * D}


# ------------------------------------------------------------------------------------ exact


def exact(case, seed):
    """The same results in 64 bits: gradients by differentiating the forward definition, the sort by counting."""
    s = prepare(case, seed)
    c = s.pop("case")
    w = {k: v.double() if v.is_floating_point() else v for k, v in s.items()}
    M, D = c["rows"], c["width"]
    if c["op"] == "norm":
        if not c["back"]:
            return _exact_norm(w["x"], w["weight"], w["bias"])
        x, weight, bias = (v.requires_grad_() for v in (w["x"], w["weight"], torch.zeros(D, dtype=torch.float64, device="cuda")))
        return torch.autograd.grad(_exact_norm(x, weight, bias)[0], (x, weight, bias), w["dy"])
    if c["op"] == "collapse":
        x = w["x"].view(M, HC, D)
        if not c["back"]:
            h = torch.einsum("mi,mid->md", w["pre"], x)
            y, mean, rstd = _exact_norm(h, w["weight"], w["bias"])
            return (y, h, mean, rstd) if c["saved"] else y
        dx, dpre = torch.autograd.grad(torch.einsum("mi,mid->md", w["pre"].requires_grad_(), x.requires_grad_()), (x, w["pre"]), w["dh"])
        return dx.reshape(M, HC * D) + w["dx_add"], dpre
    if c["op"] == "expand":
        x, y, post, comb = w["x"].view(M, HC, D), w["y"], w["post"], w["comb"]
        with torch.set_grad_enabled(c["back"]):
            inputs = [v.requires_grad_(c["back"]) for v in (x, y, post, comb)]
            out = torch.einsum("mi,md->mid", post, y) + torch.einsum("mij,mjd->mid", comb, x)
        if not c["back"]:
            return out.reshape(M, HC * D)
        dx, dy, dpost, dcomb = torch.autograd.grad(out, inputs, w["dout"].view(M, HC, D))
        return dx.reshape(M, HC * D), dy, dpost, dcomb
    if c["op"] == "dispatch" and not c["back"]:
        ids = w["ids"].cpu().reshape(-1).tolist()
        found = [[] for _ in range(c["of"])]
        for pair, e in enumerate(ids):
            if e >= 0:
                found[e].append(pair)
        source = [p for pairs in found for p in pairs]
        offsets, slots = [0], [-1] * len(ids)
        for pairs in found:
            offsets.append(offsets[-1] + len(pairs))
        for row, p in enumerate(source):
            slots[p] = row
        xs = torch.zeros(len(ids), D, dtype=torch.float64, device="cuda")
        k = w["ids"].shape[1]
        xs[: len(source)] = w["x"][torch.tensor([p // k for p in source], dtype=torch.int64, device="cuda")]
        source += [-1] * (len(ids) - len(source))
        return torch.tensor(offsets), torch.tensor(slots).view(-1, k), torch.tensor(source), xs
    # combine, and dispatch's gradient, which is combine with weights of one
    rows = torch.zeros(M, D, dtype=torch.float64, device="cuda")
    ys = w["dxs" if c["op"] == "dispatch" else "ys"]
    ways = torch.ones(w["slots"].shape, dtype=torch.float64, device="cuda") if c["op"] == "dispatch" else w["weights"]
    back = c["op"] == "combine" and c["back"]
    ys.requires_grad_(back), ways.requires_grad_(back)
    for j in range(w["slots"].shape[1]):
        t = torch.nonzero(w["slots"][:, j] >= 0).reshape(-1)
        rows = rows.index_add(0, t, ways[t, j, None] * ys[w["slots"][t, j].long()])
    return torch.autograd.grad(rows, (ys, ways), w["dy"]) if back else rows


def _exact_norm(x, weight, bias):
    mean = x.sum(1) / x.shape[1]
    rstd = 1 / torch.sqrt((x - mean[:, None]).pow(2).sum(1) / x.shape[1] + EPS)
    return (x - mean[:, None]) * rstd[:, None] * weight + bias, mean, rstd
