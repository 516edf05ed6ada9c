"""Measured cases of the operators around the LM head: layer norm, the expert-balance loss, beam selection.

`own` false: every operator in its plain form, elementary torch operations in 32 bits (64 where 32 lose what
matters).  `own` true: the framework's entry points (layer_norm, balance_loss and beam modules).
"""
import math

import torch

own = False
device = "cuda"

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


# ---------------------------------------------------------------- the cases

def _norm(name, what, rows, hidden, dtype, wtype):
    return {"name": name, "op": "norm", "what": what, "rows": rows, "hidden": hidden, "dtype": dtype, "wtype": wtype}


def _balance(name, what, groups, tokens, experts, top_k, dtype, masked):
    return {"name": name, "op": "balance", "what": what, "groups": groups, "tokens": tokens, "experts": experts,
            "top_k": top_k, "dtype": dtype, "masked": masked}


def _beam(name, items, beams, keep, vocab, dtype, masked, states=0, heads=0, length=0, room=0, dim=0):
    return {"name": name, "op": "beam", "items": items, "beams": beams, "keep": keep, "vocab": vocab, "dtype": dtype,
            "masked": masked, "states": states, "heads": heads, "length": length, "room": room, "dim": dim}


def listed():
    return [
        # the final norm of one decode step of a 4096-wide model, 16 sequences
        _norm("norm-forward-decode", "forward", 16, 4096, "bf16", "bf16"),
        # the final norm before the Qwen3-8B head on its whole batch, without a graph (evaluation)
        _norm("norm-forward-long", "forward", 131072, 4096, "bf16", "bf16"),
        # forward and backward before the Qwen3-0.6B head, fp32 master weights
        _norm("norm-train-1024", "train", 16384, 1024, "bf16", "fp32"),
        # the backward before the Qwen3-4B head, one micro-batch
        _norm("norm-backward-2560", "backward", 65536, 2560, "bf16", "bf16"),
        # an odd width and an odd number of rows, half precision
        _norm("norm-train-odd", "train", 4099, 1601, "fp16", "fp16"),
        # a small mixture (8 experts, 2 per token), fp32 router, one short batch: latency
        _balance("balance-forward-small", "forward", 1, 509, 8, 2, "fp32", False),
        # all layers of a mixture at once, loss and gradient in one call, padded tokens
        _balance("balance-fused-layers", "fused", 24, 16384, 128, 8, "bf16", True),
        # the gradient for one long packed batch, fp32 router of 256 experts
        _balance("balance-backward-long", "backward", 1, 131072, 256, 8, "fp32", False),
        # an odd number of experts
        _balance("balance-train-odd", "train", 6, 4097, 61, 4, "bf16", True),
        # one request, four beams, eight results (as many can end and four are left): latency
        _beam("beam-one-request", 1, 4, 8, 32768, "bf16", False),
        # a decode step of a batch: selection at the Qwen3 vocabulary, then the states of 8 layers' caches
        _beam("beam-step-with-caches", 8, 4, 4, 151936, "bf16", True, 16, 8, 1500, 2048, 128),
        # a large batch with fp32 logits over an odd vocabulary, banned tokens
        _beam("beam-large-odd-vocab", 64, 8, 16, 50257, "fp32", True),
    ]


def _spread(rng, low, high):
    """A whole number between the two, even over the logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(("norm", "balance", "beam"))
    if op == "norm":
        hidden = _spread(rng, 64, 8192)
        if rng.random() < 0.7:
            hidden = -(-hidden // 64) * 64
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        rows = _spread(rng, 1, max(1, min(131072, (1 << 27) // hidden)))
        case = _norm("", rng.choice(("forward", "backward", "train")), rows, hidden, dtype, rng.choice((dtype, "fp32")))
    elif op == "balance":
        experts = rng.choice((8, 16, 60, 64, 128, 160, 256, _spread(rng, 4, 512)))
        groups = _spread(rng, 1, 48)
        tokens = _spread(rng, 1, max(1, min(131072, (1 << 25) // (experts * groups))))
        case = _balance("", rng.choice(("forward", "backward", "fused", "train")), groups, tokens, experts,
                        min(experts, rng.randint(1, 8)), rng.choice(("bf16", "fp32")), rng.random() < 0.5)
    else:
        vocab = rng.choice((4096, 32768, 50257, 151936, _spread(rng, 1000, 200000)))
        beams = rng.randint(1, 16)
        items = _spread(rng, 1, max(1, min(64, (1 << 25) // (vocab * beams))))
        keep = beams * rng.randint(1, 2)
        case = _beam("", items, beams, keep, vocab, rng.choice(("bf16", "fp16", "fp32")), rng.random() < 0.5)
        if rng.random() < 0.4:
            case.update(states=2 * rng.randint(1, 4), heads=rng.choice((1, 2, 4, 8)), dim=rng.choice((64, 128)))
            token = 2 * case["states"] * items * keep * case["heads"] * case["dim"]
            case["length"] = _spread(rng, 1, max(1, min(2048, (1 << 30) // token)))
            case["room"] = case["length"] + rng.randint(0, 64)
    del case["name"]
    return case


def work(case):
    if case["op"] == "norm":
        n, h, es, ws = case["rows"], case["hidden"], BYTES[case["dtype"]], BYTES[case["wtype"]]
        forward, backward = 2 * n * h * es + 2 * h * ws, 3 * n * h * es + 8 * n + 3 * h * ws
        moved = {"forward": forward, "backward": backward, "train": forward + backward + 8 * n}[case["what"]]
        return {"bytes": moved, "flops": n * h * {"forward": 8, "backward": 14, "train": 22}[case["what"]]}
    if case["op"] == "balance":
        n, e, es = case["groups"] * case["tokens"], case["experts"], BYTES[case["dtype"]]
        mask = case["tokens"] if case["masked"] else 0
        routes = 8 * n * case["top_k"] + 8 * case["groups"] * e + mask
        forward, backward = n * e * es + routes, 2 * n * e * es + 8 * case["groups"] * e + mask
        moved = {"forward": forward, "backward": backward, "train": forward + backward, "fused": 2 * n * e * es + routes}
        return {"bytes": moved[case["what"]], "flops": n * e * {"forward": 6, "backward": 9, "train": 15, "fused": 11}[case["what"]]}
    rows, kept = case["items"] * case["beams"], case["items"] * case["keep"]
    state = case["states"] * case["heads"] * case["length"] * case["dim"] * 2  # of one row
    return {"bytes": rows * (case["vocab"] * BYTES[case["dtype"]] + 5 + state) + kept * (20 + state),
            "flops": 4 * rows * case["vocab"]}


# ---------------------------------------------------------------- the inputs

def _inputs(case, seed):
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=device).normal_(mean, std, generator=g)

    if case["op"] == "norm":
        n, h, t, w = case["rows"], case["hidden"], TYPES[case["dtype"]], TYPES[case["wtype"]]
        s = {"x": normal(n, h, std=1.5, mean=0.2, dtype=t)}  # hidden states: a scale and an offset of their own
        s["weight"], s["bias"] = normal(h, std=0.1, mean=1.0).to(w), normal(h, std=0.1).to(w)
        if case["what"] != "forward":
            s["grad_y"] = normal(n, h, std=0.5, dtype=t)
        if case["what"] == "backward":  # what a forward has left behind
            mean, rstd = [], []
            for x in s["x"].split(max(1, (1 << 24) // h)):
                x = x.double()
                mean.append(x.mean(1))
                rstd.append((x.var(1, correction=0) + EPS).rsqrt())
            s["mean"], s["rstd"] = torch.cat(mean).float(), torch.cat(rstd).float()
        return s
    if case["op"] == "balance":
        shape = case["groups"], case["tokens"], case["experts"]
        lean = normal(case["groups"], 1, case["experts"], std=0.7)  # experts that the router prefers
        logits = (normal(*shape) + lean).to(TYPES[case["dtype"]])
        s = {"logits": logits, "experts": logits.float().topk(case["top_k"], dim=-1).indices, "mask": None}
        if case["masked"]:
            s["mask"] = torch.rand(case["tokens"], device=device, generator=g) < 0.9
        if case["what"] == "backward":
            s["counts"], s["n_valid"] = _counts(s["experts"], s["mask"], case["experts"])
        s["grad_output"] = torch.full((1,), 0.01, device=device)  # the loss term's coefficient
        return s
    b, k, v = case["items"], case["beams"], case["vocab"]
    logits = normal(b, k, v, std=2.0)
    for _ in range(8):  # a few likely tokens in each row
        at = torch.randint(v, (b, k, 1), device=device, generator=g)
        logits.scatter_(2, at, normal(b, k, 1, std=2.0, mean=9.0))
    s = {"scores": -normal(b, k, std=4.0).abs(), "finished": None}
    if case["masked"]:
        logits.masked_fill_(torch.rand(v, device=device, generator=g) < 0.02, -math.inf)  # banned tokens
        s["finished"] = torch.rand(b, k, device=device, generator=g) < 0.1
    s["logits"] = logits.to(TYPES[case["dtype"]])
    shape = b * k, case["heads"], case["room"], case["dim"]
    s["states"] = [normal(*shape, dtype=torch.bfloat16) for _ in range(case["states"])]
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "beam":  # the caches have room to grow and a second set to move to; the used part is a view
        kept = case["items"] * case["keep"]
        s["other"] = [x.new_empty(kept, *x.shape[1:])[:, :, :case["length"]] for x in s["states"]]
        s["states"] = [x[:, :, :case["length"]] for x in s["states"]]
    return s


# ---------------------------------------------------------------- the plain forms

def _norm_forward(x, weight, bias):
    x = x.float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = (x.square().mean(1, keepdim=True) + EPS).rsqrt()
    return x * rstd * weight.float() + bias.float(), mean.squeeze(1), rstd.squeeze(1)


def _norm_backward(dy, x, weight, mean, rstd):
    dy, rstd = dy.float(), rstd[:, None]
    xh = (x.float() - mean[:, None]) * rstd
    g = dy * weight.float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def _counts(experts, mask, n):
    g, t, k = experts.shape
    valid = torch.ones(t, dtype=torch.bool, device=experts.device) if mask is None else mask
    at = experts + torch.arange(g, device=experts.device)[:, None, None] * n
    one = valid.to(torch.int64)[None, :, None].expand(g, t, k)
    counts = torch.zeros(g * n, dtype=torch.int64, device=experts.device).index_add_(0, at.reshape(-1), one.reshape(-1))
    return counts.view(g, n), valid.sum().expand(g).contiguous()


def _balance_share(counts, n_valid, k):
    """f: how often each expert is taken, 1 where the load is even."""
    return counts.double() * counts.shape[1] / (k * n_valid.clamp(min=1).double()[:, None])


def _balance_loss(p, counts, n_valid, mask, k):
    p = p if mask is None else p * mask[:, None]
    mean = p.sum(1, dtype=torch.float64) / n_valid.clamp(min=1).double()[:, None]
    return (_balance_share(counts, n_valid, k) * mean).sum(1).mean().float().reshape(1)


def _balance_grad(p, counts, n_valid, mask, k, grad_output):
    f = (_balance_share(counts, n_valid, k) - 1).float()[:, None]  # the ones cancel: a row of p adds up to one
    scale = grad_output / counts.shape[0] / n_valid.clamp(min=1).float()[:, None, None]
    d = scale * p * (f - (f * p).sum(2, keepdim=True))
    return d if mask is None else d * mask[:, None]


def _select(logits, scores, finished, keep, pad):
    b, k, v = logits.shape
    x = torch.nan_to_num(logits.float(), nan=-math.inf, posinf=torch.finfo(torch.float32).max, neginf=-math.inf) + 0.0
    bits = x.view(torch.int32).long()
    order = torch.where(bits < 0, -2147483648 - bits, bits)  # grows with the logit
    key = order * (1 << 32) + (v - 1 - torch.arange(v, device=x.device))  # the lower token first among equal logits
    token = key.topk(min(keep, v), dim=2).indices
    x = x.double()
    top = x.amax(2, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    lp = x.gather(2, token) - top - (x - top).exp().sum(2, keepdim=True).log()
    lp = lp.masked_fill(x.gather(2, token) == -math.inf, -math.inf)
    if finished is not None:
        first = torch.arange(token.shape[2], device=x.device) == 0
        lp = torch.where(finished[:, :, None], torch.where(first, 0.0, -math.inf), lp)
        token = torch.where(finished[:, :, None], pad, token)
    total = (scores.double()[:, :, None] + lp).reshape(b, -1)
    best, at = total.sort(dim=1, descending=True, stable=True)
    best, at = best[:, :keep], at[:, :keep]
    return {"scores": best.float(), "tokens": token.reshape(b, -1).gather(1, at), "parents": at // token.shape[2]}


def _reorder(states, parents, out):
    b = parents.shape[0]
    rows = (parents + torch.arange(b, device=parents.device)[:, None] * (states[0].shape[0] // b)).reshape(-1)
    return [o.copy_(x[rows]) for x, o in zip(states, out)]


def _run_plain(s):
    case = s["case"]
    if case["op"] == "norm":
        t, w = s["x"].dtype, s["weight"].dtype
        out = {}
        mean, rstd = s.get("mean"), s.get("rstd")
        if case["what"] != "backward":
            y, mean, rstd = _norm_forward(s["x"], s["weight"], s["bias"])
            out["y"] = y.to(t)
        if case["what"] != "forward":
            dx, dw, db = _norm_backward(s["grad_y"], s["x"], s["weight"], mean, rstd)
            out.update(grad_x=dx.to(t), grad_weight=dw.to(w), grad_bias=db.to(w))
        return out
    if case["op"] == "balance":
        out, k, mask = {}, case["top_k"], s["mask"]
        counts, n_valid = s.get("counts"), s.get("n_valid")
        p = s["logits"].float().softmax(2)
        if case["what"] != "backward":
            counts, n_valid = _counts(s["experts"], mask, case["experts"])
            out.update(loss=_balance_loss(p, counts, n_valid, mask, k), counts=counts)
        if case["what"] != "forward":
            out["grad_logits"] = _balance_grad(p, counts, n_valid, mask, k, s["grad_output"]).to(s["logits"].dtype)
        return out
    out = _select(s["logits"], s["scores"], s["finished"], case["keep"], 0)
    if s["states"]:
        out["states"] = _reorder(s["states"], out["parents"], s["other"])
    return out


# ---------------------------------------------------------------- the framework's operators

def _run_own(s):
    case = s["case"]
    if case["op"] == "norm":
        from lm_head_linear_chunked_gb300.layer_norm import layer_norm, layer_norm_backward, layer_norm_forward
        if case["what"] == "forward":
            return {"y": layer_norm(s["x"], s["weight"], s["bias"], EPS)}
        out, mean, rstd = {}, s.get("mean"), s.get("rstd")
        if case["what"] == "train":
            f = layer_norm_forward(s["x"], s["weight"], s["bias"], EPS)
            out["y"], mean, rstd = f["y"], f["mean"], f["rstd"]
        d = layer_norm_backward(s["grad_y"], s["x"], s["weight"], mean, rstd)
        out.update(grad_x=d["grad_x"], grad_weight=d["grad_weight"], grad_bias=d["grad_bias"])
        return out
    if case["op"] == "balance":
        from lm_head_linear_chunked_gb300.balance_loss import balance_backward, balance_forward, balance_fused
        if case["what"] == "fused":
            f = balance_fused(s["logits"], s["experts"], s["mask"], grad_output=s["grad_output"])
            return {"loss": f["loss"], "counts": f["counts"], "grad_logits": f["grad_logits"]}
        out, counts, n_valid = {}, s.get("counts"), s.get("n_valid")
        if case["what"] != "backward":
            f = balance_forward(s["logits"], s["experts"], s["mask"])
            counts, n_valid = f["counts"], f["n_valid"]
            out.update(loss=f["loss"], counts=counts)
        if case["what"] != "forward":
            out["grad_logits"] = balance_backward(s["logits"], counts, n_valid, case["top_k"], s["mask"],
                                                  grad_output=s["grad_output"])["grad_logits"]
        return out
    from lm_head_linear_chunked_gb300.beam import beam_reorder, beam_select
    out = dict(beam_select(s["logits"], s["scores"], case["keep"], finished=s["finished"], pad_token=0))
    if s["states"]:
        out["states"] = beam_reorder(s["states"], out["parents"], out=s["other"])
    return out


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm(s, what):
    rows = max(1, (1 << 25) // s["x"].shape[1])
    w, b = s["weight"].double(), s["bias"].double()
    y, gx, gw, gb = [], [], 0, 0
    for i in range(0, s["x"].shape[0], rows):
        x = s["x"][i:i + rows].double()
        if what == "backward":
            mean, rstd = s["mean"][i:i + rows, None].double(), s["rstd"][i:i + rows, None].double()
        else:
            mean = x.sum(1, keepdim=True) / x.shape[1]
            rstd = 1 / ((x - mean).pow(2).sum(1, keepdim=True) / x.shape[1] + EPS).sqrt()
        x = (x - mean) * rstd
        if what != "backward":
            y.append(torch.addcmul(b, x, w))
        if what != "forward":
            d = s["grad_y"][i:i + rows].double()
            gw, gb = gw + torch.einsum("rh,rh->h", d, x), gb + torch.einsum("rh->h", d)
            d = d * w
            gx.append(rstd * (d - (d.sum(1, keepdim=True) + x * (d * x).sum(1, keepdim=True)) / x.shape[1]))
    out = {} if what == "backward" else {"y": torch.cat(y)}
    if what != "forward":
        out.update(grad_x=torch.cat(gx), grad_weight=gw, grad_bias=gb)
    return out


def _exact_balance(s, case):
    groups, n, k = case["groups"], case["experts"], case["top_k"]
    keep = torch.ones(case["tokens"], dtype=torch.bool, device=device) if s["mask"] is None else s["mask"]
    total, tokens = torch.zeros(1, dtype=torch.float64, device=device), int(keep.sum())
    counts = torch.zeros(groups, n, dtype=torch.int64, device=device)
    grad = torch.zeros(s["logits"].shape, dtype=torch.float64, device=device)
    for g in range(groups):
        z = s["logits"][g].double()
        p = (z - z.logsumexp(1, keepdim=True)).exp()
        counts[g] = torch.bincount(s["experts"][g][keep].reshape(-1), minlength=n)
        if tokens:
            f = counts[g].double() * n / (k * tokens)
            total += (p[keep] @ f).sum() / tokens / groups
            d = p * (f - (p @ f)[:, None]) * (s["grad_output"].double() / groups / tokens)
            grad[g] = torch.where(keep[:, None], d, torch.zeros_like(d))
    out = {} if case["what"] == "backward" else {"loss": total, "counts": counts}
    if case["what"] != "forward":
        out["grad_logits"] = grad
    return out


def _exact_beam(s, case):
    """Item by item over the whole table of scores; the tokens, parents and states are whole values, held to the plain form's."""
    best = []
    for z, score, done in zip(s["logits"], s["scores"], s["finished"] if s["finished"] is not None else [None] * case["items"]):
        z = z.double()
        table = z - z.logsumexp(1, keepdim=True) + score.double()[:, None]
        if done is not None:
            table[done] = -math.inf
            table[done, 0] = score[done].double()
        best.append(table.reshape(-1).topk(case["keep"]).values)
    out = {"scores": torch.stack(best), "tokens": None, "parents": None}
    if case["states"]:
        out["states"] = [None] * case["states"]
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case["what"])
    if case["op"] == "balance":
        return _exact_balance(s, case)
    return _exact_beam(s, case)
