"""Measured cases of the operators between token ids and the head: RMS norm with residual, embedding, rows sorted by expert.

`own` false: every operator in its plain form, elementary torch operations in 32 bits (64 for long sums).  `own` true: the framework's
entry points (rms_norm, embedding and expert_rows modules).
"""
import math

import numpy as np
import torch

own = False
device = "cuda"

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
E4M3_MAX = 448.0
LEAST_AMAX = 2.0 ** -100  # the smallest that a group's largest magnitude counts as
ZIPF = 1.1                # of the tokens


# ---------------------------------------------------------------- the cases

def _norm(name, what, rows, hidden, dtype, wtype, residual, group=0):
    """group: columns to a scale of the 8-bit output, 0 for the whole row."""
    return {"name": name, "op": "norm", "what": what, "rows": rows, "hidden": hidden, "dtype": dtype, "wtype": wtype,
            "residual": residual, "group": group}


def _embedding(name, what, tokens, vocab, hidden, dtype, scale, padded):
    return {"name": name, "op": "embedding", "what": what, "tokens": tokens, "vocab": vocab, "hidden": hidden,
            "dtype": dtype, "scale": scale, "padded": padded}


def _experts(name, what, tokens, experts, top_k, hidden, dtype, wtype, align, masked):
    return {"name": name, "op": "experts", "what": what, "tokens": tokens, "experts": experts, "top_k": top_k,
            "hidden": hidden, "dtype": dtype, "wtype": wtype, "align": align, "masked": masked}


def listed():
    return [
        # a norm within one decode step of a 4096-wide model, 16 sequences: latency
        _norm("rms-forward-decode", "forward", 16, 4096, "bf16", "bf16", True),
        # a prompt's norm in front of 8-bit products, a scale for every 128 columns
        _norm("rms-fp8-prompt", "fp8", 32768, 4096, "bf16", "bf16", True, 128),
        # forward and backward of the norm of a 1024-wide model, with the residual's gradient, fp32 master weights
        _norm("rms-train-1024", "train", 16384, 1024, "bf16", "fp32", True),
        # the backward of the norm before a 2560-wide head, one micro-batch
        _norm("rms-backward-2560", "backward", 65536, 2560, "bf16", "bf16", False),
        # one decode step's lookup in a 151936-token vocabulary: latency
        _embedding("embedding-decode", "forward", 64, 151936, 4096, "bf16", 1.0, False),
        # a training step of the 1024-wide model: lookup and dense gradient
        _embedding("embedding-train-1024", "train", 16384, 151936, 1024, "bf16", 1.0, False),
        # the gradient for a whole batch of the 4096-wide head, padded
        _embedding("embedding-backward-long", "backward", 131072, 151936, 4096, "bf16", 1.0, True),
        # an odd vocabulary, width and number of tokens, embeddings scaled by sqrt(width)
        _embedding("embedding-train-odd", "train", 10007, 50257, 1601, "fp32", 40.0125, True),
        # one decode step of a mixture of 128 experts: sort, spread, join
        _experts("experts-decode", "forward", 32, 128, 8, 4096, "bf16", "fp32", 1, False),
        # a training step's sort, spread and join with all gradients
        _experts("experts-train-2048", "train", 16384, 128, 8, 2048, "bf16", "fp32", 1, False),
        # a long prompt through a mixture of 256, segments on whole tiles of 128 rows, padded tokens left out
        _experts("experts-prompt-aligned", "forward", 32768, 256, 6, 2560, "bf16", "bf16", 128, True),
        # odd numbers of tokens, experts and columns, half precision
        _experts("experts-train-odd", "train", 4099, 61, 3, 1601, "fp16", "fp32", 16, True),
    ]


def _spread(rng, low, high):
    """A whole number between the two, even over the logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def _width(rng, high):
    hidden = _spread(rng, 64, high)
    return -(-hidden // 64) * 64 if rng.random() < 0.7 else hidden


def draw(rng):
    op = rng.choice(("norm", "embedding", "experts"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op == "norm":
        hidden = _width(rng, 8192)
        what = rng.choice(("forward", "fp8", "backward", "train"))
        case = _norm("", what, _spread(rng, 1, max(1, min(131072, (1 << 27) // hidden))), hidden, dtype,
                     rng.choice((dtype, "fp32")), rng.random() < 0.6, rng.choice((0, 128)) if what == "fp8" else 0)
    elif op == "embedding":
        hidden = _width(rng, 4096)
        vocab = rng.choice((32768, 50257, 151936, _spread(rng, 500, 200000)))
        vocab = min(vocab, (1 << 28) // hidden)
        case = _embedding("", rng.choice(("forward", "backward", "train")), _spread(rng, 1, max(1, min(131072, (1 << 27) // hidden))),
                          vocab, hidden, dtype, rng.choice((1.0, hidden ** 0.5)), rng.random() < 0.5)
    else:
        experts = rng.choice((8, 16, 60, 64, 128, 160, 256, _spread(rng, 4, 512)))
        top_k = min(experts, rng.randint(1, 8))
        hidden = _width(rng, 4096)
        tokens = _spread(rng, 1, max(1, min(65536, (1 << 27) // (hidden * top_k))))
        case = _experts("", rng.choice(("forward", "train")), tokens, experts, top_k, hidden, dtype,
                        rng.choice((dtype, "fp32")), rng.choice((1, 1, 16, 128)) if tokens * top_k > 8 * experts else 1,
                        rng.random() < 0.5)
    del case["name"]
    return case


def _rows(case):
    """Rows that the sorted tokens may take: every expert's segment can end in align - 1 rows of padding."""
    return -(-(case["tokens"] * case["top_k"] + case["experts"] * (case["align"] - 1)) // case["align"]) * case["align"]


def _distinct(case):
    """Expected number of different tokens among those drawn."""
    p = np.arange(1, case["vocab"] + 1, dtype=np.float64) ** -ZIPF
    return float(-np.expm1(case["tokens"] * np.log1p(-p / (p.sum() * (1 + 1e-9)))).sum())


def work(case):
    es, h = BYTES[case["dtype"]], case["hidden"]
    if case["op"] == "norm":
        n, ws = case["rows"], BYTES[case["wtype"]]
        extra = 1 if case["residual"] else 0
        row = n * h * es
        forward = row * (2 + 2 * extra) + h * ws
        backward = row * (3 + extra) + 4 * n + 2 * h * ws
        groups = -(-h // case["group"]) if case["group"] else 1
        moved = {"forward": forward, "fp8": row * (1 + 2 * extra) + n * h + 4 * n * groups + h * ws, "backward": backward,
                 "train": forward + 4 * n + backward}
        return {"bytes": moved[case["what"]], "flops": n * h * {"forward": 5, "fp8": 8, "backward": 9, "train": 14}[case["what"]]}
    if case["op"] == "embedding":
        n = case["tokens"]
        forward = n * (8 + h * es) + _distinct(case) * h * es
        read = n * 0.95 if case["padded"] else n  # rows of padding carry no gradient
        backward = n * 8 + read * h * es + case["vocab"] * h * es
        moved = {"forward": forward, "backward": backward, "train": forward + backward}
        return {"bytes": moved[case["what"]], "flops": n * h * {"forward": 1, "backward": 1, "train": 2}[case["what"]]}
    t, k, r = case["tokens"], case["top_k"], _rows(case)
    plan = t * k * 12 + r * 4 + 16 * case["experts"] + (t if case["masked"] else 0)
    slots, ws = t * k * (0.9 if case["masked"] else 1), BYTES[case["wtype"]]
    spread, join = (t + r) * h * es, (t + slots) * h * es + slots * ws
    moved = {"forward": plan + spread + join, "train": plan + spread + 2 * join + (t + slots + r) * h * es + slots * ws}
    return {"bytes": moved[case["what"]], "flops": slots * h * {"forward": 2, "train": 6}[case["what"]]}


# ---------------------------------------------------------------- the inputs

def _inputs(case, seed):
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=device).normal_(mean, std, generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device=device, generator=g)

    t, h = TYPES[case["dtype"]], case["hidden"]
    if case["op"] == "norm":
        n, what = case["rows"], case["what"]
        s = {"x": normal(n, h, std=1.5, mean=0.1, dtype=t), "weight": normal(h, std=0.1, mean=1.0).to(TYPES[case["wtype"]]),
             "residual": None, "grad_sum": None}
        if case["residual"] and what != "backward":
            s["residual"] = normal(n, h, std=2.0, dtype=t)
        if what in ("backward", "train"):
            s["grad_y"] = normal(n, h, std=0.5, dtype=t)
            if case["residual"]:
                s["grad_sum"] = normal(n, h, std=0.5, dtype=t)  # what arrives along the residual
        if what == "backward":  # what a forward has left behind
            s["rstd"] = torch.cat([(x.double().square().mean(1) + EPS).rsqrt() for x in s["x"].split(max(1, (1 << 24) // h))]).float()
        return s
    if case["op"] == "embedding":
        n, v, what = case["tokens"], case["vocab"], case["what"]
        p = torch.arange(1, v + 1, dtype=torch.float64, device=device) ** -ZIPF
        cdf = p.cumsum(0) / p.sum()
        s = {"tokens": torch.searchsorted(cdf, torch.rand(n, dtype=torch.float64, device=device, generator=g)).clamp(max=v - 1),
             "padding": None}
        if case["padded"]:  # the end of the batch and a few within
            s["padding"] = v - 1
            s["tokens"].masked_fill_(uniform(n) < 0.05, v - 1)
        if what != "backward":
            s["weight"] = normal(v, h, std=0.02, dtype=t)
        if what != "forward":
            s["grad_y"] = normal(n, h, std=0.5, dtype=t)
        return s
    n, k, e = case["tokens"], case["top_k"], case["experts"]
    logits = normal(n, e) + normal(e, std=0.5)  # a few experts are preferred
    gates, experts = logits.softmax(1).topk(k, dim=1)
    s = {"x": normal(n, h, dtype=t), "experts": experts, "weights": gates.to(TYPES[case["wtype"]]), "mask": None}
    if case["masked"]:
        s["mask"] = uniform(n) < 0.9
    s["rows"] = normal(_rows(case), h, dtype=t)  # what the experts make of their rows
    if case["what"] == "train":
        s["grad_y"] = normal(n, h, std=0.5, dtype=t)
        s["grad_rows"] = normal(_rows(case), h, std=0.5, dtype=t)  # of the rows that the experts read
    return s


def prepare(case, seed):
    return {**_inputs(case, seed), "case": case}


# ---------------------------------------------------------------- the plain forms

def _norm_sum(s):
    """What is normed: x, or x with the residual, rounded to their type."""
    return s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)


def _norm_forward(x, weight):
    x = x.float()
    rstd = (x.square().mean(1, keepdim=True) + EPS).rsqrt()
    return x * rstd * weight.float(), rstd.squeeze(1)


def _norm_backward(dy, x, weight, rstd, grad_sum):
    dy, rstd = dy.float(), rstd[:, None]
    xh = x.float() * rstd
    g = dy * weight.float()
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    return dx if grad_sum is None else dx + grad_sum.float(), (dy * xh).sum(0)


def _quantized(y, group):
    """e4m3 values and the scales of y's groups of columns; the last group may be shorter."""
    n, h = y.shape
    group = group or h
    wide = torch.nn.functional.pad(y, (0, -h % group)).view(n, -1, group)
    scales = wide.abs().amax(2).clamp(min=LEAST_AMAX) / E4M3_MAX
    q = (wide / scales[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(n, -1)[:, :h]
    return q.to(torch.float8_e4m3fn), scales


def _run_norm(s):
    case, t, w = s["case"], s["x"].dtype, s["weight"].dtype
    out, x, rstd = {}, _norm_sum(s), s.get("rstd")
    if s["residual"] is not None:
        out["sum"] = x
    if case["what"] != "backward":
        y, rstd = _norm_forward(x, s["weight"])
        if case["what"] == "fp8":
            out["q"], out["scales"] = _quantized(y, case["group"])
        else:
            out["y"] = y.to(t)
    if case["what"] in ("backward", "train"):
        dx, dw = _norm_backward(s["grad_y"], x, s["weight"], rstd, s["grad_sum"])
        out.update(grad_x=dx.to(t), grad_weight=dw.to(w))
    return out


def _run_embedding(s):
    case, out, tokens = s["case"], {}, s["tokens"]
    if case["what"] != "backward":
        out["y"] = (s["weight"][tokens].float() * case["scale"]).to(s["weight"].dtype)
    if case["what"] != "forward":
        dy = s["grad_y"].float() * case["scale"]
        if s["padding"] is not None:
            dy = dy * (tokens != s["padding"])[:, None]
        if dy.dtype == s["grad_y"].dtype:
            dy = dy.double()  # thousands of rows can go into one, and the result keeps 24 bits of it
        dw = torch.zeros(case["vocab"], case["hidden"], dtype=dy.dtype, device=dy.device)
        out["grad_weight"] = dw.index_add_(0, tokens, dy).to(s["grad_y"].dtype)
    return out


def _plan(s):
    """Where each slot's row goes, which slot each row has (-1: none), the experts' counts and where their rows start."""
    case, (n, k) = s["case"], s["experts"].shape
    e, align = case["experts"], case["align"]
    flat = s["experts"].reshape(-1)
    if s["mask"] is not None:
        flat = torch.where(s["mask"][:, None].expand(n, k).reshape(-1), flat, e)  # behind all experts
    order = flat.argsort(stable=True)
    counts = torch.zeros(e + 1, dtype=torch.int64, device=flat.device).index_add_(0, flat, torch.ones_like(flat))
    padded = (counts[:e] + align - 1) // align * align
    offsets = torch.cat((padded.new_zeros(1), padded.cumsum(0)))
    first = counts.cumsum(0) - counts  # in the sorted order, without padding
    where = offsets[flat[order]] + torch.arange(n * k, device=flat.device) - first[flat[order]]
    kept = flat[order] < e
    positions = torch.empty_like(flat).scatter_(0, order, torch.where(kept, where, -1))
    slots = torch.full((_rows(case) + 1,), -1, dtype=torch.int64, device=flat.device)
    slots.scatter_(0, torch.where(kept, where, _rows(case)), torch.where(kept, order, -1))
    return positions.view(n, k).int(), slots[:-1].int(), counts[:e], offsets


def _of_slots(rows, positions):
    """The rows of every token's slots, zero where it has none: [tokens, slots, columns]."""
    got = rows[positions.clamp(min=0).long()].float()
    return got * (positions >= 0)[:, :, None]


def _run_experts(s):
    case, t = s["case"], s["x"].dtype
    positions, slots, counts, offsets = _plan(s)
    n, k = positions.shape
    taken = (slots >= 0)[:, None]
    token = slots.clamp(min=0).long() // k  # of each sorted row
    out = {"positions": positions, "slots": slots, "counts": counts, "offsets": offsets,
           "rows": torch.where(taken, s["x"][token], torch.zeros((), dtype=t, device=positions.device))}
    w = s["weights"].float()
    got = _of_slots(s["rows"], positions)
    out["y"] = (got * w[:, :, None]).sum(1).to(t)
    if case["what"] == "train":
        dy = s["grad_y"].float()
        out["grad_weights"] = (got * dy[:, None]).sum(2).to(s["weights"].dtype)
        share = w.reshape(-1)[slots.clamp(min=0).long()] * (slots >= 0)
        out["grad_rows"] = (dy[token] * share[:, None]).to(t)
        out["grad_x"] = _of_slots(s["grad_rows"], positions).sum(1).to(t)
    return out


# ---------------------------------------------------------------- the framework's operators

def _run_own(s):
    case = s["case"]
    if case["op"] == "norm":
        from lm_head_linear_chunked_gb300.rms_norm import rms_norm, rms_norm_backward, rms_norm_forward, rms_norm_fp8
        if case["what"] == "forward":
            if s["residual"] is None:
                return {"y": rms_norm(s["x"], s["weight"], eps=EPS)}
            y, total = rms_norm(s["x"], s["weight"], s["residual"], EPS)
            return {"y": y, "sum": total}
        if case["what"] == "fp8":
            f = rms_norm_fp8(s["x"], s["weight"], s["residual"], EPS, case["group"])
            out = {"q": f["q"], "scales": f["scales"]}
            return out if s["residual"] is None else {**out, "sum": f["sum"]}
        out, x, rstd = {}, s["x"], s.get("rstd")
        if case["what"] == "train":
            f = rms_norm_forward(s["x"], s["weight"], s["residual"], EPS)
            out["y"], x, rstd = f["y"], f["sum"], f["rstd"]
            if s["residual"] is not None:
                out["sum"] = x
        d = rms_norm_backward(s["grad_y"], x, s["weight"], rstd, s["grad_sum"])
        return {**out, "grad_x": d["grad_x"], "grad_weight": d["grad_weight"]}
    if case["op"] == "embedding":
        from lm_head_linear_chunked_gb300.embedding import embedding, embedding_backward
        out = {}
        if case["what"] != "backward":
            out["y"] = embedding(s["tokens"], s["weight"], case["scale"], s["padding"])
        if case["what"] != "forward":
            out["grad_weight"] = embedding_backward(s["grad_y"], s["tokens"], case["vocab"], case["scale"], s["padding"])
        return out
    from lm_head_linear_chunked_gb300.expert_rows import (combine, combine_backward, dispatch, dispatch_backward,
                                                          expert_plan)
    plan = expert_plan(s["experts"], case["experts"], s["mask"], case["align"])
    out = {k: plan[k] for k in ("positions", "slots", "counts", "offsets")}
    out["rows"] = dispatch(s["x"], plan)
    out["y"] = combine(s["rows"], s["weights"], plan)
    if case["what"] == "train":
        d = combine_backward(s["grad_y"], s["rows"], s["weights"], plan)
        out.update(grad_rows=d["grad_rows"], grad_weights=d["grad_weights"], grad_x=dispatch_backward(s["grad_rows"], plan))
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _run_norm, "embedding": _run_embedding, "experts": _run_experts}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm(s, case):
    h, what = case["hidden"], case["what"]
    w = s["weight"].double()
    lists, grad_w = {}, torch.zeros(h, dtype=torch.float64, device=device)

    def keep(name, v):
        lists.setdefault(name, []).append(v)

    step = max(1, (1 << 25) // h)
    for i in range(0, case["rows"], step):
        part = {k: s[k][i:i + step].double() for k in ("x", "residual", "grad_y", "grad_sum", "rstd") if s.get(k) is not None}
        x = part["x"]
        if "residual" in part:  # the sum takes the type of its terms before it is normed
            x = x + part["residual"]
            keep("sum", x)
            x = x.to(TYPES[case["dtype"]]).double()
        rstd = part["rstd"] if "rstd" in part else 1 / (torch.einsum("rh,rh->r", x, x) / h + EPS).sqrt()
        x = x * rstd[:, None]
        if what in ("forward", "train"):
            keep("y", x * w)
        if what == "fp8":  # before the rounding to 8 bits
            for r in range(0, h, case["group"] or h):
                y = (x * w)[:, r:r + (case["group"] or h)]
                scale = y.abs().max(1, keepdim=True).values.clamp(min=LEAST_AMAX) / E4M3_MAX
                lists.setdefault("q%d" % r, []).append(y / scale)
                lists.setdefault("s%d" % r, []).append(scale)
        if what in ("backward", "train"):
            d = part["grad_y"]
            grad_w += torch.einsum("rh,rh->h", d, x)
            d = d * w
            d = (d - x * (torch.einsum("rh,rh->r", d, x) / h)[:, None]) * rstd[:, None]
            keep("grad_x", d + part["grad_sum"] if "grad_sum" in part else d)
    groups = range(0, h, case["group"] or h) if what == "fp8" else ()
    out = {k: torch.cat(v) for k, v in lists.items() if k[0] not in "qs" or k == "sum"}
    if what == "fp8":
        out["q"] = torch.cat([torch.cat(lists["q%d" % r]) for r in groups], 1)
        out["scales"] = torch.cat([torch.cat(lists["s%d" % r]) for r in groups], 1)
    if what in ("backward", "train"):
        out["grad_weight"] = grad_w
    return out


def _exact_embedding(s, case):
    tokens, out = s["tokens"], {}
    if case["what"] != "backward":
        out["y"] = torch.index_select(s["weight"], 0, tokens).double() * case["scale"]
    if case["what"] != "forward":
        order = tokens.argsort()
        if s["padding"] is not None:
            order = order[tokens[order] != s["padding"]]
        grad = torch.zeros(case["vocab"], case["hidden"], dtype=torch.float64, device=device)
        for part in order.split(max(1, (1 << 26) // case["hidden"])):
            names, run = tokens[part].unique_consecutive(return_counts=True)
            sums = torch.segment_reduce(s["grad_y"][part].double(), "sum", lengths=run, axis=0)
            grad[names] += sums * case["scale"]
        out["grad_weight"] = grad
    return out


def _exact_experts(s, case):
    """Token by token and slot by slot, given the plan; the plan itself is whole numbers, held to the plain form's."""
    n, k, align = case["tokens"], case["top_k"], case["align"]
    names = s["experts"].cpu().numpy()
    keep = np.ones(n, bool) if s["mask"] is None else s["mask"].cpu().numpy()
    at, begin = np.full((n, k), -1, np.int64), 0
    for e in range(case["experts"]):
        t, j = np.nonzero((names == e) & keep[:, None])  # in the order of tokens, then slots
        at[t, j] = begin + np.arange(len(t))
        begin += -(-len(t) // align) * align
    at = torch.from_numpy(at).to(device)
    x, w, rows = s["x"].double(), s["weights"].double(), s["rows"]
    out = {"positions": None, "slots": None, "counts": None, "offsets": None,
           "rows": torch.zeros(_rows(case), case["hidden"], dtype=torch.float64, device=device),
           "y": torch.zeros(n, case["hidden"], dtype=torch.float64, device=device)}
    if case["what"] == "train":
        dy = s["grad_y"].double()
        out["grad_weights"] = torch.zeros(n, k, dtype=torch.float64, device=device)
        out["grad_rows"], out["grad_x"] = torch.zeros_like(out["rows"]), torch.zeros_like(out["y"])
    for j in range(k):
        t = (at[:, j] >= 0).nonzero().squeeze(1)
        p = at[t, j]
        got = rows[p].double()
        out["rows"][p] = x[t]
        out["y"][t] += got * w[t, j, None]
        if case["what"] == "train":
            out["grad_weights"][t, j] = torch.einsum("rh,rh->r", got, dy[t])
            out["grad_rows"][p] = dy[t] * w[t, j, None]
            out["grad_x"][t] += s["grad_rows"][p].double()
    return out


def exact(case, seed):
    return {"norm": _exact_norm, "embedding": _exact_embedding, "experts": _exact_experts}[case["op"]](_inputs(case, seed), case)
