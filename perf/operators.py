"""The routing, balance and gradient-clipping operators as one training or serving step calls them: inputs, the
calls, their plain form in elementary torch operations, and their definition in 64 bits.

Kinds of case:
  route      logits -> expert ids and gates (what the grouping and the combine read);
  balance    the same pass with its per-expert statistics, and the balance loss from them;
  route_bwd  gradients of gates and balance loss -> gradient of the logits;
  clip       global norm of a list of gradients, and the gradients clipped by it.
"""

import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _router(op, T, E, k, dtype="f32", score="softmax", renorm=True, scale=1.0, bias=False, padded=0.0, closed=0.0,
            alpha=0.0, **more):
    """padded: share of the rows that are padding; closed: share of the experts masked by a -inf logit."""
    return dict(op=op, T=T, E=E, k=k, dtype=dtype, score=score, renorm=renorm, scale=scale, bias=bias,
                padded=padded, closed=closed, alpha=alpha, **more)


def listed():
    return [
        # one token of one request being decoded: latency
        _router("route", 1, 384, 8, name="route-one-token"),
        # a decode batch routed by biased sigmoid scores (the balancing that needs no loss)
        _router("route", 512, 384, 8, score="sigmoid", scale=2.5, bias=True, name="route-decode-bias"),
        # a training batch with padding, biased sigmoid scores
        _router("route", 32768, 384, 8, score="sigmoid", scale=2.5, bias=True, padded=0.1, name="route-share-bias"),
        # the small expert layer's training step: 8 experts, bfloat16 logits
        _router("balance", 4096, 8, 2, dtype="bf16", renorm=False, alpha=0.01, name="balance-small"),
        # one GPU's training batch, 8 of 384 experts
        _router("balance", 32768, 384, 8, alpha=0.001, name="balance-share"),
        # odd sizes: a ragged batch with padding and experts closed
        _router("balance", 8191, 130, 6, dtype="bf16", score="sigmoid", alpha=0.01, padded=0.25, closed=0.05,
                name="balance-ragged"),
        # backward of the small expert layer's routing
        _router("route_bwd", 4096, 8, 2, dtype="bf16", renorm=False, alpha=0.01, name="bwd-small"),
        # backward of one GPU's training batch
        _router("route_bwd", 32768, 384, 8, alpha=0.001, name="bwd-share"),
        # long packed sequences over few experts
        _router("route_bwd", 262144, 64, 6, score="sigmoid", scale=2.5, alpha=0.001, name="bwd-long"),
        # the router's own weight gradient and bias of one layer: a few tensors
        dict(op="clip", sizes="384*4096,384,4096", dtype="f32", mixed=False, clip=0.5, name="clip-router"),
        # a model's many tensors of all sizes in two flat buffers, none aligned
        dict(op="clip", sizes="ragged", tensors=200, most=400000, dtype="f32", mixed=True, clip=0.1, name="clip-many"),
        # the expert share's float32 weight gradients: 48 x 1536 x 4096 of both projections
        dict(op="clip", sizes="48*1536*4096,48*4096*1536,384*4096", dtype="f32", mixed=False, clip=0.5,
             name="clip-share"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "balance", "route_bwd", "clip"])
    if op == "clip":
        n = _log_int(rng, 1, 200)
        return dict(op="clip", sizes="ragged", tensors=n, most=_log_int(rng, 1, min(400000000 // n, 40000000)),
                    dtype=rng.choice(["f32", "bf16"]), mixed=rng.random() < 0.5,
                    clip=rng.choice([0.01, 0.3, 1.0, 5.0]))
    E = rng.choice([_log_int(rng, 1, 1024), 8, 64, 384])
    k = min(E, _log_int(rng, 1, 16))
    score = rng.choice(["softmax", "sigmoid"])
    return _router(op, _log_int(rng, 1, min(262144, (1 << 24) // E)), E, k, dtype=rng.choice(["f32", "bf16"]),
                   score=score, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                   bias=score == "sigmoid" and rng.random() < 0.5, padded=rng.choice([0.0, 0.0, 0.3]),
                   closed=rng.choice([0.0, 0.0, 0.1]), alpha=rng.choice([0.001, 0.01, 0.1]))


def _sizes(case):
    """The tensors' element counts: given, or of all sizes up to `most`, spread over their logarithm."""
    if case["sizes"] != "ragged":
        return [math.prod(int(f) for f in s.split("*")) for s in case["sizes"].split(",")]
    n, most = case["tensors"], case["most"]
    return [max(1, int(most ** (((i * 0.6180339887 + 0.5) % 1.0)))) for i in range(n)]


def _dtypes(case):
    other = "bf16" if case["dtype"] == "f32" else "f32"
    return [DTYPES[other if case["mixed"] and i % 3 == 1 else case["dtype"]] for i in range(len(_sizes(case)))]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 17)
    if case["op"] == "clip":
        return _prepare_clip(case, gen)
    T, E, k = case["T"], case["E"], case["k"]
    # popular experts: an offset falling with the logarithm of an expert's rank, ranks shuffled
    rank = torch.randperm(E, generator=gen, device=DEV).float() + 1
    x = torch.randn(T, E, generator=gen, device=DEV) - 0.3 * torch.log(rank)
    if case["closed"]:
        x[:, torch.rand(E, generator=gen, device=DEV) < case["closed"]] = -math.inf
    s = dict(case=case, logits=x.to(DTYPES[case["dtype"]]), bias=None, token_mask=None)
    if case["bias"]:
        s["bias"] = 0.1 * torch.randn(E, generator=gen, device=DEV)
    if case["padded"]:
        s["token_mask"] = torch.rand(T, generator=gen, device=DEV) >= case["padded"]
    if case["op"] == "route_bwd":
        s["topk_ids"], gate = _route(s)[:2]
        s["dgate"] = torch.randn(T, k, generator=gen, device=DEV) * 1e-3
        s["counts"] = _stats(s, s["topk_ids"])[0]
        s["dloss"] = torch.full((1,), 0.5, device=DEV)
        s["dlogits"] = torch.empty_like(s["logits"])
    else:
        s["out"] = dict(topk_ids=torch.empty(T, k, dtype=torch.int32, device=DEV),
                        gate=torch.empty(T, k, device=DEV))
        if case["op"] == "balance":
            s["out"].update(counts=torch.empty(E + 1, dtype=torch.int64, device=DEV),
                            prob_sum=torch.empty(E, device=DEV))
            s["loss"] = torch.empty(1, device=DEV)
    return s


def _prepare_clip(case, gen):
    """The gradients and their clipped copies are views, one behind the other, of one flat buffer for each type."""
    sizes, types = _sizes(case), _dtypes(case)
    flat, flat_out = {}, {}
    for t in sorted(set(types), key=str):
        n = sum(m for m, u in zip(sizes, types) if u == t)
        flat[t] = torch.empty(n, dtype=t, device=DEV).normal_(0.0, 1e-2, generator=gen)
        flat_out[t] = torch.empty_like(flat[t])
    at, grads, outs = dict.fromkeys(flat, 0), [], []
    for m, t in zip(sizes, types):
        grads.append(flat[t][at[t]:at[t] + m])
        outs.append(flat_out[t][at[t]:at[t] + m])
        at[t] += m
    # clip: the bound as a share of the norm such gradients have
    s = dict(case=case, grads=grads, outs=outs, flat=flat, flat_out=flat_out,
             max_norm=case["clip"] * 1e-2 * math.sqrt(sum(sizes)), norm=torch.empty(1, device=DEV),
             sumsq=torch.empty(1, dtype=torch.float64, device=DEV))
    if own:                                   # the handles a training program makes once of its gradients
        import precision_moe_numerics_nvfp4_amd as nv
        s["grads"], s["outs"] = nv.GradList(grads), nv.GradList(outs)
    return s


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "clip":
        return _clip(s)
    if c["op"] == "route_bwd":
        return dict(dlogits=_route_bwd(s))
    ids, gate, score = _route(s)
    if c["op"] == "route":
        return dict(topk_ids=ids, gate=gate)
    counts, total = _stats(s, ids, _probabilities(score, s))
    return dict(topk_ids=ids, gate=gate, counts=counts, prob_sum=total, loss=_loss(c, counts, total))


def _run_own(s, c):
    import precision_moe_numerics_nvfp4_amd as nv
    if c["op"] == "clip":
        nv.moe_grad_sumsq(s["grads"], sumsq=s["sumsq"])
        nv.moe_grad_clip(s["grads"], s["sumsq"], s["max_norm"], outs=s["outs"], norm=s["norm"])
        return dict(norm=s["norm"], flat=[s["flat_out"][t] for t in sorted(s["flat_out"], key=str)])
    how = dict(score=c["score"], renorm=c["renorm"], scale=c["scale"])
    if c["op"] == "route_bwd":
        nv.moe_route_bwd(s["logits"], s["topk_ids"], s["dgate"], counts=s["counts"], alpha=c["alpha"],
                         dloss=s["dloss"], dlogits=s["dlogits"], **how)
        return dict(dlogits=s["dlogits"])
    o = nv.moe_route(s["logits"], c["k"], bias=s["bias"], token_mask=s["token_mask"], stats=c["op"] == "balance",
                     out=s["out"], **how)
    if c["op"] == "route":
        return dict(topk_ids=o["topk_ids"], gate=o["gate"])
    nv.moe_balance_loss(o["counts"], o["prob_sum"], c["k"], c["alpha"], loss=s["loss"])
    return dict(topk_ids=o["topk_ids"], gate=o["gate"], counts=o["counts"], prob_sum=o["prob_sum"], loss=s["loss"])


# ------------------------------------------------------------ the plain form

def _scores(x, score):
    """Scores of float32 logits (0 in rows with no expert)."""
    if score == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True).clamp_min(-1e30))
        return e / e.sum(1, keepdim=True).clamp_min(1e-38)
    return 1 / (1 + torch.exp(-x))


def _probabilities(scores, s):
    """What the balance loss sums: scores whose row sums to one, 0 in the rows that are padding."""
    p = scores if s["case"]["score"] == "softmax" else scores / scores.sum(1, keepdim=True).clamp_min(1e-38)
    return p if s["token_mask"] is None else p * s["token_mask"][:, None]


def _route(s):
    """ids int32 [T, k], gates [T, k], scores [T, E]."""
    c, k = s["case"], s["case"]["k"]
    x = s["logits"].float()
    key = x
    if s["bias"] is not None:                    # next to a border 32 bits would choose another expert
        key = 1 / (1 + torch.exp(-x.double())) + s["bias"].double()
    shut = x == -math.inf
    if s["token_mask"] is not None:
        shut = shut | ~s["token_mask"][:, None]
    key, ids = key.masked_fill(shut, -math.inf).sort(dim=1, descending=True, stable=True)
    key, ids = key[:, :k], ids[:, :k]
    there = key > -math.inf
    score = _scores(x, c["score"])
    w = score.gather(1, ids)
    if c["renorm"] and c["score"] == "softmax":  # the same quotient, from the selected logits: no tiny sums
        top = x.gather(1, ids).masked_fill(~there, -math.inf)
        w = torch.exp(top - top.amax(1, keepdim=True).clamp_min(-1e30))
    w = w * there
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-38)
    return torch.where(there, ids, -1).int(), w * c["scale"], score


def _stats(s, ids, p=None):
    """Pairs on each expert with the tokens that have one behind them, and each expert's summed probability."""
    E = s["case"]["E"]
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    flat = ids.reshape(-1).long()
    counts.scatter_add_(0, torch.where(flat < 0, E, flat), torch.ones_like(flat))
    counts[E] = (ids[:, 0] >= 0).sum()
    return counts, None if p is None else p.sum(0, dtype=torch.float64).float()


def _loss(c, counts, total):
    E = c["E"]
    n = counts[E:].double().clamp_min(1)
    return (c["alpha"] * E * ((counts[:E] / (n * c["k"])) * (total.double() / n)).sum(0, keepdim=True)).float()


def _route_bwd(s):
    c = s["case"]
    E, ids = c["E"], s["topk_ids"].long()
    x = s["logits"].float()
    score = _scores(x, c["score"])
    there = ids >= 0
    at = torch.where(there, ids, 0)
    u = s["dgate"] * c["scale"] * there                    # gradient of the selected scores before the scale
    n = s["counts"][E:].double().clamp_min(1)
    a = (c["alpha"] * E * s["counts"][:E].double() / (c["k"] * n * n)).float() * s["dloss"]
    live = there[:, :1]
    if c["score"] == "softmax":
        p = score
        dx = p * (a - (p * a).sum(1, keepdim=True)) * live
        if c["renorm"]:
            top = x.gather(1, at).masked_fill(~there, -math.inf)
            q = torch.exp(top - top.amax(1, keepdim=True).clamp_min(-1e30)) * there
            q = q / q.sum(1, keepdim=True).clamp_min(1e-38)
            dx.scatter_add_(1, at, q * (u - (q * u).sum(1, keepdim=True)))
        else:
            q = p.gather(1, at) * there
            dx.scatter_add_(1, at, q * u)
            dx -= p * (q * u).sum(1, keepdim=True)
    else:
        total = score.sum(1, keepdim=True).clamp_min(1e-38)
        p = score / total
        ds = (a - (p * a).sum(1, keepdim=True)) / total * live
        if c["renorm"]:
            q = score.gather(1, at) * there
            part = q.sum(1, keepdim=True).clamp_min(1e-38)
            u = (u - (u * q).sum(1, keepdim=True) / part) / part * there
        ds.scatter_add_(1, at, u)
        dx = ds * score * (1 - score)
    return dx.to(s["logits"].dtype)


def _clip(s):
    sumsq = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum()
    norm = sumsq.sqrt().float()
    coef = (s["max_norm"] / (norm + EPS)).clamp_max(1.0)
    done = [o.copy_(g.float() * coef) for g, o in zip(s["grads"], s["outs"])]
    assert len(done) == len(s["outs"])
    return dict(norm=norm.reshape(1), flat=[s["flat_out"][t] for t in sorted(s["flat_out"], key=str)])


# ------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "clip":
        n = [m * (4 if t == torch.float32 else 2) for m, t in zip(_sizes(case), _dtypes(case))]
        return {"bytes": 2 * sum(n), "flops": 3 * sum(_sizes(case))}
    T, E, k = case["T"], case["E"], case["k"]
    row = E * (4 if case["dtype"] == "f32" else 2)
    if case["op"] == "route_bwd":
        return {"bytes": T * (2 * row + 8 * k) + 8 * (E + 1), "flops": 8 * T * E}
    more = 12 * E + 12 if case["op"] == "balance" else 0
    return {"bytes": T * (row + 8 * k) + more, "flops": 4 * T * E}


# ------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        flat = s["flat"]
        norm = math.sqrt(sum(float(f.double().pow(2).sum()) for f in flat.values()))
        share = min(1.0, s["max_norm"] / (norm + EPS))
        return dict(norm=torch.tensor([norm], dtype=torch.float64),
                    flat=[flat[t].double().mul_(share) for t in sorted(flat, key=str)])
    x = s["logits"].double()
    T, E, k = case["T"], case["E"], case["k"]
    soft = case["score"] == "softmax"
    shut = torch.isinf(x)
    if s["token_mask"] is not None:
        shut |= torch.logical_not(s["token_mask"]).unsqueeze(1)
    live = torch.logical_not(shut.all(1))
    # scores as exp of a logarithm, padding rows as if all their logits were 0 and dropped behind
    y = torch.where(live.unsqueeze(1), torch.where(shut, -math.inf, x), 0.0)
    log_s = y - torch.logsumexp(y, 1, keepdim=True) if soft else -torch.log1p(torch.exp(-y))
    score = torch.exp(log_s) * live.unsqueeze(1)
    prob = score if soft else score / torch.where(live, score.sum(1), 1.0).unsqueeze(1)
    if case["op"] == "route_bwd":
        return dict(dlogits=_exact_bwd(s, case, score, prob, soft))
    key = x if s["bias"] is None else torch.sigmoid(x) + s["bias"].double()
    order = torch.argsort(-torch.where(shut, -math.inf, key), dim=1, stable=True)[:, :k]
    picked = torch.zeros(T, E, dtype=torch.float64, device=x.device).scatter_(1, order, 1.0) * ~shut
    part = (score * picked).sum(1, keepdim=True)
    gate = score * picked * case["scale"]
    if case["renorm"]:
        gate = gate / torch.where(part > 0, part, 1.0)
    gate = torch.gather(gate, 1, order)
    if case["op"] == "route":
        return dict(topk_ids=None, gate=gate)
    total, pairs = prob.sum(0), picked.sum(0)
    n = max(1.0, float(live.sum()))
    loss = case["alpha"] * E / (n * n * k) * torch.dot(pairs, total)
    return dict(topk_ids=None, gate=gate, counts=None, prob_sum=total, loss=loss.reshape(1))


def _exact_bwd(s, case, score, prob, soft):
    """J^T of the gates and of the loss: the derivatives of the scores first, then of the logits."""
    T, E, k = case["T"], case["E"], case["k"]
    ids = s["topk_ids"].long()
    dense = torch.zeros(T, E + 1, dtype=torch.float64, device=score.device)
    hit = dense.scatter(1, torch.where(ids < 0, E, ids), 1.0)[:, :E]
    up = dense.scatter(1, torch.where(ids < 0, E, ids), s["dgate"].double() * case["scale"])[:, :E]
    n = max(1.0, float(s["counts"][E]))
    a = case["alpha"] * E * s["counts"][:E].double() / (k * n * n) * float(s["dloss"])
    some = hit.sum(1, keepdim=True) > 0
    d_prob = torch.where(some, a.expand(T, E), 0.0)
    if case["renorm"]:
        part = (score * hit).sum(1, keepdim=True)
        part = torch.where(part > 0, part, 1.0)
        up = hit * (up - (up * score * hit).sum(1, keepdim=True) / part) / part
    if soft:
        d_score = up + d_prob
        dx = score * (d_score - (d_score * score).sum(1, keepdim=True))
    else:
        whole = score.sum(1, keepdim=True)
        d_score = up + (d_prob - (d_prob * prob).sum(1, keepdim=True)) / torch.where(whole > 0, whole, 1.0)
        dx = d_score * score * (1 - score)
    return dx
