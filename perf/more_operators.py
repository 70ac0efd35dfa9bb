"""MXFP4 (E2M1 elements, one E8M0 scale for 32) as a training or serving step meets it, and the expert layer for a
few tokens: inputs, the calls, their plain form in elementary torch operations, and their definition in 64 bits.

Kinds of case:
  quantize  rows -> MXFP4, and back to values (what a step keeps, and what it stands for);
  product   grouped product of MXFP4 rows, gathered by token, with MXFP4 expert weights;
  requant   saved MXFP4 rows or weights -> transposed MXFP8 with stochastic rounding (the gradient products' operand),
            read back to values;
  tokens    logits and activations of a few tokens -> the whole layer's output: selection, gates, up-projection,
            activation, down-projection, weighted sum; weights in MXFP4 or NVFP4.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _quantize(rows, cols, dtype, live=1.0, **more):
    """live: share of the rows that the device count covers (1: no count is given)."""
    return dict(op="quantize", rows=rows, cols=cols, dtype=dtype, live=live, **more)


def _product(T, k, experts, local, K, N, routing="uniform", dtype="bf16", **more):
    return dict(op="product", T=T, k=k, experts=experts, local=local, K=K, N=N, routing=routing, dtype=dtype, **more)


def _requant(kind, T, k, experts, local, K, N, routing="uniform", **more):
    """kind 'acts': the routed rows' [K]; 'weights': `local` experts of [N, K]."""
    return dict(op="requant", kind=kind, T=T, k=k, experts=experts, local=local, K=K, N=N, routing=routing, **more)


def _tokens(T, k, experts, local, K, F, fmt, act="silu", gated=False, score="softmax", renorm=True, scale=1.0,
            bias=False, padded=0.0, logits="f32", **more):
    return dict(op="tokens", T=T, k=k, experts=experts, local=local, K=K, F=F, fmt=fmt, act=act, gated=gated,
                score=score, renorm=renorm, scale=scale, bias=bias, padded=padded, logits=logits, **more)


def listed():
    return [
        # a decode batch's activations: latency
        _quantize(512, 4096, "bf16", name="quantize-decode"),
        # the routed intermediate of a capacity-sized buffer, float32, an odd row count, a fifth of it live
        _quantize(40009, 1536, "f32", live=0.2, name="quantize-hidden"),
        # a long stream of activations, 1 GiB
        _quantize(262144, 2048, "bf16", name="quantize-stream"),
        # a decode batch: 48 local experts with about ten rows each, weight streaming
        _product(512, 8, 384, 48, 4096, 1536, name="product-decode"),
        # the small expert layer: 8 experts of about 1024 rows, float32 output
        _product(4096, 2, 8, 8, 1024, 2048, dtype="f32", name="product-small"),
        # one GPU's share of a training batch, 8 of 384 experts, popularity falling with the rank
        _product(32768, 8, 384, 48, 4096, 1536, routing="zipf", name="product-share"),
        # the small layer's saved activations
        _requant("acts", 4096, 2, 8, 8, 1024, 2048, name="requant-small-acts"),
        # the expert share's up-projection weights
        _requant("weights", 0, 8, 384, 48, 4096, 1536, name="requant-share-weights"),
        # one token of one request being decoded, 8 of 48 experts, NVFP4 weights: latency
        _tokens(1, 8, 48, 48, 4096, 1536, "nvfp4", name="tokens-one"),
        # a few requests, gated activation, MXFP4 weights, biased sigmoid scores
        _tokens(7, 6, 48, 48, 4096, 2048, "mxfp4", gated=True, score="sigmoid", scale=2.5, bias=True,
                name="tokens-few-gated"),
        # the small layer, 16 requests on 8 experts, bfloat16 logits
        _tokens(16, 2, 8, 8, 1024, 2048, "mxfp4", act="relu2", logits="bf16", renorm=False, name="tokens-small"),
        # the largest batch on one GPU's share of the experts, some requests padding
        _tokens(64, 8, 384, 48, 4096, 1536, "nvfp4", padded=0.1, name="tokens-share"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "requant", "tokens"])
    if op == "quantize":
        cols = 32 * _log_int(rng, 1, 256)
        return _quantize(_log_int(rng, 1, (1 << 28) // cols), cols, rng.choice(["f32", "bf16"]),
                         live=rng.choice([1.0, 1.0, 0.6]))
    if op == "tokens":
        E = rng.choice([8, 48, 64, _log_int(rng, 4, 384)])
        local = rng.choice([E, max(1, E // 2), max(1, E // 8)])
        score = rng.choice(["softmax", "sigmoid"])
        K = 128 * _log_int(rng, 1, 32)
        F = 128 * _log_int(rng, 1, 16)
        while local * K * F > 48 * 4096 * 2048:
            local = max(1, local // 2)
        return _tokens(_log_int(rng, 1, 64), min(E, _log_int(rng, 1, 8)), E, local, K, F,
                       rng.choice(["mxfp4", "nvfp4"]), act=rng.choice(["none", "relu2", "silu"]),
                       gated=rng.random() < 0.5, score=score, renorm=rng.random() < 0.6,
                       scale=rng.choice([1.0, 2.5]), bias=score == "sigmoid" and rng.random() < 0.5,
                       padded=rng.choice([0.0, 0.0, 0.3]), logits=rng.choice(["f32", "bf16"]))
    E = rng.choice([8, 48, _log_int(rng, 1, 64)])
    experts = E * rng.choice([1, 1, 8])
    k = min(experts, _log_int(rng, 1, 8))
    K, N = 128 * _log_int(rng, 1, 32), 128 * _log_int(rng, 1, 16)
    routing = rng.choice(["uniform", "zipf"])
    if op == "requant":
        kind = rng.choice(["acts", "weights"])
        while kind == "weights" and E * K * N > 48 * 4096 * 1536:
            E = max(1, E // 2)
        return _requant(kind, _log_int(rng, 1, 4096) if kind == "acts" else 0, k, max(experts, E), E, K, N, routing)
    # the rows that a product may have next to the largest listed one's work, over every expert's
    most = max(1, min(32768, 31596 * 4096 * 1536 // (K * N * k)))
    return _product(_log_int(rng, 1, most), k, experts, E, K, N, routing, dtype=rng.choice(["f32", "bf16"]))


# ------------------------------------------------------------ inputs

def _randn(gen, *shape, std=1.0, outliers=False):
    x = torch.empty(shape, device=DEV).normal_(0.0, std, generator=gen)
    if outliers:                                  # one element in a thousand fifty times the others
        x = torch.where(torch.rand(shape, generator=gen, device=DEV) < 1e-3, x * 50, x)
    return x


def _route_ids(case, gen):
    """Distinct experts of each token, the popular ones dealt round the ranks: int32 [T, k], and the first local one."""
    T, k, E, local = case["T"], case["k"], case["experts"], case["local"]
    logp = torch.zeros(E, device=DEV)
    if case["routing"] == "zipf":
        logp = -1.1 * torch.log(torch.arange(1, E + 1, device=DEV).float())
    u = torch.rand(T, E, generator=gen, device=DEV).clamp_(1e-7, 1 - 1e-7)
    rank = (logp - torch.log(-torch.log(u))).topk(k, dim=1).indices
    ranks = max(1, E // local)
    ids = (rank % ranks) * local + rank // ranks if E == ranks * local else rank
    e0 = (ranks // 2 - 1) * local if ranks > 2 else 0
    return ids.int(), e0


def _group(ids, e0, local):
    """Rows by local expert, in the order of the pairs: row_token int32 [T k] (-1 past the last row), and the experts'
    row counts."""
    flat = ids.reshape(-1).long() - e0
    here = (flat >= 0) & (flat < local)
    key = torch.where(here, flat, torch.full_like(flat, local))
    order = key.sort(stable=True).indices
    counts = torch.bincount(key, minlength=local + 1)[:local]
    row_token = (order // ids.shape[1]).int()
    row_token[int(counts.sum()):] = -1
    return row_token, counts


def _offsets(counts, align=1):
    c = (counts + align - 1) // align * align
    return torch.cat([c.new_zeros(1), c.cumsum(0)])


def _mxfp4(x):
    """Codes [rows, cols/2] and scales [rows, cols/32] of x: operands that a program already holds."""
    b = x.float().reshape(x.shape[0], -1, 32)
    m, q = torch.frexp(b.abs().amax(2))
    e = torch.where(m <= 0.75, q - 3, q - 2).clamp(-127, 127)
    y = torch.ldexp(b, -e[..., None])
    return _codes(y), (e + 127).to(torch.uint8)


def _codes(y):
    """Nearest E2M1 code of blocks of values up to 6, two to a byte (the first in the low half)."""
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | ((y < 0).to(torch.uint8) << 3)).reshape(y.shape[0], -1)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _nvfp4(x, local):
    """Codes, E4M3 scales of 16 and an outer scale per expert of x [local * rows, cols]."""
    outer = x.reshape(local, -1).abs().amax(1) / 2688
    b = x.reshape(local, -1, 16)
    s = (b.abs().amax(2) / (6 * outer[:, None])).clamp(2 ** -9, 448).to(torch.float8_e4m3fn)
    y = (b / (s.float() * outer[:, None])[..., None]).clamp(-6, 6)
    return (_codes(y.reshape(x.shape[0], -1, 16)), s.view(torch.uint8).reshape(x.shape[0], -1), outer)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 9176 + 23)
    return {"quantize": _prepare_quantize, "product": _prepare_product, "requant": _prepare_requant,
            "tokens": _prepare_tokens}[case["op"]](case, gen, int(seed))


def _prepare_quantize(c, gen, seed):
    x = _randn(gen, c["rows"], c["cols"], outliers=True).to(DTYPES[c["dtype"]])
    s = dict(case=c, x=x, offsets=None)
    n = c["rows"]
    if c["live"] < 1:
        n = int(c["rows"] * c["live"])
        s["offsets"] = torch.tensor([0, n // 3, n], device=DEV)
    s["live"] = n
    s["codes"] = torch.zeros(c["rows"], c["cols"] // 2, dtype=torch.uint8, device=DEV)
    s["scales"] = torch.zeros(c["rows"], c["cols"] // 32, dtype=torch.uint8, device=DEV)
    return s


def _prepare_product(c, gen, seed):
    ids, e0 = _route_ids(c, gen)
    row_token, counts = _group(ids, e0, c["local"])
    a = _mxfp4(_randn(gen, c["T"], c["K"]).bfloat16())
    w = _mxfp4(_randn(gen, c["local"] * c["N"], c["K"], std=0.02).bfloat16())
    return dict(case=c, a=a, w=w, row_token=row_token, offsets=_offsets(counts), counts=counts.tolist(),
                y=torch.zeros(row_token.numel(), c["N"], dtype=DTYPES[c["dtype"]], device=DEV))


def _prepare_requant(c, gen, seed):
    s = dict(case=c, seed=0x5EED0000 + seed)
    if c["kind"] == "weights":
        s["q"] = _mxfp4(_randn(gen, c["local"] * c["N"], c["K"], std=0.02).bfloat16())
        s["offsets"] = s["padded"] = torch.arange(c["local"] + 1, device=DEV) * c["N"]
        s["P"], shape, s["row_token"], s["tag"] = c["local"] * c["N"], (c["local"] * c["K"], c["N"]), None, 1
    else:
        ids, e0 = _route_ids(c, gen)
        s["row_token"], counts = _group(ids, e0, c["local"])
        s["q"] = _mxfp4(_randn(gen, c["T"], c["K"]).bfloat16())
        s["offsets"], s["padded"] = _offsets(counts), _offsets(counts, 32)
        s["P"] = (ids.numel() + 31 * c["local"] + 31) // 32 * 32
        shape, s["tag"] = (c["K"], s["P"]), 0
    s["out"] = (torch.zeros(shape, dtype=torch.uint8, device=DEV),
                torch.zeros(shape[0], shape[1] // 32, dtype=torch.uint8, device=DEV))
    return s


def _prepare_tokens(c, gen, seed):
    T, E, local, K, F = c["T"], c["experts"], c["local"], c["K"], c["F"]
    quantize = _mxfp4 if c["fmt"] == "mxfp4" else lambda w: _nvfp4(w, local)
    s = dict(case=c, x=_randn(gen, T, K).bfloat16(),
             logits=(_randn(gen, T, E) - 0.2 * torch.log(torch.arange(1, E + 1, device=DEV).float())).to(
                 DTYPES[c["logits"]]),
             w1=quantize(_randn(gen, local * F * (2 if c["gated"] else 1), K, std=0.02)),
             w2=quantize(_randn(gen, local * K, F, std=0.02)),
             e0=(E // local // 2 - 1) * local if E >= 3 * local else 0, bias=None, token_mask=None)
    if c["bias"]:
        s["bias"] = 0.1 * _randn(gen, E)
    if c["padded"]:
        s["token_mask"] = torch.rand(T, generator=gen, device=DEV) >= c["padded"]
    s["out"] = dict(out=torch.empty(T, K, dtype=torch.bfloat16, device=DEV),
                    topk_ids=torch.empty(T, c["k"], dtype=torch.int32, device=DEV),
                    gate=torch.empty(T, c["k"], device=DEV))
    return s


# ------------------------------------------------------------ the calls

def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"quantize": _quantize_plain, "product": _product_plain, "requant": _requant_plain,
            "tokens": _tokens_plain}[c["op"]](s, c)


def _run_own(s, c):
    import precision_moe_numerics_nvfp4_amd as nv
    if c["op"] == "quantize":
        nv.mxfp4_quantize(s["x"], offsets=s["offsets"], codes=s["codes"], scales=s["scales"])
        return nv.mxfp4_dequantize(s["codes"], s["scales"], out_dtype=s["x"].dtype)
    if c["op"] == "product":
        return nv.moe_fwd_grouped_gemm_mxfp4(*s["a"], *s["w"], s["offsets"], row_token=s["row_token"], y=s["y"])
    if c["op"] == "requant":
        q, e = nv.mxfp8_requant_sr_mxfp4(*s["q"], s["offsets"], s["padded"], s["P"], s["seed"], s["tag"],
                                         rows_per_group=c["N"] if c["kind"] == "weights" else None,
                                         row_token=s["row_token"], out=s["out"][0], out_e8=s["out"][1])
        return nv.mxfp8_dequantize(q, e, out_dtype=torch.bfloat16)
    return nv.moe_ffn_tokens(s["x"], s["logits"], c["k"], s["w1"], s["w2"], act=c["act"], gated=c["gated"],
                             score=c["score"], renorm=c["renorm"], scale=c["scale"], bias=s["bias"],
                             token_mask=s["token_mask"], e0=s["e0"], out=s["out"])


# ------------------------------------------------------------ the plain form

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _values(q):
    """float32 values of (codes, scales) in MXFP4, or (codes, scales, outer of each expert) in NVFP4."""
    codes, scales = q[0], q[1]
    v = torch.tensor(E2M1, device=codes.device)[torch.stack([codes & 15, codes >> 4], 2).int()]
    v = v.reshape(codes.shape[0], scales.shape[1], -1)
    if len(q) == 2:
        return torch.ldexp(v, scales.int()[..., None] - 127).reshape(codes.shape[0], -1)
    v = (v * scales.view(torch.float8_e4m3fn).float()[..., None]).reshape(q[2].numel(), -1)
    return (v * q[2][:, None]).reshape(codes.shape[0], -1)


def _quantize_plain(s, c):
    """Blocks of 32 to the E2M1 grid under the smallest power of two that holds them, back at full width."""
    b = s["x"].float().reshape(c["rows"], -1, 32)
    m, q = torch.frexp(b.abs().amax(2, keepdim=True))
    e = torch.where(m <= 0.75, q - 3, q - 2).clamp(-127, 127)
    y = torch.ldexp(b, -e)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    v = torch.ldexp(torch.round(a / step) * step * torch.sign(y), e).reshape(c["rows"], c["cols"])
    v = v * (torch.arange(c["rows"], device=v.device) < s["live"])[:, None]
    return v.to(s["x"].dtype)


def _product_plain(s, c):
    """The rows in tiles of one expert each, one product over the tiles."""
    counts = s["offsets"].diff()
    most = max(s["counts"] + [1])
    h = 256 if most > 256 else 1 << (most - 1).bit_length()
    tiles = (counts + h - 1) // h
    n = sum((v + h - 1) // h for v in s["counts"])
    if n == 0:
        return torch.zeros_like(s["y"])
    expert = torch.repeat_interleave(torch.arange(c["local"], device=counts.device), tiles, output_size=n)
    first = s["offsets"][expert] + h * (torch.arange(n, device=counts.device) - (tiles.cumsum(0) - tiles)[expert])
    row = first[:, None] + torch.arange(h, device=counts.device)
    inside = row < s["offsets"][expert + 1][:, None]
    row = torch.where(inside, row, 0)
    a = _values(s["a"])[s["row_token"][row].long()]
    w = _values(s["w"]).reshape(c["local"], c["N"], c["K"])[expert]
    y = torch.zeros_like(s["y"])
    y[row[inside]] = torch.bmm(a, w.transpose(1, 2))[inside].to(y.dtype)
    return y


M32 = 0xFFFFFFFF


def _mul32(a, b):
    """(high, low) words of the product of 32-bit words held in 64 bits."""
    p, q = (a & 0xFFFF) * b, (a >> 16) * b
    q = q + (p >> 16)
    return q >> 16, ((q & 0xFFFF) << 16) | (p & 0xFFFF)


def _draws(n8, seed, tag):
    """The 16-bit draws 0 .. 8 n8 - 1 (Philox4x32 of 10 rounds: eight draws to a counter)."""
    q = torch.arange(n8, device=DEV)
    a, b, x, y = q & M32, q >> 32, torch.full_like(q, tag), torch.zeros_like(q)
    k0, k1 = seed & M32, seed >> 32
    for r in range(10):                           # the generator's rounds
        (h0, l0), (h1, l1) = _mul32(a, 0xD2511F53), _mul32(x, 0xCD9E8D57)
        a, b, x, y = h1 ^ b ^ ((k0 + r * 0x9E3779B9) & M32), l1, h0 ^ y ^ ((k1 + r * 0xBB67AE85) & M32), l0
    w = torch.stack([a, b, x, y], 1)
    return torch.stack([w & 0xFFFF, w >> 16], 2).reshape(-1).int()


def _requant_plain(s, c):
    """Transpose, block exponent, stochastic rounding to E4M3, the values it stands for."""
    v, P = _values(s["q"]), s["P"]
    if c["kind"] == "weights":
        t = v.t().contiguous()
    else:
        # output column of each row: its expert's padded start, then its place in the expert
        n = sum_rows = int(s["case"]["T"] * s["case"]["k"])
        r = torch.arange(n, device=v.device)
        live = r < s["offsets"][-1]
        g = (torch.searchsorted(s["offsets"], r, right=True) - 1).clamp_max(c["local"] - 1)
        col = torch.where(live, s["padded"][g] + r - s["offsets"][g], P)
        t = torch.zeros(c["K"], P + 1, device=v.device)
        t[:, col] = (v[s["row_token"].clamp_min(0).long()] * live[:, None]).t()
        t = t[:, :P].contiguous()
    b = t.reshape(c["K"], P // 32, 32)
    m, q = torch.frexp(b.abs().amax(2, keepdim=True))
    e = torch.where(m <= 0.875, q - 9, q - 8).clamp(-127, 127)
    a = torch.ldexp(b.abs(), -e)
    gap = torch.ldexp(torch.ones_like(a), (torch.frexp(a).exponent - 1).clamp_min(-6) - 3)
    low = torch.floor(a / gap)
    part = ((a / gap - low) * 65536).int()
    u = _draws(c["K"] * P // 8, s["seed"], s["tag"]).reshape(b.shape)
    a = (low + ((u + part) >> 16)) * gap
    v = (torch.ldexp(a, e) * torch.sign(b)).reshape(c["K"], P)
    if c["kind"] == "weights":                    # each expert's block by itself
        v = v.reshape(c["K"], c["local"], c["N"]).transpose(0, 1).reshape(c["local"] * c["K"], c["N"])
    return v.bfloat16()


def _select(s, c):
    """ids int32 [T, k] and gates [T, k], by score (with a bias: by their sum in 64 bits), lower index first."""
    x = s["logits"].float()
    key = x if s["bias"] is None else 1 / (1 + torch.exp(-x.double())) + s["bias"].double()
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    if c["score"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    gate = p.gather(1, ids)
    if c["renorm"]:
        gate = gate / gate.sum(1, keepdim=True)
    gate, ids = gate * c["scale"], ids.int()
    if s["token_mask"] is not None:
        gate = gate * s["token_mask"][:, None]
        ids = torch.where(s["token_mask"][:, None], ids, -1)
    return ids, gate


def _activate(h, act):
    if act == "silu":
        return h / (1 + torch.exp(-h))
    return h.clamp_min(0).square() if act == "relu2" else h


def _tokens_plain(s, c):
    """Pair by pair where that reads fewer experts, else every expert over every token with the others' gates zero."""
    T, k, local, K, F = c["T"], c["k"], c["local"], c["K"], c["F"]
    ids, gate = _select(s, c)
    expert = ids.long() - s["e0"]
    here = (expert >= 0) & (expert < local) & (ids >= 0)
    g = gate * here
    expert = torch.where(here, expert, 0)
    x = s["x"].float()
    rows = F * (2 if c["gated"] else 1)
    if T * k <= local:
        e = expert.reshape(-1)
        w1, w2 = ([v.reshape(local, -1, *v.shape[1:])[e].flatten(0, 1) if v.dim() > 1 else v[e] for v in w]
                  for w in (s["w1"], s["w2"]))
        n, x, g = T * k, x.repeat_interleave(k, 0)[:, None], g.reshape(-1, 1, 1)
    else:
        w1, w2, n = s["w1"], s["w2"], local
        x = x[None].expand(local, T, K)
        g = torch.zeros(T, local, device=x.device).scatter_add_(1, expert, g).t()[..., None]
    h = torch.bmm(x, _values(w1).reshape(n, rows, K).transpose(1, 2))
    h = _activate(h[..., :F], c["act"]) * h[..., F:] if c["gated"] else _activate(h, c["act"])
    y = torch.bmm(h * g, _values(w2).reshape(n, K, F).transpose(1, 2))
    y = y.reshape(T, k, K).sum(1) if T * k <= local else y.sum(0)
    return dict(out=y.bfloat16(), topk_ids=ids, gate=gate)


# ------------------------------------------------------------ what a pass cannot do without

def _rows_here(c):
    return c["T"] * c["k"] * c["local"] / c["experts"]


def work(c):
    if c["op"] == "quantize":
        n, size = c["rows"] * c["cols"] * c["live"], 2 if c["dtype"] == "bf16" else 4
        return {"bytes": int(n * (size + 17 / 32)) + int(c["rows"] * c["cols"] * (17 / 32 + size)), "flops": int(4 * n)}
    if c["op"] == "product":
        # a popularity that falls with the rank leaves this share about the uniform one's rows
        m, size = _rows_here(c), 2 if c["dtype"] == "bf16" else 4
        hit = c["local"] * (1 - (1 - c["k"] / c["experts"]) ** c["T"])
        rows = min(c["T"], m)
        return {"bytes": int((rows + hit * c["N"]) * c["K"] * 17 / 32 + m * c["N"] * size + 4 * m),
                "flops": int(2 * m * c["N"] * c["K"])}
    if c["op"] == "requant":
        if c["kind"] == "weights":
            n = c["local"] * c["N"] * c["K"]
            return {"bytes": int(n * (17 / 32 + 2 * 33 / 32 + 2)), "flops": 8 * n}
        n = int(_rows_here(c)) * c["K"]
        return {"bytes": int(min(c["T"], _rows_here(c)) * c["K"] * 17 / 32 + n * 33 / 32 +
                             c["T"] * c["k"] * c["K"] * (33 / 32 + 2)), "flops": 8 * n}
    hit = c["local"] * (1 - (1 - c["k"] / c["experts"]) ** (c["T"] * (1 - c["padded"])))
    per = c["K"] * c["F"] * (3 if c["gated"] else 2)
    byte = 17 / 32 if c["fmt"] == "mxfp4" else 9 / 16
    return {"bytes": int(hit * per * byte + c["T"] * (4 * c["K"] + c["experts"] * 4 + 8 * c["k"])),
            "flops": int(2 * _rows_here(c) * (1 - c["padded"]) * per)}


# ------------------------------------------------------------ the definition in 64 bits

def _exact_values(q):
    """Sign, exponent and mantissa of each 4-bit code taken apart, in float64."""
    c = torch.empty(q[0].shape[0], 2 * q[0].shape[1], dtype=torch.int16, device=q[0].device)
    c[:, 0::2], c[:, 1::2] = q[0] % 16, q[0] // 16
    power, half = (c // 2) % 4, (c % 2).double()
    v = torch.where(power == 0, half / 2, (1 + half / 2) * 2.0 ** (power.double() - 1))
    v = torch.where(c >= 8, -v, v)
    if len(q) == 2:
        return v * (2.0 ** (q[1].double() - 127)).repeat_interleave(32, 1)
    s = q[1].int()
    s = torch.where(s >= 8, (1 + (s % 8).double() / 8) * 2.0 ** ((s // 8).double() - 7), (s % 8).double() / 512)
    v = v * s.repeat_interleave(16, 1)
    return v * q[2].double().repeat_interleave(v.shape[0] // q[2].numel())[:, None]


def exact(case, seed):
    c = case
    if c["op"] == "requant":
        if c["K"] * c["N"] * c["local"] > 2 ** 25 if c["kind"] == "weights" else c["T"] * c["k"] * c["K"] > 2 ** 25:
            return None
    s = prepare(case, seed)
    return {"quantize": _exact_quantize, "product": _exact_product, "requant": _exact_requant,
            "tokens": _exact_tokens}[c["op"]](s, c)


def _exact_quantize(s, c):
    """The nearest of the eight magnitudes, ties to the one with an even code, slice by slice."""
    out = torch.zeros(c["rows"], c["cols"], dtype=torch.float64, device=DEV)
    grid = torch.tensor(E2M1[:8], dtype=torch.float64, device=DEV)
    mid = (grid[1:] + grid[:-1]) / 2
    step = max(1, (1 << 26) // c["cols"])
    for r in range(0, s["live"], step):
        n = min(s["live"], r + step)
        b = s["x"][r:n].double().reshape(n - r, -1, 32)
        top = b.abs().amax(2, keepdim=True)
        e = torch.ceil(torch.log2(top.clamp_min(2.0 ** -150) / 6))
        e = torch.where(top > 6 * 2.0 ** e, e + 1, torch.where(top <= 6 * 2.0 ** (e - 1), e - 1, e)).clamp_min(-127)
        a = b.abs() / 2.0 ** e
        low = torch.bucketize(a, mid)                       # a tie counts as below
        tie = a == mid[low.clamp_max(6)]
        low = torch.where(tie & (low % 2 == 1), low + 1, low)
        out[r:n] = (torch.sign(b) * grid[low] * 2.0 ** e).reshape(n - r, -1)
    return out


def _exact_product(s, c):
    a, w = _exact_values(s["a"]), s["w"]
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for g, n in enumerate(s["counts"]):
        if n:
            wg = _exact_values(tuple(t[g * c["N"]:(g + 1) * c["N"]] for t in w))
            y[at:at + n] = a[s["row_token"][at:at + n].long()] @ wg.t()
        at += n
    return y


def _exact_requant(s, c):
    v, P, K = _exact_values(s["q"]).cpu().numpy(), s["P"], c["K"]
    t = np.zeros((K, P))
    if c["kind"] == "weights":
        t[:] = v.T
    else:
        off, pad, tok = (s[n].cpu().numpy() for n in ("offsets", "padded", "row_token"))
        for g in range(c["local"]):
            m = off[g + 1] - off[g]
            t[:, pad[g]:pad[g] + m] = v[tok[off[g]:off[g] + m]].T
    top = np.abs(t).reshape(K, -1, 32).max(2)
    with np.errstate(divide="ignore"):
        e = np.where(top > 0, np.ceil(np.log2(top / 448)), -127)
    e = np.maximum(np.where(top > 448 * 2.0 ** e, e + 1, e), -127).repeat(32, 1)
    a = np.abs(t) / 2.0 ** e
    with np.errstate(divide="ignore"):
        gap = 2.0 ** (np.maximum(np.floor(np.log2(a)), -6) - 3)
    low = np.floor(a / gap)
    u64 = np.uint64
    i = np.arange(K * P // 8, dtype=u64)
    x0, x1, x2, x3 = i & u64(M32), i >> u64(32), np.full_like(i, s["tag"]), np.zeros_like(i)
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
    for _ in range(10):
        p, q = x0 * u64(0xD2511F53), x2 * u64(0xCD9E8D57)
        x0, x1, x2, x3 = ((q >> u64(32)) ^ x1 ^ u64(key[0]), q & u64(M32), (p >> u64(32)) ^ x3 ^ u64(key[1]),
                          p & u64(M32))
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    u = np.stack([x0, x0 >> u64(16), x1, x1 >> u64(16), x2, x2 >> u64(16), x3, x3 >> u64(16)], 1) & u64(0xFFFF)
    up = u.reshape(K, P).astype(np.int64) + np.floor((a / gap - low) * 65536).astype(np.int64) >= 65536
    v = torch.from_numpy(np.sign(t) * (low + up) * gap * 2.0 ** e).to(DEV)
    if c["kind"] == "weights":
        v = torch.cat(v.split(c["N"], 1))
    return v


def _exact_tokens(s, c):
    T, k, K, F = c["T"], c["k"], c["K"], c["F"]
    z = s["logits"].double()
    score = torch.softmax(z, 1) if c["score"] == "softmax" else torch.sigmoid(z)
    key = (z if s["bias"] is None else score + s["bias"].double()).tolist()
    real = [True] * T if s["token_mask"] is None else s["token_mask"].tolist()
    ids = [sorted(range(c["experts"]), key=lambda e: (-key[t][e], e))[:k] if real[t] else [-1] * k for t in range(T)]
    gate = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    for t in range(T):
        if real[t]:
            g = score[t, ids[t]]
            gate[t] = c["scale"] * (g / g.sum() if c["renorm"] else g)
    out = torch.zeros(T, K, dtype=torch.float64, device=DEV)
    x, rows = s["x"].double(), F * (2 if c["gated"] else 1)
    part = lambda w, e, n: tuple(v[e:e + 1] if v.dim() == 1 else v[e * n:(e + 1) * n] for v in w)
    for e in range(c["local"]):
        pairs = [(t, j) for t in range(T) for j in range(k) if ids[t][j] == e + s["e0"]]
        if pairs:
            at = [t for t, _ in pairs]
            h = x[at] @ _exact_values(part(s["w1"], e, rows)).t()
            a = h[:, :F]
            a = a * torch.sigmoid(a) if c["act"] == "silu" else torch.relu(a) ** 2 if c["act"] == "relu2" else a
            h = a * h[:, F:] if c["gated"] else a
            g = torch.stack([gate[p] for p in pairs])[:, None]
            out.index_add_(0, torch.tensor(at, device=DEV), g * (h @ _exact_values(part(s["w2"], e, K)).t()))
    return dict(out=out, topk_ids=None, gate=gate)
