"""Timed cases of the microscaled 4-bit and expert-routing operators.

Four operators, each in a plain form (elementary torch operations in 32 bits,
64 where the order of near-equal scores decides) and as the calls a user of
the library makes (`own`):

  quantize  a bf16 matrix to 4-bit floating point (E2M1) with one scale per
            block, and back to the values it stands for;
  linear    y = x W^T with both operands in that form, x quantized in the call;
  route     scores, groups, bias, top-k and weights of a mixture of experts;
  experts   a whole mixture-of-experts feed-forward layer on 4-bit weights.

Formats.  "mxfp4": blocks of 32 along K, scale 2^e stored as e + 127 in a byte,
e = floor(log2 max|x|) - 2.  "nvfp4": blocks of 16, scale in E4M3, and one
fp32 scale g = 2^(floor(log2 max|x|) - 10) per row.  Elements round to nearest,
ties to even, and saturate at 6.
"""
import math

import numpy as np
import torch

own = False

BLOCK = {"mxfp4": 32, "nvfp4": 16}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the activations of one decoding step's batch, before a projection
        dict(name="quantize_tokens_16x4096", op="quantize", rows=16, k=4096, fmt="mxfp4"),
        # a 70B-shaped weight matrix, quantized when a checkpoint is converted
        dict(name="quantize_weights_28672x8192", op="quantize", rows=28672, k=8192, fmt="nvfp4"),
        # one token through an 8B-shaped down projection: latency and weight bytes
        dict(name="linear_token_4096x14336", op="linear", m=1, n=4096, k=14336, fmt="mxfp4",
             out="bf16"),
        # a batch of 16 tokens through a small key/value projection
        dict(name="linear_16_tokens_1024x4096", op="linear", m=16, n=1024, k=4096, fmt="nvfp4",
             out="bf16"),
        # an odd batch through a 70B-shaped up projection
        dict(name="linear_133_tokens_28672x8192", op="linear", m=133, n=28672, k=8192,
             fmt="nvfp4", out="bf16"),
        # a prompt through an 8B-shaped up projection: dense contraction
        dict(name="linear_prompt_4096_14336x4096", op="linear", m=4096, n=14336, k=4096,
             fmt="mxfp4", out="bf16"),
        # one token's routing: latency only
        dict(name="route_token_128", op="route", t=1, experts=128, top=4, score="softmax",
             bias=False, groups=1, top_groups=1, best=1, renorm=True, scale=1.0, logits="bf16"),
        # a prompt's routing with a balance bias and groups of experts
        dict(name="route_prompt_4096x256", op="route", t=4096, experts=256, top=8,
             score="sigmoid", bias=True, groups=8, top_groups=4, best=2, renorm=True, scale=2.5,
             logits="fp32"),
        # an odd number of tokens and of experts
        dict(name="route_ragged_1021x160", op="route", t=1021, experts=160, top=6,
             score="softmax", bias=False, groups=8, top_groups=3, best=1, renorm=False,
             scale=16.0, logits="bf16"),
        # one token through eight of 64 experts: latency and weight bytes
        dict(name="experts_token_64x4096x2048", op="experts", t=1, experts=64, top=8, d=4096,
             f=2048, fmt="mxfp4"),
        # an odd decoding batch, an expert width that no tile divides
        dict(name="experts_37_tokens_60x2048x1440", op="experts", t=37, experts=60, top=4,
             d=2048, f=1440, fmt="nvfp4"),
        # a prompt through a layer of 64 experts: dense contraction
        dict(name="experts_prompt_4096_64x4096x1024", op="experts", t=4096, experts=64, top=8,
             d=4096, f=1024, fmt="mxfp4"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("quantize", "linear", "linear", "route", "experts", "experts"))
    fmt = rng.choice(("mxfp4", "nvfp4"))
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 16384), k=_log(rng, 32, 14336, 32), fmt=fmt)
    if op == "linear":
        return dict(op=op, m=_log(rng, 1, 4096), n=_log(rng, 64, 12288),
                    k=_log(rng, 128, 7168, 32), fmt=fmt, out=rng.choice(("bf16", "fp16")))
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        per = rng.randint(4, 32)
        kept = rng.randint(1, groups)
        return dict(op=op, t=_log(rng, 1, 8192), experts=groups * per,
                    top=rng.randint(1, min(8, kept * per)),
                    score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5,
                    groups=groups, top_groups=kept, best=rng.choice((1, 2)),
                    renorm=rng.random() < 0.5, scale=rng.choice((1.0, 2.5)),
                    logits=rng.choice(("bf16", "fp32")))
    e = rng.randint(4, 64)
    return dict(op=op, t=_log(rng, 1, 2048), experts=e, top=rng.randint(1, min(8, e)),
                d=_log(rng, 256, 4096, 32), f=_log(rng, 256, 1024, 32), fmt=fmt)


# ---------------------------------------------------------------- the inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _weights(g, b, n, k, fmt):
    """b matrices W[n, k] ~ N(0, 0.02) with 0.1% entries x10, quantized: what a program keeps of
    them is the packed layout; the plain form reads its two parts as codes and scales."""
    codes, scales, rows = [], [], []
    for _ in range(b):
        w = _normal(g, n, k) * 0.02
        w = torch.where(torch.rand((n, k), generator=g, device="cuda") < 1e-3, w * 10, w)
        c, s, r = _quantize(w.to(torch.bfloat16).float(), fmt)
        codes.append(c)
        scales.append(s)
        rows.append(r)
    codes, scales, rows = torch.stack(codes), torch.stack(scales), torch.stack(rows)
    return dict(codes=codes, scales=scales, rows=rows, packed=_lay_out(codes, scales, rows, fmt))


def _lay_out(codes, scales, rows, fmt):
    """The packed layout: two codes a byte row after row; the scale bytes in blocks of 128 rows x 4
    (byte 16 (r % 32) + 4 (r / 32) + j), rows padded to 128 and K to 256; nvfp4: the row scales.
    Each part is padded to 128 bytes."""
    b, n, k = codes.shape
    part = (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(b, -1)
    part = torch.nn.functional.pad(part, (0, -part.shape[1] % 128))
    g = -(-k // 256) * 256 // BLOCK[fmt]
    n_pad = -(-n // 128) * 128
    s = torch.zeros((b, n_pad, g), dtype=torch.uint8, device=codes.device)
    s[:, :n, :scales.shape[2]] = scales
    s = s.view(b, n_pad // 128, 4, 32, g // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(b, -1)
    parts = [part, s]
    if fmt == "nvfp4":
        r = torch.nn.functional.pad(rows, (0, -n % 32))
        parts.append(r.contiguous().view(torch.uint8).reshape(b, -1))
    return torch.cat(parts, 1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, st = case["op"], dict(case=case)
    if op == "quantize":
        std = 0.02 if case["rows"] > 4096 else 1.0
        x = _normal(g, case["rows"], case["k"]) * std
        st["x"] = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 1e-3, x * 10,
                              x).to(torch.bfloat16)
    elif op == "linear":
        st["x"] = _normal(g, case["m"], case["k"]).to(torch.bfloat16)
        st["w"] = _weights(g, 1, case["n"], case["k"], case["fmt"])
    elif op == "route":
        lean = _normal(g, 1, case["experts"])  # some experts are liked by every token
        logits = 1.5 * _normal(g, case["t"], case["experts"]) + 0.5 * lean
        st["logits"] = logits.to(DTYPES[case["logits"]])
        st["bias"] = 0.1 * _normal(g, case["experts"]) if case["bias"] else None
    else:
        t, e, d, f = case["t"], case["experts"], case["d"], case["f"]
        st["x"] = _normal(g, t, d).to(torch.bfloat16)
        logits = 1.5 * _normal(g, t, e) + 0.5 * _normal(g, 1, e)
        top, ids = torch.topk(logits, case["top"], dim=1)
        st["ids"] = ids.to(torch.int32)
        st["weights"] = torch.softmax(top, 1)
        st["gate"] = _weights(g, e, f, d, case["fmt"])
        st["up"] = _weights(g, e, f, d, case["fmt"])
        st["down"] = _weights(g, e, d, f, case["fmt"])
    return st


# ---------------------------------------------------------------- the plain forms

def _round_e2m1(v):
    """|v| (0 .. 6, larger saturates) to the nearest E2M1 level, ties to the even code; the code."""
    v = v.clamp(max=6.0)
    small, mid = v < 2.0, v < 4.0
    step = torch.where(small, 0.5, torch.where(mid, 1.0, 2.0))
    q = torch.round(v / step) * step
    return torch.where(q <= 2.0, q * 2, torch.where(q <= 4.0, q + 2, q * 0.5 + 4)).to(torch.uint8)


def _quantize(x, fmt):
    """x fp32 [..., K] -> codes (uint8, one a byte), scale bytes [..., K / block], row scales."""
    b = BLOCK[fmt]
    xb = x.unflatten(-1, (-1, b))
    amax = xb.abs().amax(-1, keepdim=True)
    if fmt == "mxfp4":
        e = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0)  # biased exponent of the scale
        v = xb.abs() * torch.ldexp(torch.ones_like(amax), 127 - e)
        scales, rows = e.squeeze(-1).to(torch.uint8), torch.ones_like(x[..., 0])
    else:
        top = x.abs().amax(-1, keepdim=True)
        e = (top.view(torch.int32) >> 23) - 127 - 10
        rows = torch.where(top > 0, torch.ldexp(torch.ones_like(top), e.clamp(min=-126)), 1.0)
        s8 = (amax / 6.0 / rows.unsqueeze(-1)).clamp(max=448.0).to(torch.float8_e4m3fn)
        s = s8.float() * rows.unsqueeze(-1)
        v = torch.where(s > 0, xb.abs() / torch.where(s > 0, s, 1.0), 0.0)
        scales, rows = s8.view(torch.uint8).squeeze(-1), rows.squeeze(-1)
    codes = _round_e2m1(v) | (torch.signbit(xb).to(torch.uint8) << 3)
    return codes.flatten(-2), scales, rows


def _values(codes, scales, rows, fmt):
    """The fp32 values that codes, scales and row scales stand for."""
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    v = table[codes.int()].unflatten(-1, (-1, BLOCK[fmt]))
    if fmt == "mxfp4":
        s = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    else:
        s = scales.view(torch.float8_e4m3fn).float() * rows.unsqueeze(-1)
    return (v * s.unsqueeze(-1)).flatten(-2)


def _rounded(x, fmt):
    return _values(*_quantize(x.float(), fmt), fmt)


def _route_plain(logits, bias, c):
    z = logits.double()
    if c["score"] == "softmax":
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-z))
    s = p + bias.double() if bias is not None else p
    if c["groups"] > 1:
        per = s.view(s.shape[0], c["groups"], -1)
        best = torch.sort(per, dim=2, descending=True).values[..., :c["best"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        s = torch.where(keep.unsqueeze(2), per, -math.inf).flatten(1)
    ids = torch.sort(s, dim=1, descending=True, stable=True).indices[:, :c["top"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _experts_plain(s, fmt):
    ids = s["ids"].long().flatten()
    used, to = torch.unique(ids, return_inverse=True)  # the experts that some token takes
    count = torch.bincount(to, minlength=used.numel())
    order = torch.argsort(to, stable=True)
    place = torch.empty_like(to)
    place[order] = torch.arange(to.numel(), device=to.device) - (count.cumsum(0) - count)[to[order]]
    x = _rounded(s["x"], fmt)
    rows = torch.zeros((used.numel(), int(count.max()), x.shape[1]), device=x.device)
    rows[to, place] = x.repeat_interleave(s["ids"].shape[1], 0)

    def weights(w):
        return _values(w["codes"][used], w["scales"][used], w["rows"][used], fmt).transpose(1, 2)

    gate, up = torch.bmm(rows, weights(s["gate"])), torch.bmm(rows, weights(s["up"]))
    h = (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16)
    out = torch.bmm(_rounded(h, fmt), weights(s["down"]))[to, place]
    out = out.view(*s["ids"].shape, -1) * s["weights"].unsqueeze(2)
    return out.sum(1).to(torch.bfloat16)


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import dequant_gemv_group_b200 as lq
        if op == "quantize":
            q = lq.lutq_mx_quantize(state["x"], c["fmt"])
            return lq.lutq_mx_dequantize(q, c["rows"], c["k"], c["fmt"], dtype=torch.bfloat16)
        if op == "linear":
            w, out = state["w"]["packed"], DTYPES[c["out"]]
            if c["m"] <= 16:
                return lq.lutq_mx_gemv(state["x"], w, c["n"], c["k"], c["fmt"], dtype=out)
            q = lq.lutq_mx_quantize(state["x"], c["fmt"])
            return lq.lutq_mx_gemm(q, c["m"], w, c["n"], c["k"], c["fmt"], dtype=out)
        if op == "route":
            return lq.lutq_route(state["logits"], c["top"], score=c["score"], bias=state["bias"],
                                 groups=c["groups"], top_groups=c["top_groups"],
                                 group_best=c["best"], renormalize=c["renorm"], scale=c["scale"])
        return lq.lutq_mx_experts(state["x"], state["ids"], state["weights"],
                                  state["gate"]["packed"], state["up"]["packed"],
                                  state["down"]["packed"], c["f"], c["fmt"])
    if op == "quantize":
        return _rounded(state["x"], c["fmt"]).to(torch.bfloat16)
    if op == "linear":
        w = state["w"]
        w = _values(w["codes"], w["scales"], w["rows"], c["fmt"])[0]
        return torch.matmul(_rounded(state["x"], c["fmt"]), w.t()).to(DTYPES[c["out"]])
    if op == "route":
        return _route_plain(state["logits"], state["bias"], c)
    return _experts_plain(state, c["fmt"])


# ---------------------------------------------------------------- work and exact values

def _matrix_bytes(n, k, fmt):
    return n * k / 2 + n * k / BLOCK[fmt] + (4 * n if fmt == "nvfp4" else 0)


def work(case):
    c, op = case, case["op"]
    if op == "quantize":
        # read and quantize; the packed form is written and read once; the values are written
        n = c["rows"] * c["k"]
        return dict(bytes=4 * n + 2 * _matrix_bytes(c["rows"], c["k"], c["fmt"]), flops=4 * n)
    if op == "linear":
        return dict(bytes=_matrix_bytes(c["n"], c["k"], c["fmt"]) + 2 * c["m"] * c["k"]
                    + 2 * c["m"] * c["n"], flops=2 * c["m"] * c["n"] * c["k"])
    if op == "route":
        item = 2 if c["logits"] == "bf16" else 4
        return dict(bytes=c["t"] * (c["experts"] * item + 8 * c["top"]),
                    flops=40 * c["t"] * c["experts"])
    # an expert that some token takes is read once; as if tokens chose evenly
    used = c["experts"] * (1 - (1 - c["top"] / c["experts"]) ** c["t"])
    one = 2 * _matrix_bytes(c["f"], c["d"], c["fmt"]) + _matrix_bytes(c["d"], c["f"], c["fmt"])
    return dict(bytes=used * one + c["t"] * (4 * c["d"] + 8 * c["top"]),
                flops=6 * c["t"] * c["top"] * c["d"] * c["f"])


def _exact_rounded(x, fmt):
    """The values of quantized x in 64 bits, by comparison with the midpoints between levels."""
    xb = x.double().unflatten(-1, (-1, BLOCK[fmt]))
    amax = xb.abs().amax(-1, keepdim=True)
    exponent = lambda t: torch.where(t > 0, torch.frexp(t).exponent - 1, -1000)  # noqa: E731
    one = torch.ones_like(amax)
    if fmt == "mxfp4":
        s = torch.ldexp(one, (exponent(amax) - 2).clamp(-127, 127))
    else:
        top = x.double().abs().amax(-1, keepdim=True).unsqueeze(-1)
        g = torch.where(top > 0, torch.ldexp(torch.ones_like(top),
                                             (exponent(top) - 10).clamp(min=-126)), 1.0)
        t = amax / 6.0 / g
        step = torch.ldexp(one, exponent(t).clamp(min=-6) - 3)
        s = torch.round(t / step).mul(step).clamp(max=448.0) * g
    v = torch.where(s > 0, xb.abs() / torch.where(s > 0, s, 1.0), 0.0)
    q = torch.zeros_like(v)
    for c in range(7):
        mid = (LEVELS[c] + LEVELS[c + 1]) / 2
        q += torch.where((v >= mid) if c % 2 else (v > mid), LEVELS[c + 1] - LEVELS[c], 0.0)
    return (torch.copysign(q, xb) * s).flatten(-2)


def _exact_weights(w, i, fmt):
    lv = torch.tensor(LEVELS, device="cuda", dtype=torch.float64)
    codes, s = w["codes"][i], w["scales"][i]
    v = lv[(codes & 7).long()] * (1.0 - 2.0 * (codes >> 3).double())
    if fmt == "mxfp4":
        s = torch.pow(2.0, s.double() - 127)
    else:
        e, m = (s >> 3).double(), (s & 7).double()
        s = torch.where(e > 0, torch.pow(2.0, e - 7) * (1 + m / 8), m / 512)
        s = s * w["rows"][i].double().unsqueeze(-1)
    return v * s.repeat_interleave(BLOCK[fmt], -1)


def exact(case, seed):
    c, op = case, case["op"]
    if work(case)["flops"] > 5.5e14:
        return None
    st = prepare(case, seed)
    if op == "quantize":
        return _exact_rounded(st["x"], c["fmt"])
    if op == "linear":
        return _exact_rounded(st["x"], c["fmt"]) @ _exact_weights(st["w"], 0, c["fmt"]).t()
    if op == "route":
        z = st["logits"].double().cpu().numpy()
        p = np.exp(-np.logaddexp(0.0, -z)) if c["score"] == "sigmoid" else np.exp(
            z - np.logaddexp.reduce(z, axis=1, keepdims=True))
        s = p + (0.0 if st["bias"] is None else st["bias"].double().cpu().numpy())
        if c["groups"] > 1:
            per = s.reshape(len(z), c["groups"], -1)
            best = np.sort(per, axis=2)[:, :, ::-1][:, :, :c["best"]].sum(2)
            rank = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1, kind="stable")
            s = np.where(rank[:, :, None] < c["top_groups"], per, -np.inf).reshape(len(z), -1)
        ids = np.argsort(-s, axis=1, kind="stable")[:, :c["top"]]
        w = np.take_along_axis(p, ids, 1)
        if c["renorm"]:
            w = w / w.sum(1, keepdims=True)
        return ids.astype(np.int32), w * c["scale"]
    x, y = _exact_rounded(st["x"], c["fmt"]), torch.zeros(st["x"].shape, device="cuda",
                                                          dtype=torch.float64)
    for e in range(c["experts"]):
        t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
        if not t.numel():
            continue
        gate = x[t] @ _exact_weights(st["gate"], e, c["fmt"]).t()
        up = x[t] @ _exact_weights(st["up"], e, c["fmt"]).t()
        h = _exact_rounded((gate * torch.sigmoid(gate) * up).to(torch.bfloat16), c["fmt"])
        out = h @ _exact_weights(st["down"], e, c["fmt"]).t()
        y.index_add_(0, t, out * st["weights"][t, j].double().unsqueeze(1))
    return y
