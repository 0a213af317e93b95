"""What a model's unit does between its gather and its reduce, as measured:
embedding rows read from the gathered parameters, their gradient by sorted
tokens, activations kept in 8 bits, the activation functions that keep and read
them, and the weight gradient taken from them.

A checkpoint of x (rows, cols) holds int8 codes, rows padded with zeros to
blocks of 32, and one exponent E per block:
    E = max(floor(log2 amax) + 127, E_min), q = clamp(rint(x * 2^(133 - E)), -127, 127)
and stands for q * 2^(E - 133).  E_min is 109 for fp16 (a code is then no finer
than fp16's smallest number) and 7 otherwise; a block with an infinity or a NaN
has E = 255 and codes 0 and stands for NaN.  Codes and exponents follow from x
by exact operations and are whole numbers, equal on every side.
"""
import math
import random

import torch

own = False

BLOCK = 32                        # elements per exponent of a checkpoint
PAYLOAD_BLOCK = 256               # elements per scale of an INT8 payload
FLOATS = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
KINDS = ("gelu", "gelu_tanh", "silu")
SQRT_HALF, GELU_C, GELU_A = math.sqrt(0.5), math.sqrt(2.0 / math.pi), 0.044715


def listed():
    return [
        # one token's row while a model generates: latency
        dict(name="lookup_token_bf16", op="lookup", tokens=1, vocab=32000, dim=4096, table="bf16",
             out="bf16", ranks=0, first=0, wide=True),
        # a batch's rows straight from the 8 ranks' gathered INT8 slots
        dict(name="lookup_batch_int8", op="lookup", tokens=16384, vocab=32000, dim=4096, table="int8",
             out="bf16", ranks=8, first=0, wide=True),
        # a small model's embedding gradient, every row written: latency
        dict(name="embed_grad_small_fp16", op="embed_grad", tokens=512, vocab=1000, dim=256, dy="fp16",
             grad="fp16", accumulate=False, pad=0.0, first=0, wide=True),
        # a batch's gradient into the flat bf16 gradient, every row written
        dict(name="embed_grad_batch_bf16", op="embed_grad", tokens=16384, vocab=32000, dim=4096, dy="bf16",
             grad="bf16", accumulate=False, pad=0.0, first=0, wide=True),
        # a micro-step added into fp32 gradients: odd sizes, a fifth of it padding
        dict(name="embed_grad_odd_fp32", op="embed_grad", tokens=30011, vocab=50021, dim=1001, dy="bf16",
             grad="fp32", accumulate=True, pad=0.2, first=0, wide=True),
        # the input of a block's first projections, kept for the backward pass
        dict(name="save_block_bf16", op="save", rows=16384, cols=4096, dtype="bf16", spread=1.0),
        # a kept fp32 input of odd width, taken back
        dict(name="restore_odd_fp32", op="restore", rows=4097, cols=1001, dtype="fp32", spread=2.0),
        # the gated activation between a block's projections (gate and up packed), and its backward pass
        dict(name="act_forward_block_bf16", op="forward", rows=8192, cols=11008, dtype="bf16", kind="silu",
             gated=True, spread=1.0),
        dict(name="act_backward_block_bf16", op="backward", rows=8192, cols=11008, dtype="bf16", kind="silu",
             gated=True, spread=1.0),
        # a small MLP's activation: latency
        dict(name="act_backward_mlp_fp16", op="backward", rows=512, cols=1024, dtype="fp16", kind="gelu",
             gated=False, spread=1.0),
        # the weight gradients of the same two: a few tiles over a short sum, and many over a long one
        dict(name="weight_grad_mlp_fp16", op="weight_grad", rows=512, outs=512, cols=1024, dtype="fp16",
             grad="fp16", accumulate=False, spread=1.0),
        dict(name="weight_grad_block_bf16", op="weight_grad", rows=16384, outs=11008, cols=4096, dtype="bf16",
             grad="fp32", accumulate=True, spread=1.0),
    ]


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("lookup", "embed_grad", "save", "restore", "forward", "backward", "weight_grad"))
    some = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op in ("lookup", "embed_grad"):
        dim = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            dim = max(8, dim // 8 * 8)
        d = dict(op=op, tokens=_log(rng, 1, 65536), vocab=min(_log(rng, 100, 131072), (1 << 28) // dim), dim=dim,
                 first=rng.choice((0, 0, rng.randrange(1, 5000))), wide=rng.random() < 0.7)
        d["tokens"] = min(d["tokens"], (1 << 27) // dim)
        if op == "lookup":
            d.update(table=rng.choice(("bf16", "fp16", "fp32", "int8")), out=some, ranks=0)
            if d["table"] == "int8":
                d["ranks"] = rng.choice((1, 3, 8, 64))
        else:
            d.update(dy=some, grad=rng.choice(("bf16", "fp16", "fp32")), accumulate=rng.random() < 0.5,
                     pad=rng.choice((0.0, 0.0, 0.1, 0.6)))
        return d
    if op == "weight_grad":
        d = dict(op=op, rows=_log(rng, 1, 32768), outs=_log(rng, 16, 11008), cols=_log(rng, 16, 11008),
                 dtype=rng.choice(("bf16", "bf16", "fp16")), grad=rng.choice(("fp32", "bf16", "fp16")),
                 accumulate=rng.random() < 0.5, spread=rng.choice((0.5, 1.0, 2.0)))
        if rng.random() < 0.6:
            d["outs"], d["cols"] = max(16, d["outs"] // 16 * 16), max(16, d["cols"] // 16 * 16)
        d["rows"] = max(1, min(d["rows"], (1 << 39) // (d["outs"] * d["cols"])))
        return d
    cols = _log(rng, 1, 16384)
    if rng.random() < 0.6:
        cols = max(8, cols // 8 * 8)
    d = dict(op=op, rows=min(_log(rng, 1, 65536), max(1, (1 << 26) // cols)), cols=cols, dtype=some,
             spread=rng.choice((0.0, 1.0, 2.0)))
    if op in ("forward", "backward"):
        d.update(kind=rng.choice(KINDS), gated=rng.random() < 0.5)
    return d


def _pitch(cols):
    return -(-cols // BLOCK) * BLOCK


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(case, gen, dtype=None):
    """Values as a layer's activations have them: channels of very different
    size (lognormal by `spread`), a token in 64 ten times the rest, and now and
    then a zero."""
    x = _normal(gen, case["rows"], case["cols"])
    x *= _normal(gen, case["cols"]).mul_(case["spread"]).exp_()
    x[::64] *= 10.0
    x[:, 1::13] = x[:, 1::13].clamp(min=0.0)
    if (dtype or case["dtype"]) == "fp16":
        x.clamp_(-60000.0, 60000.0)
    return x.to(FLOATS[dtype or case["dtype"]])


def _zipf(case, gen):
    """Token numbers by rank with probability ~ 1 / rank, the ranks spread over
    the vocabulary, and the ends of the sequences padded with one token."""
    n, v = case["tokens"], case["vocab"]
    rank = torch.exp(torch.rand(n, generator=gen, device="cuda", dtype=torch.float64) * math.log(v)).long() - 1
    step = next(s for s in range(int(v * 0.618) | 1, 4 * v + 8) if math.gcd(s, v) == 1)
    tok = rank.clamp(0, v - 1) * step % v
    if case.get("pad"):
        length = max(1, min(n, 512))
        tok[torch.arange(n, device="cuda") % length >= int(length * (1 - case["pad"]))] = _padding(case)
    tok += case["first"]
    if case["first"]:
        # a rank that holds some of the vocabulary's rows meets the others' tokens too
        tok[3::7] = tok[3::7] - case["first"] - 1
    return tok if case["wide"] else tok.to(torch.int32)


def _padding(case):
    return case["vocab"] // 3


def _power(k):
    """2^k in fp32, exactly, for k of -126 to 127."""
    return (k.clamp(-126, 127).to(torch.int32) + 127 << 23).view(torch.float32)


def _quantise(x, emin):
    """(codes, exponents) of a checkpoint by elementary operations."""
    rows, cols = x.shape
    p = torch.zeros(rows, _pitch(cols), device=x.device)
    p[:, :cols] = x
    p = p.view(rows, -1, BLOCK)
    top = p.abs().amax(2)
    # frexp's exponent is one more than floor(log2)
    e = torch.where(top > 0, torch.frexp(top).exponent + 126, 0).clamp(emin, 254)
    bad = ~torch.isfinite(top)
    q = torch.round(p * _power(133 - e)[:, :, None]).clamp_(-127, 127)
    q = torch.where(bad[:, :, None], 0.0, q).to(torch.int8)
    return q.view(rows, -1), torch.where(bad, 255, e).to(torch.uint8)


def _restored(codes, exps, cols):
    s = torch.where(exps == 255, math.nan, _power(exps.to(torch.int32) - 133))
    x = codes.view(codes.shape[0], -1, BLOCK).float() * s[:, :, None]
    return x.view(codes.shape[0], -1)[:, :cols]


def _emin(case):
    return 109 if case["dtype"] == "fp16" else 7


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, d = case["op"], {}
    if op in ("lookup", "embed_grad"):
        v, dim = case["vocab"], case["dim"]
        d["tokens"] = _zipf(case, gen)
        if op == "embed_grad":
            d["dy"] = _normal(gen, case["tokens"], dim).mul_(1e-2).to(FLOATS[case["dy"]])
            if case["accumulate"]:
                d["grad"] = _normal(gen, v, dim).mul_(1e-2).to(FLOATS[case["grad"]])
            else:
                d["grad"] = torch.empty(v, dim, dtype=FLOATS[case["grad"]], device="cuda")
        elif case["table"] == "int8":
            # the gathered flat parameter: the table behind 1000 other elements, slots of one size
            d["offset"] = 1000
            slot = -(-(d["offset"] + v * dim) // case["ranks"])
            slot += -slot % 8 if dim % 8 == 0 else 0
            d["slot"], blocks = slot, -(-slot // PAYLOAD_BLOCK)
            d["codes"] = torch.randint(-127, 128, (case["ranks"] * slot,), generator=gen, device="cuda",
                                       dtype=torch.int8)
            d["scales"] = _normal(gen, case["ranks"] * blocks).abs_().add_(0.5).mul_(4.7e-4)
        else:
            d["table"] = _normal(gen, v, dim).mul_(0.02).to(FLOATS[case["table"]])
        return d
    if op == "weight_grad":
        d["dy"] = _normal(gen, case["rows"], case["outs"]).mul_(1e-3).to(FLOATS[case["dtype"]])
        d["codes"], d["exps"] = _quantise(_activations(case, gen).float(), _emin(case))
        shape = case["outs"], case["cols"]
        d["grad"] = _normal(gen, *shape).mul_(1e-2).to(FLOATS[case["grad"]]) if case["accumulate"] \
            else torch.empty(shape, dtype=FLOATS[case["grad"]], device="cuda")
        return d
    x = _activations(case, gen)
    gated = case.get("gated", False)
    if gated:
        # both projections' outputs in one buffer, as one product writes them
        d["packed"] = torch.cat((x, _activations(case, gen)), 1)
        x, d["up"] = d["packed"][:, :case["cols"]], d["packed"][:, case["cols"]:]
    if op in ("save", "forward"):
        d["x"] = x
        return d
    d["codes"], d["exps"] = _quantise(x.float(), _emin(case))
    if gated:
        d["up_codes"], d["up_exps"] = _quantise(d["up"].float(), _emin(case))
    if op == "backward":
        d["dy"] = _normal(gen, case["rows"], case["cols"]).mul_(1e-2).to(FLOATS[case["dtype"]])
    return d


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    s["case"], s["scale"] = case, math.sqrt(case.get("dim", 1))
    if not own:
        return s
    import fsdp_sharded_mixed_flatparameter_amd as zf
    s["zf"] = zf
    if op in ("lookup", "embed_grad"):
        if op == "lookup":
            s["out"] = torch.empty(case["tokens"], case["dim"], dtype=FLOATS[case["out"]], device="cuda")
        return s
    rows, cols, kind = case["rows"], case["cols"], FLOATS.get(case["dtype"])

    def saved(codes=None, exps=None):
        k = zf.Saved8(rows, cols)
        if codes is not None:
            k.codes.copy_(codes)
            k.exponents.copy_(exps)
        return k

    s["saved"] = saved(s.pop("codes", None), s.pop("exps", None))
    if op == "weight_grad":
        return s
    if op in ("forward", "backward"):
        s["kind"] = {"gelu": zf.ZERO_GELU, "gelu_tanh": zf.ZERO_GELU_TANH, "silu": zf.ZERO_SILU}[case["kind"]]
    s["up_saved"] = None
    if case.get("gated"):
        s["up_saved"] = saved(s.pop("up_codes", None), s.pop("up_exps", None))
        if op == "backward":
            # one buffer for both gradients, as the next products read them
            both = torch.empty(rows, 2 * cols, dtype=kind, device="cuda")
            s["dx"], s["dup"] = both[:, :cols], both[:, cols:]
    elif op == "backward":
        s["dx"], s["dup"] = torch.empty(rows, cols, dtype=kind, device="cuda"), None
    if op in ("forward", "restore"):
        s["out"] = torch.empty(rows, cols, dtype=kind, device="cuda")
    return s


def _own(s):
    case, zf = s["case"], s["zf"]
    op = case["op"]
    if op == "lookup":
        if case["table"] == "int8":
            zf.zero_embed_lookup_int8(s["tokens"], s["codes"], s["scales"], case["ranks"], s["slot"], s["offset"],
                                      case["vocab"], s["out"], scale=s["scale"], first=case["first"])
        else:
            zf.zero_embed_lookup(s["tokens"], s["table"], s["out"], scale=s["scale"], first=case["first"])
        return s["out"]
    if op == "embed_grad":
        zf.zero_embed_grad(s["tokens"], s["dy"], s["grad"], scale=s["scale"], first=case["first"],
                           padding=_padding(case) + case["first"] if case["pad"] else None,
                           accumulate=case["accumulate"])
        return s["grad"]
    saved, up = s["saved"], s.get("up_saved")
    if op == "weight_grad":
        zf.zero_weight_grad8(s["dy"], saved, s["grad"], accumulate=case["accumulate"])
        return s["grad"]
    if op == "save":
        zf.zero_act_save8(s["x"], saved)
        return dict(codes=saved.codes, exponents=saved.exponents)
    if op == "restore":
        zf.zero_act_restore8(saved, s["out"])
        return s["out"]
    if op == "forward":
        zf.zero_act_forward8(s["kind"], s["x"], s["out"], saved, up=s.get("up"), saved_up=up)
        out = dict(y=s["out"], codes=saved.codes, exponents=saved.exponents)
        if up is not None:
            out.update(up_codes=up.codes, up_exponents=up.exponents)
        return out
    zf.zero_act_backward8(s["kind"], s["dy"], saved, s["dx"], saved_up=up, dup=s["dup"])
    return dict(dx=s["dx"]) if up is None else dict(dx=s["dx"], dup=s["dup"])


def _act(kind, x):
    """(act(x), act'(x)) in fp32."""
    if kind == "silu":
        g = 1.0 / (1.0 + torch.exp(-x))
        return x * g, g * (1.0 + x * (1.0 - g))
    if kind == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(x * SQRT_HALF))
        return x * cdf, cdf + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    t = torch.tanh(GELU_C * (x + GELU_A * x * x * x))
    return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * GELU_C * (1.0 + 3.0 * GELU_A * x * x)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("lookup", "embed_grad"):
        row = s["tokens"].long() - case["first"]
        inside = (row >= 0) & (row < case["vocab"])
    if op == "lookup":
        row = torch.where(inside, row, 0)
        if case["table"] == "int8":
            at = (s["offset"] + row * case["dim"])[:, None] + torch.arange(case["dim"], device="cuda")
            slot = at // s["slot"]
            block = slot * -(-s["slot"] // PAYLOAD_BLOCK) + (at - slot * s["slot"]) // PAYLOAD_BLOCK
            x = s["codes"][at].float() * s["scales"][block]
        else:
            x = s["table"][row].float()
        return torch.where(inside[:, None], x * s["scale"], 0.0).to(FLOATS[case["out"]])
    if op == "embed_grad":
        if case["pad"]:
            inside &= row != _padding(case)
        x = torch.zeros(case["vocab"] + 1, case["dim"], device="cuda")
        x.index_add_(0, torch.where(inside, row, case["vocab"]), s["dy"].float())
        x = x[:-1] * s["scale"]
        if case["accumulate"]:
            x += s["grad"].float()
        s["grad"] = x.to(s["grad"].dtype)
        return s["grad"]
    if op == "weight_grad":
        # the restored values in dy's type (exact where that type's range holds them)
        x = _restored(s["codes"], s["exps"], case["cols"]).to(s["dy"].dtype).float()
        x = s["dy"].float().t() @ x
        if case["accumulate"]:
            x += s["grad"].float()
        s["grad"] = x.to(s["grad"].dtype)
        return s["grad"]
    kind = FLOATS[case["dtype"]]
    if op in ("save", "forward"):
        x, out = s["x"].float(), {}
        if op == "forward":
            y = _act(case["kind"], x)[0]
            if case["gated"]:
                y = y * s["up"].float()
            out["y"] = y.to(kind)
        out["codes"], out["exponents"] = _quantise(x, _emin(case))
        if op == "forward" and case["gated"]:
            out["up_codes"], out["up_exponents"] = _quantise(s["up"].float(), _emin(case))
        return out
    x = _restored(s["codes"], s["exps"], case["cols"])
    if op == "restore":
        return x.to(kind)
    dy = s["dy"].float()
    a, da = _act(case["kind"], x)
    if not case["gated"]:
        return dict(dx=(dy * da).to(kind))
    u = _restored(s["up_codes"], s["up_exps"], case["cols"])
    return dict(dx=(dy * u * da).to(kind), dup=(dy * a).to(kind))


def run(s):
    return _own(s) if own else _plain(s)


def _size(name):
    return 1 if name == "int8" else torch.empty((), dtype=FLOATS[name]).element_size()


def work(case):
    op = case["op"]
    if op in ("lookup", "embed_grad"):
        n, v, dim = case["tokens"], case["vocab"], case["dim"]
        ids = n * (8 if case["wide"] else 4)
        if op == "lookup":
            scales = 4 / PAYLOAD_BLOCK if case["table"] == "int8" else 0
            return dict(bytes=int(n * dim * (_size(case["table"]) + scales + _size(case["out"]))) + ids,
                        flops=n * dim)
        # the rows that 1 / rank draws meet, on average
        hit = sum(-math.expm1(n * math.log1p(-math.log1p(1 / r) / math.log(v))) for r in range(1, v))
        rows = 2 * hit if case["accumulate"] else v
        return dict(bytes=int(n * (1 - case["pad"]) * dim * _size(case["dy"]) + rows * dim * _size(case["grad"])) + ids,
                    flops=n * dim)
    kept = case["rows"] * _pitch(case["cols"]) * (1 + 1 / BLOCK)
    n = case["rows"] * case["cols"]
    if op == "weight_grad":
        g = case["outs"] * case["cols"] * _size(case["grad"]) * (2 if case["accumulate"] else 1)
        return dict(bytes=int(case["rows"] * case["outs"] * 2 + kept + g), flops=2 * n * case["outs"])
    e, gates = _size(case["dtype"]), 2 if case.get("gated") else 1
    if op in ("save", "restore"):
        return dict(bytes=int(n * e + kept), flops=2 * n)
    return dict(bytes=int(n * e * (gates + 1) + kept * gates), flops=n * gates * (10 if op == "forward" else 16))


def _exact_act(kind, x):
    """(act, act') from the definitions, in 64 bits."""
    if kind == "silu":
        y = torch.sigmoid(x)
        return x * y, y + x * y * torch.sigmoid(-x)
    if kind == "gelu":
        cdf = torch.special.ndtr(x)
        return x * cdf, cdf + x * (x.square() / -2).exp() / math.sqrt(2 * math.pi)
    inner = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    # 0.5 (1 + tanh z) is the logistic function of 2 z
    y = torch.sigmoid(2 * inner)
    slope = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x ** 2)
    return x * y, y + x * y * torch.sigmoid(-2 * inner) * slope


def _exact_scales():
    """What one unit of a code stands for, by exponent."""
    return torch.tensor([2.0 ** (e - 133) for e in range(255)] + [math.nan], dtype=torch.float64, device="cuda")


def _exact_codes(x, emin):
    """A checkpoint's codes and exponents in 64 bits, by logarithm and comparison."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.double(), (0, _pitch(cols) - cols)).unflatten(1, (-1, BLOCK))
    top = x.abs().max(2, keepdim=True).values
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -200)))
    e = e - (torch.exp2(e) > top).double()
    e = e + (torch.exp2(e + 1) <= top).double()
    finite = torch.isfinite(top)
    e = (e + 127).clamp(emin, 254)
    q = torch.round(x / _exact_scales()[e.long()]).clamp(-127, 127)
    return (torch.where(finite, q, 0).to(torch.int8).flatten(1),
            torch.where(finite, e, 255).to(torch.uint8).squeeze(2))


def _exact_values(codes, exps, cols):
    scale = _exact_scales()[exps.long()]
    return (codes.double() * scale.repeat_interleave(BLOCK, 1))[:, :cols]


def exact(case, seed):
    d, op = _inputs(case, seed), case["op"]
    if op in ("lookup", "embed_grad"):
        scale, row = math.sqrt(case["dim"]), d["tokens"].long() - case["first"]
        ok = (row >= 0) & (row < case["vocab"])
    if op == "lookup":
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        if case["table"] != "int8":
            out[ok] = d["table"][row[ok]].double() * scale
            return out
        blocks = -(-d["slot"] // PAYLOAD_BLOCK)
        for r in range(0, case["tokens"], 2048):
            part = row[r:r + 2048].clamp(0, case["vocab"] - 1) * case["dim"] + d["offset"]
            at = part[:, None] + torch.arange(case["dim"], device="cuda")
            s = d["scales"][at.div(d["slot"], rounding_mode="floor") * blocks + at % d["slot"] // PAYLOAD_BLOCK]
            out[r:r + 2048] = d["codes"][at].double() * s.double() * scale
        out[~ok] = 0
        return out
    if op == "embed_grad":
        if case["pad"]:
            ok = ok & (row != _padding(case))
        out = d["grad"].double() if case["accumulate"] else torch.zeros(case["vocab"], case["dim"],
                                                                       dtype=torch.float64, device="cuda")
        return out.index_put_((row[ok],), d["dy"][ok].double() * scale, accumulate=True)
    if op == "weight_grad":
        x = _exact_values(d["codes"], d["exps"], case["cols"]).to(d["dy"].dtype).double()
        out = torch.matmul(d["dy"].double().t().contiguous(), x)
        return out + d["grad"].double() if case["accumulate"] else out
    out = {}
    if op in ("save", "forward"):
        if op == "forward":
            out["y"] = _exact_act(case["kind"], d["x"].double())[0]
            if case["gated"]:
                out["y"] = out["y"] * d["up"].double()
        out["codes"], out["exponents"] = _exact_codes(d["x"], _emin(case))
        if op == "forward" and case["gated"]:
            out["up_codes"], out["up_exponents"] = _exact_codes(d["up"], _emin(case))
        return out
    x = _exact_values(d["codes"], d["exps"], case["cols"])
    if op == "restore":
        return x
    y, slope = _exact_act(case["kind"], x)
    dy = d["dy"].double()
    if not case["gated"]:
        return dict(dx=dy * slope)
    return dict(dx=dy * slope * _exact_values(d["up_codes"], d["up_exps"], case["cols"]), dup=dy * y)
