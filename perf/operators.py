"""The operators over a list of tensors, as measured: gradient statistics
(sum of squares per tensor and over all, overflow), and the AdamW step with
32-bit states and with 8-bit states.

Every array of the step's state is an arena of rows of 256 elements: tensor k
takes ceil(n_k / 256) consecutive rows, its last row padded with zeros, so that
the plain forms work on (rows, 256) matrices.  The gradients come either as
tensors of their own or as views of one packed buffer, where odd sizes leave
them at any offset; the 16-bit parameters are always views of one packed
buffer, as unflattening a gathered flat parameter gives them.
"""
import math
import random

import torch

own = False

ROW = 256
HP = dict(lr=3e-5, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, max_grad_norm=1.0)
STEP0 = 100                       # the states are those of a run that has made 100 steps
FLOATS = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
# the 8-bit states: the format of each and its largest value
M8, M8_MAX = torch.float8_e4m3fn, 448.0
V8, V8_MAX = torch.float8_e5m2, 57344.0
V8_MIN = 2.0 ** -14               # the least code of a second moment above zero
SEED = 7                          # of the second moment's random rounding
SCALE_MIN = 2.0 ** -126
FLT_MAX = torch.finfo(torch.float32).max

# a two-layer MLP, one transformer block of 4096/11008, the same block's
# per-parameter shards on one of 8 ranks, and the flat shard of 10B over 8 ranks
MLP = (512 * 1024, 1024, 1024 * 512, 512)
BLOCK = (4096 * 4096,) * 4 + (11008 * 4096, 11008 * 4096, 4096 * 11008, 4096, 4096)
SIZES = {"mlp": MLP, "block": BLOCK, "block_n8": tuple(n // 8 for n in BLOCK),
         "shard": (1_250_000_000,)}


def _case(name, op, sizes, grad, param="none", count=0, numel=0, size_seed=0, packed=False,
          stats=True, overflow=False):
    return dict(name=name, op=op, sizes=sizes, grad=grad, param=param, count=count, numel=numel,
                size_seed=size_seed, packed=packed, stats=stats, overflow=overflow)


def listed():
    return [
        # the statistics of a small model's step: launch latency
        _case("norm_mlp_fp16", "norm", "mlp", "fp16"),
        # one transformer block's gradients before clipping
        _case("norm_block_bf16", "norm", "block", "bf16"),
        # hundreds of odd-sized fp32 gradients in one bucket (adapters, reduced in fp32)
        _case("norm_many_fp32", "norm", "random", "fp32", count=700, numel=20_000_000, size_seed=1,
              packed=True),
        # a small model's whole step: loss scale, overflow test, clip, update
        _case("adamw32_mlp_fp16", "adamw32", "mlp", "fp16", "fp16"),
        # one transformer block's whole step in bf16
        _case("adamw32_block_bf16", "adamw32", "block", "bf16", "bf16"),
        # many odd-sized tensors in one bucket, no clipping: the update alone
        _case("adamw32_many_bf16", "adamw32", "random", "bf16", "bf16", count=290,
              numel=30_000_000, size_seed=2, packed=True, stats=False),
        # per-parameter shards of a block on one of 8 ranks, gradients reduced in fp32
        _case("adamw32_block_n8_fp32", "adamw32", "block_n8", "fp32", "bf16"),
        # the same paths with 8-bit states
        _case("adamw8_mlp_fp16", "adamw8", "mlp", "fp16", "fp16"),
        _case("adamw8_block_bf16", "adamw8", "block", "bf16", "bf16"),
        _case("adamw8_many_bf16", "adamw8", "random", "bf16", "bf16", count=290,
              numel=30_000_000, size_seed=2, packed=True, stats=False),
        # fp32 parameters trained in place: no 16-bit copy
        _case("adamw8_block_n8_fp32", "adamw8", "block_n8", "fp32"),
        # the flat shard of 10B parameters over 8 ranks with 8-bit states
        _case("adamw8_shard_fp16", "adamw8", "shard", "fp16", "fp16"),
    ]


def draw(rng):
    op = rng.choice(("norm", "adamw32", "adamw8"))
    count = int(round(math.exp(rng.uniform(0.0, math.log(800.0)))))
    numel = max(count, int(math.exp(rng.uniform(math.log(1e3), math.log(2e8)))))
    grad = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    param = "none" if op == "norm" else rng.choice(("bf16", "fp16", "none"))
    stats = op == "norm" or rng.random() < 0.7
    return dict(op=op, sizes="random", grad=grad, param=param, count=count, numel=numel,
                size_seed=rng.randrange(1 << 30), packed=rng.random() < 0.5, stats=stats,
                overflow=stats and rng.random() < 0.12)


def _numels(case):
    if case["sizes"] != "random":
        return list(SIZES[case["sizes"]])
    r = random.Random(case["size_seed"])
    w = [math.exp(r.gauss(0.0, 1.5)) for _ in range(case["count"])]
    return [max(1, int(case["numel"] * x / sum(w))) for x in w]


def _mults(case, n):
    """(learning-rate factor, decay factor) per tensor: tensors of up to 4096
    elements (norms, biases) take no decay, every fifth a tenth of the rate."""
    return ([0.1 if k % 5 == 4 else 1.0 for k in range(len(n))],
            [0.0 if x <= 4096 else 1.0 for x in n])


def _loss_scale(case):
    return 65536.0 if case["grad"] == "fp16" else 1.0


def _scaled(x, most):
    """(an arena divided by one scale per row, the scales)."""
    top = x.amax(1).maximum(-x.amin(1)).clamp(max=FLT_MAX)
    scale = torch.where(top > 0, (top * (1.0 / most)).clamp(min=SCALE_MIN), 0.0)
    inv = torch.where(top > 0, 1.0 / scale, 0.0)
    return (x * inv[:, None]).clamp(-most, most), scale


def _mix(h):
    """A bijection of 32-bit numbers (in int64): xor-shifts and multiplications."""
    h = (h ^ (h >> 16)) * 0x7FEB352D & 0xFFFFFFFF
    h = (h ^ (h >> 15)) * 0x846CA68B & 0xFFFFFFFF
    return h ^ (h >> 16)


def _random16(rows, step):
    """The 16-bit numbers that the second moments of an arena are rounded with
    at a step, a function of seed, step, row and place: one 32-bit number gives
    a quad's first two, one more multiplication its last two."""
    row = torch.arange(rows, device="cuda")
    key = _mix(_mix((step.to(torch.int64) + SEED) & 0xFFFFFFFF) + row & 0xFFFFFFFF)
    h = _mix(key[:, None] + torch.arange(64, device="cuda") * 0x9E3779B9 & 0xFFFFFFFF)
    k = h * 0x2C1B3C6D & 0xFFFFFFFF
    k = k ^ (k >> 13)
    return torch.stack((h & 0xFFFF, h >> 16, k & 0xFFFF, k >> 16), 2).view(rows, ROW).to(torch.int32)


def _hold(m, v, step):
    """The 8-bit states of m (to the nearest) and v (at random, so that its mean
    moves by what one step adds, far less than the distance between codes)."""
    y, m_scale = _scaled(m, M8_MAX)
    m = y.to(M8)
    y, v_scale = _scaled(v, V8_MAX)
    y = y.clamp_(min=V8_MIN).view(torch.int32).add_(_random16(v.shape[0], step), alpha=32)
    y = (y >> 21).sub_(112 << 2).clamp_(max=0x7B)
    v = torch.where(v > 0, y, 0).to(torch.uint8).view(V8)
    return dict(m=m, m_scale=m_scale, v=v, v_scale=v_scale)


def _inputs(case, seed):
    """What the user's program holds, from the seed alone: the gradients and
    the arenas of master, m and v, of a run under way."""
    n = _numels(case)
    rows = [-(-x // ROW) for x in n]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)
    row_of = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(rows)).cuda()
    first = torch.tensor([0] + rows).cumsum(0)
    # the elements that each row holds
    left = (first[:-1] * ROW + torch.tensor(n)).cuda()[row_of] - torch.arange(sum(rows), device="cuda") * ROW
    real = torch.arange(ROW, device="cuda") < left[:, None]
    live = real.clone()
    if case["op"] != "norm":
        # rows that no gradient ever reached (an embedding's unused ones): all zero
        live[: rows[0] // 8] = False
    sigma = torch.tensor([10.0 ** host.uniform(-4, -2) for _ in n], device="cuda")[row_of][:, None]

    def normal():
        return torch.randn(sum(rows), ROW, generator=gen, device="cuda")

    g = normal().mul_(sigma).mul_(live)
    stored = g.mul(_loss_scale(case)).to(FLOATS[case["grad"]]).view(-1)
    if case["overflow"]:
        stored[int(first[len(n) // 2]) * ROW] = float("inf")
    starts = [int(x) * ROW for x in first[:-1]]
    grads = [stored[a:a + x] for a, x in zip(starts, n)]
    if case["packed"]:
        grads = list(torch.cat(grads).split(n))
    else:
        grads = [x.clone() for x in grads]
    d = dict(n=n, rows=rows, row_of=row_of, starts=starts, grads=grads)
    if case["op"] != "norm":
        d["master"] = normal().mul_(0.02).mul_(real)
        d["m"] = normal().mul_(sigma).mul_(0.3).mul_(live)
        d["v"] = normal().square_().add_(0.2).mul_(sigma * sigma).mul_(live)
        if case["op"] == "adamw8":
            d.update(_hold(d["m"], d["v"], torch.tensor(STEP0, device="cuda")))
    return d


def _pows():
    return HP["beta1"] ** STEP0, HP["beta2"] ** STEP0


def _hp(case):
    return dict(HP, max_grad_norm=HP["max_grad_norm"] if case["stats"] else 0.0)


def prepare(case, seed):
    d = _inputs(case, seed)
    n, dev = d["n"], "cuda"
    lr_mult, decay_mult = _mults(case, n)
    scale, dynamic = _loss_scale(case), case["grad"] == "fp16"
    s = dict(case=case, grads=d["grads"])
    packed = None
    if case["param"] != "none":
        packed = torch.zeros(sum(n), dtype=FLOATS[case["param"]], device=dev)
    if own:
        import fsdp_sharded_mixed_flatparameter_amd as zf
        if case["op"] == "norm":
            s["state"] = zf.StepState(scale, dynamic)
            s["plan"] = zf.MultiPlan(n, FLOATS[case["grad"]])
            s["plan"].bind(d["grads"])
            s["zf"] = zf
            s["out"] = dict(tensor_sumsq=s["plan"].tensor_sumsq, sumsq=s["state"].field("sumsq"),
                            overflow=s["state"].field("overflow"))
            return s
        masters = [d["master"].view(-1)[a:a + x] for a, x in zip(d["starts"], n)]
        opt = zf.TensorListOptimizer(masters, _hp(case), state_bits=8 if case["op"] == "adamw8" else 32,
                                     loss_scale=scale, dynamic=dynamic, lr_mult=lr_mult,
                                     decay_mult=decay_mult, statistics=case["stats"], seed=SEED,
                                     grad_dtype=FLOATS[case["grad"]],
                                     param_dtype=None if packed is None else packed.dtype)
        opt.exp_avg.copy_(d["m"].view(-1))
        opt.exp_avg_sq.copy_(d["v"].view(-1))
        if case["op"] == "adamw8":
            opt.exp_avg_scale.copy_(d["m_scale"])
            opt.exp_avg_sq_scale.copy_(d["v_scale"])
        st = opt.state.read()
        st.step, (st.beta1_pow, st.beta2_pow) = STEP0, _pows()
        opt.state.upload(st)
        opt.bind(d["grads"], None if packed is None else list(packed.split(n)))
        f = opt.state.field
        out = dict(master=opt.master, m=opt.exp_avg, v=opt.exp_avg_sq, norm=f("last_norm"),
                   step=f("step"), skipped=f("last_skipped"), loss_scale=f("loss_scale"))
        if case["op"] == "adamw8":
            out.update(m_scale=opt.exp_avg_scale, v_scale=opt.exp_avg_sq_scale)
        if packed is not None:
            out.update(param=packed)
        s.update(opt=opt, out=out)
        return s
    # the plain forms keep which row belongs to which tensor, the padding that
    # makes an arena of the gradients, and the per-tensor factors
    pads = [torch.zeros(r * ROW - x, dtype=FLOATS[case["grad"]], device=dev)
            for r, x in zip(d["rows"], n)]
    s["parts"] = [t for pair in zip(d["grads"], pads) for t in pair]
    s.update({k: d[k] for k in ("n", "rows", "row_of", "starts", "master", "m", "v", "m_scale", "v_scale")
              if k in d}, packed=packed)
    f64 = dict(dtype=torch.float64, device=dev)
    s["lr_mult"], s["decay_mult"] = torch.tensor(lr_mult, **f64), torch.tensor(decay_mult, **f64)
    b1, b2 = _pows()
    s["b1_pow"], s["b2_pow"] = torch.tensor(b1, **f64), torch.tensor(b2, **f64)
    s["scale"] = torch.tensor(scale, device=dev)
    s["slot"] = d["row_of"] * ROW + torch.arange(sum(d["rows"]), device=dev) % ROW
    s["dynamic"] = dynamic
    s["good"] = torch.zeros((), dtype=torch.int32, device=dev)
    s["step"] = torch.full((), STEP0, dtype=torch.int32, device=dev)
    return s


def _unscaled(s):
    return torch.cat(s["parts"]).float().view(-1, ROW) * (1.0 / s["scale"])


def _plain_norm(s):
    rows = _unscaled(s).double().square_().sum(1)
    # row sums into 256 sums per tensor (few rows meet in one), then those
    per = torch.zeros(len(s["n"]) * ROW, dtype=torch.float64, device=rows.device)
    per = per.index_add_(0, s["slot"], rows).view(-1, ROW).sum(1)
    total = per.sum()
    return dict(tensor_sumsq=per, sumsq=total, overflow=(~torch.isfinite(total)).to(torch.int32))


def _plain_step(s):
    case, hp, q8 = s["case"], _hp(s["case"]), s["case"]["op"] == "adamw8"
    u = _unscaled(s)
    total = u.double().square_().sum() if case["stats"] else torch.zeros_like(s["b1_pow"])
    skip = ~torch.isfinite(total)
    if case["stats"]:
        u *= (hp["max_grad_norm"] / (total.sqrt() + 1e-6)).clamp(max=1.0).float()
    b1_pow, b2_pow = s["b1_pow"] * hp["beta1"], s["b2_pow"] * hp["beta2"]
    rate = hp["lr"] * s["lr_mult"]
    keep = (1.0 - rate * (hp["weight_decay"] * s["decay_mult"])).float()[s["row_of"]][:, None]
    old = {k: s[k] for k in ("master", "m", "v", "m_scale", "v_scale") if k in s}
    m, v = old["m"], old["v"]
    if q8:
        m = m.float() * old["m_scale"][:, None]
        v = v.float() * old["v_scale"][:, None]
    m = hp["beta1"] * m + (1.0 - hp["beta1"]) * u
    v = hp["beta2"] * v + (1.0 - hp["beta2"]) * u.square_()
    del u
    new = {}
    if q8:
        rate = (rate / (1.0 - b1_pow)).float()[s["row_of"]][:, None]
        d = v.sqrt() * (1.0 / (1.0 - b2_pow).sqrt()).float() + hp["eps"]
        new["master"] = old["master"] * keep - (rate * m) / d
        del d
        new.update(_hold(m, v, s["step"] + 1))
    else:
        rate = rate.float()[s["row_of"]][:, None]
        d = (v / (1.0 - b2_pow).float()).sqrt_() + hp["eps"]
        new["master"] = old["master"] * keep - (rate * (m / (1.0 - b1_pow).float())) / d
        del d
        new["m"], new["v"] = m, v
    del m, v
    if case["stats"]:
        new = {k: torch.where(skip, old[k].view(torch.uint8), x.view(torch.uint8)).view(x.dtype)
               if x.element_size() == 1 else torch.where(skip, old[k], x) for k, x in new.items()}
    s.update(new)
    out = dict(new)
    if s["packed"] is not None:
        flat = new["master"].view(-1)
        copy = torch.cat([flat[a:a + x] for a, x in zip(s["starts"], s["n"])]).to(s["packed"].dtype)
        s["packed"] = torch.where(skip, s["packed"], copy)
        out["param"] = s["packed"]
    # the loss scaler and the counters
    s["b1_pow"], s["b2_pow"] = torch.where(skip, s["b1_pow"], b1_pow), torch.where(skip, s["b2_pow"], b2_pow)
    s["step"] = s["step"] + (~skip).to(torch.int32)
    if s["dynamic"]:
        good = torch.where(skip, 0, s["good"] + 1)
        grow = good == 1000
        s["scale"] = torch.where(skip, (s["scale"] * 0.5).clamp(min=1.0),
                                 torch.where(grow, s["scale"] * 2.0, s["scale"]))
        s["good"] = torch.where(grow, 0, good)
    out.update({k: x.view(-1) for k, x in out.items()})
    out.update(norm=total.sqrt(), step=s["step"], skipped=skip.to(torch.int32), loss_scale=s["scale"])
    return out


def run(s):
    if own:
        if s["case"]["op"] == "norm":
            s["zf"].zero_multi_unscale_norm(s["plan"], s["state"], reset=True)
        else:
            s["opt"].step()
        return s["out"]
    return _plain_norm(s) if s["case"]["op"] == "norm" else _plain_step(s)


def work(case):
    n = sum(_numels(case))
    g = torch.empty((), dtype=FLOATS[case["grad"]]).element_size()
    if case["op"] == "norm":
        return dict(bytes=n * g, flops=3 * n)
    copy = 0 if case["param"] == "none" else 2
    state = 4 if case["op"] == "adamw8" else 16
    scales = 16 * sum(-(-x // ROW) for x in _numels(case)) if case["op"] == "adamw8" else 0
    return dict(bytes=n * (g + 8 + state + copy) + scales, flops=24 * n)


def _rounded(y, bits, least, offset):
    """y in 64 bits rounded down to `bits` mantissa bits (of 2^least or more), after
    adding offset (in units of the last bit); offset None: to the nearest, ties to even."""
    e = torch.frexp(y.abs().clamp(min=2.0 ** least)).exponent - 1
    quantum = torch.ldexp(torch.ones_like(y), e - bits)
    y = y / quantum
    return (torch.round(y) if offset is None else torch.floor(y + offset)) * quantum


def exact(case, seed):
    d = _inputs(case, seed)
    hp, n, starts = _hp(case), d["n"], d["starts"]
    scale = _loss_scale(case)
    per = torch.stack([(x.double() / scale).square().sum() for x in d["grads"]])
    total = per.sum()
    bad = not math.isfinite(float(total))
    if case["op"] == "norm":
        return dict(tensor_sumsq=per, sumsq=total, overflow=int(bad))
    q8 = case["op"] == "adamw8"
    lr_mult, decay_mult = _mults(case, n)
    coef = min(1.0, hp["max_grad_norm"] / (math.sqrt(float(total)) + 1e-6)) if case["stats"] and not bad else 1.0
    t = STEP0 + 1
    out = dict(master=[], m=[], v=[], param=[], m_scale=[], v_scale=[])
    random16 = _random16(sum(d["rows"]), torch.tensor(t, device="cuda")) if q8 else None

    def scaled(x, most):
        top = x.abs().amax(1, keepdim=True)
        s = torch.where(top > 0, (top / most).clamp(min=SCALE_MIN), 1.0)
        return (x / s).clamp(-most, most), torch.where(top > 0, s, 0.0)[:, 0]

    for k, (a, x, r) in enumerate(zip(starts, n, d["rows"])):
        rows = slice(a // ROW, a // ROW + r)
        p, m, v = (d[q][rows].double() for q in ("master", "m", "v"))
        if q8:
            ms, vs = d["m_scale"][rows], d["v_scale"][rows]
            old = (p, m, v, ms, vs)
            m, v = m * ms[:, None].double(), v * vs[:, None].double()
        else:
            old = (p, m, v)
        if not bad or not case["stats"]:
            g = torch.zeros(r * ROW, dtype=torch.float64, device="cuda")
            g[:x] = d["grads"][k].double() / scale * coef
            g = g.view(r, ROW)
            lr = hp["lr"] * lr_mult[k]
            m = hp["beta1"] * m + (1 - hp["beta1"]) * g
            v = hp["beta2"] * v + (1 - hp["beta2"]) * g ** 2
            step = lr * (m / (1 - hp["beta1"] ** t)) / ((v / (1 - hp["beta2"] ** t)).sqrt() + hp["eps"])
            p = p * (1 - lr * hp["weight_decay"] * decay_mult[k]) - step
            if q8:
                (m, ms), (y, vs) = scaled(m, M8_MAX), scaled(v, V8_MAX)
                m = _rounded(m, 3, -6, None)
                y = _rounded(y.clamp(min=V8_MIN), 2, -14, random16[rows].double() / 65536)
                v = torch.where(v > 0, y.clamp(max=V8_MAX), 0.0)
            old = (p, m, v, ms, vs) if q8 else (p, m, v)
        for key, y in zip(("master", "m", "v", "m_scale", "v_scale"), old):
            out[key].append(y.reshape(-1))
        out["param"].append(torch.zeros(x, dtype=torch.float64, device="cuda") if bad and case["stats"]
                            else p.reshape(-1)[:x])
    out = {k: torch.cat(v).double() for k, v in out.items() if v}
    if case["param"] == "none":
        out.pop("param")
    # a skipped step's norm is not finite; an update without statistics has none
    out.update(norm=total.sqrt() if case["stats"] else torch.zeros_like(total), step=STEP0 + (not bad or not case["stats"]),
               skipped=int(bad and case["stats"]),
               loss_scale=scale / 2 if bad and case["stats"] and case["grad"] == "fp16" else scale)
    return out
