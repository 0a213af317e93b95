"""The step over a list of tensors in 64 bits, from its definition, with the
bounds that fp32 operations rounded one by one stay within (H = 2^-24 per
rounding; the bounds add the roundings of each term, first order, and take 1%
on top for the products of them)."""
import numpy as np

H = 2.0 ** -24
ROW = 256
MOST4, MOST5 = 448.0, 57344.0
SCALE_MIN = 2.0 ** -126
SLACK = 1.01
TINY = 2.0 ** -140                     # a few fp32 subnormal steps


def mix(h):
    h = ((h ^ (h >> np.uint64(16))) * np.uint64(0x7FEB352D)) & np.uint64(0xFFFFFFFF)
    h = ((h ^ (h >> np.uint64(15))) * np.uint64(0x846CA68B)) & np.uint64(0xFFFFFFFF)
    return h ^ (h >> np.uint64(16))


def random16(rows, t, seed):
    """(rows, 256) 16-bit numbers of step t, from the documented definition."""
    m32 = np.uint64(0xFFFFFFFF)
    base = mix(np.array([(t + seed) & 0xFFFFFFFF], np.uint64))
    key = mix((base + np.arange(rows, dtype=np.uint64)) & m32)
    q = np.arange(64, dtype=np.uint64) * np.uint64(0x9E3779B9)
    h = mix((key[:, None] + q) & m32)
    k = (h * np.uint64(0x2C1B3C6D)) & m32
    k = k ^ (k >> np.uint64(13))
    lo = np.uint64(0xFFFF)
    return np.stack((h & lo, h >> np.uint64(16), k & lo, k >> np.uint64(16)),
                    2).reshape(rows, ROW).astype(np.float64)


def nearest_e4m3(y):
    """To the nearest e4m3 value, ties to even, on 64-bit values."""
    e = np.maximum(np.frexp(np.abs(y))[1] - 1, -6)
    q = np.ldexp(1.0, e - 3)
    return np.clip(np.rint(y / q) * q, -MOST4, MOST4)


def random_e5m2(y, r16):
    """Cut to e5m2 after adding r16 / 65536 of a step; 0 stays 0."""
    z = np.maximum(y, 2.0 ** -14)
    q = np.ldexp(1.0, np.frexp(z)[1] - 1 - 2)
    return np.where(y > 0, np.minimum(np.floor(z / q + r16 / 65536.0) * q, MOST5), 0.0)


class ListReference:
    """Arenas in 64 bits and the step state of a list, stepped beside the
    library's (whose rounded states each step starts from)."""

    def __init__(self, numels, hp, loss_scale=1.0, lr_mult=None, decay_mult=None, seed=0):
        self.n = list(numels)
        self.rows = [-(-x // ROW) for x in self.n]
        self.row0 = np.concatenate(([0], np.cumsum(self.rows))).astype(int)
        self.hp = hp
        self.lr_mult = np.ones(len(self.n)) if lr_mult is None else np.asarray(lr_mult, float)
        self.decay_mult = np.ones(len(self.n)) if decay_mult is None else np.asarray(decay_mult, float)
        self.seed = seed

    def arena(self, tensors):
        out = np.zeros(int(self.row0[-1]) * ROW)
        for k, t in enumerate(tensors):
            a = int(self.row0[k]) * ROW
            out[a:a + self.n[k]] = t
        return out

    def per_row(self, x):
        return np.repeat(np.repeat(np.asarray(x, float), self.rows), ROW)

    def step(self, grads, p, m, v, t, loss_scale, bits, m_scale=None, v_scale=None):
        """One applied step t (from 1) on arenas of the library's own values:
        the new values and the bounds of each."""
        hp = self.hp
        sums = [float(np.sum((np.asarray(g, float) / loss_scale) ** 2)) for g in grads]
        total = float(np.sum(sums))
        coef = 1.0
        if hp["max_grad_norm"] > 0:
            coef = min(1.0, hp["max_grad_norm"] / (np.sqrt(total) + 1e-6))
        g = self.arena(grads) / loss_scale * coef
        b1, b2 = hp["beta1"], hp["beta2"]
        held = 0 if bits == 32 else 1                    # the product code * scale
        if bits == 8:
            m = m * np.repeat(m_scale.astype(float), ROW)
            v = v * np.repeat(v_scale.astype(float), ROW)
        # coefficient, product, sum (and the held value); g: coef and its product
        m_err = H * ((3 + held) * np.abs(b1 * m) + 5 * np.abs((1 - b1) * g)) * SLACK + TINY
        v_err = H * ((3 + held) * b2 * v + 8 * (1 - b2) * g * g) * SLACK + TINY
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g * g
        lr = self.per_row(hp["lr"] * self.lr_mult)
        keep = 1 - lr * hp["weight_decay"] * self.per_row(self.decay_mult)
        bc1, bc2 = 1 - b1 ** t, 1 - b2 ** t
        d = np.sqrt(v / bc2) + hp["eps"]
        upd = lr * (m / bc1) / d
        # sqrt halves the relative error of v; then bc2, its quotient, the root
        # and the sum (32 bits), or the root to 2 ulp, the factor and its
        # product, and the sum (8 bits); TINY may be all there is of v
        with np.errstate(divide="ignore", invalid="ignore"):
            root = np.where(v > 0, np.minimum(0.5 * v_err / v, 1.0), 0.0)
        d_rel = root + (3 if bits == 32 else 7) * H
        d_rel = np.where(np.sqrt(v / bc2) < 1e-3 * hp["eps"], 1e-3, d_rel)
        upd_err = lr / bc1 / d * m_err + np.abs(upd) * (d_rel + (6 if bits == 32 else 7) * H)
        new = p * keep - upd
        p_err = (H * 3 * np.abs(p * keep) + upd_err + H * np.abs(new)) * SLACK + TINY
        return dict(p=new, m=m, v=v, p_err=p_err, m_err=m_err, v_err=v_err,
                    norm=np.sqrt(total), sums=sums, coef=coef)

    def check_codes(self, ref, t, m, v, m_scale, v_scale):
        """The 8-bit states: scales of each row's largest value, and every code
        between the roundings of the ends of its value's interval."""
        R = int(self.row0[-1])
        for name, x, err, sc, most in (("m", ref["m"], ref["m_err"], m_scale, MOST4),
                                       ("v", ref["v"], ref["v_err"], v_scale, MOST5)):
            x, err = x.reshape(R, ROW), err.reshape(R, ROW)
            top = np.abs(x).max(1)
            at = np.abs(x).argmax(1)
            sc = sc.astype(float)
            want = np.maximum(top / most, SCALE_MIN)
            tol = np.maximum(err.max(1), err[np.arange(R), at]) / most + 3 * H * want
            zero = top == 0
            assert np.all(sc[zero] == 0), "%s: a row of zeros has a scale" % name
            bad = np.abs(sc - want) > tol
            assert not np.any(bad & ~zero), "%s scales: %d rows off" % (name, int(np.sum(bad & ~zero)))
        r16 = random16(R, t, self.seed)
        for name, x, err, sc, code, rnd in (
                ("m", ref["m"], ref["m_err"], m_scale, m, lambda y: nearest_e4m3(y)),
                ("v", ref["v"], ref["v_err"], v_scale, v, lambda y: random_e5m2(y, r16))):
            x, err = x.reshape(R, ROW), err.reshape(R, ROW)
            inv = np.where(sc > 0, 1 / np.where(sc > 0, sc, 1).astype(float), 0.0)[:, None]
            y, dy = x * inv, err * inv + 3 * H * np.abs(x * inv)
            lo, hi = rnd(np.maximum(y - dy, 1e-300) if name == "v" else y - dy), rnd(y + dy)
            code = code.reshape(R, ROW)
            live = x != 0
            ok = (code >= lo) & (code <= hi) | (~live & (code == 0))
            assert np.all(ok), "%s codes: %d off, first %s" % (
                name, int(np.sum(~ok)), [(y[i], code[i], lo[i], hi[i]) for i in
                                         [tuple(np.argwhere(~ok)[0])]])


def hold_in_fp32(g, m, v, m_scale, v_scale, hp, inv_coef, t, seed):
    """The 8-bit states after step t by fp32 operations rounded one by one, on
    arenas of gradients and codes: (m codes, v codes, m scales, v scales)."""
    f = np.float32
    R = len(m_scale)
    g = g.astype(f).reshape(R, ROW) * f(inv_coef)
    m, v = m.astype(f).reshape(R, ROW), v.astype(f).reshape(R, ROW)
    m = f(hp["beta1"]) * (m * m_scale[:, None]) + f(1 - hp["beta1"]) * g
    v = f(hp["beta2"]) * (v * v_scale[:, None]) + f(1 - hp["beta2"]) * (g * g)

    def scaled(x, most):
        top = np.minimum(np.abs(x).max(1), np.finfo(f).max)
        sc = np.where(top > 0, np.maximum(top * f(1.0 / most), f(SCALE_MIN)), f(0))
        inv = np.where(sc > 0, f(1) / np.where(sc > 0, sc, f(1)), f(0))
        return x * inv[:, None], sc
    ym, ms = scaled(m, MOST4)
    yv, vs = scaled(v, MOST5)
    assert ym.dtype == yv.dtype == ms.dtype == vs.dtype == f
    y = np.maximum(yv, f(2.0 ** -14)).view(np.uint32).astype(np.int64)
    code = np.minimum(((y + 32 * random16(R, t, seed).astype(np.int64)) >> 21) - 448, 0x7B)
    code = np.where(v > 0, code, 0)
    val = np.ldexp(np.where(code >> 2, 4 + (code & 3), code & 3).astype(np.float64),
                   np.maximum(code >> 2, 1) - 17)
    return nearest_e4m3(ym.astype(np.float64)).reshape(-1), val.reshape(-1), ms, vs
