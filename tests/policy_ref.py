"""Plain 64-bit forms of the policy operators (include/policy.h), with bounds
on what a 32-bit evaluation of the same formulas may be off.

A bound carries, beside each value, the sum of the magnitudes that formed it
(what the roundings are relative to) through the same recurrence.  u is half
a step of fp32; half(dtype) that of the stored type."""
import numpy as np

U = 2.0 ** -24
# half a step of each stored type, relative, and of its smallest values
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
# (fp32: an exponential below 2^-126 counts as 0)
TINY = {"f32": 2.0 ** -125, "bf16": 2.0 ** -125, "f16": 2.0 ** -24}


def half(name, x):
    """Largest rounding of |x| to the stored type."""
    return HALF[name] * np.abs(x) + TINY[name]


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1 / (1 + e), e / (1 + e))


# Roundings of one step, each at most u of the step's magnitudes: the
# sigmoid (its exponent's product and what it rounds off 2, exp2 2, 1 + E 1,
# reciprocal 2, product 1) 8, b's product 1, the fused multiply-add 1; the map's
# slope takes the same 8 and a product; joining the maps of slots and tiles adds
# at most 2 per 8 steps.  12 covers a step.
STEP = 12


def recurrence(x, gate, h0, dones, sig, name):
    """x, gate [L, N, D], h0 [N, D] or None, dones [L, N] or None, float64 in
    and out: dict of h, h_last, the states entering each step, and bounds."""
    L, N, D = x.shape
    a = sigmoid(gate) if sig else gate
    keep = sigmoid(-gate) if sig else None
    b = keep * x if sig else x
    m = np.ones((L + 1, N, 1), bool)
    if dones is not None:
        m[1:] = (dones == 0)[:, :, None]
    state = np.zeros((N, D)) if h0 is None else h0.copy()
    mag, err = np.abs(state), np.zeros((N, D))
    h, prev, eh, eprev = (np.zeros((L, N, D)) for _ in range(4))
    for t in range(L):
        state, mag, err = (np.where(m[t], v, 0.0) for v in (state, mag, err))
        prev[t], eprev[t] = state, err
        state = a[t] * state + b[t]
        mag = np.abs(a[t]) * mag + np.abs(b[t])
        err = np.abs(a[t]) * err + STEP * U * mag
        h[t], eh[t] = state, err
    last = np.where(m[L], state, 0.0)
    return dict(h=h, h_last=last, prev=prev, eprev=eprev, a=a, keep=keep, m=m,
                eh=eh + half(name, np.abs(h) + eh),
                elast=np.where(m[L], err, 0.0) + half("f32", last))


def recurrence_grad(x, gate, h0, dones, dh, dh_last, sig, name):
    """The formula's gradient and its bounds; the state entering a step is
    taken as the stored h, so its rounding to the stored type counts."""
    f = recurrence(x, gate, h0, dones, sig, name)
    L, N, D = x.shape
    a, keep, m = f["a"], f["keep"], f["m"]
    G = np.zeros((N, D)) if dh_last is None else np.where(m[L], dh_last, 0.0)
    mag, err = np.abs(G), np.zeros((N, D))
    dx, dg, edx, edg = (np.zeros((L, N, D)) for _ in range(4))
    for t in range(L - 1, -1, -1):
        d = dh[t] + G
        dmag = np.abs(dh[t]) + mag
        derr = err + 2 * U * dmag
        p = f["prev"][t]
        # stored state: rounded once to the type, except h0 itself
        ep = f["eprev"][t] + (half(name, np.abs(p) + f["eprev"][t]) if t else 0.0)
        ep = np.where(m[t], ep, 0.0)
        if sig:
            dx[t] = keep[t] * d
            e = keep[t] * derr + 10 * U * np.abs(keep[t]) * dmag
            dg[t] = a[t] * dx[t] * (p - x[t])
            edg[t] = a[t] * ((np.abs(dx[t]) + e) * (ep + U * (np.abs(p) + np.abs(x[t]))) +
                             e * np.abs(p - x[t])) + 12 * U * np.abs(dg[t])
        else:
            dx[t], e = d, derr
            dg[t] = d * p
            edg[t] = (np.abs(d) + derr) * ep + derr * np.abs(p) + 2 * U * np.abs(dg[t])
        edx[t] = e + half(name, np.abs(dx[t]) + e)
        edg[t] += half(name, np.abs(dg[t]) + edg[t])
        G = np.where(m[t], a[t] * d, 0.0)
        mag = np.where(m[t], np.abs(a[t]) * dmag, 0.0)
        err = np.where(m[t], np.abs(a[t]) * derr + STEP * U * np.abs(a[t]) * dmag, 0.0)
    return dict(f, dx=dx, dgate=dg, dh0=G, edx=edx, edg=edg, edh0=err + half("f32", G))


def embed(weight, index, scale, name):
    V = weight.shape[0]
    known = (index >= 0) & (index < V)
    out = np.where(known[..., None], weight[np.where(known, index, 0)] * scale, 0.0) if V else \
        np.zeros(index.shape + (weight.shape[1],))
    return out, U * np.abs(out) + half(name, out)


def embed_grad(dout, index, V, scale, name):
    """Summing n values in any order in 32 bits is off by at most n - 1
    roundings of the sum of their magnitudes; the scale is one more."""
    index, dout = index.reshape(-1), dout.reshape(-1, dout.shape[-1])
    known = (index >= 0) & (index < V)
    dw, mag = np.zeros((2, V, dout.shape[1]))
    np.add.at(dw, index[known], dout[known])
    np.add.at(mag, index[known], np.abs(dout[known]))
    n = np.bincount(index[known], minlength=V)[:, None] if V else np.zeros((0, 1))
    err = (n + 1) * U * mag * abs(scale)
    dw = dw * scale
    return dw, err + half(name, np.abs(dw) + err)


def logits(z, name, bias=None, history=None, history_len=None, repetition=1.0, presence=0.0,
           frequency=0.0, allowed=None, dout=None):
    """[R, V] float64 in and out: out and its bound (division, presence,
    frequency's product and difference, bias: 5 roundings of the magnitudes),
    and with dout the gradients and theirs."""
    R, V = z.shape
    count = np.zeros((R, V))
    if history is not None:
        H = history.shape[1]
        lens = np.full(R, H) if history_len is None else np.clip(history_len, 0, H)
        for r in range(R):
            for v in history[r, :lens[r]]:
                if 0 <= v < V:
                    count[r, v] += 1
    rho, alpha, beta = (np.broadcast_to(np.asarray(x, np.float64).reshape(-1, 1), (R, V))
                        for x in (repetition, presence, frequency))
    seen = count > 0
    with np.errstate(invalid="ignore"):
        factor = np.where(seen, np.where(z > 0, 1 / rho, rho), 1.0)
        y = z * factor
        b = 0.0 if bias is None else np.broadcast_to(bias, (R, V))
        out = y - alpha * seen - beta * count + b
        mag = np.abs(y) + np.abs(alpha) * seen + np.abs(beta) * count + np.abs(b)
        err = 5 * U * mag
        bound = err + half(name, np.abs(out) + err)
    ok = np.ones((R, V), bool) if allowed is None else np.broadcast_to(allowed, (R, V))
    res = dict(out=np.where(ok, out, -np.inf), eout=np.where(ok, bound, 0.0))
    if dout is not None:
        g = np.where(ok, dout, 0.0)
        res["dlogits"] = g * np.where(ok, factor, 1.0)
        res["edl"] = U * np.abs(res["dlogits"]) + half(name, res["dlogits"])
        res["dbias"] = g.sum(0)
        res["edb"] = R * U * np.abs(g).sum(0) + half("f32", res["dbias"])
    return res
