"""Plain 64-bit forms of the operators of a residual block (include/block.h),
with bounds on what a 32-bit evaluation of the same formulas may be off.

u is half a step of fp32.  Beside each value goes a bound of its error to first
order (products of two errors are below 1e-6 of the bounds; SLACK covers them):
a rounding adds u times the magnitudes that were added, an error passes on by
the derivative."""
import numpy as np

from policy_ref import U, half, sigmoid

SLACK = 1.02
TINY = 2.0 ** -120  # products whose factors underflow


def fin(name, value, err):
    """The bound of a stored value: its error and one rounding to the type."""
    err = SLACK * err + TINY
    return err + half(name, np.abs(value) + err)


def e_sigmoid(z):
    """Relative error of sigmoid(z): the exponent's product and its constant
    (|z| log2(e) u each, times ln 2), exp2 2 u, 1 + E, reciprocal 2 u."""
    return U * (2 * np.abs(z) + 6)


def silu_slope(z):
    s = sigmoid(z)
    return s * (1 + z * (1 - s))


def e_silu_slope(z):
    """s (1 + z (1 - s)): s by its relative error, 1 - s by s's and a rounding,
    the product and the sum one rounding each of at most 1 + |z|."""
    s = sigmoid(z)
    return s * (1 + np.abs(z)) * (e_sigmoid(z) * 2 + 4 * U)


# --------------------------------------------------------------- convolution
def conv(x, weight, bias, state, dones, silu, name, dy=None, dnew=None):
    """[L, N, D], [D, W], [D] or None, [N, W - 1, D] or None, [L, N] or None."""
    L, N, D = x.shape
    W = weight.shape[1]
    bias = np.zeros(D) if bias is None else bias
    state = np.zeros((N, W - 1, D)) if state is None else state
    past = np.concatenate([state.transpose(1, 0, 2), x])  # step t at W - 1 + t
    episode = np.zeros((L + W, N), int)
    if dones is not None:
        episode[W:] = np.cumsum(dones != 0, 0)  # row W - 1 + t: dones before step t
    same = lambda t, j: (episode[t + j] == episode[t + W - 1])[:, None]  # tap j of step t
    p, mag = np.zeros((2, L, N, D))
    for t in range(L):
        p[t] = bias
        mag[t] = np.abs(bias)
        for j in range(W):
            v = np.where(same(t, j), past[t + j], 0.0) * weight[:, j]
            p[t] += v
            mag[t] += np.abs(v)
    ep = (W + 1) * U * mag
    s = sigmoid(p)
    y = p * s if silu else p
    ey = 1.1 * ep + np.abs(y) * (e_sigmoid(p) + U) if silu else ep
    left = np.stack([np.where((episode[L + j] == episode[L + W - 1])[:, None], past[L + j], 0.0)
                     for j in range(W - 1)], 1) if W > 1 else np.zeros((N, 0, D))
    res = dict(y=y, ey=fin(name, y, ey), new_state=left)
    if dy is None:
        return res
    dp = dy * silu_slope(p) if silu else dy
    # the slope's own slope is below 1/2
    edp = np.abs(dy) * (0.5 * ep + e_silu_slope(p)) + U * np.abs(dp) if silu else np.zeros_like(dy)
    dpast, epast, mpast = np.zeros((3,) + past.shape)
    dw, edw, mdw = np.zeros((3, D, W))
    for t in range(L):
        for j in range(W):
            ok = same(t, j)
            dpast[t + j] += np.where(ok, dp[t] * weight[:, j], 0.0)
            mpast[t + j] += np.where(ok, np.abs(dp[t] * weight[:, j]), 0.0)
            epast[t + j] += np.where(ok, edp[t] * np.abs(weight[:, j]), 0.0)
            v = np.where(ok, past[t + j], 0.0)
            dw[:, j] += (dp[t] * v).sum(0)
            mdw[:, j] += np.abs(dp[t] * v).sum(0)
            edw[:, j] += (edp[t] * np.abs(v)).sum(0)
    if dnew is not None:
        for j in range(W - 1):
            ok = (episode[L + j] == episode[L + W - 1])[:, None]
            dpast[L + j] += np.where(ok, dnew[:, j], 0.0)
            mpast[L + j] += np.where(ok, np.abs(dnew[:, j]), 0.0)
    epast += (W + 1) * U * mpast
    # a sum's longest chain: a thread's steps, a workgroup's rows (at most
    # 256), column sums (at most 64 / 4 + 8, twice)
    n = L + 256 + 48
    db = dp.sum((0, 1))
    edb = edp.sum((0, 1)) + n * U * np.abs(dp).sum((0, 1))
    dstate = dpast[:W - 1].transpose(1, 0, 2)
    res.update(dx=dpast[W - 1:], edx=fin(name, dpast, epast)[W - 1:], dweight=dw,
               edweight=fin("f32", dw, edw + n * U * mdw), dbias=db, edbias=fin("f32", db, edb), dstate=dstate,
               edstate=fin(name, dpast, epast)[:W - 1].transpose(1, 0, 2))
    return res


# ---------------------------------------------------------------------- scan
def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def scan(x, delta, rate, b, c, skip, gate, bias, state, dones, soft, name, dy=None, dnew=None):
    """x, delta, gate [L, N, D]; b, c [L, N, G, S]; rate [D, S]; float64."""
    L, N, D = x.shape
    S, G = rate.shape[1], b.shape[2]
    zero = np.zeros(D)
    skip, bias = (zero if v is None else v for v in (skip, bias))
    wide = lambda t: np.repeat(t, D // G, 1)  # [N, G, S] as the channels meet it
    v = delta + bias
    ev = U * (np.abs(delta) + np.abs(bias))
    if soft:
        dt, sg = softplus(v), sigmoid(v)
        # log(1 + E): E by sigmoid's count, 16 roundings of the series and sums
        edt = ev * sg + U * (2 * np.abs(v) + 16) * softplus(-np.abs(v)) + U * dt
        esg = sg * (e_sigmoid(v) + ev)
    else:
        dt, sg, edt, esg = v, np.ones_like(v), ev, np.zeros_like(v)
    m = np.ones((L + 1, N, 1, 1), bool)
    if dones is not None:
        m[1:] = (dones == 0)[:, :, None, None]
    h = np.zeros((N, D, S)) if state is None else state.copy()
    eh = np.zeros_like(h)
    # A chunk's decay comes from the sum of its D_t: at most 8 ceil(L / 8)
    # additions of it, as if each D_t were off by as many roundings.
    chain = 8 * ((L + 7) // 8) if L > 32 else 0
    hs, ehs, prev, eprev, a, ea, hb, ehb = (np.zeros((L, N, D, S)) for _ in range(8))
    for t in range(L):
        h, eh = np.where(m[t], h, 0.0), np.where(m[t], eh, 0.0)
        prev[t], eprev[t] = h, eh
        a[t] = np.exp(dt[t][..., None] * rate)
        ea[t] = a[t] * (np.abs(rate) * (edt[t][..., None] + (3 + chain) * U * np.abs(dt[t][..., None])) + 2 * U) + TINY
        bt = wide(b[t])
        hb[t] = (dt[t] * x[t])[..., None] * bt
        ehb[t] = (edt[t] * np.abs(x[t]))[..., None] * np.abs(bt) + 2 * U * np.abs(hb[t])
        eh = a[t] * eh + ea[t] * np.abs(h) + ehb[t] + 2 * U * (np.abs(a[t] * h) + np.abs(hb[t]))
        h = a[t] * h + hb[t]
        hs[t], ehs[t] = h, eh
    cs = np.stack([wide(c[t]) for t in range(L)]) if L else np.zeros((0, N, D, S))
    bs = np.stack([wide(b[t]) for t in range(L)]) if L else np.zeros((0, N, D, S))
    y = (cs * hs).sum(-1) + skip * x
    mag = np.abs(cs * hs).sum(-1) + np.abs(skip * x)
    ey = (np.abs(cs) * ehs).sum(-1) + (S + 4) * U * mag
    if gate is None:
        out, eo, fac, efac = y, ey, np.ones_like(y), np.zeros_like(y)
    else:
        fac = gate * sigmoid(gate)
        efac = np.abs(fac) * (e_sigmoid(gate) + U)
        out, eo = y * fac, np.abs(fac) * ey + np.abs(y) * efac + U * np.abs(y * fac)
    last, elast = np.where(m[L], h, 0.0), np.where(m[L], eh, 0.0)
    res = dict(y=out, ey=fin(name, out, eo), new_state=last, enew_state=fin("f32", last, elast))
    if dy is None:
        return res
    w, ew = dy * fac, np.abs(dy) * efac + U * np.abs(dy * fac)
    Gr = np.zeros((N, D, S)) if dnew is None else np.where(m[L], dnew, 0.0)
    eG = np.zeros_like(Gr)
    d, ed, q, eq = (np.zeros((L, N, D, S)) for _ in range(4))
    for t in range(L - 1, -1, -1):
        d[t] = cs[t] * w[t][..., None] + Gr
        ed[t] = np.abs(cs[t]) * ew[t][..., None] + eG + U * (np.abs(cs[t] * w[t][..., None]) + np.abs(Gr))
        g = a[t] * d[t]
        eg = a[t] * ed[t] + ea[t] * np.abs(d[t]) + U * np.abs(g)
        q[t] = g * prev[t]
        eq[t] = eg * np.abs(prev[t]) + np.abs(g) * eprev[t] + U * np.abs(q[t])
        Gr, eG = np.where(m[t], g, 0.0), np.where(m[t], eg, 0.0)
    dth, edth = dt[..., None], edt[..., None]
    du, edu = dt * x, edt * np.abs(x) + U * np.abs(dt * x)
    groups = lambda t: t.reshape(L, N, G, D // G, S).sum(3)
    n = D // G + 8  # a lane's channels, lanes, blocks: at most all of them
    db = groups(d * du[..., None])
    edb = groups(ed * np.abs(du[..., None]) + np.abs(d) * edu[..., None]) + n * U * groups(np.abs(d * du[..., None]))
    dc = groups(w[..., None] * hs)
    edc = groups(np.abs(w[..., None]) * ehs + ew[..., None] * np.abs(hs)) + n * U * groups(np.abs(w[..., None] * hs))
    s1 = (bs * d).sum(-1)
    es1 = (np.abs(bs) * ed).sum(-1) + (S + 2) * U * np.abs(bs * d).sum(-1)
    s2 = (rate * q).sum(-1)
    es2 = (np.abs(rate) * eq).sum(-1) + (S + 5) * U * np.abs(rate * q).sum(-1)
    dD = x * s1 + s2
    edD = np.abs(x) * es1 + es2 + 2 * U * (np.abs(x * s1) + np.abs(s2))
    dd = dD * sg
    edd = sg * edD + np.abs(dD) * esg + U * np.abs(dd)
    dx = dt * s1 + skip * w
    edx = edt * np.abs(s1) + np.abs(dt) * es1 + np.abs(skip) * ew + 2 * U * (np.abs(dt * s1) + np.abs(skip * w))
    n = L + 48  # a wave's steps, column sums
    over = lambda t: t.sum((0, 1))
    drate = over(dth * q)
    edrate = over(edth * np.abs(q) + np.abs(dth) * eq) + n * U * over(np.abs(dth * q))
    dskip, edskip = over(w * x), over(ew * np.abs(x)) + n * U * over(np.abs(w * x))
    dbias, edbias = over(dd), over(edd) + n * U * over(np.abs(dd))
    f32 = lambda v, e: fin("f32", v, e)
    res.update(dx=dx, edx=fin(name, dx, edx), ddelta=dd, eddelta=fin(name, dd, edd), db=db, edb=fin(name, db, edb),
               dc=dc, edc=fin(name, dc, edc), drate=drate, edrate=f32(drate, edrate), dskip=dskip,
               edskip=f32(dskip, edskip), ddelta_bias=dbias, eddelta_bias=f32(dbias, edbias), dstate=Gr,
               edstate=f32(Gr, eG))
    if gate is not None:
        f, ef = dy * silu_slope(gate), np.abs(dy) * e_silu_slope(gate) + 2 * U * np.abs(dy * silu_slope(gate))
        dg = f * y
        res.update(dgate=dg, edgate=fin(name, dg, ef * np.abs(y) + np.abs(f) * ey + U * np.abs(dg)))
    return res


# ---------------------------------------------------------------------- norm
ACT = {"none": (lambda g: g, lambda g: np.ones_like(g), lambda g: 0 * g, lambda g: 0 * g),
       "sigmoid": (sigmoid, lambda g: sigmoid(g) * (1 - sigmoid(g)), lambda g: sigmoid(g) * e_sigmoid(g),
                   lambda g: sigmoid(g) * (2 * e_sigmoid(g) + 2 * U)),
       "silu": (lambda g: g * sigmoid(g), silu_slope, lambda g: np.abs(g) * sigmoid(g) * (e_sigmoid(g) + U),
                e_silu_slope)}
TERMS = 40  # roundings on the way of a term of a row's sum, at most: 16 of a thread, 6 of a wave, 8 of waves


def norm(residual, branch, weight, branch_weight, gate, name, act="none", rs=1.0, bs=1.0, branch_norm=True,
         eps=1e-6, kept=None, scale=1.0, dstream=None, dnormed=None):
    """[R, D]; kept [R, D] of truth values or None; float64."""
    R, D = residual.shape
    one = np.ones(D)
    w, bw = (one if v is None else v for v in (weight, branch_weight))
    s = rs * residual
    es = U * np.abs(s)
    if branch is not None:
        if branch_norm:
            ib = 1 / np.sqrt((branch ** 2).mean(-1, keepdims=True) + eps)
            eib = ib * (TERMS / 2 + 4) * U
        else:
            ib, eib = np.ones((R, 1)), np.zeros((R, 1))
        uh = branch * ib
        euh = np.abs(branch) * eib + U * np.abs(uh)
        v = uh * bw
        ev = euh * np.abs(bw) + U * np.abs(v)
        g = np.ones((R, D)) if gate is None else np.broadcast_to(gate, (R, D))
        A, dA, eA, edA = (f(g) for f in (ACT["none"] if gate is None else ACT[act]))
        z = v * A
        ez = ev * np.abs(A) + np.abs(v) * eA + U * np.abs(z)
        on = np.ones((R, D), bool) if kept is None else kept
        z, ez = np.where(on, z * scale, 0.0), np.where(on, ez * scale + 2 * U * np.abs(z * scale), 0.0)
        es = es + np.abs(bs) * ez + 2 * U * (np.abs(s) + np.abs(bs * z))
        s = s + bs * z
    ss = (s ** 2).mean(-1, keepdims=True) + eps
    inv = 1 / np.sqrt(ss)
    einv = inv * ((np.abs(s) * es).mean(-1, keepdims=True) / ss + (TERMS / 2 + 4) * U)
    nh = s * inv
    enh = es * inv + np.abs(s) * einv + U * np.abs(nh)
    y = nh * w
    res = dict(stream=s, estream=fin(name, s, es), normed=y, enormed=fin(name, y, np.abs(w) * enh + 2 * U * np.abs(y)))
    if dstream is None and dnormed is None:
        return res
    d, ed = (np.zeros((2, R, D)) if dstream is None else (dstream, np.zeros((R, D))))
    n = R + 48
    if dnormed is not None:
        gg = dnormed * w
        mean = (gg * nh).mean(-1, keepdims=True)
        emean = (np.abs(gg) * enh).mean(-1, keepdims=True) + TERMS * U * np.abs(gg * nh).mean(-1, keepdims=True)
        inner = gg - nh * mean
        einner = np.abs(nh) * emean + np.abs(mean) * enh + 2 * U * (np.abs(gg) + np.abs(nh * mean))
        ed = inv * einner + einv * np.abs(inner) + 2 * U * (np.abs(d) + inv * np.abs(inner))
        d = d + inv * inner
        dw = (dnormed * nh).sum(0)
        edw = (np.abs(dnormed) * enh).sum(0) + n * U * np.abs(dnormed * nh).sum(0)
        res.update(dweight=dw, edweight=fin("f32", dw, edw))
    else:
        res.update(dweight=np.zeros(D), edweight=np.full(D, TINY))
    res.update(dresidual=rs * d, edresidual=fin(name, rs * d, np.abs(rs) * ed + U * np.abs(rs * d)))
    if branch is None:
        return res
    dz = bs * d
    edz = np.abs(bs) * ed + U * np.abs(dz)
    dz, edz = np.where(on, dz * scale, 0.0), np.where(on, edz * scale + 2 * U * np.abs(dz * scale), 0.0)
    da = dz * v
    eda = edz * np.abs(v) + np.abs(dz) * ev + U * np.abs(da)
    dg = da * dA
    edg = eda * np.abs(dA) + np.abs(da) * edA + U * np.abs(dg)
    du = dz * A
    edu = edz * np.abs(A) + np.abs(dz) * eA + U * np.abs(du)
    dbw = (du * uh).sum(0)
    edbw = (edu * np.abs(uh) + np.abs(du) * euh).sum(0) + n * U * np.abs(du * uh).sum(0)
    e = du * bw
    ee = edu * np.abs(bw) + U * np.abs(e)
    if branch_norm:
        mean = (e * uh).mean(-1, keepdims=True)
        emean = (ee * np.abs(uh) + np.abs(e) * euh).mean(-1, keepdims=True) + \
            TERMS * U * np.abs(e * uh).mean(-1, keepdims=True)
        inner = e - uh * mean
        einner = ee + np.abs(uh) * emean + np.abs(mean) * euh + 2 * U * (np.abs(e) + np.abs(uh * mean))
        e, ee = ib * inner, ib * einner + eib * np.abs(inner) + U * np.abs(ib * inner)
    res.update(dbranch=e, edbranch=fin(name, e, ee), dbranch_weight=dbw, edbranch_weight=fin("f32", dbw, edbw))
    if gate is not None and gate.ndim == 1:
        total = dg.sum(0)
        res.update(dgate=total, edgate=fin("f32", total, edg.sum(0) + n * U * np.abs(dg).sum(0)))
    elif gate is not None:
        res.update(dgate=dg, edgate=fin(name, dg, edg))
    return res


# ------------------------------------------------------------------- dropout
def philox(counter, key):
    """Philox4x32-10 on Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xffffffff, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xffffffff]
        k = [(k[0] + 0x9E3779B9) & 0xffffffff, (k[1] + 0xBB67AE85) & 0xffffffff]
    return c


def kept(count, p, seed, offset=0, start=0):
    """Whether the elements start .. start + count - 1 are kept, and the scale."""
    drop = int(np.floor(65536 * p + 0.5))
    seed &= (1 << 64) - 1
    res = np.zeros(count, bool)
    block = None
    for i in range(start, start + count):
        if i // 8 != block:
            block = i // 8
            words = philox((block & 0xffffffff, block >> 32, offset, 0x44524f50), (seed & 0xffffffff, seed >> 32))
        res[i - start] = (words[i % 8 // 2] >> (16 * (i % 2))) & 0xffff >= drop
    return res, 65536 / (65536 - drop) if drop < 65536 else 0.0
