"""fp64 oracle of the block around the scan: the gated linear recurrence, the
norms with gate and residual scale, and the 8-bit form (test infrastructure).

Plain numpy, token after token and row after row, written from the formulas;
shares no code with the library.  Every function that a kernel is compared
with also returns a bound on the error of fp32 arithmetic: each value comes
with a majorant (the same expression over absolute values, nothing cancels),
and one rounding to fp32 is off by at most U of it.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24                       # half a step of fp32
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
KEEP = 64                            # tokens between kept states
GROUP = 64                           # channels per 8-bit scale


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1 / (1 + e), e / (1 + e))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


# ----------------------------------------------------------------- 8 bits ---

def pack8(x):
    """x [rows, D] (float32 values) -> q int8, scale float32, in the fp32
    arithmetic that defines the form."""
    x = np.asarray(x, np.float32)
    rows, D = x.shape
    q = np.zeros((rows, D), np.int8)
    scale = np.zeros((rows, -(-D // GROUP)), np.float32)
    for g in range(scale.shape[1]):
        v = x[:, g * GROUP:(g + 1) * GROUP]
        amax = np.max(np.abs(v), axis=1) if v.size else np.zeros(rows, np.float32)
        fine = np.isfinite(v).all(axis=1)
        some = fine & (amax >= np.float32(2.0 ** -100))
        scale[fine & ~some, g] = 0
        scale[~fine, g] = np.nan
        with np.errstate(all="ignore"):
            scale[some, g] = amax[some] / np.float32(127)
            inv = np.float32(127) / amax[some]
            q[some, g * GROUP:(g + 1) * GROUP] = np.rint(v[some] * inv[:, None]).astype(np.int8)
    return q, scale


def unpack8(q, scale):
    return q.astype(np.float64) * np.repeat(scale.astype(np.float64), GROUP, axis=1)[:, : q.shape[1]]


def held8(x):
    """The values 8 bits hold of x [..., D], float64."""
    flat = np.asarray(x, np.float32).reshape(-1, x.shape[-1])
    return unpack8(*pack8(flat)).reshape(x.shape)


# ------------------------------------------------------------- recurrence ---

def gate_values(gate, x, f, i, lam, c):
    """a, b and what the backward needs of them, elementwise."""
    if gate == "decay":
        return dict(a=f, b=x)
    if gate == "sigmoid":
        return dict(a=sigmoid(f), na=sigmoid(-f), b=sigmoid(-f) * x)
    la = -c * softplus(lam) * sigmoid(f)
    v = -np.expm1(2 * la)
    u = np.sqrt(v)
    return dict(a=np.exp(la), la=la, u=u, si=sigmoid(i), b=u * sigmoid(i) * x)


# Roundings that a step's decay and input take (relative, in units of U): a
# value given is exact; exp(-|f|) by the hardware's exponential is within 2
# units in the last place (4 U) and 1.2 |f| more for its argument, |f| <= 10
# in the tests, then a sum, a reciprocal and products: 32.  The lru input adds a
# second logistic, the series, a root: 96 for a log-decay up to 1 in size.  A
# relative error d of the log-decay la is la d of a = exp(la), so that a's
# roundings grow by the factor 1 + |la|.
STEP = {"decay": 4, "sigmoid": 40, "lru": 96}


def step_error(gate, g):
    return STEP[gate] * U * (1 + np.abs(g["la"]) if gate == "lru" else 1)


def valid_mask(B, L, lens):
    n = np.full(B, L) if lens is None else np.clip(np.asarray(lens), 0, L)
    return np.arange(L)[None, :] < n[:, None]


def gated_scan(gate, x, f, i=None, lam=None, c=8.0, h0=None, reset=None, lens=None, restart=None):
    """y, h_last, kept states, h_{t-1} of every token, each with its error
    bound: dict of float64 arrays.  restart: kept states from which pieces of
    64 tokens start (what the backward does; the state before a piece's first
    token is the last of the piece before)."""
    x, f = np.asarray(x, np.float64), np.asarray(f, np.float64)
    B, L, D = x.shape
    i = None if i is None else np.asarray(i, np.float64)
    lam = None if lam is None else np.asarray(lam, np.float64)
    ok = valid_mask(B, L, lens)
    K = -(-L // KEEP)
    out = {k: np.zeros((B, L, D)) for k in ("y", "y_err", "prev", "prev_err", "prev_maj")}
    out["states"] = np.zeros((B, K, D))
    out["states_err"] = np.zeros((B, K, D))
    h = np.zeros((B, D)) if h0 is None else np.asarray(h0, np.float64).copy()
    H, e = np.abs(h), np.zeros((B, D))
    for t in range(L):
        m = ok[:, t][:, None]
        r = np.zeros((B, 1), bool) if reset is None else (np.asarray(reset)[:, t] != 0)[:, None] & m
        if restart is not None and t == 0:
            h, H = restart[:, 0].copy(), np.abs(restart[:, 0])
        out["prev"][:, t], out["prev_err"][:, t], out["prev_maj"][:, t] = (np.where(r, 0, v) for v in (h, e, H))
        if t % KEEP == 0:
            if restart is not None:
                h, H, e = restart[:, t // KEEP].copy(), np.abs(restart[:, t // KEEP]), np.zeros((B, D))
            out["states"][:, t // KEEP], out["states_err"][:, t // KEEP] = h, e + U * np.abs(h)
        h, H, e = np.where(r, 0, h), np.where(r, 0, H), np.where(r, 0, e)
        with np.errstate(all="ignore"):
            g = gate_values(gate, x[:, t], f[:, t], None if i is None else i[:, t], lam, c)
            hn = g["a"] * h + g["b"]
            Hn = np.abs(g["a"]) * H + np.abs(g["b"])
            en = np.abs(g["a"]) * e + step_error(gate, g) * Hn
        h, H, e = np.where(m, hn, h), np.where(m, Hn, H), np.where(m, en, e)
        out["y"][:, t] = np.where(m, h, 0)
        out["y_err"][:, t] = np.where(m, e, 0)
    out["h_last"], out["h_last_err"] = h, e + U * np.abs(h)
    return out


def gated_backward(gate, x, f, i=None, lam=None, c=8.0, h0=None, reset=None, lens=None, dy=None, dh_last=None,
                   states=None):
    """dx, df, di, dlam, dh0 with error bounds.  states: the forward's kept
    states where x, f, i are not exactly what it ran on (8-bit copies)."""
    x, f, dy = (np.asarray(v, np.float64) for v in (x, f, dy))
    B, L, D = x.shape
    fw = gated_scan(gate, x, f, i, lam, c, h0, reset, lens, restart=states)
    i = None if i is None else np.asarray(i, np.float64)
    lam = None if lam is None else np.asarray(lam, np.float64)
    ok = valid_mask(B, L, lens)
    d = np.zeros((B, D)) if dh_last is None else np.asarray(dh_last, np.float64).copy()
    M, E = np.abs(d), np.zeros((B, D))
    out = {n: np.zeros((B, L, D)) for n in ("dx", "df", "di", "dx_err", "df_err", "di_err")}
    tot, tot_err = np.zeros(D), np.zeros(D)
    for t in range(L - 1, -1, -1):
        m = ok[:, t][:, None]
        with np.errstate(all="ignore"):
            g = gate_values(gate, x[:, t], f[:, t], None if i is None else i[:, t], lam, c)
            k = step_error(gate, g)
            dn, Mn = d + dy[:, t], M + np.abs(dy[:, t])
            En = E + k * Mn
            p, P, pe = fw["prev"][:, t], fw["prev_maj"][:, t], fw["prev_err"][:, t]
            a = g["a"]
            if gate == "decay":
                w = {"dx": np.ones_like(a), "df": p}
                W = {"dx": (np.ones_like(a), 0), "df": (P, pe)}
            elif gate == "sigmoid":
                s = a * g["na"]
                w = {"dx": g["na"], "df": s * (p - x[:, t])}
                W = {"dx": (g["na"], 0), "df": (s * (P + np.abs(x[:, t])), s * pe)}
            else:
                xt, u, si, la = x[:, t], g["u"], g["si"], g["la"]
                slope = si * sigmoid(-i[:, t])
                inner = np.where(u > 0, si * xt * a * a / np.where(u > 0, u, 1), 0)
                q, Q = la * (a * p - inner), -la * (a * P + np.abs(inner))
                nf = sigmoid(-f[:, t])
                w = {"dx": u * si, "di": u * xt * slope, "df": q * nf, "q": q}
                W = {"dx": (u * si, 0), "di": (u * np.abs(xt) * slope, 0), "df": (Q * nf, -la * a * pe * nf),
                     "q": (Q, -la * a * pe)}
            for n, v in w.items():
                big, we = W[n]
                val = v * dn
                # a factor's own roundings, its error through h, and the error of d
                err = (k * big + we) * Mn + big * En
                if n == "q":
                    tot += np.where(m, val, 0).sum(0)
                    tot_err += np.where(m, err + 64 * U * big * Mn, 0).sum(0)
                else:
                    out[n][:, t] = np.where(m, val, 0)
                    out[n + "_err"][:, t] = np.where(m, err, 0)
            keep = np.ones_like(a) if reset is None else (np.asarray(reset)[:, t] == 0)[:, None]
            dp, Mp, Ep = (np.where(keep, np.abs(a) if j else a, 0) * v for j, v in enumerate((dn, Mn, En)))
            Ep = Ep + k * Mp
        d, M, E = np.where(m, dp, d), np.where(m, Mp, M), np.where(m, Ep, E)
    out["dh0"], out["dh0_err"] = d, E + U * M
    if gate == "lru":
        ratio = sigmoid(lam) / softplus(lam)
        out["dlam"], out["dlam_err"] = tot * ratio, tot_err * ratio + 16 * U * np.abs(tot * ratio)
    else:
        for n in ("di", "di_err"):
            del out[n]
    return out


# ------------------------------------------------------------------ block ---

# Roundings behind a norm's output: a tree sum of squares over a row (at most
# 8 terms in a thread, 5 + 4 levels across), the reciprocal root, products and
# the gate's logistic; one constant for all of them, relative to majorants.
NORM_ROUNDINGS = 96


def _norm(kind, v, maj, w, b, eps):
    """n = N(v) w + b with hat, 1/sd and the majorants of hat and n; maj: |v| or a majorant of it."""
    if kind == "layer":
        mean = v.mean(-1, keepdims=True)
        v, maj = v - mean, maj + maj.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    hat, HAT = v * rstd, maj * rstd
    n = hat * w + b
    return n, hat, rstd, HAT, HAT * np.abs(w) + np.abs(b)


def _act(act, g):
    if act == "none":
        return 1.0, 0.0, 1.0, 0.0
    s, ns = sigmoid(g), sigmoid(-g)
    if act == "sigmoid":
        return s, s * ns, s, s * ns
    return g * s, s * (1 + g * ns), np.abs(g) * s, s * (1 + np.abs(g) * ns)


def _params(D, w_y, b_y, s, w_z, b_z):
    one, zero = np.ones(D), np.zeros(D)
    return [np.asarray(v, np.float64) if v is not None else d
            for v, d in ((w_y, one), (b_y, zero), (s, one), (w_z, one), (b_z, zero))]


def block_norm(kind, act, r, y=None, g=None, w_y=None, b_y=None, s=None, w_z=None, b_z=None, eps=1e-6, res_scale=1.0):
    """r, z and their error bounds before the final rounding."""
    r = np.asarray(r, np.float64)
    w_y, b_y, s, w_z, b_z = _params(r.shape[-1], w_y, b_y, s, w_z, b_z)
    k, R = NORM_ROUNDINGS * U, np.abs(r)
    if y is not None:
        y = np.asarray(y, np.float64)
        n, _, _, _, N = _norm(kind, y, np.abs(y), w_y, b_y, eps)
        a, _, A, _ = _act(act, None if g is None else np.asarray(g, np.float64))
        r = r + res_scale * s * a * n
        R = R + np.abs(res_scale * s) * A * N
    z, _, _, _, Z = _norm(kind, r, R, w_z, b_z, eps)
    return {"r": r, "r_err": k * R, "z": z, "z_err": 2 * k * Z}


def block_backward(kind, act, r=None, y=None, g=None, dr_out=None, dz=None, w_y=None, b_y=None, s=None, w_z=None,
                   eps=1e-6, res_scale=1.0):
    """dr, dy, dg and the parameters' sums, with error bounds."""
    ref = np.asarray(dz if dz is not None else dr_out, np.float64)
    w_y, b_y, s, w_z, _ = _params(ref.shape[-1], w_y, b_y, s, w_z, None)
    k = NORM_ROUNDINGS * U
    mean = lambda v: v.mean(-1, keepdims=True)  # noqa: E731
    e = np.zeros_like(ref) if dr_out is None else np.asarray(dr_out, np.float64)
    M = np.abs(e)
    out = {}

    def norm_back(u, UU, hat, HAT, rstd):
        t = u - hat * mean(u * hat)
        T = UU + HAT * mean(UU * HAT)
        if kind == "layer":
            t, T = t - mean(u), T + mean(UU)
        return rstd * t, rstd * T

    def sums(name, v, V):
        out[name], out[name + "_err"] = v.sum(0), 4 * k * V.sum(0)

    if dz is not None:
        dz = np.asarray(dz, np.float64)
        r = np.asarray(r, np.float64)
        _, hat, rstd, HAT, _ = _norm(kind, r, np.abs(r), w_z, 0.0, eps)
        t, T = norm_back(dz * w_z, np.abs(dz * w_z), hat, HAT, rstd)
        e, M = e + t, M + T
        sums("dw_z", dz * hat, np.abs(dz) * HAT)
        sums("db_z", dz, np.abs(dz))
    out["dr"], out["dr_err"] = e, 2 * k * M
    if y is None:
        return out
    y = np.asarray(y, np.float64)
    n, hat, rstd, HAT, N = _norm(kind, y, np.abs(y), w_y, b_y, eps)
    a, da, A, DA = _act(act, None if g is None else np.asarray(g, np.float64))
    sums("ds", res_scale * e * a * n, np.abs(res_scale) * M * A * N)
    dm, DM = res_scale * s * e, np.abs(res_scale * s) * M
    if act != "none":
        out["dg"], out["dg_err"] = dm * n * da, 4 * k * DM * N * DA
    dn, DN = dm * a, DM * A
    sums("dw_y", dn * hat, DN * HAT)
    sums("db_y", dn, DN)
    t, T = norm_back(dn * w_y, DN * np.abs(w_y), hat, HAT, rstd)
    out["dy"], out["dy_err"] = t, 4 * k * T
    return out
