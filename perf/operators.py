"""What a recurrent block is made of, as measured: the gated linear recurrence
(forward, training, single tokens), the norms around a block with its gate and
residual scale, and activations kept in 8 bits between the two passes.

The plain forms below are elementary torch operations in fp32, rounded once at
the end; with `own` set, `run` makes the calls a user of the library makes.

Recurrence, per channel (B sequences of L tokens, D channels):
    h_t = a_t h_{t-1} + b_t,   y_t = h_t
    decay    a = f,                              b = x
    sigmoid  a = s(f),                           b = (1 - a) x
    lru      a = exp(-c softplus(lam) s(f)),     b = sqrt(1 - a^2) s(i) x
reset[b, t] != 0 starts a new sequence at t (h_{t-1} counts as zero); tokens at
or past lens[b] are padding: y and the gradients are zero there and the state
stays as it was.

Block, per row:  r' = r + rs * s * act(g) * (N(y) w_y + b_y),  z = N(r') w_z + b_z.

8 bits: per row and run of 64 channels, scale = amax / 127 and
q = rint(x * (127 / amax)), both in fp32; the value held is q * scale.  The
recurrence's backward recomputes h_{t-1} from its inputs as they were kept,
started anew at every 64th token from the forward's own state there.
"""
import math

import torch

own = False

C_LRU = 8.0
EPS = 1e-6
RES_SCALE = 0.5
GROUP = 64          # channels that share an 8-bit scale
KEPT_EVERY = 64     # tokens between the forward states kept for the backward
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _mru():
    from linear_rnn_scan_b200 import mru
    return mru


# ---------------------------------------------------------------- cases ---

def _scan(name, gate, dtype, B, L, D, train=False, packed=False, ragged=False):
    d = {"op": "scan", "gate": gate, "dtype": dtype, "B": B, "L": L, "D": D, "train": train, "packed": packed,
         "ragged": ragged}
    return dict(d, name=name) if name else d


def _block(name, norm, act, dtype, rows, D, train=False, packed=False):
    d = {"op": "block", "norm": norm, "act": act, "dtype": dtype, "rows": rows, "D": D, "train": train,
         "packed": packed}
    return dict(d, name=name) if name else d


def _pack(name, dtype, rows, D):
    d = {"op": "pack", "dtype": dtype, "rows": rows, "D": D}
    return dict(d, name=name) if name else d


def listed():
    return [
        # one new token for each of 64 running sequences (serving; latency)
        _scan("scan_step_b64_bf16", "lru", "bf16", 64, 1, 2048),
        # the smallest sequence workload: one head of 4 x 4, 1024 tokens
        _scan("scan_short_f32", "decay", "f32", 1, 1024, 16),
        # prefill of eight prompts, width of 8 heads of 16 x 16
        _scan("scan_prefill_lru_bf16", "lru", "bf16", 8, 4096, 2048),
        # one very long sequence: little to do side by side, the carry decides
        _scan("scan_long_f32", "decay", "f32", 1, 262144, 2048),
        # a training step at 16 heads of 32 x 32: forward and backward
        _scan("scan_train_sigmoid_bf16", "sigmoid", "bf16", 4, 8192, 16384, train=True),
        # packed and padded documents, odd width, every gradient, fp32
        _scan("scan_train_lru_ragged_f32", "lru", "f32", 3, 1237, 1001, train=True, ragged=True),
        # a training step that keeps its inputs in 8 bits between the passes
        _scan("scan_train_8bit_bf16", "lru", "bf16", 8, 4096, 2048, train=True, packed=True),
        # the block's ends for one token of 64 sequences (serving; latency)
        _block("block_step_bf16", "rms", "silu", "bf16", 64, 2048),
        # a training step of the block's ends, 8 sequences of 4096 tokens
        _block("block_train_bf16", "rms", "silu", "bf16", 32768, 2048, train=True),
        # odd width, layer norm with biases, fp32
        _block("block_train_layer_odd_f32", "layer", "sigmoid", "f32", 3711, 1001, train=True),
        # wide rows (4 heads of 64 x 64), saved in 8 bits between the passes
        _block("block_train_8bit_wide_bf16", "rms", "silu", "bf16", 16384, 16384, train=True, packed=True),
        # activations of a layer put away in 8 bits and brought back
        _pack("pack_bf16", "bf16", 32768, 2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, most):
    d = _log_int(rng, 16, most)
    return d if rng.random() < 0.4 else max(16, d // 16 * 16)


def draw(rng):
    largest = work(listed()[4])["bytes"]
    while True:
        kind = rng.choice(["scan", "scan", "scan", "block", "block", "pack"])
        dtype = rng.choice(["bf16", "f32"])
        D = _width(rng, 16384)
        if kind == "scan":
            case = _scan(None, rng.choice(["decay", "sigmoid", "lru"]), dtype, _log_int(rng, 1, 64),
                         _log_int(rng, 1, 262144), D, train=rng.random() < 0.6, packed=rng.random() < 0.4,
                         ragged=rng.random() < 0.4)
            case["packed"] = case["packed"] and case["train"]
        elif kind == "block":
            case = _block(None, rng.choice(["rms", "layer"]), rng.choice(["silu", "sigmoid", "none"]), dtype,
                          _log_int(rng, 1, 65536), D, train=rng.random() < 0.7, packed=rng.random() < 0.4)
            case["packed"] = case["packed"] and case["train"]
        else:
            case = _pack(None, dtype, _log_int(rng, 1, 65536), D)
        # within the largest case's cost, and what the fp32 temporaries of the plain forms hold on the device
        if work(case)["bytes"] <= largest and _elements(case) <= 1 << 29:
            return case


def _elements(case):
    return case["D"] * (case["B"] * case["L"] if case["op"] == "scan" else case["rows"])


def work(case):
    """A training pass is two calls with the rest of the model between them:
    what each call reads and writes counts once per call."""
    n = _elements(case)
    e = 4 if case["dtype"] == "f32" else 2
    p8 = 1 + 4.0 / GROUP                                   # a value and its share of the scale
    if case["op"] == "pack":
        return {"bytes": int(n * (2 * e + 2 * p8)), "flops": 4 * n}
    if case["op"] == "scan":
        k = 3 if case["gate"] == "lru" else 2              # x, f (, i)
        by, fl = n * (k + 1) * e, 8 * n
        if case["train"]:
            by += n * ((k * (2 * p8) if case["packed"] else k * e) + (1 + k) * e)
            fl += 24 * n
        return {"bytes": int(by), "flops": fl}
    k = 2 if case["act"] == "none" else 3                  # r, y (, g)
    by, fl = n * (k + 2) * e, 12 * n
    if case["train"]:
        by += n * ((k * (2 * p8) if case["packed"] else k * e) + (2 + k) * e)
        fl += 40 * n
    return {"bytes": int(by), "flops": fl}


# --------------------------------------------------------------- inputs ---

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = DT[case["dtype"]]

    def normal(*shape, mean=0.0, std=1.0, dtype=dt):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(mean, std, generator=gen)

    st = {"case": case}
    if case["op"] == "pack":
        # activations: unit scale, with some channels much larger than the rest
        x = normal(case["rows"], case["D"])
        x[:, :: 97] *= 20.0
        st["x"] = x
        return st
    D = case["D"]
    if case["op"] == "block":
        R = case["rows"]
        st["r"], st["y"] = normal(R, D), normal(R, D, std=0.5)
        st["g"] = None if case["act"] == "none" else normal(R, D)
        for k in ("w_y", "w_z"):
            st[k] = normal(D, mean=1.0, std=0.1, dtype=torch.float32)
        for k in ("b_y", "b_z"):
            st[k] = normal(D, std=0.1, dtype=torch.float32) if case["norm"] == "layer" else None
        st["s"] = normal(D, mean=0.5, std=0.1, dtype=torch.float32)
        if case["train"]:
            # gradients lie partly along the activations, as a training loss's do: sums over rows do not cancel out
            st["dr"] = normal(R, D)
            st["dz"] = normal(R, D).add_(st["r"], alpha=0.25)
        return st
    B, L = case["B"], case["L"]
    st["x"] = normal(B, L, D)
    st["i"] = st["lam"] = None
    if case["gate"] == "decay":
        st["f"] = torch.sigmoid(normal(B, L, D, mean=3.0))
    elif case["gate"] == "sigmoid":
        st["f"] = normal(B, L, D, mean=2.0, std=1.5)
    else:
        st["f"], st["i"] = normal(B, L, D), normal(B, L, D)
        # channels whose decay at an open gate is spread over 0.9 .. 0.999
        a0 = torch.empty(D, device=dev).uniform_(0.9, 0.999, generator=gen)
        st["lam"] = torch.log(torch.expm1(-torch.log(a0) / C_LRU))
    st["h0"] = normal(B, D, dtype=torch.float32)
    st["reset"] = st["lens"] = None
    if case["ragged"]:
        st["reset"] = (torch.empty((B, L), device=dev).uniform_(0, 1, generator=gen) < 1 / 200).to(torch.uint8)
        lens = torch.empty(B, device=dev).uniform_(0, 1, generator=gen) * (L + 1)
        st["lens"] = lens.floor().clamp(0, L).to(torch.int32)
        st["lens"][0] = L
    if case["train"]:
        st["dy"], st["dh_last"] = normal(B, L, D), normal(B, D, dtype=torch.float32)
    return st


# ------------------------------------------------------------------ run ---

def run(state):
    case = state["case"]
    if case["op"] == "scan":
        return _run_scan(state, case)
    if case["op"] == "block":
        return _run_block(state, case)
    return _run_pack(state, case)


def _run_scan(st, case):
    kw = {k: st[k] for k in ("lam", "reset", "lens")}
    if own:
        mru = _mru()
        p = mru.gated_problem(case["B"], case["L"], case["D"], gate=case["gate"], x_dtype=case["dtype"], c=C_LRU)
        save = ("int8" if case["packed"] else "full") if case["train"] else None
        y, h_last, saved = mru.gated_scan_t(p, st["x"], st["f"], i=st["i"], h0=st["h0"], save=save, **kw)
        out = {"y": y, "h_last": h_last}
        if case["train"]:
            ins = {} if case["packed"] else {"x": st["x"], "f": st["f"], "i": st["i"]}
            gr = mru.gated_scan_backward_t(p, st["dy"], saved, dh_last=st["dh_last"], **ins, **kw)
            out.update(dx=gr.dx, df=gr.df, di=gr.di, dlam=gr.dlam, dh0=gr.dh0)
        return {k: v for k, v in out.items() if v is not None}
    dt = DT[case["dtype"]]
    valid, keep = _masks(st, case)
    a, b = _plain_gates(case, st["x"], st["f"], st["i"], st["lam"], valid, keep)
    b[:, 0].addcmul_(a[:, 0], st["h0"])
    h = _plain_scan(a, b)
    out = {"h_last": h[:, -1].clone()}
    out["y"] = (h if valid is None else h * valid).to(dt)
    if not case["train"]:
        return out
    x, f, i = st["x"], st["f"], st["i"]
    if case["packed"]:
        del a, b
        x, f, i = (_plain_unpack(*_plain_pack(v)) if v is not None else None for v in (x, f, i))
        a, b = _plain_gates(case, x, f, i, st["lam"], valid, keep)
        h = _plain_scan_from_kept(a, b, torch.cat([st["h0"][:, None], h[:, KEPT_EVERY - 1:-1:KEPT_EVERY]], 1))
    del b
    hp = torch.cat([st["h0"][:, None], h[:, :-1]], 1)
    del h
    if keep is not None:
        hp *= keep
    dy = st["dy"].float()
    if valid is not None:
        dy = dy * valid
    else:
        dy = dy.clone() if dy is st["dy"] else dy
    dy[:, -1] += st["dh_last"]
    # d_t = dy_t + a_{t+1} d_{t+1}: the scan on the reversed sequence, with the decays one step later
    an = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    d = _plain_scan(an.flip(1), dy.flip(1)).flip(1)
    del an, dy
    out["dh0"] = a[:, 0] * d[:, 0]
    del a
    if valid is not None:
        d = d * valid
    x, f = x.float(), f.float()
    if case["gate"] == "decay":
        out["dx"], out["df"] = d.to(dt), (d * hp).to(dt)
    elif case["gate"] == "sigmoid":
        na = torch.sigmoid(-f)
        out["dx"] = (na * d).to(dt)
        out["df"] = (torch.sigmoid(f) * na * (hp - x) * d).to(dt)
    else:
        sp = torch.nn.functional.softplus(st["lam"])
        sf, si = torch.sigmoid(f), torch.sigmoid(i.float())
        la = -C_LRU * sp * sf
        beta = torch.sqrt(-torch.expm1(2 * la))
        out["dx"] = (d * beta * si).to(dt)
        out["di"] = (d * beta * x * si * torch.sigmoid(-i.float())).to(dt)
        q = d * (torch.exp(la) * hp * la - si * x * torch.exp(2 * la) * la / beta)
        del d, hp, beta, la, si
        out["df"] = (q * torch.sigmoid(-f)).to(dt)
        out["dlam"] = (q.sum((0, 1), dtype=torch.float64) * torch.sigmoid(st["lam"]) / sp).float()
    return out


def _masks(st, case):
    """Tokens that are not padding, and those whose previous state counts."""
    valid = keep = None
    if st["lens"] is not None:
        valid = (torch.arange(case["L"], device=st["x"].device) < st["lens"][:, None]).float()[..., None]
    if st["reset"] is not None:
        keep = (st["reset"] == 0).float()[..., None]
    return valid, keep


def _plain_gates(case, x, f, i, lam, valid, keep):
    x, f = x.float(), f.float()
    if case["gate"] == "decay":
        a, b = f.clone(), x.clone()
    elif case["gate"] == "sigmoid":
        a, b = torch.sigmoid(f), torch.sigmoid(-f) * x
    else:
        la = torch.sigmoid(f) * (-C_LRU * torch.nn.functional.softplus(lam))
        a = torch.exp(la)
        b = torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(i.float()) * x
    if keep is not None:
        a = a * keep
    if valid is not None:
        a = torch.where(valid != 0, a, torch.ones_like(a))
        b = b * valid
    return a, b


def _plain_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 (h_{-1} = 0) by doubling."""
    L, step = a.shape[1], 1
    while step < L:
        hb = b.clone()
        hb[:, step:].addcmul_(a[:, step:], b[:, :-step])
        b = hb
        if 2 * step < L:
            ha = a.clone()
            ha[:, step:].mul_(a[:, :-step])
            a = ha
        step *= 2
    return b


def _plain_scan_from_kept(a, b, kept):
    """The states of pieces of KEPT_EVERY tokens, each from its kept state (kept [B, pieces, D])."""
    B, L, D = a.shape
    pad = -L % KEPT_EVERY
    a = torch.nn.functional.pad(a, (0, 0, 0, pad)).view(-1, KEPT_EVERY, D)
    b = torch.nn.functional.pad(b, (0, 0, 0, pad)).view(-1, KEPT_EVERY, D)
    b[:, 0].addcmul_(a[:, 0], kept.reshape(-1, D))
    return _plain_scan(a, b).view(B, -1, D)[:, :L]


def _plain_norm(case, v, w, b):
    if case["norm"] == "layer":
        v = v - v.mean(-1, keepdim=True)
    rstd = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    hat = v * rstd
    out = hat * w
    return (out if b is None else out + b), hat, rstd


def _plain_act(case, g):
    """The gate's value and derivative."""
    if case["act"] == "none":
        return 1.0, None
    sg = torch.sigmoid(g.float())
    if case["act"] == "sigmoid":
        return sg, sg * (1 - sg)
    return g.float() * sg, sg * (1 + g.float() * (1 - sg))


def _plain_norm_backward(case, dn, w, hat, rstd):
    dh = dn * w
    t = hat * (dh * hat).mean(-1, keepdim=True)
    if case["norm"] == "layer":
        t = t + dh.mean(-1, keepdim=True)
    return (dh - t) * rstd


def _run_block(st, case):
    if own:
        mru = _mru()
        p = mru.block_problem(case["rows"], case["D"], norm=case["norm"], act=case["act"], x_dtype=case["dtype"],
                              eps=EPS, res_scale=RES_SCALE)
        w = {k: st[k] for k in ("w_y", "b_y", "s", "w_z")}
        r_out, z, saved = mru.block_norm_t(p, st["r"], y=st["y"], g=st["g"], b_z=st["b_z"],
                                           save="int8" if case["packed"] else None, **w)
        out = {"r": r_out, "z": z}
        if case["train"]:
            ins = {"saved": saved} if case["packed"] else {"r_out": r_out, "y": st["y"], "g": st["g"]}
            gr = mru.block_norm_backward_t(p, dr_out=st["dr"], dz=st["dz"], **ins, **w)
            out.update(dr=gr.dr, dy=gr.dy, dg=gr.dg, dw_y=gr.dw_y, ds=gr.ds, dw_z=gr.dw_z)
            if case["norm"] == "layer":
                out.update(db_y=gr.db_y, db_z=gr.db_z)
        return {k: v for k, v in out.items() if v is not None}
    dt = DT[case["dtype"]]
    s = st["s"] * RES_SCALE
    n, _, _ = _plain_norm(case, st["y"].float(), st["w_y"], st["b_y"])
    act, _ = _plain_act(case, st["g"])
    r2 = st["r"].float() + s * (act * n)
    z, _, _ = _plain_norm(case, r2, st["w_z"], st["b_z"])
    out = {"r": r2.to(dt), "z": z.to(dt)}
    del r2, z, n, act
    if not case["train"]:
        return out
    r2, y, g = out["r"], st["y"], st["g"]
    if case["packed"]:
        r2, y, g = (_plain_unpack(*_plain_pack(v)) if v is not None else None for v in (r2, y, g))
    dz = st["dz"].float()
    _, hat, rstd = _plain_norm(case, r2.float(), st["w_z"], None)
    e = st["dr"].float() + _plain_norm_backward(case, dz, st["w_z"], hat, rstd)
    out["dr"] = e.to(dt)
    out["dw_z"] = (dz * hat).sum(0, dtype=torch.float64).float()
    out["db_z"] = dz.sum(0, dtype=torch.float64).float()
    del dz, hat
    n, hat, rstd = _plain_norm(case, y.float(), st["w_y"], st["b_y"])
    act, dact = _plain_act(case, g)
    out["ds"] = (RES_SCALE * (e * act * n)).sum(0, dtype=torch.float64).float()
    dm = e * s
    del e
    if dact is not None:
        out["dg"] = (dm * n * dact).to(dt)
    dn = dm * act
    del dm, dact, act, n
    out["dw_y"] = (dn * hat).sum(0, dtype=torch.float64).float()
    out["db_y"] = dn.sum(0, dtype=torch.float64).float()
    out["dy"] = _plain_norm_backward(case, dn, st["w_y"], hat, rstd).to(dt)
    if case["norm"] == "rms":
        del out["db_y"], out["db_z"]
    return out


def _plain_pack(x):
    """q (whole numbers, as int8) and the scales of runs of 64 channels."""
    D = x.shape[-1]
    pad = -D % GROUP
    v = torch.nn.functional.pad(x.float(), (0, pad)).unflatten(-1, (-1, GROUP))
    amax = v.abs().amax(-1, keepdim=True)
    # tensor by tensor: a division by or of a number is a product with a rounded reciprocal in torch
    top = torch.full_like(amax, 127.0)
    inv = torch.where(amax > 0, top / amax, torch.zeros_like(amax))
    return torch.round(v * inv).to(torch.int8).flatten(-2)[..., :D], (amax / top).squeeze(-1)


def _plain_unpack(q, scale):
    return q.float() * scale.repeat_interleave(GROUP, -1)[..., : q.shape[-1]]


def _run_pack(st, case):
    if own:
        mru = _mru()
        q, scale = mru.pack8_t(st["x"])
        return {"scale": scale, "x": mru.unpack8_t(q, scale, dtype=DT[case["dtype"]])}
    q, scale = _plain_pack(st["x"])
    return {"scale": scale, "x": _plain_unpack(q, scale).to(DT[case["dtype"]])}


# ---------------------------------------------------------------- exact ---

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "pack":
        return _exact_pack(st["x"])
    if case["op"] == "block":
        return _exact_block(st, case)
    # the sequential loop makes a few small launches per token
    if case["L"] * (3 if case["train"] else 1) > 600000:
        return None
    return _exact_scan(st, case)


def _held(x):
    """The values 8 bits hold of x, in 64 bits (the quantiser itself is
    defined in fp32)."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c in range(0, x.shape[-1], GROUP):
        v = x[..., c:c + GROUP].to(torch.float32)
        top = v.abs().max(-1, keepdim=True).values
        step = torch.div(top, torch.full_like(top, 127.0))
        q = (v * torch.div(torch.full_like(top, 127.0), top)).round()
        out[..., c:c + GROUP] = torch.where(top > 0, q.double() * step.double(), torch.zeros_like(v).double())
    return out


def _exact_pack(x):
    D = x.shape[-1]
    scale = [x[..., c:c + GROUP].double().abs().max(-1).values / 127.0 for c in range(0, D, GROUP)]
    return {"scale": torch.stack(scale, -1), "x": _held(x)}


def _exact_ab(case, x, f, i, lam):
    """Decay, input coefficient (b = coefficient * x) and log-decay of one token, 64 bits."""
    if case["gate"] == "decay":
        return f, torch.ones_like(f), None, None
    if case["gate"] == "sigmoid":
        return 1 / (1 + torch.exp(-f)), 1 / (1 + torch.exp(f)), None, None
    sp = torch.clamp(lam, min=0) + torch.log1p(torch.exp(-lam.abs()))
    la = -C_LRU * sp / (1 + torch.exp(-f))
    gain = torch.sqrt(-torch.expm1(2 * la))
    return torch.exp(la), gain / (1 + torch.exp(-i)), la, gain


def _exact_scan(st, case):
    B, L, D = case["B"], case["L"], case["D"]
    lam = None if st["lam"] is None else st["lam"].double()
    lens = st["lens"].tolist() if st["lens"] is not None else [L] * B
    on = torch.ones((L, B, 1), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        on[n:, b] = 0
    carry = on.new_ones((L, B, 1))
    if st["reset"] is not None:
        carry = (st["reset"] == 0).double().t()[..., None]

    def coefficients(x, f, i):
        """Time-major decay and input, gates and masks applied token block by token block."""
        a = torch.empty((L, B, D), dtype=torch.float64, device="cuda")
        u = torch.empty_like(a)
        for t in range(0, L, 2048):
            s = slice(t, t + 2048)
            xs, fs = x[:, s].double(), f[:, s].double()
            av, cv, _, _ = _exact_ab(case, xs, fs, None if i is None else i[:, s].double(), lam)
            m = on[s]
            a[s] = av.transpose(0, 1) * carry[s] * m + (1 - m)
            u[s] = (cv * xs).transpose(0, 1) * m
        return a, u

    def forward(a, u, kept=None):
        h = st["h0"].double()
        for t in range(L):
            if kept is not None and t > 0 and t % KEPT_EVERY == 0:
                h = kept[t // KEPT_EVERY - 1]
            u[t].addcmul_(a[t], h)                         # in place: u becomes h
            h = u[t]
        return u

    x, f, i = st["x"], st["f"], st["i"]
    a, u = coefficients(x, f, i)
    h = forward(a, u)
    out = {"h_last": h[-1].clone(), "y": (h * on).transpose(0, 1).contiguous()}
    if not case["train"]:
        return out
    if case["packed"]:
        kept = h[KEPT_EVERY - 1::KEPT_EVERY].clone()
        del a, u, h
        x, f, i = (_held(v) if v is not None else None for v in (x, f, i))
        a, u = coefficients(x, f, i)
        h = forward(a, u, kept)
    d = st["dy"].transpose(0, 1).double() * on
    d[-1] += st["dh_last"].double()
    for t in range(L - 2, -1, -1):
        d[t].addcmul_(a[t + 1], d[t + 1])
    out["dh0"] = a[0] * d[0]
    del a
    prev = torch.cat([st["h0"].double()[None], h[:-1]]) * carry
    del h, u
    d, prev = (d * on).transpose(0, 1), prev.transpose(0, 1)
    out["dx"] = torch.empty((B, L, D), dtype=torch.float64, device="cuda")
    out["df"] = torch.empty_like(out["dx"])
    if case["gate"] == "lru":
        out["di"] = torch.empty_like(out["dx"])
        total = torch.zeros(D, dtype=torch.float64, device="cuda")
    for t in range(0, L, 2048):
        s = slice(t, t + 2048)
        xs, fs, ds, ps = x[:, s].double(), f[:, s].double(), d[:, s], prev[:, s]
        iv = None if i is None else i[:, s].double()
        av, cv, la, gain = _exact_ab(case, xs, fs, iv, lam)
        out["dx"][:, s] = ds * cv
        if case["gate"] == "decay":
            out["df"][:, s] = ds * ps
        elif case["gate"] == "sigmoid":
            out["df"][:, s] = ds * (ps - xs) * av * (1 - av)
        else:
            inner = 1 / (1 + torch.exp(-iv))
            out["di"][:, s] = ds * gain * xs * inner * (1 - inner)
            dla = ds * (av * ps - xs * inner * av * av / gain)
            out["df"][:, s] = dla * la * (1 - 1 / (1 + torch.exp(-fs)))
            slope = 1 / (1 + torch.exp(-lam))              # d softplus
            total += (dla * (-C_LRU / (1 + torch.exp(-fs)))).sum((0, 1)) * slope
    if case["gate"] == "lru":
        out["dlam"] = total
    return out


def _exact_block(st, case):
    """Row blocks of the definition in 64 bits, gradients by differentiation."""
    names = ["w_y", "b_y", "s", "w_z", "b_z"]
    par = {k: None if st[k] is None else st[k].double().requires_grad_(case["train"]) for k in names}
    rows = max(1, (1 << 24) // case["D"])
    dims = case["D"]

    def norm(v, w, b):
        if case["norm"] == "layer":
            v = v - v.sum(-1, keepdim=True) / dims
        v = v / torch.sqrt((v * v).sum(-1, keepdim=True) / dims + EPS) * w
        return v if b is None else v + b

    def gate(g):
        if g is None:
            return 1.0
        one = 1 / (1 + torch.exp(-g))
        return one if case["act"] == "sigmoid" else g * one

    parts = {}
    for at in range(0, case["rows"], rows):
        cut = {k: None if st[k] is None else st[k][at:at + rows] for k in ("r", "y", "g")}
        with torch.no_grad():
            r2 = cut["r"].double() + RES_SCALE * par["s"] * gate(None if cut["g"] is None else cut["g"].double()) * \
                norm(cut["y"].double(), par["w_y"], par["b_y"])
            got = {"r": r2, "z": norm(r2, par["w_z"], par["b_z"])}
        if case["train"]:
            # the backward's inputs are what is kept: the stored sum, and 8-bit values where asked for
            kept = {"r": r2.float().to(DT[case["dtype"]]), "y": cut["y"], "g": cut["g"]}
            kept = {k: v if v is None else (_held(v) if case["packed"] else v.double()) for k, v in kept.items()}
            kept = {k: v if v is None else v.requires_grad_(True) for k, v in kept.items()}
            z = norm(kept["r"], par["w_z"], par["b_z"])
            (z * st["dz"][at:at + rows].double()).sum().backward()
            got["dr"] = kept["r"].grad + st["dr"][at:at + rows].double()
            m = RES_SCALE * par["s"] * gate(kept["g"]) * norm(kept["y"], par["w_y"], par["b_y"])
            (m * got["dr"]).sum().backward()
            got["dy"] = kept["y"].grad
            if kept["g"] is not None:
                got["dg"] = kept["g"].grad
        for k, v in got.items():
            parts.setdefault(k, []).append(v)
    out = {k: torch.cat(v) for k, v in parts.items()}
    if case["train"]:
        out.update({"d" + k: v.grad for k, v in par.items() if v is not None})
    return out
