"""Timed and checked cases of the operators around linear attention: the gated linear
recurrence, layer norm and rotary positions with several axes.

`own` chooses what `run` computes: False, the operators' plain form in elementary torch
operations; True, the library's own kernels through its public calls.
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # --- gated linear recurrence: a [T, H, d] (gate), b [T, H, d], fp32 states [nseq, H, d]
        # one token for each sequence of a small serving batch
        dict(name="step_small", op="step", T=3, H=16, d=64, a="f32", b="bf16"),
        # the library's long single sequence (B=1, H=16, N=65536), gates kept in fp32
        dict(name="scan_long", op="scan", T=65536, H=16, d=64, nseq=1, ragged=False, state=False, a="f32", b="bf16"),
        # packed sequences of mixed lengths that continue from carried states
        dict(name="scan_ragged", op="scan", T=40009, H=8, d=64, nseq=64, ragged=True, state=True, a="f32", b="f32"),
        # a training batch (B=8, H=8, N=4096) in bf16: gradients of gates and inputs
        dict(name="scan_bwd_batch", op="scan_bwd", T=32768, H=8, d=64, nseq=8, ragged=False, state=False,
             a="bf16", b="bf16"),
        # a short packed batch whose rows are not a multiple of any vector, gradients of the states too
        dict(name="scan_bwd_odd", op="scan_bwd", T=2051, H=5, d=37, nseq=7, ragged=True, state=True, a="f32", b="f32"),
        # --- layer norm: rows [T, H] of d values, weight and bias [H, d] or [d] in fp32
        # the attention output of the long sequence, every head with its own weight
        dict(name="norm_heads", op="norm", T=65536, H=16, d=64, groups=16, b="bf16"),
        # fp32 rows of an odd width, one weight for all
        dict(name="norm_odd", op="norm", T=1025, H=1, d=1023, groups=1, b="f32"),
        # gradients of the per-head norm of a training batch
        dict(name="norm_bwd_heads", op="norm_bwd", T=32768, H=8, d=64, groups=8, b="bf16"),
        # gradients of a norm over a whole model row
        dict(name="norm_bwd_wide", op="norm_bwd", T=8192, H=1, d=4096, groups=1, b="bf16"),
        # --- rotary positions: q, k [T, H, d], positions [T, axes], frequencies [sum(pairs)]
        # a long video token sequence: time, height and width
        dict(name="rotary_video", op="rotary", T=65536, H=16, d=64, pairs="8,12,12", interleaved=False, inverse=False,
             b="bf16"),
        # an image batch in fp32 with neighbouring pairs, an odd head size whose tail is not rotated: the gradient
        dict(name="rotary_odd", op="rotary", T=4099, H=7, d=83, pairs="20,19", interleaved=True, inverse=True, b="f32"),
        # one token for each sequence of a serving batch, at far positions
        dict(name="rotary_step", op="rotary", T=16, H=16, d=64, pairs="32", interleaved=False, inverse=False, b="bf16"),
    ]


# A drawn case holds and moves no more than the long listed ones do.
_MAX_ELEMENTS = 65536 * 16 * 64
_MAX_BYTES = 8 * _MAX_ELEMENTS


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "scan_bwd", "scan_bwd", "norm", "norm_bwd", "rotary", "rotary"])
    kind = rng.choice(["f32", "bf16"])
    case = dict(op=op, b=kind)
    if op in ("step", "scan", "scan_bwd"):
        case["a"] = rng.choice(["f32", kind])
        case["H"] = rng.randint(1, 16)
        case["d"] = rng.choice([32, 64, 64, 128, _log_int(rng, 1, 256)])
        limit = _MAX_ELEMENTS // (case["H"] * case["d"]) // (1 if op != "scan_bwd" else 2)
        case["T"] = _log_int(rng, 1, 512 if op == "step" else min(65536, limit))
        if op != "step":
            case["ragged"] = rng.random() < 0.5
            case["nseq"] = _log_int(rng, 1, 64)
            if not case["ragged"]:
                case["T"] = max(1, case["T"] // case["nseq"]) * case["nseq"]
            case["state"] = rng.random() < 0.5
    elif op in ("norm", "norm_bwd"):
        heads = rng.random() < 0.5
        case["H"] = rng.randint(1, 16) if heads else 1
        case["d"] = rng.choice([32, 64, 128, 256, _log_int(rng, 1, 256)]) if heads else _log_int(rng, 256, 8192)
        case["groups"] = rng.choice([1, case["H"]])
        limit = _MAX_ELEMENTS // (case["H"] * case["d"]) // (1 if kind == "bf16" and op == "norm" else 2)
        case["T"] = _log_int(rng, 1, min(65536, limit))
    else:
        case["H"] = rng.randint(1, 16)
        case["d"] = rng.choice([32, 64, 64, 128, _log_int(rng, 2, 256)])
        axes = rng.randint(1, min(3, max(1, case["d"] // 2)))
        total = rng.choice([case["d"] // 2, rng.randint(axes, case["d"] // 2)])
        cuts = sorted(rng.randint(0, total) for _ in range(axes - 1))
        case["pairs"] = ",".join(str(y - x) for x, y in zip([0] + cuts, cuts + [total]))
        case["interleaved"] = rng.random() < 0.5
        case["inverse"] = rng.random() < 0.5
        limit = _MAX_ELEMENTS // (case["H"] * case["d"]) // (1 if kind == "bf16" else 2)
        case["T"] = _log_int(rng, 1, min(65536, limit))
    while work(case)["bytes"] > _MAX_BYTES:
        case["T"] = case["T"] // 2 // case.get("nseq", 1) * case.get("nseq", 1)
    return case


def _elements(case):
    return case["T"] * case["H"] * case["d"]


def work(case):
    n, sb = _elements(case), SIZE[case["b"]]
    op = case["op"]
    if op in ("step", "scan", "scan_bwd"):
        sa = SIZE[case["a"]]
        states = 4 * case.get("nseq", case["T"]) * case["H"] * case["d"]
        if op == "step":
            return {"bytes": n * (sa + 2 * sb) + 2 * states, "flops": 2 * n}
        if op == "scan":
            return {"bytes": n * (sa + 2 * sb) + (2 * states if case["state"] else 0), "flops": 2 * n}
        return {"bytes": n * (2 * sa + 3 * sb) + (3 * states if case["state"] else 0), "flops": 3 * n}
    if op in ("norm", "norm_bwd"):
        rows, params = case["T"] * case["H"], 4 * case["groups"] * case["d"]
        if op == "norm":
            return {"bytes": 2 * n * sb + 8 * rows + 2 * params, "flops": 8 * n}
        return {"bytes": 3 * n * sb + 8 * rows + 3 * params, "flops": 14 * n}
    pairs = [int(p) for p in case["pairs"].split(",")]
    return {"bytes": 4 * n * sb + 4 * case["T"] * len(pairs) + 4 * sum(pairs),
            "flops": 2 * case["T"] * case["H"] * 6 * sum(pairs)}


def _lengths(case, g):
    """Sequence boundaries of a packed batch (empty sequences occur), as a list on the host."""
    T, nseq = case["T"], case["nseq"]
    if not case["ragged"]:
        return [s * (T // nseq) for s in range(nseq + 1)]
    cuts = torch.randint(0, T + 1, (nseq - 1,), generator=g).sort().values.tolist()
    return [0] + cuts + [T]


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    T, H, d = case["T"], case["H"], case["d"]
    tb = DTYPES[case["b"]]
    st = {"case": case}
    op = case["op"]
    if op in ("step", "scan", "scan_bwd"):
        # forget gates near one, as a sigmoid of a shifted projection gives them
        st["a"] = torch.sigmoid(2.0 + 1.5 * normal(T, H, d)).to(DTYPES[case["a"]])
        st["b"] = normal(T, H, d).to(tb)
        if op == "step":
            st["state"] = 2.0 * normal(T, H, d)
            return st
        cu = _lengths(case, cpu)
        st["cu_list"] = cu
        st["cu"] = torch.tensor(cu, dtype=torch.int32).cuda() if case["ragged"] else None
        # what the plain form indexes by: the sequences that have rows, their first and last rows
        live = [s for s in range(case["nseq"]) if cu[s + 1] > cu[s]]
        st["live"] = torch.tensor(live).cuda()
        st["heads"] = torch.tensor([cu[s] for s in live]).cuda()
        st["tails"] = torch.tensor([cu[s + 1] - 1 for s in live]).cuda()
        st["first"] = torch.zeros(T, 1, 1, dtype=torch.bool, device="cuda").index_fill_(0, st["heads"], True)
        st["last"] = torch.zeros(T, 1, 1, dtype=torch.bool, device="cuda").index_fill_(0, st["tails"], True)
        if case["state"]:
            st["state"] = 2.0 * normal(case["nseq"], H, d)
        if op == "scan_bwd":
            h = _plain_scan(st["a"].float(), st["b"].float(), st)
            st["h"] = h.to(tb)
            st["dh"] = normal(T, H, d).to(tb)
            if case["state"]:
                st["dstate"] = normal(case["nseq"], H, d)
            del st["b"]
        return st
    if op in ("norm", "norm_bwd"):
        # rows of very different size, as unnormalised attention outputs have them
        st["x"] = ((normal(T, H, d) + 0.25) * torch.exp(normal(T, H, 1))).to(tb)
        G = case["groups"]
        st["weight"] = 1.0 + 0.1 * normal(G, d)
        st["bias"] = 0.1 * normal(G, d)
        if G == 1:
            st["weight"], st["bias"] = st["weight"][0].contiguous(), st["bias"][0].contiguous()
        st["eps"] = 1e-5
        if op == "norm_bwd":
            x = st["x"].float()
            mean = x.mean(-1, keepdim=True)
            st["mean"] = mean.squeeze(-1).contiguous()
            st["rstd"] = torch.rsqrt(((x - mean) ** 2).mean(-1) + st["eps"]).contiguous()
            st["dy"] = normal(T, H, d).to(tb)
        return st
    pairs = [int(p) for p in case["pairs"].split(",")]
    st["pairs"] = pairs
    st["q"], st["k"] = normal(T, H, d).to(tb), normal(T, H, d).to(tb)
    # every axis has its own ladder of frequencies, from one radian a step downwards
    st["freq"] = torch.cat([10000.0 ** (-torch.arange(p, dtype=torch.float64) / max(p, 1)) for p in pairs]).float().cuda()
    if len(pairs) == 1:      # a token's place in its sequence, far ones among them
        pos = torch.randint(0, 1 << 20, (T, 1), generator=cpu)
    else:                    # frames of rows and columns
        side = 32
        idx = torch.arange(T) + int(torch.randint(0, 1 << 18, (1,), generator=cpu))
        pos = torch.stack([idx // (side * side), idx // side % side, idx % side], 1)[:, -len(pairs):]
    st["pos"] = pos.to(torch.int32).contiguous().cuda()
    st["axis"] = torch.repeat_interleave(torch.arange(len(pairs)), torch.tensor(pairs)).cuda()   # for the plain form
    return st


# --------------------------------------------------------------------------- plain forms

def _doubling(a, b):
    """Inclusive scan of h_t = a_t h_{t-1} + b_t over dimension 0 by recursive doubling."""
    n, s = a.shape[0], 1
    while s < n:
        b = torch.cat([b[:s], b[s:] + a[s:] * b[:-s]])
        if 2 * s < n:
            a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return b


def _plain_scan(a, b, st):
    if "state" in st:
        heads = st["heads"]
        b = b.index_copy(0, heads, b[heads] + a[heads] * st["state"][st["live"]])
    return _doubling(torch.where(st["first"], 0.0, a), b)


def _plain(st):
    case = st["case"]
    op = case["op"]
    tb = DTYPES[case["b"]]
    if op == "step":
        s = st["a"].float() * st["state"] + st["b"].float()
        return s.to(tb), s
    if op == "scan":
        h = _plain_scan(st["a"].float(), st["b"].float(), st)
        if not case["state"]:
            return h.to(tb)
        return h.to(tb), st["state"].index_copy(0, st["live"], h[st["tails"]])
    if op == "scan_bwd":
        a, h, dh = st["a"].float(), st["h"].float(), st["dh"].float()
        if case["state"]:
            dh = dh.index_add(0, st["tails"], st["dstate"][st["live"]])
        nxt = torch.cat([a[1:], torch.zeros_like(a[:1])])          # a_{t+1}, nothing behind a last row
        g = _doubling(torch.where(st["last"], 0.0, nxt).flip(0), dh.flip(0)).flip(0)
        before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
        before = torch.where(st["first"], 0.0, before)
        if case["state"]:
            before = before.index_copy(0, st["heads"], st["state"][st["live"]])
        da, db = (g * before).to(DTYPES[case["a"]]), g.to(tb)
        if not case["state"]:
            return da, db
        return da, db, st["dstate"].index_copy(0, st["live"], a[st["heads"]] * g[st["heads"]])
    if op == "norm":
        x = st["x"].float()
        mean = x.mean(-1, keepdim=True)
        c = x - mean
        rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + st["eps"])
        return (c * rstd * st["weight"] + st["bias"]).to(tb), mean.squeeze(-1), rstd.squeeze(-1)
    if op == "norm_bwd":
        x, dy = st["x"].float(), st["dy"].float()
        xh = (x - st["mean"].unsqueeze(-1)) * st["rstd"].unsqueeze(-1)
        gy = dy * st["weight"]
        dx = st["rstd"].unsqueeze(-1) * (gy - gy.mean(-1, keepdim=True) - xh * (gy * xh).mean(-1, keepdim=True))
        over = (0,) if case["groups"] > 1 else (0, 1)
        return (dx.to(tb), (dy * xh).sum(over, dtype=torch.float64).float(), dy.sum(over, dtype=torch.float64).float())
    P = sum(st["pairs"])
    angle = st["pos"].double()[:, st["axis"]] * st["freq"].double()      # 64 bits: far positions turn many times
    c, s = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    if case["inverse"]:
        s = -s
    outs = []
    for x in (st["q"], st["k"]):
        x = x.float()
        y = x.clone()
        i0, i1 = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if case["interleaved"] else (slice(0, P), slice(P, 2 * P))
        y[..., i0] = x[..., i0] * c - x[..., i1] * s
        y[..., i1] = x[..., i1] * c + x[..., i0] * s
        outs.append(y.to(tb))
    return tuple(outs)


# --------------------------------------------------------------------------- the library's calls

def _own(st):
    import kernelized_linear_attention_gb300 as la
    case = st["case"]
    op = case["op"]
    if op == "step":
        out = torch.empty_like(st["state"])
        return la.la_gated_step(st["a"], st["b"], st["state"], state_out=out), out
    if op in ("scan", "scan_bwd"):
        seqs = dict(cu_seqlens=st["cu"], nseq=None if case["ragged"] else case["nseq"])
    if op == "scan":
        return la.la_gated_scan(st["a"], st["b"], state_in=st.get("state"), return_state=case["state"], **seqs)
    if op == "scan_bwd":
        return la.la_gated_scan_backward(st["a"], st["h"], st["dh"], state_in=st.get("state"),
                                         dstate_out=st.get("dstate"), return_dstate=case["state"], **seqs)
    if op == "norm":
        return la.la_layer_norm(st["x"], st["weight"], st["bias"], eps=st["eps"], return_stats=True)
    if op == "norm_bwd":
        return la.la_layer_norm_backward(st["x"], st["dy"], st["mean"], st["rstd"], st["weight"])
    return la.la_rotary(st["q"], st["k"], st["freq"], st["pos"], st["pairs"], interleaved=case["interleaved"],
                        inverse=case["inverse"])


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "step":
        s = torch.addcmul(st["b"].to(f64), st["a"].to(f64), st["state"].to(f64))
        return s, s
    if op in ("scan", "scan_bwd"):
        cu = st["cu_list"]
        spans = [(s, cu[s], cu[s + 1]) for s in range(case["nseq"])]
        a = st["a"].to(f64)
        zero = torch.zeros_like(a[0])
        s_in = st["state"].to(f64) if case["state"] else None
    if op == "scan":                                   # the recurrence itself, token by token
        h = st["b"].to(f64)
        s_out = s_in.clone() if case["state"] else None
        for s, lo, hi in spans:
            prev = s_in[s] if case["state"] else zero
            for t in range(lo, hi):
                prev = h[t].addcmul_(a[t], prev)
            if case["state"]:
                s_out[s] = prev
        return (h, s_out) if case["state"] else h
    if op == "scan_bwd":                               # its adjoint, from every last token backwards
        g = st["dh"].to(f64)
        h = st["h"].to(f64)
        da = torch.zeros_like(a)
        ds = st["dstate"].to(f64) if case["state"] else None
        for s, lo, hi in spans:
            carry = ds[s].clone() if case["state"] else zero   # gradient that reaches h_t from behind t
            for t in range(hi - 1, lo - 1, -1):
                g[t] += carry
                carry = a[t] * g[t]
                if t > lo:
                    da[t] = g[t] * h[t - 1]
                elif case["state"]:
                    da[t] = g[t] * s_in[s]
            if case["state"]:
                ds[s] = carry
        return (da, g, ds) if case["state"] else (da, g)
    if op == "norm":
        x = st["x"].to(f64)
        var, mean = torch.var_mean(x, dim=-1, correction=0)
        rstd = 1.0 / torch.sqrt(var + st["eps"])
        y = (x - mean[..., None]) * rstd[..., None] * st["weight"].to(f64) + st["bias"].to(f64)
        return y, mean, rstd
    if op == "norm_bwd":
        d = case["d"]
        x, dy, w = st["x"].to(f64), st["dy"].to(f64), st["weight"].to(f64)
        r = st["rstd"].to(f64)[..., None]
        c = x - st["mean"].to(f64)[..., None]
        u = dy * w
        dx = r * u - r * u.sum(-1, keepdim=True) / d - r ** 3 * c * (u * c).sum(-1, keepdim=True) / d
        rows = (dy * c * r), dy
        if case["groups"] > 1:
            return dx, rows[0].sum(0), rows[1].sum(0)
        return dx, rows[0].reshape(-1, d).sum(0), rows[1].reshape(-1, d).sum(0)
    # rotary: each pair as a complex number times a unit phase
    P = sum(st["pairs"])
    pos = torch.cat([st["pos"][:, i:i + 1].expand(-1, p) for i, p in enumerate(st["pairs"])], 1).to(f64)
    turn = torch.polar(torch.ones_like(pos), pos * st["freq"].to(f64))
    if case["inverse"]:
        turn = turn.conj()
    outs = []
    for x in (st["q"].to(f64), st["k"].to(f64)):
        y = x.clone()
        rot = x[..., :2 * P]
        if case["interleaved"]:
            z = torch.view_as_complex(rot.reshape(*rot.shape[:-1], P, 2).contiguous()) * turn[:, None]
            y[..., :2 * P] = torch.view_as_real(z).reshape(rot.shape)
        else:
            z = torch.complex(rot[..., :P].contiguous(), rot[..., P:].contiguous()) * turn[:, None]
            y[..., :2 * P] = torch.cat([z.real, z.imag], -1)
        outs.append(y)
    return tuple(outs)
