"""Timed and checked cases of linear attention with a decay for each head (prompts, single tokens,
gradients) and of the norm of queries and keys with their rotation in the same pass.

`own` chooses what `run` computes: False, the operators' plain form in elementary torch
operations; True, the library's own kernels through its public calls.
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # --- decayed linear attention: q, k [T, H, dk], v [T, H, dv], log decays [H], fp32 states [nseq, H, dk, dv]
        # the library's serving batch: one token for each of 256 sequences
        dict(name="decay_step_batch", op="step", T=256, H=16, dk=64, dv=64, b="bf16"),
        # one long prompt (B=1, H=16, N=65536)
        dict(name="decay_long", op="decay", T=65536, H=16, dk=64, dv=64, nseq=1, ragged=False, state=False, b="bf16"),
        # packed prompts of mixed lengths that continue from carried states
        dict(name="decay_ragged", op="decay", T=40009, H=8, dk=64, dv=64, nseq=64, ragged=True, state=True, b="bf16"),
        # prompts of a model with wide heads, whose states the decoding goes on from
        dict(name="decay_wide", op="decay", T=16384, H=16, dk=128, dv=128, nseq=4, ragged=False, state=True, b="bf16"),
        # fp32 rows of odd sizes, few tokens: latency
        dict(name="decay_odd", op="decay", T=1025, H=3, dk=37, dv=53, nseq=3, ragged=True, state=True, b="f32"),
        # a training batch (B=8, H=8, N=4096): gradients of queries, keys and values
        dict(name="decay_bwd_batch", op="decay_bwd", T=32768, H=8, dk=64, dv=64, nseq=8, ragged=False, state=False,
             b="bf16"),
        # gradients in fp32 through carried states
        dict(name="decay_bwd_states", op="decay_bwd", T=4099, H=4, dk=64, dv=64, nseq=7, ragged=True, state=True, b="f32"),
        # --- norm of queries and keys with the rotation: q [T, Hq, d], k [T, Hk, d]
        # the long prompt, three axes (time, height, width), every head with its own weight
        dict(name="qk_long", op="qk", T=65536, H=16, Hk=16, d=64, groups=True, pairs="8,12,12", interleaved=False,
             fused=False, b="bf16"),
        # shared key heads of 128, rows of one fused projection's output
        dict(name="qk_fused", op="qk", T=16384, H=16, Hk=4, d=128, groups=False, pairs="64", interleaved=False,
             fused=True, b="bf16"),
        # one token for each sequence of a serving batch
        dict(name="qk_step", op="qk", T=16, H=16, Hk=4, d=64, groups=False, pairs="32", interleaved=False, fused=True,
             b="bf16"),
        # gradients of a training batch
        dict(name="qk_bwd_batch", op="qk_bwd", T=32768, H=8, Hk=8, d=64, groups=False, pairs="32", interleaved=False,
             fused=False, b="bf16"),
        # fp32 gradients, neighbouring pairs, an odd head size whose tail is not rotated
        dict(name="qk_bwd_odd", op="qk_bwd", T=4099, H=7, Hk=7, d=83, groups=True, pairs="20,19", interleaved=True,
             fused=False, b="f32"),
    ]


# A drawn case holds and moves no more than the long listed ones do.
_MAX_ELEMENTS = 65536 * 16 * 64
_MAX_BYTES = 8 * _MAX_ELEMENTS


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["step", "decay", "decay", "decay", "decay_bwd", "decay_bwd", "qk", "qk", "qk_bwd", "qk_bwd"])
    kind = rng.choice(["f32", "bf16", "bf16"])
    case = dict(op=op, b=kind, H=rng.randint(1, 16))
    if op in ("step", "decay", "decay_bwd"):
        case["dk"] = rng.choice([32, 64, 64, 128, _log_int(rng, 1, 128)])
        case["dv"] = rng.choice([case["dk"], case["dk"], _log_int(rng, 1, 128)])
        per = case["H"] * max(case["dk"], case["dv"])
        if op == "step":
            case["T"] = _log_int(rng, 1, min(512, _MAX_ELEMENTS // (case["H"] * case["dk"] * case["dv"])))
        else:
            # fp32 and gradients over fewer tokens
            limit = _MAX_ELEMENTS // per // ((4 if kind == "f32" else 1) * (2 if op == "decay_bwd" else 1))
            case["T"] = _log_int(rng, 1, min(65536, limit))
            case["ragged"] = rng.random() < 0.5
            case["nseq"] = _log_int(rng, 1, 64)
            if not case["ragged"]:
                case["T"] = max(1, case["T"] // case["nseq"]) * case["nseq"]
            case["state"] = rng.random() < 0.5
    else:
        case["Hk"] = rng.choice([case["H"], rng.randint(1, case["H"])])
        case["d"] = rng.choice([32, 64, 64, 128, _log_int(rng, 2, 256)])
        axes = rng.randint(1, min(3, max(1, case["d"] // 2)))
        total = rng.choice([case["d"] // 2, rng.randint(axes, case["d"] // 2)])
        cuts = sorted(rng.randint(0, total) for _ in range(axes - 1))
        case["pairs"] = ",".join(str(y - x) for x, y in zip([0] + cuts, cuts + [total]))
        case["interleaved"] = rng.random() < 0.5
        case["groups"] = rng.random() < 0.5
        case["fused"] = rng.random() < 0.5
        limit = _MAX_ELEMENTS // (case["H"] * case["d"]) // (1 if kind == "bf16" and op == "qk" else 2)
        case["T"] = _log_int(rng, 1, min(65536, limit))
    while work(case)["bytes"] > _MAX_BYTES and case["T"] > case.get("nseq", 1):
        case["T"] = max(case.get("nseq", 1), case["T"] // 2 // case.get("nseq", 1) * case.get("nseq", 1))
    return case


def work(case):
    T, H, s, op = case["T"], case["H"], SIZE[case["b"]], case["op"]
    if op in ("step", "decay", "decay_bwd"):
        dk, dv = case["dk"], case["dv"]
        state = 4 * case.get("nseq", T) * H * dk * dv
        if op == "step":
            return {"bytes": T * H * 2 * (dk + dv) * s + 2 * state + 4 * H, "flops": 5 * T * H * dk * dv}
        # the recurrence's own operations: an update and a readout for each product with a state
        if op == "decay":
            return {"bytes": T * H * 2 * (dk + dv) * s + (2 * state if case["state"] else 0) + 4 * H,
                    "flops": 5 * T * H * dk * dv}
        return {"bytes": T * H * (4 * dk + 3 * dv) * s + (3 * state if case["state"] else 0) + 4 * H,
                "flops": 12 * T * H * dk * dv}
    d, rows = case["d"], T * (H + case["Hk"])
    pairs = [int(p) for p in case["pairs"].split(",")]
    params = 4 * d * (H + case["Hk"] if case["groups"] else 2)
    table = 4 * T * len(pairs) + 4 * sum(pairs)
    if op == "qk":
        return {"bytes": 2 * rows * d * s + 4 * rows + params + table, "flops": 7 * rows * d}
    return {"bytes": 3 * rows * d * s + 4 * rows + 2 * params + table, "flops": 14 * rows * d}


_CHUNK = 128      # tokens of a chunk of the plain form


def _lengths(case, g):
    """Sequence boundaries of a packed batch (empty sequences occur), as a list on the host."""
    T, nseq = case["T"], case["nseq"]
    if not case["ragged"]:
        return [s * (T // nseq) for s in range(nseq + 1)]
    cuts = torch.randint(0, T + 1, (nseq - 1,), generator=g).sort().values.tolist()
    return [0] + cuts + [T]


def _chunks(cu):
    """What the plain form indexes by: every sequence cut into chunks, as (sequence, first token, one past the
    last token, place of the first token in its sequence)."""
    rows = [(s, lo + c, min(lo + c + _CHUNK, hi), c) for s, (lo, hi) in enumerate(zip(cu, cu[1:]))
            for c in range(0, hi - lo, _CHUNK)]
    seq, start, end, place = torch.tensor(rows).T.contiguous().cuda()
    at = start[:, None] + torch.arange(_CHUNK, device="cuda")
    return dict(seq=seq, place=place, n=end - start, at=at.clamp(max=int(cu[-1]) - 1), live=at < end[:, None])


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    T, H, op, tb = case["T"], case["H"], case["op"], DTYPES[case["b"]]
    st = {"case": case}
    if op in ("step", "decay", "decay_bwd"):
        dk, dv = case["dk"], case["dv"]
        st["q"] = (normal(T, H, dk) * dk ** -0.25).to(tb)
        st["k"] = (normal(T, H, dk) * dk ** -0.25).to(tb)
        st["v"] = normal(T, H, dv).to(tb)
        # heads from a memory of two tokens to one of thousands
        reach = 1.0 + 10.0 * (torch.arange(H, device="cuda") + torch.rand(H, generator=g, device="cuda")) / H
        st["log_decay"] = torch.log1p(-(2.0 ** -reach.double())).float()
        st["scale"] = dk ** -0.5
        if op == "step":
            st["state"] = 2.0 * normal(T, H, dk, dv)
            return st
        cu = _lengths(case, cpu)
        st["cu_list"] = cu
        st["cu"] = torch.tensor(cu, dtype=torch.int32).cuda() if case["ragged"] else None
        st["chunks"] = _chunks(cu)
        if case["state"]:
            st["state"] = 2.0 * normal(case["nseq"], H, dk, dv)
        if op == "decay_bwd":
            st["dout"] = normal(T, H, dv).to(tb)
            if case["state"]:
                st["dstate"] = normal(case["nseq"], H, dk, dv)
        return st
    Hk, d = case["Hk"], case["d"]
    pairs = [int(p) for p in case["pairs"].split(",")]
    st["pairs"] = pairs
    # rows of very different size, as projections of a residual stream have them
    if case["fused"]:        # queries, keys and values side by side
        rows = (normal(T, H + 2 * Hk, d) * torch.exp(0.5 * normal(T, H + 2 * Hk, 1))).to(tb)
        st["q"], st["k"] = rows[:, :H], rows[:, H:H + Hk]
    else:
        st["q"] = (normal(T, H, d) * torch.exp(0.5 * normal(T, H, 1))).to(tb)
        st["k"] = (normal(T, Hk, d) * torch.exp(0.5 * normal(T, Hk, 1))).to(tb)
    st["qw"] = 1.0 + 0.1 * (normal(H, d) if case["groups"] else normal(d))
    st["kw"] = 1.0 + 0.1 * (normal(Hk, d) if case["groups"] else normal(d))
    st["eps"] = 1e-6
    st["freq"] = torch.cat([10000.0 ** (-torch.arange(p, dtype=torch.float64) / max(p, 1)) for p in pairs]).float().cuda()
    if len(pairs) == 1:      # a token's place in its sequence, far ones among them
        pos = torch.randint(0, 1 << 20, (T, 1), generator=cpu)
    else:                    # frames of rows and columns
        side = 32
        idx = torch.arange(T) + int(torch.randint(0, 1 << 18, (1,), generator=cpu))
        pos = torch.stack([idx // (side * side), idx // side % side, idx % side], 1)[:, -len(pairs):]
    st["pos"] = pos.to(torch.int32).contiguous().cuda()
    st["axis"] = torch.repeat_interleave(torch.arange(len(pairs)), torch.tensor(pairs)).cuda()   # for the plain form
    if op == "qk_bwd":
        st["qr"], st["kr"] = (torch.rsqrt((st[x].float() ** 2).mean(-1) + st["eps"]) for x in "qk")
        st["dq_out"], st["dk_out"] = normal(T, H, d).to(tb), normal(T, Hk, d).to(tb)
    return st


# --------------------------------------------------------------------------- plain forms

def _powers(st, n):
    """decay^n for whole n >= 0 [...], as fp32 [..., H]: the exponents in 64 bits."""
    return torch.exp(n.double()[..., None] * st["log_decay"].double()).float()


def _chunked(st, x):
    """x [T, H, d] as fp32 [chunks, H, tokens of a chunk, d], nothing behind a sequence's end."""
    c = st["chunks"]
    return torch.where(c["live"][..., None, None], x.float()[c["at"]], 0.0).transpose(1, 2)


def _unchunked(st, y):
    return y.transpose(1, 2)[st["chunks"]["live"]]


def _between(st):
    """[H, chunk, earlier chunk]: the decay from behind the earlier one to the first token of the other."""
    c = st["chunks"]
    gap = c["place"][:, None] - (c["place"] + c["n"])[None, :]
    use = (c["seq"][:, None] == c["seq"][None, :]) & (gap >= 0)
    return torch.where(use[..., None], _powers(st, gap.clamp(min=0)), 0.0).permute(2, 0, 1)


def _states(st, parts, first, decay_to_first, between):
    """The state that enters each chunk: other chunks' parts, and what enters the sequence."""
    s = torch.einsum("hcb,bhkv->chkv", between, parts)
    if first is not None:
        s = s + first[st["chunks"]["seq"]] * decay_to_first[..., None, None]
    return s


def _decay_parts(st):
    i = torch.arange(_CHUNK, device="cuda")
    c = st["chunks"]
    ahead = torch.where((i[:, None] >= i[None, :])[..., None], _powers(st, (i[:, None] - i[None, :]).clamp(min=0)), 0.0)
    into = _powers(st, i + 1).T[None, :, :, None]                                   # [1, H, i, 1]: from the entering state
    to_end = _powers(st, (c["n"][:, None] - 1 - i).clamp(min=0)).permute(0, 2, 1)[..., None]
    return ahead.permute(2, 0, 1), into, to_end


def _sequence_sum(st, parts, weight, carried, kept):
    """Per sequence: sum of weight x parts over its chunks, and the carried state times `kept`."""
    out = torch.zeros(st["case"]["nseq"], *parts.shape[1:], device="cuda")
    out = out.index_add(0, st["chunks"]["seq"], parts * weight[..., None, None])
    return out if carried is None else out + carried * kept[..., None, None]


def _plain(st):
    case = st["case"]
    op, tb = case["op"], DTYPES[case["b"]]
    if op == "step":
        g = torch.exp(st["log_decay"].double()).float()[:, None, None]
        s = g * st["state"] + st["k"].float()[..., :, None] * st["v"].float()[..., None, :]
        return (st["scale"] * (st["q"].float()[..., :, None] * s).sum(-2)).to(tb), s
    if op in ("decay", "decay_bwd"):
        c = st["chunks"]
        q, k, v = (_chunked(st, st[x]) for x in "qkv")
        ahead, into, to_end = _decay_parts(st)
        between = _between(st)
        length = torch.zeros(case["nseq"], dtype=torch.long, device="cuda").index_add(0, c["seq"], c["n"])
        behind = _powers(st, length[c["seq"]] - c["place"] - c["n"])                # from a chunk's end to the sequence's
        before = _powers(st, c["place"])
        whole = _powers(st, length)
        parts = (k * to_end).transpose(-1, -2) @ v
        s = _states(st, parts, st.get("state"), before, between)
    if op == "decay":
        out = ((q @ k.transpose(-1, -2)) * ahead) @ v + (q * into) @ s
        out = _unchunked(st, st["scale"] * out).to(tb)
        if not case["state"]:
            return out
        return out, _sequence_sum(st, parts, behind, st["state"], whole)
    if op == "decay_bwd":
        do = _chunked(st, st["dout"])
        back = ahead.transpose(-1, -2)
        dq = ((do @ v.transpose(-1, -2)) * ahead) @ k + (do * into) @ s.transpose(-1, -2)
        rparts = st["scale"] * ((q * into).transpose(-1, -2) @ do)
        r = _states(st, rparts, st.get("dstate"), behind, between.transpose(-1, -2))  # what enters from behind
        dk = st["scale"] * ((v @ do.transpose(-1, -2)) * back) @ q + (v * to_end) @ r.transpose(-1, -2)
        dv = st["scale"] * ((k @ q.transpose(-1, -2)) * back) @ do + (k * to_end) @ r
        grads = tuple(_unchunked(st, x).to(tb) for x in (st["scale"] * dq, dk, dv))
        if not case["state"]:
            return grads
        return grads + (_sequence_sum(st, rparts, before, st["dstate"], whole),)
    P = sum(st["pairs"])
    angle = st["pos"].double()[:, st["axis"]] * st["freq"].double()      # 64 bits: far positions turn many times
    c, s = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    i0, i1 = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if case["interleaved"] else (slice(0, P), slice(P, 2 * P))

    def rotate(u, s):
        y = u.clone()
        y[..., i0] = u[..., i0] * c - u[..., i1] * s
        y[..., i1] = u[..., i1] * c + u[..., i0] * s
        return y

    def forward(x, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"])
        return rotate(x * r * w, s).to(tb), r.squeeze(-1)

    def backward(x, r, dy, w):
        du = rotate(dy.float(), -s)
        xh = x.float() * r[..., None]
        dx = r[..., None] * (du * w - xh * (du * w * xh).mean(-1, keepdim=True))
        return dx.to(tb), (du * xh).sum((0,) if case["groups"] else (0, 1), dtype=torch.float64).float()

    if op == "qk":
        (qo, qr), (ko, kr) = forward(st["q"], st["qw"]), forward(st["k"], st["kw"])
        return qo, ko, qr, kr
    (dq, dqw), (dk, dkw) = (backward(st["q"], st["qr"], st["dq_out"], st["qw"]),
                            backward(st["k"], st["kr"], st["dk_out"], st["kw"]))
    return dq, dk, dqw, dkw


# --------------------------------------------------------------------------- the library's calls

def _own(st):
    import kernelized_linear_attention_gb300 as la
    case = st["case"]
    op = case["op"]
    if op == "step":
        new = torch.empty_like(st["state"])
        return la.la_decay_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"], scale=st["scale"],
                                state_out=new), new
    if op in ("decay", "decay_bwd"):
        seqs = dict(cu_seqlens=st["cu"], nseq=None if case["ragged"] else case["nseq"])
    if op == "decay":
        return la.la_decay_attention(st["q"], st["k"], st["v"], st["log_decay"], scale=st["scale"],
                                     state_in=st.get("state"), return_state=case["state"], **seqs)
    if op == "decay_bwd":
        return la.la_decay_attention_backward(st["q"], st["k"], st["v"], st["dout"], st["log_decay"],
                                              scale=st["scale"], state_in=st.get("state"),
                                              dstate_out=st.get("dstate"), return_dstate=case["state"], **seqs)
    turn = dict(freq=st["freq"], positions=st["pos"], pairs=st["pairs"], interleaved=case["interleaved"])
    if op == "qk":
        return la.la_qk_norm_rotary(st["q"], st["k"], st["qw"], st["kw"], eps=st["eps"], return_rstd=True, **turn)
    return la.la_qk_norm_rotary_backward(st["q"], st["k"], st["qr"], st["kr"], st["dq_out"], st["dk_out"], st["qw"],
                                         st["kw"], **turn)


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64

    def walk(cu, reverse):
        """Tokens place by place, all sequences side by side: yields (sequences that have the place, their tokens)."""
        lengths = [hi - lo for lo, hi in zip(cu, cu[1:])]
        first = torch.tensor(cu[:-1]).cuda()
        n = torch.tensor(lengths).cuda()
        same = len(set(lengths)) == 1
        every = torch.arange(len(lengths)).cuda()
        for t in range(max(lengths)):
            live = every if same else torch.nonzero(n > t).squeeze(-1)
            yield live, (first[live] + n[live] - 1 - t if reverse else first[live] + t)

    if op in ("step", "decay", "decay_bwd"):
        q, k, v = (st[x].to(f64) for x in "qkv")
        g = st["log_decay"].to(f64).exp()[:, None, None]
        scale = st["scale"]
    if op == "step":
        s = torch.baddbmm(st["state"].to(f64).flatten(0, 1), k.flatten(0, 1)[..., None], v.flatten(0, 1)[:, None, :],
                          beta=0) + (g * st["state"].to(f64)).flatten(0, 1)
        out = scale * torch.bmm(q.flatten(0, 1)[:, None, :], s).squeeze(1)
        return out.view(v.shape), s.view(st["state"].shape)
    if op in ("decay", "decay_bwd"):                  # the recurrence itself, token by token
        cu = st["cu_list"]
        s = st["state"].to(f64) if case["state"] else torch.zeros(case["nseq"], case["H"], case["dk"], case["dv"],
                                                                  dtype=f64, device="cuda")
        res = torch.empty_like(v if op == "decay" else q)
        do = st["dout"].to(f64) if op == "decay_bwd" else None
        for live, t in walk(cu, False):
            new = g * s[live] + k[t][..., :, None] * v[t][..., None, :]
            s[live] = new
            res[t] = scale * ((q[t][..., None, :] @ new).squeeze(-2) if op == "decay" else
                              (new @ do[t][..., :, None]).squeeze(-1))
        if op == "decay":
            return (res, s) if case["state"] else res
        r = st["dstate"].to(f64) if case["state"] else torch.zeros_like(s)   # what enters from behind: decay x gradient
        dk, dv = torch.empty_like(k), torch.empty_like(v)
        for live, t in walk(cu, True):
            new = r[live] + scale * q[t][..., :, None] * do[t][..., None, :]
            dk[t] = (new @ v[t][..., :, None]).squeeze(-1)
            dv[t] = (k[t][..., None, :] @ new).squeeze(-2)
            r[live] = g * new
        return (res, dk, dv, r) if case["state"] else (res, dk, dv)
    P, d = sum(st["pairs"]), case["d"]
    pos = torch.cat([st["pos"][:, i:i + 1].expand(-1, p) for i, p in enumerate(st["pairs"])], 1).to(f64)
    turn = torch.polar(torch.ones_like(pos), pos * st["freq"].to(f64))[:, None]

    def rotated(x, turn):                              # each pair as a complex number times a unit phase
        y, rot = x.clone(), x[..., :2 * P]
        if case["interleaved"]:
            z = torch.view_as_complex(rot.reshape(*rot.shape[:-1], P, 2).contiguous()) * turn
            y[..., :2 * P] = torch.view_as_real(z).reshape(rot.shape)
        else:
            z = torch.complex(rot[..., :P].contiguous(), rot[..., P:].contiguous()) * turn
            y[..., :2 * P] = torch.cat([z.real, z.imag], -1)
        return y

    outs, more = [], []
    for x, w, r, dy in (("q", "qw", "qr", "dq_out"), ("k", "kw", "kr", "dk_out")):
        x, w = st[x].to(f64), st[w].to(f64)
        if op == "qk":
            r = 1.0 / torch.sqrt(x.square().sum(-1) / d + st["eps"])
            outs.append(rotated(x * r[..., None] * w, turn))
            more.append(r)
        else:
            r = st[r].to(f64)[..., None]
            du = rotated(st[dy].to(f64), turn.conj())
            u = du * w
            outs.append(r * u - r ** 3 * x * (u * x).sum(-1, keepdim=True) / d)
            dw = (du * x * r).sum(0)
            more.append(dw if case["groups"] else dw.sum(0))
    return tuple(outs + more)
