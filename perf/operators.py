"""The selective state-space mixer's operators, as cases to measure.

Four operators, each in the directions a user calls:

  prologue   u = silu(conv(xbc) + bias) (causal, depthwise, per sequence), step = softplus(delta + delta_bias),
             g = a * step; and the gradients of all inputs and parameters
  scan       H_t = e^{g_t} H_{t-1} + step_t B_t x_t^T, y_t = H_t^T C_t + D x_t per head; and its gradients
  decode     one token of prologue and scan against pools of convolution states and states
  norm       p = post . t / rms_group(t) with t = x . silu(z), r = residual + scale . p, n = pre . r / rms(r);
             and its gradients

`run` computes them from elementary torch operations in 32 bits, or, where `own` is true, by the framework's calls.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------------------------------------------------
# cases

def _mix(name, op, lens, H, G, P, N, dtype, packed=False, state=False, **more):
    return {"name": name, "op": op, "lens": lens, "H": H, "G": G, "P": P, "N": N, "dtype": dtype, "packed": packed,
            "state": state, **more}


def _norm(name, op, rows, d, groups, dtype, gate, post, residual, scale, pre):
    return {"name": name, "op": op, "rows": rows, "d": d, "groups": groups, "dtype": dtype, "gate": gate, "post": post,
            "residual": residual, "scale": scale, "pre": pre}


def listed():
    return [
        # a training batch's input side: 64 heads of 64, 8 groups of 128 states
        _mix("prologue-2x4096-bf16", "prologue", "4096,4096", 64, 8, 64, 128, "bf16"),
        # gradients of a packed batch: documents of any length, one of them empty, one a single token
        _mix("prologue-grad-packed-bf16", "prologue_grad", "1777,64,1,0,3025,512", 40, 1, 64, 128, "bf16", packed=True),
        # a short prompt in full precision: latency counts
        _mix("scan-77-f32", "scan", "77", 8, 2, 64, 64, "f32", state=True),
        # the training shape: four sequences of 2048
        _mix("scan-4x2048-bf16", "scan", "2048,2048,2048,2048", 32, 1, 64, 128, "bf16"),
        # a long prefill that hands its state to decoding
        _mix("scan-2x32768-bf16", "scan", "32768,32768", 32, 4, 64, 128, "bf16", state=True),
        # a serving step that prefills several prompts, each continuing from a state
        _mix("scan-packed-bf16", "scan", "1900,1,0,4096,333,27,129,2048", 48, 8, 64, 128, "bf16", packed=True, state=True),
        # the training shape's gradients
        _mix("scan-grad-4x2048-bf16", "scan_grad", "2048,2048,2048,2048", 32, 1, 64, 128, "bf16"),
        # gradients in full precision through given states, packed and ragged
        _mix("scan-grad-packed-f32", "scan_grad", "1000,1,63,300", 8, 2, 64, 64, "f32", packed=True, state=True),
        # one sequence decoding: latency
        _mix("decode-1-bf16", "decode", "1", 48, 8, 64, 128, "bf16", slots=4, state_dtype="f32"),
        # a decoding batch out of a larger pool: the state's bytes
        _mix("decode-64-bf16", "decode", "64", 48, 8, 64, 128, "bf16", slots=96, state_dtype="f32"),
        # the residual stream of a prefill: gated norm after the block, scaled residual, norm before the next block
        _norm("norm-16384x4096-bf16", "norm", 16384, 4096, 8, "bf16", True, True, True, True, True),
        # its gradients on a training batch
        _norm("norm-grad-8192x2048-bf16", "norm_grad", 8192, 2048, 1, "bf16", True, True, True, True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, total):
    """`total` tokens in 1 to 12 sequences of uneven lengths, empty ones among them."""
    n = rng.randint(1, 12)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def draw(rng):
    op = rng.choice(("prologue", "prologue_grad", "scan", "scan", "scan_grad", "scan_grad", "decode", "norm", "norm_grad"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op.startswith("norm"):
        d = 64 * _log(rng, 8, 80)
        d += 64 if d == 3072 else 0
        groups = rng.choice([k for k in (1, 2, 4, 8) if d % (8 * k) == 0])
        flag = lambda: rng.random() < 0.6  # noqa: E731
        pre, residual = flag(), flag()
        post = flag() or not pre
        c = _norm("", op, _log(rng, 1, 16384), d, groups if post else 1, dtype, flag(), post, residual, residual and flag(), pre)
    else:
        G = rng.choice((1, 2, 4, 8))
        H = G * rng.choice((1, 2, 3, 5, 8))
        P, N = rng.choice(((64, 128), (64, 128), (64, 64), (128, 128)))
        if op == "decode":
            B = _log(rng, 1, 200)
            c = _mix("", op, str(B), H, G, P, N, dtype, slots=B + rng.randint(0, B), state_dtype=rng.choice(("f32", "f32", "bf16")))
        else:
            total = _log(rng, 1, 8192 if dtype == "bf16" else 4096)
            packed = rng.random() < 0.5
            lens = _split(rng, total) if packed else [max(1, total // rng.choice((1, 1, 2, 3)))] * rng.choice((1, 2, 3))
            c = _mix("", op, ",".join(map(str, lens)), H, G, P, N, dtype, packed=packed, state=op.startswith("scan") and rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------------------------------
# inputs

def _lens(c):
    return [int(v) for v in c["lens"].split(",")]


def _channels(c):
    return c["H"] * c["P"] + 2 * c["G"] * c["N"]


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DT[c["dtype"]]
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    uniform = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    s = {"case": dict(c)}
    if c["op"].startswith("norm"):
        R, d = c["rows"], c["d"]
        s["x"] = normal(R, d).to(dt)
        s["z"] = normal(R, d).to(dt) if c["gate"] else None
        s["post"] = 1 + 0.1 * normal(d) if c["post"] else None
        s["residual"] = (2 * normal(R, d)).to(dt) if c["residual"] else None
        s["scale"] = 0.5 + uniform(d) if c["scale"] else None
        s["pre"] = 1 + 0.1 * normal(d) if c["pre"] else None
        if c["op"] == "norm_grad":
            s["d_r"] = normal(R, d).to(dt) if c["residual"] or not c["pre"] else None
            s["d_n"] = normal(R, d).to(dt) if c["pre"] else None
        return s
    lens, H, G, P, N, ch = _lens(c), c["H"], c["G"], c["P"], c["N"], _channels(c)
    a = -(1 + 15 * uniform(H))  # decay rates, and steps of 0.001 to 0.1: heads that forget in ten tokens and in thousands
    step0 = torch.exp(math.log(1e-3) + uniform(H) * math.log(100.0))
    delta_bias = step0 + torch.log(-torch.expm1(-step0))
    weight, bias = 0.4 * normal(ch, 4), 0.1 * normal(ch)
    skip = 1 + 0.1 * normal(H)
    if c["op"] == "decode":
        B, slots = lens[0], c["slots"]
        row = normal(B, ch + H).to(dt)  # the token's projection; the operator reads slices of its rows
        s.update(xbc=row[:, :ch], delta=row[:, ch:], weight=weight, bias=bias, a=a, delta_bias=delta_bias, skip=skip,
                 conv_state=normal(slots, 3, ch), state=(0.3 * normal(slots, H, N, P)).to(DT[c["state_dtype"]]),
                 slots=torch.randperm(slots, generator=gen, device="cuda")[:B].to(torch.int32))
        return s
    lead = (sum(lens),) if c["packed"] else (len(lens), lens[0])
    if c["packed"]:
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    else:
        s["offsets"] = None
    if c["op"].startswith("prologue"):
        row = normal(*lead, ch + H).to(dt)
        s.update(xbc=row[..., :ch], delta=row[..., ch:], weight=weight, bias=bias, a=a, delta_bias=delta_bias)
        if c["op"] == "prologue_grad":
            s.update(du=normal(*lead, ch).to(dt), dstep=normal(*lead, H).to(dt), dg=normal(*lead, H).to(dt))
        return s
    u = normal(*lead, ch)
    u = (u * torch.sigmoid(u)).to(dt)  # what the convolution leaves: x, B and C side by side
    step = torch.nn.functional.softplus(0.5 * normal(*lead, H) + delta_bias)
    s.update(x=u[..., :H * P].unflatten(-1, (H, P)), bm=u[..., H * P:H * P + G * N].unflatten(-1, (G, N)),
             cm=u[..., H * P + G * N:].unflatten(-1, (G, N)), step=step.to(dt), g=(a * step).to(dt), skip=skip,
             s0=0.3 * normal(len(lens), H, N, P) if c["state"] else None)
    if c["op"] == "scan_grad":
        s.update(dy=normal(*lead, H, P).to(dt), ds1=0.3 * normal(len(lens), H, N, P) if c["state"] else None)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# plain forms, in 32 bits

def _grid(c, offsets):
    """For packed tokens: [sequence, position] -> token, and whether there is one."""
    at = torch.arange(max(max(_lens(c)), 1), device="cuda")
    idx = offsets[:-1, None].long() + at
    return idx.clamp(max=max(sum(_lens(c)) - 1, 0)), at < (offsets[1:] - offsets[:-1])[:, None]


def _pad(t, grid):
    """Packed tokens as [sequence, position, ...], zeros where there is none."""
    idx, there = grid
    if t.shape[0] == 0:
        return t.new_zeros(*idx.shape, *t.shape[1:])
    return torch.where(there.reshape(*there.shape, *[1] * (t.dim() - 1)), t[idx], t.new_zeros(()))


def _conv(x, weight, bias, before):
    """x [S, T, ch] after `before` [S, 3, ch] -> its causal convolution and the convolution's SiLU."""
    T, full = x.shape[1], torch.cat([before, x], 1)
    v = bias + sum(weight[:, j] * full[:, j:j + T] for j in range(4))
    return v, v * torch.sigmoid(v)


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _prologue(s):
    c, dt = s["case"], s["xbc"].dtype
    x, delta = s["xbc"].float(), s["delta"].float()
    grid = _grid(c, s["offsets"]) if c["packed"] else None
    xp = _pad(x, grid) if c["packed"] else x
    _, u = _conv(xp, s["weight"], s["bias"], xp.new_zeros(xp.shape[0], 3, xp.shape[2]))
    if c["packed"]:
        u = u[grid[1]]
    step = _softplus(delta + s["delta_bias"])
    return {"u": u.to(dt), "step": step.to(dt), "g": (s["a"] * step).to(dt)}


def _prologue_grad(s):
    c, dt = s["case"], s["xbc"].dtype
    x, delta, du = s["xbc"].float(), s["delta"].float(), s["du"].float()
    dstep, dg = s["dstep"].float(), s["dg"].float()
    if c["packed"]:
        grid = _grid(c, s["offsets"])
        x, du = _pad(x, grid), _pad(du, grid)
    T = x.shape[1]
    zeros = x.new_zeros(x.shape[0], 3, x.shape[2])
    v, _ = _conv(x, s["weight"], s["bias"], zeros)
    sig = torch.sigmoid(v)
    dv = du * sig * (1 + v * (1 - sig))
    before, after = torch.cat([zeros, x], 1), torch.cat([dv, zeros], 1)
    dx = sum(s["weight"][:, j] * after[:, 3 - j:3 - j + T] for j in range(4))
    dweight = torch.stack([(dv * before[:, j:j + T]).sum((0, 1)) for j in range(4)], 1)
    dbias = dv.sum((0, 1))
    if c["packed"]:
        dx = dx[grid[1]]
    w = delta + s["delta_bias"]
    dw = (dstep + s["a"] * dg) * torch.sigmoid(w)
    lead = tuple(range(delta.dim() - 1))
    return {"dxbc": dx.to(dt), "ddelta": dw.to(dt), "dweight": dweight, "dbias": dbias, "da": (dg * _softplus(w)).sum(lead),
            "ddelta_bias": dw.sum(lead)}


def _segment_sums(t):
    """[..., n] -> [..., n, n]: the sum of t over (j, i] for j <= i, and -inf for j > i."""
    n = t.shape[-1]
    below = torch.ones(n, n, dtype=torch.bool, device=t.device).tril(-1)
    sums = torch.where(below, t[..., :, None], t.new_zeros(())).cumsum(-2)
    return torch.where(below | torch.eye(n, dtype=torch.bool, device=t.device), sums, t.new_full((), -math.inf))


def _scan_padded(x, step, g, bm, cm, skip, s0):
    """x [S, T, H, P], step and g [S, T, H], bm and cm [S, T, G, N], s0 [S, H, N, P] -> y and the last state: within chunks of
    64 tokens as products of matrices, and over the chunks by their decays."""
    S, T, H, P = x.shape
    G, N = bm.shape[2:]
    Q = 64
    short = -T % Q
    chunked = lambda t: torch.nn.functional.pad(t, [0, 0] * (t.dim() - 2) + [0, short]).unflatten(1, (-1, Q))  # noqa: E731
    heads = lambda t: t.repeat_interleave(H // G, 3)  # noqa: E731
    xc, sc, gc, bc, cc = chunked(x), chunked(step), chunked(g).movedim(3, 2), chunked(bm), chunked(cm)
    within = torch.exp(_segment_sums(gc))                                                    # [S, c, H, i, j]
    scores = torch.einsum("scign,scjgn->scgij", cc, bc).repeat_interleave(H // G, 2)
    xs = xc * sc[..., None]
    y = torch.einsum("schij,scjhp->scihp", scores * within, xs)
    to_end = within[..., -1, :].movedim(2, 3)                                                # [S, c, j, H]
    added = torch.einsum("scjhn,scjhp->schnp", heads(bc), xs * to_end[..., None])
    decay = torch.exp(_segment_sums(torch.nn.functional.pad(gc.sum(-1).movedim(1, 2), [1, 0])))  # [S, H, c + 1, c + 1]
    every = torch.einsum("shij,sjhnp->sihnp", decay, torch.cat([s0[:, None], added], 1))     # states at chunk ends
    from_start = torch.exp(gc.cumsum(-1)).movedim(2, 3)
    y = y + torch.einsum("scihn,schnp->scihp", heads(cc), every[:, :-1]) * from_start[..., None]
    return (y + skip[:, None] * xc).flatten(1, 2)[:, :T], every[:, -1]


def _scan_f32(s, t):
    """The scan of tensors `t` in 32 bits: y in the tokens' own layout and the last states."""
    c = s["case"]
    grid = _grid(c, s["offsets"]) if c["packed"] else None
    tok = [_pad(t[k], grid) if c["packed"] else t[k] for k in ("x", "step", "g", "bm", "cm")]
    s0 = t["s0"] if t["s0"] is not None else tok[0].new_zeros(tok[0].shape[0], c["H"], c["N"], c["P"])
    y, s1 = _scan_padded(*tok, t["skip"], s0)
    return (y[grid[1]] if c["packed"] else y), s1


def _scan(s):
    t = {k: s[k].float() if s[k] is not None else None for k in ("x", "step", "g", "bm", "cm", "skip", "s0")}
    y, s1 = _scan_f32(s, t)
    return {"y": y.to(s["x"].dtype), **({"state": s1} if s["case"]["state"] else {})}


def _scan_grad(s):
    names = ["x", "step", "g", "bm", "cm", "skip"] + (["s0"] if s["s0"] is not None else [])
    t = {k: s[k].float().detach().requires_grad_() for k in names}
    with torch.enable_grad():
        y, s1 = _scan_f32(s, {"s0": None, **t})
        outs, ups = [y], [s["dy"].float()]
        if s["ds1"] is not None:
            outs, ups = outs + [s1], ups + [s["ds1"]]
        got = torch.autograd.grad(outs, [t[k] for k in names], ups)
    return {"d" + k: v if k in ("skip", "s0") else v.to(s["x"].dtype) for k, v in zip(names, got)}


def _decode(s):
    c, dt = s["case"], s["xbc"].dtype
    H, G, P, N = c["H"], c["G"], c["P"], c["N"]
    at = s["slots"].long()
    x = s["xbc"].float()
    before = s["conv_state"][at]
    _, u = _conv(x[:, None], s["weight"], s["bias"], before)
    s["conv_state"][at] = torch.cat([before[:, 1:], x[:, None]], 1)
    xs, bm, cm = u[:, 0].split([H * P, G * N, G * N], 1)
    xs = xs.reshape(-1, H, P)
    bm, cm = (t.reshape(-1, G, N).repeat_interleave(H // G, 1) for t in (bm, cm))
    step = _softplus(s["delta"].float() + s["delta_bias"])
    h = torch.exp(s["a"] * step)[..., None, None] * s["state"][at].float() + bm[..., None] * (step[..., None] * xs)[:, :, None]
    s["state"][at] = h.to(s["state"].dtype)
    y = (h * cm[..., None]).sum(2) + s["skip"][:, None] * xs
    return {"y": y.to(dt), "state": s["state"], "conv_state": s["conv_state"]}


def _norm_parts(s):
    c = s["case"]
    x, d = s["x"].float(), c["d"]
    sig = torch.sigmoid(s["z"].float()) if c["gate"] else None
    t = x * (s["z"].float() * sig) if c["gate"] else x
    inv_t, p = None, t
    if c["post"]:
        tg = t.unflatten(1, (c["groups"], -1))
        inv_t = torch.rsqrt(tg.square().mean(-1, keepdim=True) + EPS)
        p = (tg * inv_t).flatten(1) * s["post"]
    r = p * s["scale"] if c["scale"] else p
    r = r + s["residual"].float() if c["residual"] else r
    inv_r = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) if c["pre"] else None
    return x, sig, t, inv_t, p, r, inv_r


def _norm_run(s):
    c, dt = s["case"], s["x"].dtype
    *_, r, inv_r = _norm_parts(s)
    return {**({"r": r.to(dt)} if c["residual"] or not c["pre"] else {}), **({"n": (r * inv_r * s["pre"]).to(dt)} if c["pre"] else {})}


def _norm_grad(s):
    c, dt = s["case"], s["x"].dtype
    x, sig, t, inv_t, p, r, inv_r = _norm_parts(s)
    got = {}
    dr = s["d_r"].float() if s["d_r"] is not None else torch.zeros_like(r)
    if c["pre"]:
        dn, nh = s["d_n"].float(), r * inv_r
        got["dpre"] = (dn * nh).sum(0)
        k = dn * s["pre"]
        dr = dr + inv_r * (k - nh * (k * nh).mean(-1, keepdim=True))
    if c["residual"]:
        got["dresidual"] = dr.to(dt)
    dp = dr
    if c["scale"]:
        got["dscale"] = (dr * p).sum(0)
        dp = dr * s["scale"]
    dtt = dp
    if c["post"]:
        th = t.unflatten(1, (c["groups"], -1)) * inv_t
        got["dpost"] = (dp * th.flatten(1)).sum(0)
        k = (dp * s["post"]).unflatten(1, (c["groups"], -1))
        dtt = (inv_t * (k - th * (k * th).mean(-1, keepdim=True))).flatten(1)
    if c["gate"]:
        z = s["z"].float()
        got["dz"] = (dtt * x * sig * (1 + z * (1 - sig))).to(dt)
        dtt = dtt * (z * sig)
    got["dx"] = dtt.to(dt)
    return got


PLAIN = {"prologue": _prologue, "prologue_grad": _prologue_grad, "scan": _scan, "scan_grad": _scan_grad, "decode": _decode,
         "norm": _norm_run, "norm_grad": _norm_grad}


# ---------------------------------------------------------------------------------------------------------------------
# the framework's calls

def _own(s):
    import gated_deltanet_mixer_gdn2_gb300 as gdn2

    c, op = s["case"], s["case"]["op"]
    if op == "prologue":
        u, step, g = gdn2.ssm_prologue(s["xbc"], s["delta"], s["weight"], s["bias"], s["a"], s["delta_bias"], offsets=s["offsets"])
        return {"u": u, "step": step, "g": g}
    if op == "prologue_grad":
        got = gdn2.ssm_prologue_backward(s["xbc"], s["delta"], s["weight"], s["bias"], s["a"], s["delta_bias"], s["du"],
                                         s["dstep"], s["dg"], offsets=s["offsets"])
        return dict(zip(("dxbc", "ddelta", "dweight", "dbias", "da", "ddelta_bias"), got))
    if op == "scan":
        y, s1 = gdn2.ssm_chunk_fwd(s["x"], s["step"], s["g"], s["bm"], s["cm"], s["skip"], s["s0"], offsets=s["offsets"],
                                   output_final_state=c["state"])
        return {"y": y, **({"state": s1} if c["state"] else {})}
    if op == "scan_grad":
        got = gdn2.ssm_backward(s["x"], s["step"], s["g"], s["bm"], s["cm"], s["dy"], s["skip"], s["s0"], s["ds1"],
                                offsets=s["offsets"])
        return {k: v for k, v in zip(("dx", "dstep", "dg", "dbm", "dcm", "dskip", "ds0"), got) if v is not None}
    if op == "decode":
        y = gdn2.ssm_decode_step(s["xbc"], s["delta"], s["weight"], s["bias"], s["a"], s["delta_bias"], s["skip"],
                                 s["conv_state"], s["state"], s["slots"])
        return {"y": y, "state": s["state"], "conv_state": s["conv_state"]}
    if op == "norm":
        r, n = gdn2.block_norm(s["x"], s["z"], s["post"], s["residual"], s["scale"], s["pre"], groups=c["groups"], eps=EPS)
        return {**({"r": r} if r is not None else {}), **({"n": n} if n is not None else {})}
    got = gdn2.block_norm_backward(s["x"], s["z"], s["post"], s["residual"], s["scale"], s["pre"], s["d_r"], s["d_n"],
                                   groups=c["groups"], eps=EPS)
    return {k: v for k, v in zip(("dx", "dz", "dpost", "dresidual", "dscale", "dpre"), got) if v is not None}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c, e = case, SIZE[case["dtype"]]
    if c["op"].startswith("norm"):
        n = c["rows"] * c["d"]
        reads = 1 + c["gate"] + c["residual"]
        if c["op"] == "norm":
            writes = (c["residual"] or not c["pre"]) + c["pre"]
            return {"bytes": n * e * (reads + writes), "flops": n * 12}
        ups = (c["residual"] or not c["pre"]) + c["pre"]
        return {"bytes": n * e * (reads + ups + 1 + c["gate"] + c["residual"]), "flops": n * 30}
    H, G, P, N, ch = c["H"], c["G"], c["P"], c["N"], _channels(c)
    if c["op"] == "decode":
        B, se = int(c["lens"]), SIZE[c["state_dtype"]]
        return {"bytes": B * (H * N * P * se * 2 + ch * 3 * 4 * 2 + (ch + H + H * P) * e) + ch * 20,
                "flops": B * (H * N * P * 5 + ch * 12)}
    toks, n = sum(_lens(c)), len(_lens(c))
    if c["op"] == "prologue":
        return {"bytes": toks * e * (2 * ch + 3 * H) + ch * 20, "flops": toks * (ch * 14 + H * 10)}
    if c["op"] == "prologue_grad":
        return {"bytes": toks * e * (3 * ch + 4 * H) + ch * 40, "flops": toks * (ch * 36 + H * 20)}
    states = n * H * N * P * 4 * 2 if c["state"] else 0
    if c["op"] == "scan":
        return {"bytes": toks * e * (2 * H * P + 2 * H + 2 * G * N) + states, "flops": toks * H * N * P * 4}
    return {"bytes": toks * e * (3 * H * P + 4 * H + 4 * G * N) + 2 * states, "flops": toks * H * N * P * 12}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_norm(s):
    """Norms through float64 autograd of the forward definition."""
    c, f = s["case"], lambda t: t.double().requires_grad_() if t is not None else None
    v = {k: f(s[k]) for k in ("x", "z", "post", "residual", "scale", "pre")}
    with torch.enable_grad():
        t = v["x"] / (1 + torch.exp(-v["z"])) * v["z"] if c["gate"] else v["x"]
        if c["post"]:
            w = c["d"] // c["groups"]
            ms = (t ** 2).reshape(-1, w).sum(1) / w
            t = (t.reshape(-1, w) / torch.sqrt(ms + EPS)[:, None]).reshape(t.shape) * v["post"][None]
        if c["scale"]:
            t = t * v["scale"][None]
        if c["residual"]:
            t = t + v["residual"]
        n = t / torch.sqrt((t ** 2).sum(1, keepdim=True) / c["d"] + EPS) * v["pre"][None] if c["pre"] else None
        if c["op"] == "norm":
            return {**({"r": t.detach()} if c["residual"] or not c["pre"] else {}), **({"n": n.detach()} if c["pre"] else {})}
        loss = (t * s["d_r"].double()).sum() if s["d_r"] is not None else 0
        loss = loss + (n * s["d_n"].double()).sum() if c["pre"] else loss
        names = [k for k in v if v[k] is not None]
        return {"d" + k: g for k, g in zip(names, torch.autograd.grad(loss, [v[k] for k in names]))}


def _sequences(s):
    c = s["case"]
    lens = _lens(c)
    starts = np.concatenate([[0], np.cumsum(lens)])
    return [(int(starts[i]), int(starts[i + 1])) for i in range(len(lens))]


def _exact_prologue(s):
    """One sequence after the other, the convolution as a sum over shifted copies."""
    flat = lambda t: t.reshape(-1, t.shape[-1]).double()  # noqa: E731
    x, delta, w, b = flat(s["xbc"]), flat(s["delta"]), s["weight"].double(), s["bias"].double()
    shape = s["xbc"].shape
    v = b[None].repeat(x.shape[0], 1)
    for lo, hi in _sequences(s):
        for back in range(min(4, hi - lo)):
            v[lo + back:hi] += w[:, 3 - back] * x[lo:hi - back]
    z = delta + s["delta_bias"].double()
    step = torch.where(z > 30, z, torch.log1p(torch.exp(z.clamp(max=30))))
    a = s["a"].double()
    back_to = lambda t: t.reshape(*shape[:-1], t.shape[-1])  # noqa: E731
    if s["case"]["op"] == "prologue":
        return {"u": back_to(v / (1 + torch.exp(-v))), "step": back_to(step), "g": back_to(a * step)}
    du, dstep, dg = flat(s["du"]), flat(s["dstep"]), flat(s["dg"])
    e = 1 / (1 + torch.exp(-v))
    dv = du * (e + v * e * (1 - e))
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for lo, hi in _sequences(s):
        for back in range(min(4, hi - lo)):
            dx[lo:hi - back] += w[:, 3 - back] * dv[lo + back:hi]
            dw[:, 3 - back] += (dv[lo + back:hi] * x[lo:hi - back]).sum(0)
    dz = (dstep + a * dg) / (1 + torch.exp(-z))
    return {"dxbc": back_to(dx), "ddelta": back_to(dz), "dweight": dw, "dbias": dv.sum(0), "da": (dg * step).sum(0),
            "ddelta_bias": dz.sum(0)}


def _exact_scan(s):
    """Token by token over all sequences at once (a missing token leaves the state as it is); gradients by walking back
    through states recomputed from one kept every 64 tokens."""
    c = s["case"]
    H, G, P, N = c["H"], c["G"], c["P"], c["N"]
    spans = _sequences(s)
    S, T = len(spans), max(1, max(hi - lo for lo, hi in spans))

    def laid(t):
        t = t.reshape(-1, *t.shape[(1 if c["packed"] else 2):]).double()
        out = t.new_zeros(T, S, *t.shape[1:])
        for i, (lo, hi) in enumerate(spans):
            out[:hi - lo, i] = t[lo:hi]
        return out

    def back(t, like):
        return torch.cat([t[:hi - lo, i] for i, (lo, hi) in enumerate(spans)]).reshape(like.shape)

    x, step, g, bm, cm = (laid(s[k]) for k in ("x", "step", "g", "bm", "cm"))
    alpha, skip, r = torch.exp(g)[..., None, None], s["skip"].double()[:, None], H // G
    xs = (step[..., None] * x).reshape(T, S, G, r, 1, P)
    b6, c6 = bm.reshape(T, S, G, 1, N, 1), cm.reshape(T, S, G, 1, 1, N)
    h = s["s0"].double() if s["s0"] is not None else x.new_zeros(S, H, N, P)

    def forth(h, t):
        return (alpha[t] * h).reshape(S, G, r, N, P).addcmul(b6[t], xs[t]).reshape(S, H, N, P)

    if c["op"] == "scan":
        y = torch.zeros_like(x)
        for t in range(T):
            h = forth(h, t)
            y[t] = (c6[t] @ h.reshape(S, G, r, N, P)).reshape(S, H, P)
        y += skip * x
        return {"y": back(y, s["x"]), **({"state": h} if c["state"] else {})}
    dy = laid(s["dy"])
    kept = []
    for t in range(T):
        if t % 64 == 0:
            kept.append(h)
        h = forth(h, t)
    dx, dstep, dg, dbm, dcm = (torch.zeros_like(t) for t in (x, step, g, bm, cm))
    dh = s["ds1"].double() if s["ds1"] is not None else torch.zeros_like(h)
    for lo in range(64 * (len(kept) - 1), -1, -64):
        hs = [kept[lo // 64]]
        for t in range(lo, min(lo + 64, T)):
            hs.append(forth(hs[-1], t))
        for t in range(min(lo + 64, T) - 1, lo - 1, -1):
            before, now = hs[t - lo], hs[t - lo + 1]
            dh = dh + (cm[t].reshape(S, G, 1, N, 1) * dy[t].reshape(S, G, r, 1, P)).reshape(S, H, N, P)
            dcm[t] = (now @ dy[t][..., None])[..., 0].reshape(S, G, r, N).sum(2)
            q = (bm[t].reshape(S, G, 1, 1, N) @ dh.reshape(S, G, r, N, P)).reshape(S, H, P)
            dbm[t] = (step[t][..., None] * (dh @ x[t][..., None])[..., 0]).reshape(S, G, r, N).sum(2)
            dx[t] = step[t][..., None] * q + skip * dy[t]
            dstep[t] = (x[t] * q).sum(-1)
            dh_a = alpha[t] * dh
            dg[t] = (dh_a * before).sum((-1, -2))
            dh = dh_a
    got = {"dx": back(dx, s["x"]), "dstep": back(dstep, s["step"]), "dg": back(dg, s["g"]), "dbm": back(dbm, s["bm"]),
           "dcm": back(dcm, s["cm"]), "dskip": (x * dy).sum((0, 1, 3))}
    return {**got, **({"ds0": dh} if s["s0"] is not None else {})}


def _exact_decode(s):
    """Row by row of the pools."""
    c = s["case"]
    H, G, P, N = c["H"], c["G"], c["P"], c["N"]
    conv, state = s["conv_state"].double(), s["state"].double()
    at = s["slots"].long()
    hist = torch.cat([conv[at], s["xbc"].double()[:, None]], 1)                    # [B, 4, ch]
    v = torch.einsum("bjc,cj->bc", hist, s["weight"].double()) + s["bias"].double()
    u = v / (1 + torch.exp(-v))
    x, bm, cm = u[:, :H * P].reshape(-1, H, P), u[:, H * P:H * P + G * N].reshape(-1, G, N), u[:, H * P + G * N:].reshape(-1, G, N)
    z = s["delta"].double() + s["delta_bias"].double()
    step = torch.log1p(torch.exp(-z.abs())) + z.clamp(min=0)
    of = torch.arange(H, device=x.device) // (H // G)
    h = torch.exp(s["a"].double() * step)[..., None, None] * state[at] + torch.einsum("bhn,bhp,bh->bhnp", bm[:, of], x, step)
    y = torch.einsum("bhn,bhnp->bhp", cm[:, of], h) + s["skip"].double()[:, None] * x
    state[at], conv[at] = h, hist[:, 1:]
    return {"y": y, "state": state, "conv_state": conv}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return (_exact_norm if op.startswith("norm") else _exact_prologue if op.startswith("prologue") else
            _exact_decode if op == "decode" else _exact_scan)(s)
