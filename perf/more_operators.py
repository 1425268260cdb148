"""The operators of a stack's attention layers, as cases to measure.

Three operators, each in the forms a user calls:

  prologue   q, k = rotation(norm(q), norm(k)) per head: training (and its gradients), or serving, where k and v go into the
             pages of a cache in the same pass
  attend     attention of a row's newest tokens over its pages: o = softmax(scale q K^T over the visible tokens) V
  pages      forking rows of a cache (full pages shared and counted, the last one copied), making room for their next token,
             and copying rows of pools

`run` computes them from elementary torch operations in 32 bits, or, where `own` is true, by the framework's calls.
"""
import math

import torch

own = False

EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------------------------------------------------
# cases

def _prologue_case(name, op, lens, Hq, Hkv, d, rot, dtype, packed=False, norm=True, pairs=False, start=0, **more):
    return {"name": name, "op": op, "lens": lens, "Hq": Hq, "Hkv": Hkv, "d": d, "rot": rot, "dtype": dtype, "packed": packed,
            "norm": norm, "pairs": pairs, "start": start, **more}


def _attend_case(name, lens, N, Hq, Hkv, d, page, dtype, window=0):
    return {"name": name, "op": "attend", "lens": lens, "N": N, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "dtype": dtype,
            "window": window}


def listed():
    ragged = ",".join(str(n) for n in [0, 1, 16384] + [(i * i * 1237 + 331 * i) % 16000 for i in range(1, 62)])
    return [
        # a training batch: 32 query and 8 key heads of 128, rotated whole
        _prologue_case("prologue-4x4096-bf16", "prologue", "4096,4096,4096,4096", 32, 8, 128, 128, "bf16"),
        # one sequence decoding: latency; heads of 256 of which a quarter is rotated
        _prologue_case("prologue-decode-1-bf16", "prologue_paged", "1", 16, 2, 256, 64, "bf16", page=64, past="4095"),
        # a serving step that takes in prompts of several rows, some of them behind what the cache holds already
        _prologue_case("prologue-prompts-bf16", "prologue_paged", "1900,1,0,4096,333,27,129,2048", 32, 8, 128, 128, "bf16",
                       packed=True, page=32, past="0,700,64,0,5,8191,0,77"),
        # a training batch's gradients
        _prologue_case("prologue-grad-4x2048-bf16", "prologue_grad", "2048,2048,2048,2048", 16, 2, 128, 128, "bf16"),
        # gradients in full precision: packed documents, far positions, neighbouring elements rotated
        _prologue_case("prologue-grad-packed-f32", "prologue_grad", "1000,1,0,63,300", 6, 3, 96, 48, "f32", packed=True,
                       pairs=True, start=900000),
        # one short sequence decoding: latency
        _attend_case("attend-77-bf16", "77", 1, 16, 4, 64, 16, "bf16"),
        # one long sequence: the cache's bytes, split over its length
        _attend_case("attend-131072-bf16", "131072", 1, 32, 8, 128, 64, "bf16"),
        # a decoding batch of uneven lengths, an empty row and a row of one token among them; two key heads of 256
        _attend_case("attend-64-ragged-bf16", ragged, 1, 16, 2, 256, 64, "bf16"),
        # drafted tokens checked four at a time
        _attend_case("attend-draft-16x4-bf16", ",".join(str(8192 - 37 * i) for i in range(16)), 4, 32, 4, 128, 32, "bf16"),
        # full precision, a window, pages of no power of two
        _attend_case("attend-window-f32", "1,0,700,63,4097", 1, 6, 2, 96, 24, "f32", window=512),
        # a step of a beam search: eight rows continue from others, with their pages and recurrent states
        {"name": "fork-8-of-16", "op": "fork", "lens": ",".join(str(500 + 211 * i) for i in range(16)), "forks": 8, "page": 32,
         "spare": 200, "layers": 2, "Hkv": 4, "d": 128, "dtype": "bf16", "state": 64},
        # recurrent states of a batch handed to other rows of their pools
        {"name": "copy-states-64", "op": "copy", "rows": 160, "n": 64, "width": 32 * 128 * 128, "layers": 2, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, total):
    """`total` tokens in 1 to 12 sequences of uneven lengths, empty ones among them."""
    n = rng.randint(1, 12)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def draw(rng):
    op = rng.choice(("prologue", "prologue_paged", "prologue_grad", "prologue_grad", "attend", "attend", "attend", "attend", "fork", "copy"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    text = lambda v: ",".join(map(str, v))  # noqa: E731
    Hkv, G, d = rng.choice((1, 2, 3, 4, 8)), rng.choice((1, 2, 3, 4, 7, 8, 16)), rng.choice((64, 80, 96, 128, 128, 256))
    Hq = Hkv * G
    if op.startswith("prologue"):
        rot = rng.choice([r for r in (16, 32, 48, 64, 80, 96, 128, 256) if r <= d])
        total = _log(rng, 1, min(16384, max(64, (1 << 25) // ((Hq + Hkv) * d))))
        packed = rng.random() < 0.5
        lens = _split(rng, total) if packed else [max(1, total // rng.choice((1, 1, 2, 3)))] * rng.choice((1, 2, 3))
        c = _prologue_case("", op, text(lens), Hq, Hkv, d, rot, dtype, packed=packed, norm=rng.random() < 0.8,
                           pairs=rng.random() < 0.3, start=rng.choice((0, 0, _log(rng, 1, 1 << 20))))
        if op == "prologue_paged":
            c.update(page=rng.choice((8, 16, 24, 32, 64, 128)), past=text(rng.choice((0, _log(rng, 1, 5000))) for _ in lens), start=0)
    elif op == "attend":
        B, N = _log(rng, 1, 128), rng.choice((1, 1, 1, 2, 4))
        most = max(16, min(65536, 60_000_000 // (B * Hkv * d * max(1, N * G // 32))))
        lens = [rng.choice((0, N, _log(rng, 1, most), _log(rng, 1, most), most)) for _ in range(B)]
        c = _attend_case("", text(lens), N, Hq, Hkv, d, rng.choice((8, 16, 24, 32, 64, 128)), dtype, rng.choice((0, 0, 0, _log(rng, 1, 4096))))
    elif op == "fork":
        n = _log(rng, 1, 64)
        c = {"op": op, "lens": text(_log(rng, 1, 3000) for _ in range(n + rng.randint(1, 32))), "forks": n, "page": rng.choice((8, 16, 24, 32, 64)),
             "spare": rng.choice((0, 2, 100, 2000)), "layers": rng.choice((1, 2)), "Hkv": min(Hkv, 4), "d": min(d, 128), "dtype": dtype,
             "state": rng.choice((32, 64))}
    else:
        rows, layers = _log(rng, 4, 300), rng.choice((1, 2, 3))
        n = _log(rng, 1, rows // 2)
        c = {"op": op, "rows": rows, "n": n, "width": 8 * _log(rng, 16, min(65536, 8_000_000 // (n * layers))), "layers": layers, "dtype": dtype}
    c.pop("name", None)
    return c


# ---------------------------------------------------------------------------------------------------------------------
# inputs

def _ints(text):
    return [int(v) for v in text.split(",")]


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(gen, held, page, spare, extra):
    """A cache of which row i holds held[i] tokens on pages of no order: table, lengths, references and number of pages."""
    per = [-(-n // page) for n in held]
    pages, wide = sum(per) + spare, max(max(per) + extra, 1)
    order = torch.randperm(max(pages, 1), generator=gen, device="cuda").to(torch.int32)
    per_row = torch.tensor(per, device="cuda")
    at = torch.arange(wide, device="cuda") < per_row[:, None]
    table = torch.full((len(held), wide), -1, dtype=torch.int32, device="cuda")
    table[at] = order[:sum(per)]
    refs = torch.zeros(max(pages, 1), dtype=torch.int32, device="cuda")
    refs[order[:sum(per)].long()] = 1
    return table, _int32(held), refs, max(pages, 1)


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DT[c["dtype"]]
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=dt)  # noqa: E731
    s = {"case": dict(c)}
    if c["op"] == "copy":
        order = torch.randperm(c["rows"], generator=gen, device="cuda").to(torch.int32)
        s.update(pools=[normal(c["rows"], c["width"]) for _ in range(c["layers"])], src=order[:c["n"]].clone(),
                 dst=order[c["rows"] - c["n"]:].clone())
        return s
    Hkv, d, page = c["Hkv"], c["d"], c.get("page")
    if c["op"] == "fork":
        lens = _ints(c["lens"])
        slots = len(lens)
        table, lengths, refs, pages = _table(gen, lens, page, c["spare"], 2)
        order = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32)
        sources = order[c["forks"]:]
        pick = torch.randint(len(sources), (c["forks"],), generator=gen, device="cuda")
        s.update(table=table, lengths=lengths, refs=refs, src=sources[pick], dst=order[:c["forks"]].clone(),
                 pools=[normal(pages, Hkv, page, d) for _ in range(2 * c["layers"])],
                 states=[torch.randn(slots, Hkv, c["state"], c["state"], generator=gen, device="cuda") for _ in range(c["layers"])])
        return s
    Hq = c["Hq"]
    if c["op"] == "attend":
        lens = _ints(c["lens"])
        B = len(lens)
        order = torch.randperm(B + 3, generator=gen, device="cuda")[:B]  # the rows' places in a pool that holds others too
        held = [5] * (B + 3)
        for b, at in enumerate(order.tolist()):
            held[at] = lens[b]
        table, lengths, refs, pages = _table(gen, held, page, 7, 1)
        s.update(q=normal(B, c["N"], Hq, d), k_pages=normal(pages, Hkv, page, d), v_pages=normal(pages, Hkv, page, d), table=table,
                 lengths=lengths, slots=order.to(torch.int32))
        return s
    lens = _ints(c["lens"])
    lead = (sum(lens),) if c["packed"] else (len(lens), lens[0])
    starts = [sum(lens[:i]) for i in range(len(lens) + 1)]
    row = normal(*lead, (Hq + 2 * Hkv) * d)  # the token's projection; the operator reads slices of its rows
    weight = lambda: 1 + 0.1 * torch.randn(d, generator=gen, device="cuda") if c["norm"] else None  # noqa: E731
    s.update(q=row[..., :Hq * d].unflatten(-1, (Hq, d)), k=row[..., Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d)),
             v=row[..., (Hq + Hkv) * d:].unflatten(-1, (Hkv, d)), q_weight=weight(), k_weight=weight(),
             inv_freq=torch.exp(torch.arange(c["rot"] // 2, device="cuda") * (-math.log(1e6) * 2 / c["rot"])),
             offsets=_int32(starts) if c["packed"] else None, positions=None)
    if c["start"]:
        s["positions"] = _int32([c["start"] + t for n in lens for t in range(n)]).reshape(lead)
    if c["op"] == "prologue_grad":
        s.update(dq=normal(*lead, Hq, d), dk=normal(*lead, Hkv, d))
    if c["op"] == "prologue_paged":
        past, B = _ints(c["past"]), len(lens)
        order = torch.randperm(B + 2, generator=gen, device="cuda")[:B]
        held = [3] * (B + 2)
        for b, at in enumerate(order.tolist()):
            held[at] = past[b] + lens[b]
        table, lengths, refs, pages = _table(gen, held, page, 5, 1)
        s.update(k_pages=normal(pages, Hkv, page, d), v_pages=normal(pages, Hkv, page, d), table=table, lengths=lengths,
                 slots=order.to(torch.int32))
    return s


# ---------------------------------------------------------------------------------------------------------------------
# plain forms, in 32 bits

def _row_of(s):
    """Of every token, flat: its sequence and its place in it."""
    lens = _ints(s["case"]["lens"])
    rows = s["q"].shape[0] if s["offsets"] is not None else s["q"].shape[0] * s["q"].shape[1]
    at = torch.arange(rows, device="cuda")
    if s["offsets"] is None:
        return at // lens[0], at % lens[0]
    seq = torch.searchsorted(s["offsets"].long(), at, right=True) - 1
    return seq, at - s["offsets"].long()[seq]


def _angles(s):
    """cos and sin of every token's angles [rows, 1, rot / 2]: formed in 64 bits, since positions reach a million."""
    if s["positions"] is not None:
        pos = s["positions"].reshape(-1)
    else:
        seq, pos = _row_of(s)
        if "lengths" in s:
            n = torch.zeros(s["slots"].shape[0], dtype=torch.long, device="cuda").index_add_(0, seq, torch.ones_like(seq))
            pos = s["lengths"].long()[s["slots"].long()[seq]] - n[seq] + pos
    a = pos.double()[:, None] * s["inv_freq"].double()
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _turn(x, cos, sin, pairs):
    """x [rows, H, d]: its first 2 * cos.shape[-1] elements rotated, by halves or by neighbours."""
    r = 2 * cos.shape[-1]
    if pairs:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., r:]], -1)
    a, b = x[..., :r // 2], x[..., r // 2:r]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1)


def _heads(t):
    return t.reshape(-1, *t.shape[-2:]).float()


def _norm_turn(x, w, cos, sin, pairs):
    x = _heads(x)
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    return _turn(x, cos, sin, pairs)


def _prologue(s):
    c, dt = s["case"], s["q"].dtype
    cos, sin = _angles(s)
    return {n: _norm_turn(s[n], s[n + "_weight"], cos, sin, c["pairs"]).reshape(s[n].shape).to(dt) for n in ("q", "k")}


def _prologue_paged(s):
    c, got = s["case"], _prologue(s)
    seq, at = _row_of(s)
    n = torch.zeros(s["slots"].shape[0], dtype=torch.long, device="cuda").index_add_(0, seq, torch.ones_like(seq))
    slot = s["slots"].long()[seq]
    at = s["lengths"].long()[slot] - n[seq] + at
    page = s["table"].long()[slot, at // c["page"]]
    s["k_pages"][page, :, at % c["page"]] = got["k"].reshape(-1, c["Hkv"], c["d"])
    s["v_pages"][page, :, at % c["page"]] = s["v"].reshape(-1, c["Hkv"], c["d"])
    return {"q": got["q"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _prologue_grad(s):
    c, dt, got = s["case"], s["q"].dtype, {}
    cos, sin = _angles(s)
    for n in ("q", "k"):
        dn, w = _turn(_heads(s["d" + n]), cos, -sin, c["pairs"]), s[n + "_weight"]
        if w is not None:
            x = _heads(s[n])
            inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
            xh = x * inv
            got["d" + n + "_weight"] = (dn * xh).sum((0, 1))
            dn = dn * w
            dn = inv * (dn - xh * (dn * xh).mean(-1, keepdim=True))
        got["d" + n] = dn.reshape(s[n].shape).to(dt)
    return got


def _attend(s):
    c, q = s["case"], s["q"].float()
    B, N, Hq, d = q.shape
    Hkv, page = c["Hkv"], c["page"]
    used = max(1, -(-max(_ints(c["lens"])) // page))
    slot = s["slots"].long()
    table, length = s["table"].long()[slot, :used], s["lengths"].long()[slot]
    there = torch.arange(used * page, device="cuda")
    visible = there <= (length[:, None] - N + torch.arange(N, device="cuda"))[..., None]           # [B, N, T]
    if c["window"]:
        visible = visible & (there > (length[:, None] - N + torch.arange(N, device="cuda") - c["window"])[..., None])
    some = (visible.any(1) & (table >= 0).repeat_interleave(page, 1))[:, None, :, None]
    laid = lambda pool: pool[table.clamp(min=0)].movedim(2, 1).reshape(B, Hkv, used * page, d).float()  # noqa: E731
    k = torch.where(some, laid(s["k_pages"]), 0.0)
    v = torch.where(some, laid(s["v_pages"]), 0.0)
    qg = q.reshape(B, N, Hkv, Hq // Hkv, d).movedim(1, 2).reshape(B, Hkv, -1, d)
    score = (qg @ k.transpose(-1, -2) * d ** -0.5).reshape(B, Hkv, N, Hq // Hkv, -1)
    score = torch.where(visible[:, None, :, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, Hkv, N * (Hq // Hkv), -1) @ v).reshape(B, Hkv, N, Hq // Hkv, d)
    o = o / torch.where(total == 0, 1.0, total)
    return {"o": o.movedim(2, 1).reshape(B, N, Hq, d).to(s["q"].dtype)}


def _release(s, slots):
    held = s["table"][slots]
    there = (held >= 0).flatten()
    s["refs"].scatter_add_(0, held.flatten().clamp(min=0).long(), -there.to(torch.int32))
    s["table"][slots] = -1
    s["lengths"][slots] = 0


def _free(s):
    """The free pages, lowest first (then the others), and how many there are."""
    return torch.sort((s["refs"] > 0).to(torch.int32), stable=True).indices.to(torch.int32), (s["refs"] <= 0).sum()


def _fork(s):
    c, src, dst = s["case"], s["src"].long(), s["dst"].long()
    table, lengths, refs, page = s["table"], s["lengths"], s["refs"], c["page"]
    _release(s, dst)
    # the last page of each source, where it is not full, goes to a free page as long as there are some
    order, free = _free(s)
    part = lengths[src] % page != 0
    number = part.long().cumsum(0)
    ok = ~part | (number <= free)
    fresh = order[(number - 1).clamp(min=0, max=len(order) - 1)]
    full = (lengths[src] // page).long()
    columns = torch.arange(table.shape[1], device="cuda")
    shared = torch.where((columns < full[:, None]) & ok[:, None], table[src], -1)
    refs.scatter_add_(0, shared.flatten().clamp(min=0).long(), (shared >= 0).flatten().to(torch.int32))
    copied = part & ok
    last = table[src].gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    copy_from, copy_to = torch.where(copied, last, -1), torch.where(copied, fresh, -1)
    refs.scatter_add_(0, copy_to.clamp(min=0).long(), copied.to(torch.int32))
    table[dst] = torch.where(copied[:, None] & (columns == full[:, None]), fresh[:, None], shared)
    lengths[dst] = torch.where(ok, lengths[src], 0)
    # pages and states; lists without gaps, or the copied rows would be written twice
    for pool in s["pools"]:
        pool[copy_to[copied].long()] = pool[copy_from[copied].long()]
    for pool in s["states"]:
        pool[dst] = pool[src]
    # room for the next token of the new rows
    order, free = _free(s)
    wanted = lengths[dst] // page
    new = (lengths[dst] % page == 0) & (wanted < table.shape[1])
    number = new.long().cumsum(0)
    more = (~new | (number <= free)) & (wanted < table.shape[1])
    taken = new & more
    fresh = order[(number - 1).clamp(min=0, max=len(order) - 1)]
    refs.scatter_add_(0, fresh.long(), taken.to(torch.int32))
    table[dst] = torch.where(taken[:, None] & (columns == wanted[:, None]), fresh[:, None], table[dst])
    lengths[dst] += more.to(torch.int32)
    return {"table": table, "lengths": lengths, "refs": refs, "from": copy_from, "to": copy_to, "forked": ok.to(torch.int32),
            "appended": more.to(torch.int32), "pools": s["pools"], "states": s["states"]}


def _copy(s):
    for pool in s["pools"]:
        pool[s["dst"].long()] = pool[s["src"].long()]
    return {"pools": s["pools"]}


PLAIN = {"prologue": _prologue, "prologue_paged": _prologue_paged, "prologue_grad": _prologue_grad, "attend": _attend, "fork": _fork,
         "copy": _copy}


# ---------------------------------------------------------------------------------------------------------------------
# the framework's calls

def _own(s):
    import gated_deltanet_mixer_gdn2_gb300 as gdn2

    c, op = s["case"], s["case"]["op"]
    if op == "prologue":
        q, k = gdn2.attn_prologue(s["q"], s["k"], s["q_weight"], s["k_weight"], s["inv_freq"], s["positions"], s["offsets"],
                                  interleaved=c["pairs"], eps=EPS)
        return {"q": q, "k": k}
    if op == "prologue_paged":
        q = gdn2.attn_prologue_paged(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["slots"],
                                     s["q_weight"], s["k_weight"], s["inv_freq"], s["positions"], s["offsets"],
                                     interleaved=c["pairs"], eps=EPS)
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "prologue_grad":
        dq, dk, dqw, dkw = gdn2.attn_prologue_backward(s["q"], s["k"], s["dq"], s["dk"], s["q_weight"], s["k_weight"], s["inv_freq"],
                                                       s["positions"], s["offsets"], interleaved=c["pairs"], eps=EPS)
        return {**({"dq_weight": dqw} if c["norm"] else {}), "dq": dq, **({"dk_weight": dkw} if c["norm"] else {}), "dk": dk}
    if op == "attend":
        return {"o": gdn2.attn_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["slots"], window=c["window"])}
    if op == "copy":
        gdn2.pages_copy(s["pools"], s["src"], s["dst"])
        return {"pools": s["pools"]}
    copy_from, copy_to, forked = gdn2.pages_fork(s["table"], s["lengths"], s["refs"], s["src"], s["dst"], page=c["page"])
    gdn2.pages_copy(s["pools"], copy_from, copy_to)
    gdn2.pages_copy(s["states"], s["src"], s["dst"])
    appended = gdn2.pages_append(s["table"], s["lengths"], s["refs"], s["dst"], 1, page=c["page"])
    return {"table": s["table"], "lengths": s["lengths"], "refs": s["refs"], "from": copy_from, "to": copy_to, "forked": forked,
            "appended": appended, "pools": s["pools"], "states": s["states"]}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c, e, op = case, SIZE[case["dtype"]], case["op"]
    if op == "copy":
        n = c["n"] * c["width"] * c["layers"]
        return {"bytes": 2 * n * e, "flops": n}
    lens = _ints(c["lens"])
    if op == "fork":
        copied = c["forks"] * 2 * c["layers"] * c["Hkv"] * c["page"] * c["d"]
        states = c["forks"] * c["layers"] * c["Hkv"] * c["state"] ** 2
        pages = sum(-(-n // c["page"]) for n in lens)
        return {"bytes": 2 * copied * e + 2 * states * 4 + 8 * pages, "flops": copied + states}
    if op == "attend":
        keys = sum(min(n, c["window"] + c["N"] - 1) if c["window"] else n for n in lens)
        qo = 2 * len(lens) * c["N"] * c["Hq"] * c["d"]
        return {"bytes": 2 * keys * c["Hkv"] * c["d"] * e + qo * e, "flops": max(1, 4 * keys * c["N"] * c["Hq"] * c["d"])}
    n, weights = sum(lens) * c["d"], 4 * c["d"] * (2 + 2 * (op == "prologue_grad")) if c["norm"] else 0
    if op == "prologue_grad":
        return {"bytes": n * (c["Hq"] + c["Hkv"]) * e * (3 if c["norm"] else 2) + weights, "flops": 22 * n * (c["Hq"] + c["Hkv"])}
    heads = c["Hq"] + c["Hkv"] + (c["Hkv"] if op == "prologue_paged" else 0)
    return {"bytes": 2 * n * heads * e + weights, "flops": 9 * n * (c["Hq"] + c["Hkv"])}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _spans(c):
    lens = _ints(c["lens"])
    return [(sum(lens[:i]), sum(lens[:i + 1])) for i in range(len(lens))]


def _exact_turned(s, x, w, first):
    """x [rows, H, d] as complex numbers turned by e^{i position freq}; `first`: the position of each sequence's first token."""
    c = s["case"]
    half, spans = c["rot"] // 2, _spans(c)
    if s["positions"] is not None:
        pos = s["positions"].reshape(-1).double()
    else:
        pos = torch.cat([torch.arange(f, f + hi - lo, device="cuda", dtype=torch.float64) for f, (lo, hi) in zip(first, spans)])
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + EPS) * w
    turn = torch.polar(torch.ones(len(pos), 1, half, dtype=torch.float64, device="cuda"), torch.outer(pos, s["inv_freq"].double())[:, None])
    if c["pairs"]:
        z = torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:-1], half, 2).contiguous()) * turn
        lead = torch.view_as_real(z).reshape(*x.shape[:-1], 2 * half)
    else:
        z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
        lead = torch.cat([z.real, z.imag], -1)
    return torch.cat([lead, x[..., 2 * half:]], -1)


def _exact_prologue(s):
    c, wide = s["case"], lambda t: t.reshape(-1, *t.shape[-2:]).double()  # noqa: E731
    weight = lambda n: s[n + "_weight"].double() if c["norm"] else None  # noqa: E731
    spans = _spans(c)
    if c["op"] == "prologue_grad":
        got = {}
        for n in ("q", "k"):
            x, w = wide(s[n]).requires_grad_(), weight(n)
            if w is not None:
                w.requires_grad_()
            with torch.enable_grad():
                loss = (_exact_turned(s, x, w, [0] * len(spans)) * wide(s["d" + n])).sum()
            grads = torch.autograd.grad(loss, [x] + ([w] if w is not None else []))
            if w is not None:
                got["d" + n + "_weight"] = grads[1]
            got["d" + n] = grads[0].reshape(s[n].shape)
        return got
    slots = s["slots"].tolist() if c["op"] == "prologue_paged" else None
    ends = s["lengths"].tolist() if slots is not None else None
    first = [ends[slots[i]] - (hi - lo) for i, (lo, hi) in enumerate(spans)] if slots is not None else [0] * len(spans)
    q, k = (_exact_turned(s, wide(s[n]), weight(n), first) for n in ("q", "k"))
    if slots is None:
        return {"q": q.reshape(s["q"].shape), "k": k.reshape(s["k"].shape)}
    v, kp, vp = wide(s["v"]), s["k_pages"].double(), s["v_pages"].double()
    page, table = c["page"], s["table"].tolist()
    for i, (lo, hi) in enumerate(spans):
        t = lo
        while t < hi:  # page by page
            at = first[i] + t - lo
            n = min(hi - t, page - at % page)
            where = table[slots[i]][at // page]
            kp[where, :, at % page:at % page + n] = k[t:t + n].movedim(0, 1)
            vp[where, :, at % page:at % page + n] = v[t:t + n].movedim(0, 1)
            t += n
    return {"q": q.reshape(s["q"].shape), "k_pages": kp, "v_pages": vp}


def _exact_attend(s):
    """Row by row, token by token."""
    c = s["case"]
    B, N, Hq, d = s["q"].shape
    G = Hq // c["Hkv"]
    o = torch.zeros(B, N, Hq, d, dtype=torch.float64, device="cuda")
    lens, slots = _ints(c["lens"]), s["slots"].tolist()
    for b in range(B):
        for n in range(N):
            end = lens[b] - N + n + 1
            lo = max(0, end - c["window"]) if c["window"] else 0
            if end <= lo:
                continue
            first, last = lo // c["page"], -(-end // c["page"])
            held = s["table"][slots[b], first:last].long()
            k, v = (pool[held].transpose(1, 2).flatten(0, 1)[lo - first * c["page"]:end - first * c["page"]].double()
                    for pool in (s["k_pages"], s["v_pages"]))                                          # [tokens, Hkv, d]
            q = s["q"][b, n].double().reshape(c["Hkv"], G, d)
            w = torch.softmax(torch.bmm(q, k.permute(1, 2, 0)) / math.sqrt(d), -1)
            o[b, n] = torch.bmm(w, v.transpose(0, 1)).reshape(Hq, d)
    return {"o": o}


def _exact_fork(s):
    """Row by row on the host, as written."""
    c, page = s["case"], s["case"]["page"]
    table, lengths, refs = s["table"].tolist(), s["lengths"].tolist(), s["refs"].tolist()
    wide, src, dst = len(table[0]), s["src"].tolist(), s["dst"].tolist()
    for row in dst:
        for p in table[row]:
            if p >= 0:
                refs[p] -= 1
        table[row], lengths[row] = [-1] * wide, 0
    free = [p for p, n in enumerate(refs) if n <= 0]
    copy_from, copy_to, forked, appended, asked = [], [], [], [], 0
    for a, b in zip(src, dst):
        part, full = lengths[a] % page != 0, lengths[a] // page
        asked += part
        ok = not part or asked <= len(free)
        forked.append(int(ok))
        copy_from.append(table[a][full] if ok and part else -1)
        copy_to.append(free[asked - 1] if ok and part else -1)
        if ok:
            table[b][:full], lengths[b] = table[a][:full], lengths[a]
            for p in table[a][:full]:
                refs[p] += 1
            if part:
                table[b][full] = copy_to[-1]
                refs[copy_to[-1]] += 1
    free, asked = [p for p, n in enumerate(refs) if n <= 0], 0
    for b in dst:
        at = lengths[b] // page
        new = lengths[b] % page == 0 and at < wide
        asked += new
        ok = (not new or asked <= len(free)) and at < wide
        appended.append(int(ok))
        if new and ok:
            table[b][at] = free[asked - 1]
            refs[free[asked - 1]] += 1
        lengths[b] += ok
    pools, states = [p.double() for p in s["pools"]], [p.double() for p in s["states"]]
    for a, b in zip(copy_from, copy_to):
        if b >= 0:
            for p in pools:
                p[b] = p[a]
    for a, b in zip(src, dst):
        for p in states:
            p[b] = p[a]
    return {"table": _int32(table), "lengths": _int32(lengths), "refs": _int32(refs), "from": _int32(copy_from), "to": _int32(copy_to),
            "forked": _int32(forked), "appended": _int32(appended), "pools": pools, "states": states}


def _exact_copy(s):
    pools = [p.double() for p in s["pools"]]
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        for p in pools:
            p[b] = p[a]
    return {"pools": pools}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return (_exact_attend if op == "attend" else _exact_fork if op == "fork" else _exact_copy if op == "copy" else _exact_prologue)(s)
