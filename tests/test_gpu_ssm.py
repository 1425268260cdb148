"""The selective state-space mixer on the GPU against its fp64 reference (oracle/ssm.py), both kernel families
through the public calls.

Tolerances, fixed from the arithmetic before any run: a result stored in bf16 carries one rounding of 2^-9,
and on the tensor-core path operands of two products (pair matrix, states) one more each; 1e-2 = five
such roundings of the largest value. fp32 results sum up to a few thousand terms, each with a handful of
2^-24 roundings and an exponential of an argument of up to ~16: 1e-5 = 170 roundings of 2^-24. fp32 results of
the tensor-core path (states) are formed from operands split so that nothing above 2^-24 is dropped: same bound.
"""
import numpy as np
import pytest

import synth
from oracle import max_rel_err, ssm

pytestmark = pytest.mark.gpu

TOL = {"bf16": 1e-2, "f32": 1e-5}


@pytest.fixture(scope="module")
def g2():
    import gated_deltanet_mixer_gdn2_gb300 as mod

    return mod


def _dev(a, dtype):
    return synth.to_torch(np.ascontiguousarray(a, dtype=np.float32), dtype, "cuda")


def _f32(a):
    import torch

    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _r32(a):
    return np.asarray(a, dtype=np.float32).astype(np.float64)


def _close(name, got, want, tol):
    got = _np(got).reshape(want.shape)
    assert np.isfinite(got).all(), name
    if want.size:
        e = max_rel_err(got, want)
        assert e <= tol, (name, e)


def _offsets(lens):
    import torch

    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


class Scan:
    """Inputs of one scan as stored values in fp64 and as device tensors: x, B and C as slices of one row."""

    def __init__(self, dtype, lens, packed, H, G, P, N, seed, states=True, decay=1.0, d=True):
        rng = np.random.default_rng(seed)
        rd = lambda *s: synth.round_to(rng.standard_normal(s), dtype).astype(np.float64)
        self.dtype, self.packed, self.H, self.G, self.P, self.N = dtype, packed, H, G, P, N
        rows = sum(lens)
        self.lens, self.rows, self.B = lens, rows, len(lens)
        off = np.concatenate([[0], np.cumsum(lens)])
        self.seqs = ssm.spans(len(lens), lens[0] if lens else 0, off if packed else None)
        self.row = rd(rows, H * P + 2 * G * N)
        self.x, self.bm, self.cm = self.split(self.row)
        self.step = synth.round_to(rng.uniform(0.01, 0.5, (rows, H)), dtype).astype(np.float64)
        rate = np.exp(rng.uniform(-6, 1, H))
        self.g = synth.round_to(-decay * rate * rng.uniform(0.2, 1, (rows, H)), dtype).astype(np.float64)
        self.d = _r32(1 + 0.1 * rng.standard_normal(H)) if d else None
        self.s0 = _r32(0.3 * rng.standard_normal((self.B, H, N, P))) if states else None
        self.dy = rd(rows, H, P)
        self.ds1 = _r32(0.3 * rng.standard_normal((self.B, H, N, P))) if states else None

    def split(self, row):
        a, b = self.H * self.P, self.H * self.P + self.G * self.N
        return (row[:, :a].reshape(-1, self.H, self.P), row[:, a:b].reshape(-1, self.G, self.N),
                row[:, b:].reshape(-1, self.G, self.N))

    def lead(self, a):
        return a if self.packed else a.reshape(self.B, self.lens[0], *a.shape[1:])

    def device(self):
        row = _dev(self.lead(self.row), self.dtype)
        a, b = self.H * self.P, self.H * self.P + self.G * self.N
        x, bm, cm = (row[..., :a].unflatten(-1, (self.H, self.P)), row[..., a:b].unflatten(-1, (self.G, self.N)),
                     row[..., b:].unflatten(-1, (self.G, self.N)))
        return (x, _dev(self.lead(self.step), self.dtype), _dev(self.lead(self.g), self.dtype), bm, cm)

    def offsets(self):
        return _offsets(self.lens) if self.packed else None

    def ref(self):
        return ssm.scan(self.x, self.step, self.g, self.bm, self.cm, self.d, self.s0, self.seqs)

    def ref_grad(self):
        return ssm.scan_grad(self.x, self.step, self.g, self.bm, self.cm, self.d, self.s0, self.seqs, self.dy, self.ds1)

    def run(self, g2, **kw):
        x, step, g, bm, cm = self.device()
        return g2.ssm_chunk_fwd(x, step, g, bm, cm, _f32(self.d), _f32(self.s0), self.offsets(), **kw)

    def run_grad(self, g2, **kw):
        x, step, g, bm, cm = self.device()
        return g2.ssm_backward(x, step, g, bm, cm, _dev(self.lead(self.dy), self.dtype), _f32(self.d), _f32(self.s0),
                               _f32(self.ds1), self.offsets(), **kw)


# (lens, packed, H, G, P, N): single tokens, one token past every tile and chunk length, lengths that are no
# multiple of anything, groups of one and of several heads, every state size, values of 8 to 200 channels
SHAPES = [
    ([1], False, 1, 1, 64, 128),
    ([33, 33], False, 2, 1, 64, 64),
    ([130], False, 4, 2, 64, 128),
    ([257], False, 3, 3, 128, 128),
    ([64, 64], False, 2, 2, 16, 16),
    ([100], False, 2, 1, 8, 32),
    ([70], False, 2, 1, 200, 256),
    ([0, 5, 128, 129, 1, 0, 200, 0], True, 4, 2, 64, 128),
    ([127], True, 6, 1, 64, 64),
    ([3, 1, 1], True, 5, 5, 32, 128),
    ([300, 70], True, 2, 1, 128, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
def test_scan(g2, dtype, shape):
    c = Scan(dtype, *shape, seed=11)
    y, s1 = c.run(g2)
    ry, rs = c.ref()
    _close("y", y, c.lead(ry), TOL[dtype])
    _close("state", s1, rs, TOL["f32"])
    assert g2.gdn2_last_device_status() == g2.GDN2_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
def test_scan_gradients(g2, dtype, shape):
    c = Scan(dtype, *shape, seed=12)
    got, want = c.run_grad(g2), c.ref_grad()
    for name, a, b in zip(("dx", "dstep", "dg", "dbm", "dcm"), got, want):
        _close(name, a, c.lead(b), TOL[dtype])
    _close("dd", got[5], want[5], TOL["f32"])
    _close("ds0", got[6], want[6], TOL["f32"])
    assert g2.gdn2_last_device_status() == g2.GDN2_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_without_states_or_skip(g2, dtype):
    c = Scan(dtype, [90, 90], False, 2, 1, 64, 128, seed=13, states=False, d=False)
    y, s1 = c.run(g2, output_final_state=False)
    assert s1 is None
    _close("y", y, c.lead(c.ref()[0]), TOL[dtype])
    got, want = c.run_grad(g2), c.ref_grad()
    for name, a, b in zip(("dx", "dstep", "dg", "dbm", "dcm"), got, want):
        _close(name, a, c.lead(b), TOL[dtype])
    assert got[5] is None and got[6] is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_decay_extremes(g2, dtype):
    """No decay at all, decays that forget a chunk within a token, and full resets (g = -inf)."""
    c = Scan(dtype, [200], False, 4, 2, 64, 128, seed=14)
    c.g[:, 0] = 0.0
    c.g[:, 1] = -60.0
    c.g[50, 2] = c.g[128, 2] = c.g[0, 3] = -np.inf
    y, s1 = c.run(g2)
    ry, rs = c.ref()
    _close("y", y, c.lead(ry), TOL[dtype])
    _close("state", s1, rs, TOL["f32"])
    got, want = c.run_grad(g2), c.ref_grad()
    for name, a, b in zip(("dx", "dstep", "dg", "dbm", "dcm"), got, want):
        _close(name, a, c.lead(b), TOL[dtype])
    _close("ds0", got[6], want[6], TOL["f32"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_cut_into_units(g2, dtype):
    """Few heads and a long sequence: the sequence is cut and its parts joined by their states."""
    c = Scan(dtype, [1500, 37, 0, 700], True, 1, 1, 64, 128, seed=15, decay=0.05)
    y, s1 = c.run(g2)
    ry, rs = c.ref()
    _close("y", y, ry, TOL[dtype])
    _close("state", s1, rs, TOL["f32"])
    got, want = c.run_grad(g2), c.ref_grad()
    for name, a, b in zip(("dx", "dstep", "dg", "dbm", "dcm"), got, want):
        _close(name, a, b, TOL[dtype])
    _close("ds0", got[6], want[6], TOL["f32"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_split_equals_whole(g2, dtype):
    """The final state of the first part as the second part's initial state; it may be updated in place."""
    import torch

    c = Scan(dtype, [300], False, 4, 1, 64, 128, seed=16, states=False)
    x, step, g, bm, cm = c.device()
    d = _f32(c.d)
    y, s1 = g2.ssm_chunk_fwd(x, step, g, bm, cm, d)
    st = torch.zeros_like(s1)
    parts = []
    for lo, hi in ((0, 37), (37, 38), (38, 300)):
        ya = torch.empty((1, hi - lo, 4, 64), dtype=x.dtype, device="cuda")
        g2.gdn2_ssm_chunk_fwd(x[:, lo:hi], step[:, lo:hi].contiguous(), g[:, lo:hi].contiguous(), bm[:, lo:hi], cm[:, lo:hi], ya,
                              d, st, st)
        parts.append(ya)
    ry, rs = c.ref()
    _close("y", torch.cat(parts, 1), c.lead(ry), TOL[dtype])
    _close("state", st, rs, TOL["f32"])
    _close("state", s1, rs, TOL["f32"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_sequences_do_not_mix(g2, dtype):
    """Infinities and NaN in one packed sequence, and in rows of no sequence, leave the others bit for bit."""
    import torch

    lens = [100, 60, 140, 3]
    c = Scan(dtype, lens, True, 2, 1, 64, 128, seed=17)
    y, s1 = c.run(g2)
    grads = c.run_grad(g2)
    c.row[100:160] = np.nan
    c.row[110:112] = np.inf
    c.dy[100:160] = np.nan
    yb, sb = c.run(g2)
    gradsb = c.run_grad(g2)
    keep = np.r_[0:100, 160:303]
    assert torch.equal(y[keep], yb[keep])
    assert torch.equal(s1[[0, 2, 3]], sb[[0, 2, 3]])
    for a, b in zip(grads[:5], gradsb[:5]):
        assert torch.equal(a[keep], b[keep])
    assert torch.equal(grads[6][[0, 2, 3]], gradsb[6][[0, 2, 3]])
    # rows past the last offset belong to no sequence: not read into any, not written
    x, step, g, bm, cm = c.device()
    off = _offsets([100])
    out = torch.full((303, 2, 64), 7.0, dtype=x.dtype, device="cuda")
    g2.gdn2_ssm_chunk_fwd(x, step, g, bm, cm, out, _f32(c.d), _f32(c.s0[:1]), None, off)
    assert torch.equal(out[:100], y[:100]) and bool((out[100:] == 7).all())


def test_scan_is_deterministic_and_follows_its_stream(g2):
    import torch

    c = Scan("bf16", [700, 20], True, 4, 1, 64, 128, seed=18)
    ya, sa = c.run(g2)
    ga = c.run_grad(g2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        yb, sb = c.run(g2)
        gb = c.run_grad(g2)
    side.synchronize()
    assert torch.equal(ya, yb) and torch.equal(sa, sb)
    for a, b in zip(ga, gb):
        assert torch.equal(a, b)


def test_scan_empty_calls(g2):
    import torch

    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    s0 = torch.randn(2, 2, 64, 64, device="cuda")
    y, s1 = g2.ssm_chunk_fwd(z(2, 0, 2, 64), z(2, 0, 2), z(2, 0, 2), z(2, 0, 1, 64), z(2, 0, 1, 64), None, s0)
    assert y.numel() == 0 and torch.equal(s1, s0)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    got = g2.ssm_backward(z(0, 2, 64), z(0, 2), z(0, 2), z(0, 1, 64), z(0, 1, 64), z(0, 2, 64), torch.ones(2, device="cuda"), s0,
                          2 * s0, off)
    assert torch.equal(got[6], 2 * s0) and bool((got[5] == 0).all())
    y, s1 = g2.ssm_chunk_fwd(z(0, 4, 2, 64), z(0, 4, 2), z(0, 4, 2), z(0, 4, 1, 64), z(0, 4, 1, 64))
    assert y.shape == (0, 4, 2, 64) and s1.shape[0] == 0


def test_scan_gradient_against_differences(g2):
    """<GPU gradient, v> against a central difference of the fp64 forward along v, for every input. fp32 inputs: the
    gradient's own error is 1e-5 of its size, which the random direction averages; 1e-4 of the sum's scale."""
    c = Scan("f32", [40, 25], True, 2, 1, 32, 32, seed=19)
    got = c.run_grad(g2)
    rng = np.random.default_rng(20)
    names = ("x", "step", "g", "bm", "cm", "d", "s0")
    args = [getattr(c, n) for n in names]

    def f(a):
        y, s1 = ssm.scan(*a, c.seqs)
        return (y * c.dy).sum() + (s1 * c.ds1).sum()

    for i, n in enumerate(names):
        v = rng.standard_normal(args[i].shape)
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - 1e-5 * v, args[i] + 1e-5 * v
        want = (f(hi) - f(lo)) / 2e-5
        have = _np(got[i]).reshape(v.shape) * v
        assert abs(have.sum() - want) <= 1e-4 * np.sqrt((have ** 2).sum()) + 1e-6 * abs(want), n


def test_scan_past_32_bit_offsets(g2):
    """More than 2^31 values in x and y: the last tokens, whose state forgets within a few hundred tokens (e^-0.5 a
    token: 600 tokens leave e^-300), equal those of a call on the tail alone."""
    import torch

    T, H, P, N, tail = 540000, 64, 64, 64, 1280
    torch.manual_seed(0)
    x = torch.randn(1, T, H, P, device="cuda", dtype=torch.bfloat16)
    bm, cm = (torch.randn(1, T, 1, N, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    step = torch.rand(1, T, H, device="cuda").to(torch.bfloat16)
    g = torch.full_like(step, -0.5)
    assert x.numel() > 2 ** 31
    y, s1 = g2.ssm_chunk_fwd(x, step, g, bm, cm)
    cut = [t[:, -tail:].contiguous() for t in (x, step, g, bm, cm)]
    yt, st = g2.ssm_chunk_fwd(*cut)
    d = (y[:, -256:].float() - yt[:, -256:].float()).abs().max() / yt.float().abs().max()
    assert float(d) <= 1e-2
    assert float((s1 - st).abs().max() / st.abs().max()) <= 1e-5
    assert g2.gdn2_last_device_status() == g2.GDN2_OK


# ---- prologue -------------------------------------------------------------------------------------------

def _prologue_inputs(dtype, lens, ch, H, seed, pad=0):
    rng = np.random.default_rng(seed)
    rows = sum(lens)
    rd = lambda *s: synth.round_to(rng.standard_normal(s), dtype).astype(np.float64)
    return dict(row=rd(rows, ch + 8 * -(-H // 8) + pad), w=_r32(0.4 * rng.standard_normal((ch, 4))), bias=_r32(rng.standard_normal(ch)),
                a=_r32(-rng.uniform(0.5, 4, H)), db=_r32(rng.standard_normal(H)), conv=_r32(rng.standard_normal((len(lens), 3, ch))),
                du=rd(rows, ch), dstep=rd(rows, H), dg=rd(rows, H))


PRO = [([1], False, 8, 1), ([2, 2, 2], False, 264, 3), ([131], False, 2048, 24), ([0, 1, 2, 3, 4, 0, 50, 17], True, 1032, 8),
       ([3, 0, 400, 5], True, 136, 40)]
# columns behind the channels and gates: rows on 16-, 8-, 4- and 2-byte (bf16) boundaries
PADS = [0, 4, 2, 1]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,packed,ch,H", PRO)
@pytest.mark.parametrize("pad", PADS)
@pytest.mark.parametrize("states,silu", [(True, True), (False, False)])
def test_prologue(g2, dtype, lens, packed, ch, H, pad, states, silu):
    """u and the gates; the new convolution states are stored samples, so exact."""
    p = _prologue_inputs(dtype, lens, ch, H, 21, pad)
    lead = (lambda t: t) if packed else (lambda t: t.unflatten(0, (len(lens), lens[0])))
    row = lead(_dev(p["row"], dtype))
    conv = _f32(p["conv"]) if states else None
    off = _offsets(lens) if packed else None
    u, step, g = g2.ssm_prologue(row[..., :ch], row[..., ch:ch + H], _f32(p["w"]), _f32(p["bias"]), _f32(p["a"]), _f32(p["db"]), conv,
                                 off, silu=silu)
    seqs = ssm.spans(len(lens), lens[0], np.concatenate([[0], np.cumsum(lens)]) if packed else None)
    want = ssm.prologue(p["row"][:, :ch], p["row"][:, ch:ch + H], p["w"], p["bias"], p["a"], p["db"], seqs,
                        p["conv"] if states else None, silu)
    for name, a, b in zip(("u", "step", "g"), (u, step, g), want):
        _close(name, a, b, TOL[dtype])
    if states:
        assert np.array_equal(_np(conv), want[3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,packed,ch,H", PRO)
@pytest.mark.parametrize("pad", PADS)
@pytest.mark.parametrize("silu", [True, False])
def test_prologue_gradients(g2, dtype, lens, packed, ch, H, pad, silu):
    p = _prologue_inputs(dtype, lens, ch, H, 22, pad)
    lead = (lambda t: t) if packed else (lambda t: t.unflatten(0, (len(lens), lens[0])))
    row = lead(_dev(p["row"], dtype))
    off = _offsets(lens) if packed else None
    got = g2.ssm_prologue_backward(row[..., :ch], row[..., ch:ch + H], _f32(p["w"]), _f32(p["bias"]), _f32(p["a"]), _f32(p["db"]),
                                   *(lead(_dev(p[k], dtype)) for k in ("du", "dstep", "dg")), off, silu=silu)
    seqs = ssm.spans(len(lens), lens[0], np.concatenate([[0], np.cumsum(lens)]) if packed else None)
    want = ssm.prologue_grad(p["row"][:, :ch], p["row"][:, ch:ch + H], p["w"], p["bias"], p["a"], p["db"], p["du"], p["dstep"],
                             p["dg"], seqs, silu)
    for name, a, b in zip(("dxbc", "ddelta", "dweight", "dbias", "da", "ddelta_bias"), got, want):
        _close(name, a, b, TOL[dtype] if name in ("dxbc", "ddelta") else TOL["f32"])


def test_prologue_runs_are_seamless(g2):
    """Long enough that rows are cut into many runs, at lengths around their edges: every output equals the
    reference's at the seams too (bf16 elementwise: one rounding of 2^-9 and fp32 noise)."""
    lens = [1000, 63, 1, 2, 0, 905, 64]
    p = _prologue_inputs("bf16", lens, 512, 8, 23)
    row, off = _dev(p["row"], "bf16"), _offsets(lens)
    seqs = ssm.spans(0, 0, np.concatenate([[0], np.cumsum(lens)]))
    args = [_f32(p[k]) for k in ("w", "bias", "a", "db")]
    u, _, _ = g2.ssm_prologue(row[:, :512], row[:, 512:520], *args, None, off)
    want, _, _, _ = ssm.prologue(p["row"][:, :512], p["row"][:, 512:520], p["w"], p["bias"], p["a"], p["db"], seqs)
    np.testing.assert_allclose(_np(u), want, rtol=2 ** -8, atol=1e-6)
    got = g2.ssm_prologue_backward(row[:, :512], row[:, 512:520], *args, *(_dev(p[k], "bf16") for k in ("du", "dstep", "dg")), off)
    ref = ssm.prologue_grad(p["row"][:, :512], p["row"][:, 512:520], p["w"], p["bias"], p["a"], p["db"], p["du"], p["dstep"],
                            p["dg"], seqs)
    np.testing.assert_allclose(_np(got[0]), ref[0], rtol=2 ** -8, atol=1e-5)


# ---- decode ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,state_dtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("B,H,G,P,N", [(1, 1, 1, 64, 128), (3, 6, 2, 64, 64), (2, 17, 1, 16, 16), (2, 8, 1, 128, 256), (5, 40, 1, 32, 128)])
def test_decode_step(g2, dtype, state_dtype, B, H, G, P, N):
    """Three tokens against pools of states; inactive rows and unnamed pool rows keep every bit."""
    import torch

    rng = np.random.default_rng(31)
    ch, slots = H * P + 2 * G * N, 2 * B + 1
    rd = lambda *s: synth.round_to(rng.standard_normal(s), dtype).astype(np.float64)
    w, bias, a, db, d = (_r32(v) for v in (0.4 * rng.standard_normal((ch, 4)), rng.standard_normal(ch), -rng.uniform(0.5, 4, H),
                                          rng.standard_normal(H) - 2, rng.standard_normal(H)))
    conv, st = _f32(rng.standard_normal((slots, 3, ch))), _dev(rng.standard_normal((slots, H, N, P)), state_dtype)
    at = rng.permutation(slots)[:B].astype(np.int32)
    if B > 2:
        at[1] = -1 if B == 3 else slots
    active = [i for i in range(B) if 0 <= at[i] < slots]
    dev_at = torch.from_numpy(at).cuda()
    for _ in range(3):
        row = rd(B, ch + H)
        before_c, before_s = _np(conv), _np(st)
        drow = _dev(row, dtype)
        y = torch.full((B, H, P), 5.0, dtype=drow.dtype, device="cuda")
        g2.gdn2_ssm_decode_step(drow[:, :ch], drow[:, ch:], _f32(w), _f32(bias), _f32(a), _f32(db), _f32(d), conv, st, y, dev_at)
        ids = at[active]
        ry, rc, rs = ssm.decode(row[active][:, :ch], row[active][:, ch:], w, bias, a, db, d, before_c[ids], before_s[ids])
        _close("y", y[active], ry, TOL[dtype])
        _close("state", st[torch.from_numpy(ids).long().cuda()], rs, TOL[state_dtype])
        assert np.array_equal(_np(conv)[ids], rc)
        rest = np.setdiff1d(np.arange(slots), ids)
        assert np.array_equal(_np(st)[rest], before_s[rest]) and np.array_equal(_np(conv)[rest], before_c[rest])
        for i in set(range(B)) - set(active):
            assert bool((y[i] == 5).all())


def test_decode_step_without_slots_in_a_graph(g2):
    """The step can be captured; replays advance the states as calls do."""
    import torch

    torch.manual_seed(1)
    B, H, G, P, N = 4, 8, 2, 64, 128
    ch = H * P + 2 * G * N
    f = lambda *s: torch.randn(*s, device="cuda")
    xbc, delta = f(B, ch).bfloat16(), f(B, H).bfloat16()
    w, bias, a, db, d = 0.4 * f(ch, 4), f(ch), -f(H).abs(), f(H), f(H)
    c1, s1 = f(B, 3, ch), f(B, H, N, P)
    c2, s2 = c1.clone(), s1.clone()
    for _ in range(3):
        y1 = g2.ssm_decode_step(xbc, delta, w, bias, a, db, d, c1, s1)
    y2 = torch.empty_like(y1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g2.gdn2_ssm_decode_step(xbc, delta, w, bias, a, db, d, c2, s2, y2)  # warm: one step
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2.gdn2_ssm_decode_step(xbc, delta, w, bias, a, db, d, c2, s2, y2)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y1, y2) and torch.equal(s1, s2) and torch.equal(c1, c2)


def test_mixer_prompt_then_tokens(g2):
    """prologue -> scan -> gated norm over a packed prompt, then tokens by decode steps from its states, against the
    reference over all tokens."""
    import torch

    rng = np.random.default_rng(41)
    lens, new, H, G, P, N = [70, 0, 131], 3, 4, 2, 64, 128
    ch = H * P + 2 * G * N
    rd = lambda *s: synth.round_to(rng.standard_normal(s), "bf16").astype(np.float64)
    w, bias, a, db, d = (_r32(v) for v in (0.4 * rng.standard_normal((ch, 4)), 0.1 * rng.standard_normal(ch), -rng.uniform(0.5, 4, H),
                                          rng.standard_normal(H) - 3, rng.standard_normal(H)))
    dw = [_f32(t) for t in (w, bias, a, db, d)]
    toks = [rd(n + new, ch + H) for n in lens]
    prompt = _dev(np.concatenate([t[:n] for t, n in zip(toks, lens)]), "bf16")
    conv = torch.zeros(3, 3, ch, device="cuda")
    off = _offsets(lens)
    u, step, g = g2.ssm_prologue(prompt[:, :ch], prompt[:, ch:], *dw[:4], conv, off)
    x, bm, cm = u[:, :H * P].unflatten(-1, (H, P)), u[:, H * P:H * P + G * N].unflatten(-1, (G, N)), u[:, H * P + G * N:].unflatten(-1, (G, N))
    y, st = g2.ssm_chunk_fwd(x, step, g, bm, cm, dw[4], None, off)
    z, post = rd(sum(lens), H * P), _r32(1 + 0.1 * rng.standard_normal(H * P))
    out, _ = g2.block_norm(y.flatten(1), _dev(z, "bf16"), _f32(post), groups=G)
    outs = []
    for t in range(new):
        tok = _dev(np.stack([k[n + t] for k, n in zip(toks, lens)]), "bf16")
        outs.append(g2.ssm_decode_step(tok[:, :ch], tok[:, ch:], *dw, conv, st))
    tol = 2e-2  # u, step and g stored in bf16 between the calls add three roundings of 2^-9 to TOL
    at = 0
    for b, (t, n) in enumerate(zip(toks, lens)):
        u, step, g, _ = ssm.prologue(t[:, :ch], t[:, ch:], w, bias, a, db, [(0, n + new)])
        sp = lambda v: (v[:, :H * P].reshape(-1, H, P), v[:, H * P:H * P + G * N].reshape(-1, G, N), v[:, H * P + G * N:].reshape(-1, G, N))
        x, bm, cm = sp(u)
        ry, _ = ssm.scan(x, step, g, bm, cm, d, None, [(0, n + new)])
        for k in range(new):
            _close("token", outs[k][b], ry[n + k], tol)
        if n:
            ro, _ = ssm.block_norm(ry[:n].reshape(n, -1), z[at:at + n], post, None, None, None, groups=G)
            _close("block", out[at:at + n], ro, tol)
        at += n


# ---- block norm -----------------------------------------------------------------------------------------

FLAGS = [(1, 1, 1, 1, 1), (0, 0, 1, 0, 1), (1, 1, 0, 0, 0), (0, 1, 1, 1, 0), (1, 0, 0, 1, 1), (0, 0, 0, 0, 1), (1, 0, 1, 0, 0)]


def _norm_inputs(dtype, rows, d, flags, seed):
    rng = np.random.default_rng(seed)
    rd = lambda: synth.round_to(rng.standard_normal((rows, d)), dtype).astype(np.float64)
    wt = lambda: _r32(1 + 0.2 * rng.standard_normal(d))
    gate, post, residual, scale, pre = flags
    return ([rd(), rd() if gate else None, wt() if post else None, 2 * rd() if residual else None, wt() if scale else None,
             wt() if pre else None], rd(), rd() if pre else None)


def _norm_dev(args, dtype):
    return [None if a is None else _f32(a) if a.ndim == 1 else _dev(a, dtype) for a in args]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d,groups", [(1, 8, 1), (5, 520, 5), (700, 64, 2), (3, 4096, 8), (2, 5000, 1), (3, 8192, 4)])
@pytest.mark.parametrize("flags", FLAGS)
def test_block_norm(g2, dtype, rows, d, groups, flags):
    args, d_r, d_n = _norm_inputs(dtype, rows, d, flags, 51)
    groups = groups if flags[1] else 1
    dev = _norm_dev(args, dtype)
    r, n = g2.block_norm(*dev, groups=groups)
    rr, rn = ssm.block_norm(*args, groups=groups)
    if r is not None:
        _close("r", r, rr, TOL[dtype])
    assert (n is None) == (rn is None)
    if n is not None:
        _close("n", n, rn, TOL[dtype])
    if r is None:
        d_r = None
    got = g2.block_norm_backward(*dev, None if d_r is None else _dev(d_r, dtype), None if d_n is None else _dev(d_n, dtype), groups=groups)
    want = ssm.block_norm_grad(*args, d_r, d_n, groups=groups)
    for name, a, b, given in zip(("dx", "dz", "dpost", "dresidual", "dscale", "dpre"), got, want, args):
        assert (a is None) == (given is None), name
        if a is not None:
            _close(name, a, b, TOL["f32"] if given.ndim == 1 else TOL[dtype])


def test_block_norm_rows_of_zeros_and_aliases(g2):
    """A row of zeros has a finite norm (eps), and r and n may replace their inputs."""
    import torch

    args, _, _ = _norm_inputs("bf16", 6, 256, (0, 1, 1, 0, 1), 52)
    args[0][2] = 0
    args[3][2] = 0
    x, _, post, res, _, pre = _norm_dev(args, "bf16")
    r, n = g2.block_norm(x, None, post, res, None, pre)
    assert bool((n[2] == 0).all())
    g2.gdn2_block_norm(x, None, post, res, None, pre, res, x)
    assert torch.equal(res, r) and torch.equal(x, n)


def test_block_norm_past_32_bit_offsets(g2):
    import torch

    rows, d = 540000, 4096
    torch.manual_seed(0)
    x = torch.randn(rows, d, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(d, device="cuda")
    _, n = g2.block_norm(x, pre_weight=w)
    _, tail = g2.block_norm(x[-100:].contiguous(), pre_weight=w)
    assert torch.equal(n[-100:], tail)


# ---- refusals -------------------------------------------------------------------------------------------

def test_refusals(g2):
    """Wrong types, shapes and layouts are refused before anything is enqueued."""
    import torch

    c = Scan("bf16", [16], False, 2, 1, 64, 64, seed=61)
    x, step, g, bm, cm = c.device()
    ok = lambda **k: g2.ssm_chunk_fwd(*{**dict(x=x, step=step, g=g, bm=bm, cm=cm), **k}.values())
    ok()
    with pytest.raises(TypeError):
        ok(step=step.float())
    with pytest.raises(TypeError):
        g2.ssm_chunk_fwd(x.half(), step.half(), g.half(), bm.half(), cm.half())
    with pytest.raises(ValueError):
        ok(step=step[:, :8])
    with pytest.raises(ValueError):
        ok(x=x.transpose(-1, -2))
    with pytest.raises(ValueError):
        ok(step=step.expand(2, 16, 2)[:1].transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        ok(x=x.cpu())
    with pytest.raises(TypeError):
        g2.ssm_chunk_fwd(x[0], step[0], g[0], bm[0], cm[0], offsets=torch.tensor([0, 16], device="cuda"))
    with pytest.raises(ValueError):
        g2.ssm_chunk_fwd(x, step, g, bm, cm, initial_state=torch.zeros(1, 2, 64, 32, device="cuda"))
    with pytest.raises(TypeError):
        g2.ssm_chunk_fwd(x, step, g, bm, cm, initial_state=torch.zeros(1, 2, 64, 64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(g2.Gdn2Error) as e:  # a state size that is not built
        ok(bm=bm[..., :24].contiguous(), cm=cm[..., :24].contiguous())
    assert e.value.status == g2.GDN2_ERR_UNSUPPORTED
    wide = torch.zeros(1, 16, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(g2.Gdn2Error) as e:  # rows 264 bytes apart
        ok(x=wide[..., :128].unflatten(-1, (2, 64)))
    assert e.value.status == g2.GDN2_ERR_MISALIGNED
    with pytest.raises(g2.Gdn2Error) as e:
        g2.gdn2_block_norm(torch.zeros(2, 12, device="cuda"), None, None, None, None, None, torch.zeros(2, 12, device="cuda"), None)
    assert e.value.status == g2.GDN2_ERR_UNSUPPORTED
    with pytest.raises(g2.Gdn2Error) as e:  # groups without a norm after the block
        g2.block_norm(torch.zeros(2, 16, device="cuda"), groups=2)
    assert e.value.status == g2.GDN2_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        g2.ssm_decode_step(torch.zeros(2, 100, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 2, dtype=torch.bfloat16, device="cuda"),
                           None, None, None, None, None, None, torch.zeros(2, 2, 64, 64, device="cuda"))
