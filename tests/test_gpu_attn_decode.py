"""Attention of the newest tokens over a paged cache on the GPU, against the fp64 reference (oracle/attn.py; for longer caches the same in
torch fp64).

Tolerances, fixed from the arithmetic before any run. A result is within half a step of its type (2^-8 bf16, 2^-24 fp32, relative) of the fp32
value; that one's error counts against A = sum of p |v|: a score's error of scale sum |q k| d 2^-24 enters its weight once and the sum once; a
weight's exponential is within 2^-21; in bf16 a weight goes into its product as two parts, 2^-17; sums over keys run 2^-24 per key at worst.
Together 2 d 2^-24 S + 2^-15 + keys 2^-24 for bf16 (S: the largest scale sum |q k|), 2 d 2^-24 S + 2^-19 + keys 2^-24 for fp32."""
import numpy as np
import pytest

from oracle import attn
from tests.test_gpu_attn_prologue import HALF, _cache, _dev, _int32, _np, g2  # noqa: F401

pytestmark = pytest.mark.gpu


def _reach(q, k_pages, scale, keys, dtype):
    d = q.shape[-1]
    s = abs(scale) * d * np.abs(q).mean() * np.abs(k_pages[np.isfinite(k_pages)]).mean() * 4  # some four times the mean sum of |q k|
    return 2 * d * 2.0 ** -24 * s + (2.0 ** -15 if dtype == "bf16" else 2.0 ** -19) + keys * 2.0 ** -24


def _check(got, want, mag, reach, dtype):
    live = ~np.isnan(want)
    assert np.isfinite(got[live]).all()
    off = np.abs(got - want) - (HALF[dtype] * np.abs(want) * (1 + 2.0 ** -7) + reach * mag + 1e-30)
    assert (off[live] <= 0).all(), float(off[live].max())


class Case:
    def __init__(self, lens, N, Hq, Hkv, d, page, dtype, seed=0, extra=2):
        rng = np.random.default_rng(seed)
        B, rows = len(lens), len(lens) + extra
        self.slots = rng.permutation(rows)[:B]
        self.lengths = np.full(rows, 3)
        self.lengths[self.slots] = lens
        self.table, self.pools = _cache(rng, self.lengths, page, Hkv, d, dtype)
        self.q = _dev(rng.standard_normal((B, N, Hq, d)), dtype)
        self.scale, self.dtype, self.N, self.page = d ** -0.5, dtype, N, page

    def run(self, g2, **k):  # noqa: F811
        return g2.attn_decode(self.q, *self.pools, _int32(self.table), _int32(self.lengths), _int32(self.slots), scale=self.scale, **k)

    def check(self, got, window=0):
        q, k, v = _np(self.q), _np(self.pools[0]), _np(self.pools[1])
        want, mag = attn.attend(q, k, v, self.table, self.lengths, self.slots, self.scale, window)
        _check(_np(got), want, mag, _reach(q, k, self.scale, int(max(self.lengths.max(), 1)), self.dtype), self.dtype)


CASES = [  # lens, N, Hq, Hkv, d, page, window
    ([1], 1, 1, 1, 16, 16, 0),
    ([0], 1, 2, 1, 64, 16, 0),
    ([77, 0, 1, 16, 17], 1, 8, 2, 64, 16, 0),
    ([200, 3, 65], 1, 6, 3, 80, 24, 0),
    ([130, 500], 1, 16, 1, 128, 32, 0),
    ([513, 64, 2], 1, 8, 2, 256, 64, 0),
    ([300, 4, 2, 0, 63], 4, 4, 2, 64, 8, 0),
    ([257, 129], 4, 16, 2, 128, 48, 0),
    ([90], 3, 20, 1, 96, 7, 0),
    ([700, 10, 33], 1, 4, 2, 128, 16, 64),
    ([700, 10, 1], 3, 12, 2, 64, 24, 5),
    ([400, 90], 2, 32, 2, 256, 128, 100),
    ([64, 65], 2, 2, 2, 128, 1, 1),
    ([100, 30, 500], 40, 4, 2, 64, 16, 0),   # more tokens than a few: some see little or nothing of what the last one sees
    ([100, 300], 33, 6, 2, 128, 24, 20),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES)
def test_decode(g2, case, dtype):  # noqa: F811
    lens, N, Hq, Hkv, d, page, window = case
    c = Case(lens, N, Hq, Hkv, d, page, dtype, seed=len(lens) + d)
    got = c.run(g2, window=window)
    c.check(got, window)
    assert got.equal(c.run(g2, window=window))  # the same bits every time


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,window", [(1, 0), (4, 0), (1, 9), (4, 9), (2, 40)])
@pytest.mark.parametrize("G", [1, 4, 16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_hidden_does_not_count(g2, N, window, G, dtype, bad):  # noqa: F811
    """Keys and values that a token does not see hold what is not finite: the rest of a page, other pages, those before the window, and those
    of later tokens of the same call."""
    import torch

    c = Case([41, 18, 100], N, 2 * G, 2, 64, 16, dtype, seed=G)
    want = c.run(g2, window=window)
    c.check(want, window)
    mine = torch.zeros(c.pools[0].shape[0], 16, dtype=torch.bool, device="cuda")
    for b, s in enumerate(c.slots):
        lo, last = attn.visible(int(c.lengths[s]), N, 0, window)[0], attn.visible(int(c.lengths[s]), N, N - 1, window)[1]
        for t in range(lo, last + 1):
            mine[c.table[s, t // 16], t % 16] = True
    for p in c.pools:
        p.masked_fill_(~mine[:, None, :, None], bad)
    assert c.run(g2, window=window).equal(want)
    if N > 1:  # the newest token's key and value: all but the newest token are as before
        for b, s in enumerate(c.slots):
            t = int(c.lengths[s]) - 1
            for p in c.pools:
                p[c.table[s, t // 16], :, t % 16] = bad
        got = c.run(g2, window=window)
        assert got[:, :-1].equal(want[:, :-1]) and not bool(got[:, -1].isfinite().any())
        if window:  # the first token's oldest key: later tokens do not see it
            c = Case([41, 18, 100], N, 2 * G, 2, 64, 16, dtype, seed=G)
            for s in c.slots:
                t = attn.visible(int(c.lengths[s]), N, 0, window)[0]
                if t > 0:
                    for p in c.pools:
                        p[c.table[s, t // 16], :, t % 16] = bad
            got = c.run(g2, window=window)
            for b, s in enumerate(c.slots):
                if int(c.lengths[s]) - N - window + 1 > 0:
                    assert got[b, 1:].equal(want[b, 1:]) and not bool(got[b, 0].isfinite().any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_and_rows_that_are_not_there(g2, dtype):  # noqa: F811
    import torch

    c = Case([100, 90, 64, 33], 2, 4, 2, 64, 16, dtype)
    a, b, s, _ = c.slots
    c.table[a, 2], c.table[a, 4], c.table[b, :] = -1, 10 ** 6, -3
    c.table[s, :3] = -1  # its tokens' own page is left
    slots = c.slots.copy()
    slots[3] = 99
    o = torch.full_like(c.q, 7.0)
    g2.gdn2_attn_decode(c.q, *c.pools, _int32(c.table), _int32(c.lengths), o, _int32(slots), scale=c.scale)
    assert bool((o[3] == 7).all()) and bool((o[1] == 0).all())
    c.slots = slots
    c.check(o)
    c.lengths[c.slots[:3]] = [-5, 2 ** 31 - 1, -2 ** 31]  # clamped
    o = torch.full_like(c.q, 7.0)
    g2.gdn2_attn_decode(c.q, *c.pools, _int32(c.table), _int32(c.lengths), o, _int32(slots), scale=c.scale)
    assert bool((o[:3] == 0).all()) and bool((o[3] == 7).all())
    # no pages at all
    empty = [p[:0].contiguous() for p in c.pools]
    o = g2.attn_decode(c.q, *empty, _int32(c.table), _int32(c.lengths), _int32(c.slots[:4] * 0))
    assert bool((o == 0).all())


def _attend64(q, k_pages, v_pages, table, lengths, slots, scale):
    """One token a row, on the device in fp64."""
    import torch

    B, _, Hq, d = q.shape
    _, Hkv, page, _ = k_pages.shape
    o, mag = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(lengths[slots[b]])
        if n:
            at = torch.as_tensor(table[slots[b], :-(-n // page)], device="cuda").long()
            k, v = (p[at].transpose(0, 1).flatten(1, 2)[:, :n].double() for p in (k_pages, v_pages))
            w = torch.softmax(q[b, 0].double().reshape(Hkv, -1, d) @ k.transpose(1, 2) * scale, -1)
            o[b, 0], mag[b, 0] = (w @ v).reshape(Hq, d), (w @ v.abs()).reshape(Hq, d)
    return o.cpu().numpy(), mag.cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,Hq,Hkv,d,page", [
    ([50000], 8, 1, 64, 16), ([20011], 4, 4, 128, 40), ([30000, 5, 1000], 16, 2, 256, 64),
    ([(37 * i * i) % 900 if i % 5 else 0 for i in range(300)], 4, 2, 64, 32), ([3] * 700, 2, 1, 128, 4),
    ([0] * 400 + [5] * 30 + [0] * 200 + [4000] + [0] * 300, 4, 2, 64, 16),                       # long runs of empty rows
    ([2000] + [(7 * i) % 23 if i % 3 else 0 for i in range(4999)], 2, 1, 64, 8)])
def test_long_rows_and_many_rows(g2, lens, Hq, Hkv, d, page, dtype):  # noqa: F811
    c = Case(lens, 1, Hq, Hkv, d, page, dtype, seed=len(lens))
    got = c.run(g2)
    want, mag = _attend64(c.q, *c.pools, c.table, c.lengths, c.slots, c.scale)
    _check(_np(got), want, mag, _reach(_np(c.q), _np(c.pools[0][:50]), c.scale, max(lens), dtype), dtype)


def test_sharp_and_flat_scores(g2):  # noqa: F811
    """Scores a hundred apart: one key takes all; all equal: the mean."""
    import torch

    c = Case([300, 300], 1, 4, 2, 64, 16, "bf16")
    c.scale = 60.0
    got = c.run(g2)
    assert bool(got.isfinite().all())
    want, _ = attn.attend(_np(c.q), _np(c.pools[0]), _np(c.pools[1]), c.table, c.lengths, c.slots, c.scale)
    # a score of 60 * 64 * |q k| is known to 64 * 2^-24 of the sum of its terms (some 60 * 64 * 0.64 * 2): 0.02 of a weight's logarithm
    assert np.abs(_np(got) - want).max() <= 0.05 * np.abs(_np(c.pools[1])).max()
    c.pools[0].zero_()
    c.check(c.run(g2))
    c.scale = 0.0
    c.check(c.run(g2))
    assert isinstance(got, torch.Tensor)


def test_single_token_form_and_slices(g2):  # noqa: F811
    """q [B, H, d], out of a wider row; without slots."""
    import torch

    c = Case([70, 5], 1, 4, 2, 64, 16, "bf16", extra=0)
    order = np.argsort(c.slots)
    row = torch.randn(2, 4 * 64 + 128, device="cuda").bfloat16()
    row[:, 64:320] = c.q[order].flatten(1)
    got = g2.attn_decode(row[:, 64:320].unflatten(-1, (4, 64)), *c.pools, _int32(c.table), _int32(c.lengths))
    assert got.shape == (2, 4, 64) and got.equal(c.run(g2)[order][:, 0])


def test_far_pages(g2):  # noqa: F811
    """Pools of more than 2^31 elements: a page behind the 32-bit range is written and read."""
    import torch

    pages, Hkv, page, d = 140_000, 4, 32, 128
    pools = [torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table, lengths = _int32([[pages - 1, 3, pages - 2]]), _int32([80])
    qkv = torch.randn(1, 80, 16, d, device="cuda").bfloat16()
    q = g2.attn_prologue_paged(qkv[:, :, :8], qkv[:, :, 8:12], qkv[:, :, 12:], *pools, table, lengths)
    assert q.equal(qkv[:, :, :8].contiguous())
    for at, p in enumerate((pages - 1, 3, pages - 2)):
        n = min(32, 80 - 32 * at)
        assert pools[0][p, :, :n].equal(qkv[0, 32 * at:32 * at + n, 8:12].transpose(0, 1))
        assert pools[1][p, :, :n].equal(qkv[0, 32 * at:32 * at + n, 12:].transpose(0, 1))
    near = [torch.stack([p[pages - 1], p[3], p[pages - 2]]) for p in pools]
    o = g2.attn_decode(q[:, -1:], *pools, table, lengths)
    assert o.equal(g2.attn_decode(q[:, -1:], *near, _int32([[0, 1, 2]]), lengths))


def test_captured_and_replayed(g2):  # noqa: F811
    """A graph follows lengths, tables and slots that change on the device; two graphs and eager calls beside each other."""
    import torch

    c = Case([900, 20, 300], 1, 8, 2, 128, 16, "bf16")
    c.table = np.concatenate([c.table, np.full((5, 40), -1)], 1)
    table, lengths, slots = _int32(c.table), _int32(c.lengths), _int32(c.slots)
    f = lambda: g2.attn_decode(c.q, *c.pools, table, lengths, slots)  # noqa: E731
    f()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = f()
        graphs.append((graph, got))
    for lens in ([1, 1, 1], [900, 20, 300], [0, 19, 299], [640, 0, 17]):
        c.lengths[c.slots] = lens
        lengths.copy_(_int32(c.lengths))
        want = f()
        streams = [torch.cuda.Stream() for _ in graphs]
        torch.cuda.synchronize()
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(got.equal(want) for _, got in graphs)
        c.check(want)


def test_two_streams_at_once(g2):  # noqa: F811
    import torch

    c = [Case([9000, 40], 1, 8, 2, 128, 16, "bf16", seed=i) for i in range(2)]
    args = [(x.q, *x.pools, _int32(x.table), _int32(x.lengths), _int32(x.slots)) for x in c]
    want = [g2.attn_decode(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in c]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [g2.attn_decode(*a, stream=s) for a, s in zip(args, streams)]
    torch.cuda.synchronize()
    assert all(x.equal(y) for x, y in zip(got, want))


def _dense64(q, k_pages, v_pages, table, lengths, slots, scale, window):
    """Any shape, on the device in fp64: rows of inactive slots NaN; and the sums of p |v|."""
    import torch

    B, N, Hq, d = q.shape
    pages, Hkv, page, _ = k_pages.shape
    wide = table.shape[1]
    o = torch.full(q.shape, float("nan"), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(o)
    for b in range(B):
        s = int(slots[b])
        if not 0 <= s < len(table):
            continue
        entries = torch.as_tensor(table[s].astype(np.int64), device="cuda")
        there = ((entries >= 0) & (entries < pages)).repeat_interleave(page)
        k, v = (p[entries.clamp(0, pages - 1)].transpose(0, 1).flatten(1, 2).double() for p in (k_pages, v_pages))
        length = min(max(int(lengths[s]), 0), wide * page)
        key = torch.arange(wide * page, device="cuda")
        last = length - N + torch.arange(N, device="cuda")[:, None]
        see = there & (key <= last) & ((key > last - window) if window else True)                     # [N, keys]
        z = (q[b].double().reshape(N, Hkv, -1, d).transpose(0, 1) @ k[:, None].transpose(-1, -2)) * scale  # [Hkv, N, G, keys]
        w = torch.softmax(z.masked_fill(~see[None, :, None], -float("inf")), -1).nan_to_num(0.0)
        o[b], mag[b] = ((w @ x[:, None]).transpose(0, 1).reshape(N, Hq, d) for x in (v, v.abs()))
    return o.cpu().numpy(), mag.cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seed", range(30))
def test_any_shape(g2, seed, dtype):  # noqa: F811
    """Sizes, holes, shared pages, inactive rows, lengths past the table and windows by chance; rows of inactive slots stay."""
    import torch

    rng = np.random.default_rng(100 + seed)
    B, rows, Hkv, G, N = rng.integers(1, 40), 45, rng.integers(1, 5), int(rng.choice([1, 2, 3, 5, 8, 16, 20])), int(rng.choice([1, 1, 2, 3, 6]))
    d, page = 16 * int(rng.integers(1, 17)), int(rng.choice([1, 3, 8, 16, 24, 32, 48, 64]))
    wide = max(1, int(rng.choice([100, 400, 1500, 3000]) // page))
    pages = wide + 5
    table = rng.integers(0, pages, (rows, wide))  # pages that rows share
    table[rng.random(table.shape) < 0.1] = rng.choice([-1, pages, 2 ** 30])
    top = wide * page
    lengths = np.where(rng.random(rows) < 0.3, rng.choice([-1, 0, 1, N, top, top + 1, 2 ** 31 - 1], rows), rng.integers(0, top + 1, rows))
    slots = rng.permutation(rows + 6)[:B] - 3
    window = int(rng.choice([0, 0, 1, 7, 100, 10 ** 6, 2 ** 31 - 1]))
    pools = [_dev(rng.standard_normal((pages, Hkv, page, d)), dtype) for _ in range(2)]
    q, scale = _dev(rng.standard_normal((B, N, Hkv * G, d)), dtype), float(rng.choice([d ** -0.5, -0.05, 1.0 / d]))
    o = torch.full_like(q, 7.0)
    g2.gdn2_attn_decode(q, *pools, _int32(table), _int32(lengths), o, _int32(slots), scale=scale, window=window)
    want, mag = _dense64(q, *pools, table, lengths, slots, scale, window)
    dead = np.isnan(want[:, 0, 0, 0])
    assert bool((o[torch.as_tensor(dead, device="cuda")] == 7).all())
    _check(_np(o), want, mag, _reach(_np(q), _np(pools[0]), scale, top, dtype), dtype)
