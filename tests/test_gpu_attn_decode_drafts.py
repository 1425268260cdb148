"""Several tokens a row (drafts) whose query rows fill more than one tile: the form of bf16 caches wider than 64 that keeps its products in tensor
memory, and the joining of its parts. Reference and tolerances are those of the other decode tests."""
import numpy as np
import pytest

from oracle import attn
from tests.test_gpu_attn_decode import Case, _check, _dense64, _reach
from tests.test_gpu_attn_prologue import _dev, _int32, _np, g2  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,N,Hq,Hkv,d,page,window", [
    ([1], 17, 1, 1, 80, 16, 0),                      # more tokens than keys: rows that see nothing
    ([127, 128, 129, 0, 2], 4, 16, 2, 128, 16, 0),   # around a step
    ([255, 256, 257], 5, 8, 2, 256, 32, 0),
    ([384, 5], 3, 14, 1, 96, 24, 0),                 # pages that no group of keys fits
    ([700, 130, 1], 4, 16, 2, 144, 7, 0),            # pages of single keys' copies, a width between the panels
    ([1000, 90, 17], 6, 12, 2, 128, 48, 130),        # windows over steps' edges
    ([400, 33], 20, 4, 2, 256, 16, 3),               # windows shorter than the tokens
    ([513, 64, 1100], 40, 4, 2, 128, 64, 0),         # several units a key head
    ([300], 70, 2, 1, 192, 16, 100),
    ([2000, 3, 900], 4, 32, 4, 128, 1024, 0),        # one page a row, or two
])
def test_drafts(g2, lens, N, Hq, Hkv, d, page, window):  # noqa: F811
    c = Case(lens, N, Hq, Hkv, d, page, "bf16", seed=N + d)
    got = c.run(g2, window=window)
    c.check(got, window)
    assert got.equal(c.run(g2, window=window))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("N,window", [(4, 0), (4, 9), (9, 4), (4, 200), (40, 0)])
@pytest.mark.parametrize("d,page", [(128, 16), (96, 24), (256, 16)])
def test_what_is_hidden_does_not_count(g2, d, page, N, window, bad):  # noqa: F811
    """The rest of a page, other pages, keys before the window, and those of later tokens of the same call hold what is not finite."""
    import torch

    c = Case([141, 58, 400, 129], N, 16, 2, d, page, "bf16", seed=N)
    want = c.run(g2, window=window)
    c.check(want, window)
    mine = torch.zeros(c.pools[0].shape[0], page, dtype=torch.bool, device="cuda")
    for s in c.slots:
        lo, last = attn.visible(int(c.lengths[s]), N, 0, window)[0], attn.visible(int(c.lengths[s]), N, N - 1, window)[1]
        for t in range(lo, last + 1):
            mine[c.table[s, t // page], t % page] = True
    for p in c.pools:
        p.masked_fill_(~mine[:, None, :, None], bad)
    assert c.run(g2, window=window).equal(want)
    for s in c.slots:  # the newest token's key and value
        t = int(c.lengths[s]) - 1
        for p in c.pools:
            p[c.table[s, t // page], :, t % page] = bad
    got = c.run(g2, window=window)
    assert got[:, :-1].equal(want[:, :-1]) and not bool(got[:, -1].isfinite().any())
    if window:  # the first token's oldest key
        c = Case([141, 58, 400, 129], N, 16, 2, d, page, "bf16", seed=N)
        for s in c.slots:
            t = attn.visible(int(c.lengths[s]), N, 0, window)[0]
            if t > 0:
                for p in c.pools:
                    p[c.table[s, t // page], :, t % page] = bad
        got = c.run(g2, window=window)
        for b, s in enumerate(c.slots):
            if int(c.lengths[s]) - N - window + 1 > 0:
                assert got[b, 1:].equal(want[b, 1:]) and not bool(got[b, 0].isfinite().any())


@pytest.mark.parametrize("seed", range(24))
def test_any_shape(g2, seed):  # noqa: F811
    """Sizes, holes, shared pages, inactive rows and windows by chance, more than 16 query rows a key head."""
    import torch

    rng = np.random.default_rng(500 + seed)
    B, rows, Hkv, G = rng.integers(1, 50), 45, rng.integers(1, 5), int(rng.choice([1, 3, 4, 8, 16, 20]))
    N = int(16 // G + 1 + rng.integers(0, 5))
    d, page = 16 * int(rng.integers(5, 17)), int(rng.choice([1, 8, 16, 24, 32, 64, 128]))
    wide = max(1, int(rng.choice([100, 400, 1500, 6000]) // page))
    pages = wide + 5
    table = rng.integers(0, pages, (rows, wide))
    table[rng.random(table.shape) < 0.1] = rng.choice([-1, pages, 2 ** 30])
    top = wide * page
    lengths = np.where(rng.random(rows) < 0.3, rng.choice([-1, 0, 1, N, top, top + 1, 2 ** 31 - 1], rows), rng.integers(0, top + 1, rows))
    slots = rng.integers(0, rows + 6, B) - 3  # the same slot more than once
    window = int(rng.choice([0, 0, 1, 7, 100, 10 ** 6]))
    pools = [_dev(rng.standard_normal((pages, Hkv, page, d)), "bf16") for _ in range(2)]
    q, scale = _dev(rng.standard_normal((B, N, Hkv * G, d)), "bf16"), float(rng.choice([d ** -0.5, -0.05, 0.0]))
    o = torch.full_like(q, 7.0)
    g2.gdn2_attn_decode(q, *pools, _int32(table), _int32(lengths), o, _int32(slots), scale=scale, window=window)
    want, mag = _dense64(q, *pools, table, lengths, slots, scale, window)
    dead = np.isnan(want[:, 0, 0, 0])
    assert bool((o[torch.as_tensor(dead, device="cuda")] == 7).all())
    _check(_np(o), want, mag, _reach(_np(q), _np(pools[0]), scale, top, "bf16"), "bf16")


@pytest.mark.parametrize("lens,N,Hq,Hkv,d,page", [
    ([60000], 4, 8, 1, 128, 64), ([30000, 5, 1000], 4, 16, 2, 256, 64), ([(37 * i * i) % 900 if i % 5 else 0 for i in range(300)], 3, 12, 2, 128, 32),
    ([20011], 20, 4, 4, 112, 40), ([0] * 300 + [5] * 30 + [4000] + [0] * 300, 5, 4, 1, 128, 16)])
def test_long_rows_and_many_rows(g2, lens, N, Hq, Hkv, d, page):  # noqa: F811
    c = Case(lens, N, Hq, Hkv, d, page, "bf16", seed=len(lens))
    got = c.run(g2)
    want, mag = _dense64(c.q, *c.pools, c.table, c.lengths, c.slots, c.scale, 0)
    _check(_np(got), want, mag, _reach(_np(c.q), _np(c.pools[0][:50]), c.scale, max(lens), "bf16"), "bf16")


def test_rising_scores(g2):  # noqa: F811
    """Scores that grow along the row by far more than the slack of the running maximum, and fall: every step moves the reference, or none."""
    c = Case([1500, 1500], 3, 8, 1, 128, 16, "bf16")
    for down in (False, True):
        k = c.pools[0]
        ramp = np.zeros(k.shape, np.float32)
        for s in c.slots:
            for t in range(1500):
                ramp[c.table[s, t // 16], :, t % 16, 0] = (1500 - t if down else t) / 4
        c.pools[0] = _dev(ramp + 0.25 * _np(k), "bf16")
        c.q[..., 0] = 4.0
        # scores reach 4 * 375 * scale = 133; a sum of their terms is known to 128 * 2^-24 of 1500 scale
        c.check(c.run(g2))


def test_captured_and_two_streams(g2):  # noqa: F811
    """Graphs follow lengths that change on the device; two of them at once on two streams, each with a workspace of its own."""
    import torch

    cases = [Case([900, 20, 300], 4, 16, 2, d, 16, "bf16", seed=d) for d in (128, 256)]
    fs = []
    for c in cases:
        c.table = np.concatenate([c.table, np.full((5, 40), -1)], 1)
        fs.append((_int32(c.table), _int32(c.lengths), _int32(c.slots)))
    call = lambda c, a: g2.attn_decode(c.q, *c.pools, *a)  # noqa: E731
    graphs = []
    for c, a in zip(cases, fs):
        call(c, a)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call(c, a)
        graphs.append((graph, got))
    for lens in ([900, 20, 300], [4, 4, 4], [0, 19, 299], [640, 0, 17]):
        want = []
        for c, a in zip(cases, fs):
            c.lengths[c.slots] = lens
            a[1].copy_(_int32(c.lengths))
            want.append(call(c, a))
        streams = [torch.cuda.Stream() for _ in graphs]
        torch.cuda.synchronize()
        for _ in range(10):
            for (graph, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for (_, got), w, c in zip(graphs, want, cases):
            assert got.equal(w)
            c.check(w)


@pytest.mark.parametrize("d,page", [(128, 16), (128, 24), (256, 16)])
def test_timeout_then_correct(g2, d, page):  # noqa: F811
    """Waits that give up at once: the call ends, the status says so, and the next call is right."""
    import torch

    c = Case([3000, 500, 7], 4, 16, 2, d, page, "bf16")
    g2.gdn2_set_wait_limit(0)
    try:
        c.run(g2)
        torch.cuda.synchronize()
        assert g2.gdn2_last_device_status() == g2.GDN2_ERR_TIMEOUT
    finally:
        g2.gdn2_set_wait_limit(-1)
    assert g2.gdn2_last_device_status() == g2.GDN2_OK
    c.check(c.run(g2))


@pytest.mark.parametrize("page", [32, 24])
def test_far_pages(g2, page):  # noqa: F811
    """Pools of more than 2^31 elements: pages behind the 32-bit range are read, by tensor copies and key by key."""
    import torch

    pages, Hkv, d = 140_000 * 32 // page, 4, 128
    pools = [torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    at, length = [pages - 1, 3, pages - 2], 3 * page - 5
    near = [torch.randn(3, Hkv, page, d, device="cuda").bfloat16() for _ in range(2)]
    for p, n in zip(pools, near):
        p[at] = n
    q = torch.randn(1, 5, 32, d, device="cuda").bfloat16()
    o = g2.attn_decode(q, *pools, _int32([at]), _int32([length]))
    assert o.equal(g2.attn_decode(q, *near, _int32([[0, 1, 2]]), _int32([length])))
    want, mag = _dense64(q, *near, np.array([[0, 1, 2]]), np.array([length]), [0], d ** -0.5, 0)
    _check(_np(o), want, mag, _reach(_np(q), _np(near[0]), d ** -0.5, length, "bf16"), "bf16")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G", [2, 8])
def test_scores_below_all_numbers(g2, G, d):  # noqa: F811
    """Scores that overflow to -inf, a whole step of them first: no weight, and the others as ever."""
    c = Case([700, 300], 4, 2 * G, 2, d, 16, "bf16")
    k = _np(c.pools[0]).copy()
    k[..., 0] = 0.0
    for s in c.slots:
        for t in range(260):
            k[c.table[s, t // 16], :, t % 16, 0] = -1e30
    c.pools[0] = _dev(k, "bf16")
    c.q[..., 0] = 1e10
    got = c.run(g2)
    rest = _np(c.q).copy()  # the reference's magnitudes without the part that overflows, which adds nothing to the other scores
    rest[..., 0] = 1.0
    want, mag = attn.attend(_np(c.q), k, _np(c.pools[1]), c.table, c.lengths, c.slots, c.scale)
    k[..., 0] = 0.0
    _check(_np(got), want, mag, _reach(rest, k, c.scale, 700, "bf16"), "bf16")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G", [2, 8])
def test_rows_do_not_touch_each_other(g2, G, d):  # noqa: F811
    """The newest token's key has one infinite component: its scores are infinite, and the other tokens' results keep their bits."""
    c = Case([700, 300, 131], 4, 2 * G, 2, d, 16, "bf16")
    want = c.run(g2)
    for s in c.slots:
        t = int(c.lengths[s]) - 1
        c.pools[0][c.table[s, t // 16], :, t % 16, 0] = float("inf")
    assert c.run(g2)[:, :-1].equal(want[:, :-1])
