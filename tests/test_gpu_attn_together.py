"""The attention layers' operators as a server uses them, together: rows are admitted, take prompts of several lengths, decode, are forked,
go on apart, and are given back, with two layers' pools and a mixer's states on the same slots. Each layer's output is compared with
attention over the row's whole history in fp64.

Tolerance: queries and keys are taken as the prologue stored them, so what is compared is one attention, as in test_gpu_attn_decode: half a
step of bf16 of the result, and 2^-13 of sum p |v| (d = 64, scores up to some 20: 2 * 64 * 2^-24 * 20, 2^-15 of the weights' parts, keys of
at most 300)."""
import numpy as np
import pytest

from tests.test_gpu_attn_prologue import _int32, g2  # noqa: F401

pytestmark = pytest.mark.gpu

SLOTS, PAGE, PAGES, WIDE, HQ, HKV, D, LAYERS = 10, 16, 90, 20, 4, 2, 64, 2


class Server:
    def __init__(self, g2):  # noqa: F811
        import torch

        self.g2, self.torch = g2, torch
        torch.manual_seed(0)
        self.table = torch.full((SLOTS, WIDE), -1, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(SLOTS, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        self.pools = [[torch.full((PAGES, HKV, PAGE, D), float("nan"), device="cuda").bfloat16() for _ in range(2)] for _ in range(LAYERS)]
        self.states = torch.zeros(SLOTS, 2, 16, 16, device="cuda")
        self.freq = 1e4 ** -(torch.arange(D // 2, device="cuda") / (D / 2))
        self.w = [1 + 0.1 * torch.randn(2, D, device="cuda") for _ in range(LAYERS)]
        self.past = {}  # slot -> per layer (keys, values) of its tokens, as stored

    def cache(self):
        return self.table, self.lengths, self.refs

    def feed(self, slots, counts):
        """counts[i] new tokens for slots[i]: packed when they differ; the newest tokens' outputs of each layer are checked where the counts are
        alike."""
        t = self.torch
        ok = self.g2.pages_append(*self.cache(), _int32(slots), _int32(counts), page=PAGE)
        assert bool(ok.all())
        at = _int32(slots)
        offsets = _int32(np.concatenate([[0], np.cumsum(counts)]))
        alike = len(set(counts)) == 1
        for layer in range(LAYERS):
            row = t.randn(sum(counts), (HQ + 2 * HKV) * D, device="cuda").bfloat16()
            q, k, v = (x.unflatten(-1, (-1, D)) for x in row.split([HQ * D, HKV * D, HKV * D], -1))
            args = (*self.pools[layer], self.table, self.lengths, at, *self.w[layer], self.freq)
            if alike:
                q, k, v = (x.unflatten(0, (len(slots), counts[0])) for x in (q, k, v))
                turned = self.g2.attn_prologue_paged(q, k, v, *args)
            else:
                turned = self.g2.attn_prologue_paged(q, k, v, *args, offsets=offsets)
            # what the cache should hold: the same keys by the prologue that keeps no cache
            flat = k.reshape(1, -1, HKV, D)
            pos = np.concatenate([np.arange(n) + len(self.past[s][layer][0]) for s, n in zip(slots, counts)])
            _, keys = self.g2.attn_prologue(flat[:, :, :1].expand(-1, -1, HQ, -1).contiguous(), flat, None, self.w[layer][1], self.freq, _int32(pos)[None])
            lo = 0
            for s, n in zip(slots, counts):
                kk, vv = self.past[s][layer]
                self.past[s][layer] = (t.cat([kk, keys[0, lo:lo + n]]), t.cat([vv, v.reshape(-1, HKV, D)[lo:lo + n]]))
                lo += n
            if alike:
                self.check(self.g2.attn_decode(turned, *args[:5]), turned, slots, layer, counts[0])
        self.states[at.long()] += 1.0 + at[:, None, None, None]

    def check(self, o, q, slots, layer, n):
        t = self.torch
        for i, s in enumerate(slots):
            k, v = (x.double().transpose(0, 1) for x in self.past[s][layer])
            total = k.shape[1]
            for j in range(n):
                seen = total - n + j + 1
                w = t.softmax(q[i, j].double().reshape(HKV, HQ // HKV, D) @ k[:, :seen].transpose(1, 2) / D ** 0.5, -1)
                want, mag = (w @ v[:, :seen]).reshape(HQ, D), (w @ v[:, :seen].abs()).reshape(HQ, D)
                assert bool(((o[i, j].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -13 * mag).all())

    def admit(self, slot):
        empty = lambda: self.torch.zeros(0, HKV, D, device="cuda").bfloat16()  # noqa: E731
        self.past[slot] = [(empty(), empty()) for _ in range(LAYERS)]
        self.states[slot] = 0

    def fork(self, src, dst):
        a, b, ok = self.g2.pages_fork(*self.cache(), _int32(src), _int32(dst), page=PAGE)
        assert bool(ok.all())
        self.g2.pages_copy([p for layer in self.pools for p in layer], a, b)
        self.g2.pages_copy([self.states], _int32(src), _int32(dst))
        for s, d in zip(src, dst):
            self.past[d] = list(self.past[s])

    def leave(self, slots):
        self.g2.pages_release(*self.cache(), _int32(slots))
        for s in slots:
            del self.past[s]


def test_a_server(g2):  # noqa: F811
    rng = np.random.default_rng(0)
    s = Server(g2)
    for slot in (3, 0, 7):
        s.admit(slot)
    s.feed([3, 0, 7], [20, 1, 65])
    for _ in range(3):
        s.feed([7, 3, 0], [1, 1, 1])
    s.fork([7, 7, 0], [1, 9, 4])
    s.feed([1, 9, 4, 7], [1, 1, 1, 1])        # they go on apart
    s.feed([1, 9], [4, 4])                    # four drafted tokens at once
    states = s.states.clone()
    s.fork([9, 3], [7, 0])                    # rows that held something else
    assert s.torch.equal(s.states[7], states[9]) and s.torch.equal(s.states[0], states[3])
    s.feed([7, 0, 9, 3], [2, 2, 2, 2])
    s.leave([1, 4])
    s.admit(5)
    s.feed([5], [130])
    s.feed([5, 9, 7], [1, 1, 1])
    for _ in range(20):
        live = sorted(s.past)
        spare = [x for x in range(SLOTS) if x not in s.past]
        kind = rng.integers(4)
        if kind == 0 and spare and len(live) < 7:
            s.fork([int(rng.choice(live))], [spare[0]])
        elif kind == 1 and len(live) > 3:
            s.leave([int(rng.choice(live))])
        else:
            s.feed([int(x) for x in rng.permutation(live)], [int(rng.integers(1, 4))] * len(live))
    s.leave(sorted(s.past))
    assert bool((s.refs == 0).all()) and bool((s.table == -1).all()) and bool((s.lengths == 0).all())


def test_a_step_in_a_graph(g2):  # noqa: F811
    """One decode step, from room in the cache to the output, captured once and replayed over a page's end."""
    import torch

    a, b = Server(g2), Server(g2)
    for s in (a, b):
        for slot in (2, 6):
            s.admit(slot)
        torch.manual_seed(5)
        s.feed([2, 6], [14, 30])
    slots = _int32([2, 6])
    row = torch.zeros(2, (HQ + 2 * HKV) * D, dtype=torch.bfloat16, device="cuda")

    def step(s):
        g2.pages_append(*s.cache(), slots, 1, page=PAGE)
        q, k, v = (x.unflatten(-1, (-1, D)).unsqueeze(1) for x in row.split([HQ * D, HKV * D, HKV * D], -1))
        q = g2.attn_prologue_paged(q, k, v, *s.pools[0], s.table, s.lengths, slots, *s.w[0], s.freq)
        return g2.attn_decode(q, *s.pools[0], s.table, s.lengths, slots)

    rows = [torch.randn_like(row) for _ in range(8)]
    row.copy_(rows[0])
    want = [step(a)]
    row.copy_(rows[0])
    step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(b)
    assert torch.equal(b.lengths, a.lengths)  # a capture runs nothing
    for r in rows[1:]:
        row.copy_(r)
        want.append(step(a))
        graph.replay()
        assert torch.equal(got, want[-1])
    assert all(torch.equal(x, y) for x, y in zip(a.cache(), b.cache()))


def _calls(g2):  # noqa: F811
    """Every call that allocates, on given inputs."""
    import torch

    torch.manual_seed(1)
    q, k, v = (torch.randn(3, 5, h, D, device="cuda").bfloat16() for h in (HQ, HKV, HKV))
    w, freq = torch.rand(D, device="cuda"), torch.rand(D // 2, device="cuda")
    pools = [torch.randn(40, HKV, PAGE, D, device="cuda").bfloat16() for _ in range(2)]
    table = torch.arange(36, device="cuda", dtype=torch.int32).reshape(3, 12)
    lengths = _int32([190, 40, 7])
    spare = []

    def pages(call):
        def run(**kw):
            spare.append((torch.full((6, 12), -1, dtype=torch.int32, device="cuda"), _int32([0] * 6), _int32([0] * 40)))
            spare[-1][0][:3] = table
            spare[-1][1][:3] = lengths
            spare[-1][2][:36] = 1
            torch.cuda.synchronize()
            return call(*spare[-1], **kw)
        return run

    return {
        "prologue": lambda **kw: g2.attn_prologue(q, k, w, w, freq, **kw),
        "prologue gradients": lambda **kw: g2.attn_prologue_backward(q, k, q, k, w, w, freq, **kw),
        "prologue into pages": lambda **kw: (g2.attn_prologue_paged(q, k, v, *pools, table, lengths, None, w, w, freq, **kw),),
        "decode": lambda **kw: (g2.attn_decode(q, *pools, table, lengths, **kw),),
        "fork": pages(lambda *c, **kw: g2.pages_fork(*c, _int32([0, 1]), _int32([4, 5]), page=PAGE, **kw)),
        "append": pages(lambda *c, **kw: (g2.pages_append(*c, _int32([0, 4]), 3, page=PAGE, **kw),)),
    }


@pytest.mark.parametrize("name", ["prologue", "prologue gradients", "prologue into pages", "decode", "fork", "append"])
def test_stream_argument(g2, name):  # noqa: F811
    """A call on another stream takes its memory from that stream's pool, and its results are those of the caller's own stream."""
    import torch

    call = _calls(g2)[name]
    want = [t.clone() for t in call() if t is not None]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(10_000_000)
        got = call(stream=side)
        mine = [torch.full((1 << 20,), -1, dtype=torch.uint8, device="cuda") for _ in range(8)]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([t for t in got if t is not None], want)) and len(mine) == 8
