"""Requests for room that are turned down in mid-step: the rows take no part in the step's other calls and hold what they held, whether the step is
called or replayed."""
import numpy as np
import pytest

from tests.test_gpu_attn_decode import _check, _dense64, _reach
from tests.test_gpu_attn_prologue import _dev, _int32, _np, g2  # noqa: F401
from tests.test_gpu_pages import Both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 7, 1500])
def test_rows_that_take_part(g2, n):  # noqa: F811
    rng = np.random.default_rng(n)
    b = Both(g2, 2 * n + 2, 4, 2 * n, 8)
    for _ in range(6):
        slots, active = rng.permutation(2 * n + 4)[:n] - 1, _int32(np.full(n, 77))
        tokens = rng.integers(-1, 20, n)
        got = g2.pages_append(*b.dev, _int32(slots), _int32(tokens), page=8, active=active)
        ok = b.ref.append(list(map(int, slots)), list(map(int, tokens)))
        b.same((got, ok), (active, np.where(np.array(ok) > 0, slots, -1)))
        order = rng.permutation(2 * n + 4) - 1
        m = n // 2
        src, dst, active = order[:m], order[m:2 * m], _int32(np.full(m, 77))
        got = g2.pages_fork(*b.dev, _int32(src), _int32(dst), page=8, active=active)
        want = b.ref.fork(list(map(int, src)), list(map(int, dst)))
        b.same(*zip(got, want), (active, np.where(np.array(want[2], dtype=int) > 0, dst, -1)))
        b.release(order[:max(n // 3, 1)])
    assert g2.pages_append(*b.dev, _int32([]), 1, page=8, active=_int32([])).shape == (0,)


def test_a_step_without_room(g2):  # noqa: F811
    """Three rows decode, captured once; pages run out under one of them, which waits until another leaves, and goes on as if nothing had been."""
    import torch

    page, d, Hq, Hkv = 16, 64, 4, 2
    rng = np.random.default_rng(5)
    b = Both(g2, 5, 8, 7, page)
    b.append([0, 3, 4], [47, 31, 14])  # pages of three, two and one; one is left
    pools = [_dev(rng.standard_normal((7, Hkv, page, d)), "bf16") for _ in range(2)]
    slots, active = _int32([4, 3, 0]), _int32([-1] * 3)
    rows = torch.zeros(3, 1, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(3, 1, Hq, d, dtype=torch.bfloat16, device="cuda")
    states = torch.zeros(5, Hq, d, d, device="cuda")
    table, lengths, _ = b.dev
    tokens = lambda: torch.rand(3, 1, Hq, d, device="cuda").bfloat16()  # noqa: E731
    qm, km, vm, gm, bm, wm = (tokens() for _ in range(6))
    om = torch.empty_like(vm)

    def step():
        ok = g2.pages_append(*b.dev, slots, 1, page=page, active=active)
        q = g2.attn_prologue_paged(rows[:, :, :Hq], rows[:, :, Hq:Hq + Hkv], rows[:, :, Hq + Hkv:], *pools, table, lengths, active)
        g2.gdn2_attn_decode(q, *pools, table, lengths, o, active)
        g2.gdn2_recurrent_update(qm, km, vm, -gm, bm, wm, states, om, active)  # a mixer's states by the same slots
        return ok

    kept = [t.clone() for t in (*b.dev, *pools, states)]
    step()
    for t, k in zip((*b.dev, *pools, states), kept):
        t.copy_(k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ok = step()
    waited = 0
    for i in range(29):
        rows.copy_(torch.randn_like(rows))
        o.fill_(7)
        was, had = [p.clone() for p in pools], states.clone()
        graph.replay()
        met = b.ref.append([4, 3, 0], [1, 1, 1])
        b.same((ok, met))
        live = [s if m else -1 for s, m in zip([4, 3, 0], met)]
        for j, s in enumerate(live):
            if s >= 0:
                n = b.ref.lengths[s] - 1
                for p, part in zip(was, (rows[j, 0, Hq:Hq + Hkv], rows[j, 0, Hq + Hkv:])):
                    p[b.ref.table[s][n // page], :, n % page] = part
            else:
                waited += 1
                assert bool((o[j] == 7).all())
        assert all(p.equal(w) for p, w in zip(pools, was))  # the tokens of rows that take part, and nothing else
        moved = [not torch.equal(states[s], had[s]) for s in range(5)]
        assert moved == [s in live for s in range(5)]
        q = rows[:, :, :Hq].contiguous()
        want, mag = _dense64(q, *pools, np.array(b.ref.table), np.array(b.ref.lengths), live, d ** -0.5, 0)
        _check(_np(o), want, mag, _reach(_np(q), _np(pools[0]), d ** -0.5, 100, "bf16"), "bf16")
        if i == 12:
            assert waited == 12 + 11
            b.release([3])
    assert waited == 12 + 11 and b.ref.lengths == [64, 0, 0, 16, 32]
