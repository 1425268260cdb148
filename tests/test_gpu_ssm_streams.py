"""The selective state-space calls on a stream that is given to them: their memory is that stream's."""
import pytest

from tests.test_gpu_ssm import g2  # noqa: F401

pytestmark = pytest.mark.gpu


def _int32(v):
    import torch

    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _calls(g2):
    """Every call that allocates, on given inputs: name -> (call, its results on the current stream)."""
    import torch

    torch.manual_seed(3)
    f = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    rows, H, G, P, N = 300, 4, 1, 64, 64
    ch = H * P + 2 * G * N
    off = _int32([0, 200, rows])
    xbc, delta = f(rows, ch).bfloat16(), f(rows, H).bfloat16()
    w, bias, a, db, d = 0.4 * f(ch, 4), f(ch), -f(H).abs(), f(H), f(H)
    u, step, g = g2.ssm_prologue(xbc, delta, w, bias, a, db, None, off)
    x, bm, cm = u[:, :H * P].unflatten(-1, (H, P)), u[:, H * P:H * P + N].unflatten(-1, (1, N)), u[:, H * P + N:].unflatten(-1, (1, N))
    dy, s0, ds1 = f(rows, H, P).bfloat16(), f(2, H, N, P), f(2, H, N, P)
    wide = [t.unsqueeze(0) for t in (x, step, g, bm, cm)]  # one sequence of few heads, long enough to be cut
    long = [torch.cat([t] * 8, 1) for t in wide]
    z, r, dr, dn = (f(rows, H * P).bfloat16() for _ in range(4))
    post, scale, pre = (f(H * P) for _ in range(3))
    y = x.flatten(1).contiguous()
    fresh, used = [(torch.ones(5, 3, ch, device="cuda"), torch.ones(5, H, N, P, device="cuda")) for _ in range(4)], []

    def decode(**k):
        used.append(fresh.pop())  # kept: the call may still be waiting when it returns
        return (g2.ssm_decode_step(xbc[:5], delta[:5], w, bias, a, db, d, *used[-1], **k),)

    calls = {
        "prologue": lambda **k: g2.ssm_prologue(xbc, delta, w, bias, a, db, None, off, **k),
        "prologue gradients": lambda **k: g2.ssm_prologue_backward(xbc, delta, w, bias, a, db, u, step, g, off, **k),
        "scan": lambda **k: g2.ssm_chunk_fwd(x, step, g, bm, cm, d, s0, off, **k),
        "scan, cut": lambda **k: g2.ssm_chunk_fwd(*long, d, **k),
        "scan gradients": lambda **k: g2.ssm_backward(x, step, g, bm, cm, dy, d, s0, ds1, off, **k),
        "decode": decode,
        "norm": lambda **k: g2.block_norm(y, z, post, r, scale, pre, **k),
        "norm gradients": lambda **k: g2.block_norm_backward(z, r, post, dr, scale, pre, dr, dn, **k),
    }
    return calls


STREAM_CALLS = ["prologue", "prologue gradients", "scan", "scan, cut", "scan gradients", "decode", "norm", "norm gradients"]
CYCLES = 40_000_000  # some 20 ms: far longer than the host takes to queue what follows


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_stream_argument_keeps_its_memory(g2, name, monkeypatch):  # noqa: F811
    """A call on a stream that is busy is still waiting when it returns: what the caller's stream allocates meanwhile is no
    memory of the call's, and its results are those of a call on the caller's own stream."""
    import torch

    call = _calls(g2)[name]
    want = [t.clone() for t in call() if t is not None]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    taken, empty = [], torch.empty

    def spy(*args, **kw):
        t = empty(*args, **kw)
        taken.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()))
        return t

    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    monkeypatch.setattr(torch, "empty", spy)
    got = call(stream=side)
    monkeypatch.setattr(torch, "empty", empty)
    mine = [empty(hi - lo, dtype=torch.uint8, device="cuda") for lo, hi in taken for _ in range(2)]
    for t in mine:
        at = t.data_ptr()
        assert all(at + t.numel() <= lo or at >= hi for lo, hi in taken if hi > lo), name
    side.synchronize()
    for a, b in zip([t for t in got if t is not None], want):
        assert torch.equal(a, b), name


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_stream_argument_waits_for_no_memory_in_use(g2, name):  # noqa: F811
    """Memory that the caller's stream has let go of but still works on is not the call's: results come from its own stream."""
    import torch

    call = _calls(g2)[name]
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() for t in call() if t is not None]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    kept = [t.clone() for t in old]
    del old
    got = call(stream=side)
    torch.cuda.synchronize()
    assert all(bool((t == 3).all()) for t in kept) and got is not None


def test_results_of_a_stream_are_kept_for_the_caller(g2):  # noqa: F811
    """A result that the caller's stream still reads when it is let go of is not given to the next call on that stream."""
    import torch

    call = _calls(g2)["prologue"]
    side = torch.cuda.Stream()
    want = call()[0].clone()
    first = call(stream=side)
    side.synchronize()
    torch.cuda._sleep(CYCLES)
    kept = first[0].clone()
    del first
    with torch.cuda.stream(side):
        again = [torch.zeros_like(want) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and len(again) == 4
