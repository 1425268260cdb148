"""A small stack of selective state-space mixers on the operators: trained on packed sequences of unequal length, then
prompted and decoded token by token from the states that the prompt left.

    python examples/ssm_mixer.py [--steps 150]

Per block, with r the residual stream and n its norm:
    z, xbc, delta = n W_in                            (library products)
    u, step, g    = ssm_prologue(xbc, delta)          u = x | B | C
    y             = ssm_chunk_fwd(x, step, g, B, C)   one token: ssm_decode_step in place of both
    p             = block_norm(y, z)                  gated norm over groups of heads
    r, n          = block_norm(p W_out, residual = r) residual and the next block's norm
The task: each sequence repeats a random word of up to eight letters, and the next letter is asked for.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import gated_deltanet_mixer_gdn2_gb300 as g2

D, H, G, P, N, LETTERS, BLOCKS = 128, 4, 1, 64, 64, 24, 2
INNER, CH = H * P, H * P + 2 * G * N


class Prologue(torch.autograd.Function):
    @staticmethod
    def forward(ctx, xbc, delta, w, bias, a, delta_bias, offsets):
        ctx.save_for_backward(xbc, delta, w, bias, a, delta_bias, offsets)
        return g2.ssm_prologue(xbc, delta, w, bias, a, delta_bias, None, offsets)

    @staticmethod
    def backward(ctx, du, dstep, dg):
        xbc, delta, w, bias, a, delta_bias, offsets = ctx.saved_tensors
        grads = g2.ssm_prologue_backward(xbc, delta, w, bias, a, delta_bias, du.contiguous(), dstep, dg, offsets)
        return (*grads, None)


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, step, g, d, offsets):
        ctx.save_for_backward(u, step, g, d, offsets)
        return g2.ssm_chunk_fwd(*split(u, step, g), d, None, offsets, output_final_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        u, step, g, d, offsets = ctx.saved_tensors
        du = torch.empty_like(u)  # dx, dB and dC are slices of one row
        x, step, g, bm, cm = split(u, step, g)
        dx, _, _, db, dc = split(du, step, g)
        dstep, dg, dd = torch.empty_like(step), torch.empty_like(g), torch.empty_like(d)
        g2.gdn2_ssm_backward(x, step, g, bm, cm, dy.contiguous(), dx, dstep, dg, db, dc, dd, d, offsets=offsets)
        return du, dstep, dg, dd, None


class Norm(torch.autograd.Function):
    """r, n of block_norm; those that it does not return are None."""

    @staticmethod
    def forward(ctx, x, z, post, residual, pre, groups):
        ctx.save_for_backward(x, z, post, residual, pre)
        ctx.groups = groups
        return g2.block_norm(x, z, post, residual, None, pre, groups=groups)

    @staticmethod
    def backward(ctx, dr, dn):
        x, z, post, residual, pre = ctx.saved_tensors
        whole = lambda t: t.contiguous() if t is not None else None
        dx, dz, dpost, dres, _, dpre = g2.block_norm_backward(x, z, post, residual, None, pre, whole(dr), whole(dn), groups=ctx.groups)
        return dx, dz, dpost, dres, dpre, None


def split(u, step, g):
    return (u[..., :INNER].unflatten(-1, (H, P)), step, g, u[..., INNER:INNER + G * N].unflatten(-1, (G, N)),
            u[..., INNER + G * N:].unflatten(-1, (G, N)))


class Mixer(torch.nn.Module):
    """One block's parameters: fp32, its matrices used in bf16."""

    def __init__(self):
        super().__init__()
        new = lambda *s, std: torch.nn.Parameter(std * torch.randn(*s))
        self.w_in = new(D, INNER + CH + H, std=D ** -0.5)
        self.w_out = new(INNER, D, std=INNER ** -0.5)
        self.conv = new(CH, 4, std=0.5)
        self.conv_bias = torch.nn.Parameter(torch.zeros(CH))
        self.log_rate = torch.nn.Parameter(torch.linspace(-2, 1, H))
        self.delta_bias = torch.nn.Parameter(torch.linspace(-4, -1, H))
        self.d = torch.nn.Parameter(torch.ones(H))
        self.post = torch.nn.Parameter(torch.ones(INNER))
        self.next = torch.nn.Parameter(torch.ones(D))  # the norm before the next block

    def project(self, n):
        z, xbc, delta = (n @ self.w_in.to(n.dtype)).split([INNER, CH, H], -1)
        return z.contiguous(), xbc, delta

    def train_pass(self, r, n, offsets):
        z, xbc, delta = self.project(n)
        u, step, g = Prologue.apply(xbc, delta, self.conv, self.conv_bias, -torch.exp(self.log_rate), self.delta_bias, offsets)
        y = Scan.apply(u, step, g, self.d, offsets)
        p, _ = Norm.apply(y.flatten(-2), z, self.post, None, None, G)
        return Norm.apply(p @ self.w_out.to(p.dtype), None, None, r, self.next, 1)

    @torch.no_grad()
    def prompt(self, r, n, offsets, state):
        z, xbc, delta = self.project(n)
        u, step, g = g2.ssm_prologue(xbc, delta, self.conv, self.conv_bias, -torch.exp(self.log_rate), self.delta_bias,
                                     state["conv"], offsets)
        y, state["ssm"] = g2.ssm_chunk_fwd(*split(u, step, g), self.d, None, offsets)
        return self.leave(y, z, r)

    @torch.no_grad()
    def token(self, r, n, state):
        z, xbc, delta = self.project(n)
        y = g2.ssm_decode_step(xbc, delta, self.conv, self.conv_bias, -torch.exp(self.log_rate), self.delta_bias, self.d,
                               state["conv"], state["ssm"])
        return self.leave(y, z, r)

    def leave(self, y, z, r):
        p, _ = g2.block_norm(y.flatten(-2), z, self.post, groups=G)
        return g2.block_norm(p @ self.w_out.to(p.dtype), residual=r, pre_weight=self.next)


class Model(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.embed = torch.nn.Parameter(torch.randn(LETTERS, D))
        self.first = torch.nn.Parameter(torch.ones(D))
        self.blocks = torch.nn.ModuleList(Mixer() for _ in range(BLOCKS))
        self.head = torch.nn.Parameter(D ** -0.5 * torch.randn(D, LETTERS))

    def enter(self, letters):
        return self.embed[letters].to(torch.bfloat16)

    def logits(self, n):
        return n.float() @ self.head

    def forward(self, letters, offsets):
        r = self.enter(letters)
        _, n = Norm.apply(r, None, None, None, self.first, 1)
        for b in self.blocks:
            r, n = b.train_pass(r, n, offsets)
        return self.logits(n)

    @torch.no_grad()
    def prompt(self, letters, offsets):
        """The logits after every token of the packed prompts and the states they leave."""
        rows = offsets.numel() - 1
        states = [{"conv": torch.zeros(rows, 3, CH, device=letters.device)} for _ in self.blocks]
        r = self.enter(letters)
        _, n = g2.block_norm(r, pre_weight=self.first)
        for b, s in zip(self.blocks, states):
            r, n = b.prompt(r, n, offsets, s)
        return self.logits(n), states

    @torch.no_grad()
    def token(self, letters, states):
        r = self.enter(letters)
        _, n = g2.block_norm(r, pre_weight=self.first)
        for b, s in zip(self.blocks, states):
            r, n = b.token(r, n, s)
        return self.logits(n)


def words(rng, rows, device, lo=17, hi=80):
    """Packed sequences, each a word repeated: letters, offsets, and each sequence's word."""
    seqs, spelled = [], []
    for _ in range(rows):
        word = torch.randint(LETTERS, (int(torch.randint(2, 9, (1,), generator=rng)),), generator=rng)
        n = int(torch.randint(lo, hi, (1,), generator=rng))
        seqs.append(word.repeat(n // len(word) + 1)[:n])
        spelled.append(word)
    off = torch.tensor([0] + [len(s) for s in seqs]).cumsum(0)
    return torch.cat(seqs).to(device), off.to(device=device, dtype=torch.int32), spelled


def train(model, rng, steps, rows=48):
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3, weight_decay=0.0)
    losses = []
    for _ in range(steps):
        letters, off, _ = words(rng, rows, "cuda")
        logits = model(letters, off)
        ask = torch.ones(len(letters), dtype=torch.bool, device="cuda")
        ask[off[1:].long() - 1] = False  # a sequence's last letter asks for nothing
        loss = torch.nn.functional.cross_entropy(logits[:-1][ask[:-1]], letters[1:][ask[:-1]])
        opt.zero_grad(set_to_none=True)
        loss.backward()
        torch.nn.utils.clip_grad_norm_(model.parameters(), 1.0)
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def spell(model, rng, rows=32, tokens=24):
    """Greedy continuation of prompts: the share of letters that continue the prompt's word."""
    letters, off, spelled = words(rng, rows, "cuda")
    lens = off.diff().tolist()
    logits, states = model.prompt(letters, off)
    at = logits[off[1:].long() - 1]
    right = 0
    for t in range(tokens):
        guess = at.argmax(-1)
        want = torch.tensor([int(w[(n + t) % len(w)]) for w, n in zip(spelled, lens)], device="cuda")
        right += int((guess == want).sum())
        at = model.token(guess, states)
    return right / (rows * tokens)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=150)
    steps = ap.parse_args().steps
    torch.manual_seed(0)
    rng = torch.Generator().manual_seed(1)
    model = Model().cuda()
    losses = train(model, rng, steps)
    print("loss: first %.3f, last %.3f" % (losses[0], sum(losses[-10:]) / len(losses[-10:])))
    print("letters continued: %.1f%%" % (100 * spell(model, rng)))


if __name__ == "__main__":
    main()
