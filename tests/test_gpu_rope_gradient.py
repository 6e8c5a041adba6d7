"""Gradients of queries and keys that are turned and then attended, element by
element against automatic differentiation in 64 bits and along a direction against
differences.

Reference: the loss sum(O dO) as a function of q and k before the rotation, with what
the rounding of the turned rows moved them by added as a constant, so that both sides
have their gradient at the same rows.  Bound: the attention's backward is off by
2^-6 A + 2^-8 |gradient of the turned row| (A: its terms' absolute values, as its own
tests have it, and its result's rounding); rope_backward adds two of its elements, each
times its cos or sin, and rounds once more, 2^-8 of the result."""
import pytest
import torch

import exact_attention_forward_04_gb300 as fa
from exact_attention_forward_04_gb300.inputs import make_qkv
from tests.test_gpu_backward import _term_scales

pytestmark = pytest.mark.gpu

DEV = "cuda"


def turn(x, cs, interleaved, transposed=False):
    """x [B, H, N, d] by cs [.., N, rot / 2, 2], in x's type; differentiable."""
    rot = 2 * cs.shape[-2]
    c, s = cs[..., 0], -cs[..., 1] if transposed else cs[..., 1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * c - b * s, b * c + a * s
    y = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((y, x[..., rot:]), -1)


def attend(q, k, v, scale, causal):
    s = scale * (q @ k.transpose(-1, -2))
    if causal:
        n = s.shape[-1]
        s = s.masked_fill(torch.arange(n) > torch.arange(n)[:, None], float("-inf"))
    return torch.softmax(s, -1) @ v


def references(q, k, v, g, qr, kr, o, lse, cs, interleaved, scale, causal):
    """Gradients of q and k, their bounds, and the loss."""
    q, k, v, g, qr, kr = (t.double() for t in (q, k, v, g, qr, kr))
    moved = [r - turn(x, cs, interleaved) for x, r in ((q, qr), (k, kr))]

    def loss(a, b):
        at = [turn(x, cs, interleaved) + m for x, m in zip((a, b), moved)]
        return (attend(*at, v, scale, causal) * g).sum()

    leaves = [q.clone().requires_grad_(), k.clone().requires_grad_()]
    want = torch.autograd.grad(loss(*leaves), leaves)
    turned = [qr.clone().requires_grad_(), kr.clone().requires_grad_()]
    of_turned = torch.autograd.grad((attend(*turned, v, scale, causal) * g).sum(), turned)
    bounds = []
    size = torch.stack((cs[..., 0].abs(), -cs[..., 1].abs()), -1)      # |c| u + |s| v, |c| v + |s| u below
    for a, w, r in zip(_term_scales(qr, kr, v, o, lse, g, scale, causal), want, of_turned):
        b = 2.0 ** -6 * a + 2.0 ** -8 * r.abs()
        rot = 2 * cs.shape[-2]
        sums = turn(b, size, interleaved)
        if interleaved:
            sums[..., 1:rot:2] += 2 * b[..., 0:rot:2] * cs[..., 1].abs()
        else:
            sums[..., rot // 2:rot] += 2 * b[..., :rot // 2] * cs[..., 1].abs()
        bounds.append(sums * (1 + 2.0 ** -8) + 2.0 ** -8 * w.abs())
    return want, of_turned, bounds, loss


def case(B, H, N, d, rot, interleaved, causal, per_batch):
    q, k, v = make_qkv(B, H, N, d, seed=300 + N + d + rot)
    g = make_qkv(B, H, N, d, seed=400 + N + d + rot)[0]
    table = fa.rope_table(3 * N, rot, device="cpu")
    gen = torch.Generator().manual_seed(N)
    pos = torch.stack([torch.randperm(3 * N, generator=gen)[:N] for _ in range(B)]).int()
    pos = pos if per_batch else pos[0]
    cs = table[(pos[:, None] if per_batch else pos).long()].double()
    return q, k, v, g, table, pos, cs


CASES = [(1, 2, 70, 64, 64, False, True, False), (2, 2, 133, 64, 32, True, False, True),
         (2, 1, 70, 128, 128, True, True, False), (1, 2, 200, 128, 48, False, False, True)]


@pytest.mark.parametrize("B,H,N,d,rot,interleaved,causal,per_batch", CASES)
def test_turned_attended_and_turned_back(B, H, N, d, rot, interleaved, causal, per_batch):
    q, k, v, g, table, pos, cs = case(B, H, N, d, rot, interleaved, causal, per_batch)
    p, t, scale = pos.to(DEV), table.to(DEV), d ** -0.5
    qr, kr = (fa.rope(x.to(DEV), p, t, interleaved=interleaved) for x in (q, k))
    o, lse = fa.forward(qr, kr, v.to(DEV), causal=causal)
    dqr, dkr, _ = fa.backward(qr, kr, v.to(DEV), o, lse, g.to(DEV), causal=causal)
    got = [fa.rope_backward(x, p, t, interleaved=interleaved).cpu().double() for x in (dqr, dkr)]
    fa.check_errors()
    compare(got, references(q, k, v, g, qr.cpu(), kr.cpu(), o.cpu(), lse.cpu(), cs, interleaved, scale, causal),
          (q, k), cs, interleaved)


def compare(got, refs, before, cs, interleaved):
    want, of_turned, bounds, loss = refs
    for which, (x, w, r, b) in enumerate(zip(got, want, of_turned, bounds)):
        over = ((x - w).abs() / b).max().item()
        assert over <= 1, f"{'qk'[which]}: {over:.2f} of the bound"
        # the bound tells what is wrong: nothing, not turned back, turned the other way
        for wrong in (torch.zeros_like(w), r, turn(r, cs, interleaved)):
            assert ((wrong - w).abs() > b).double().mean() > 0.05
        # along the gradient itself, where no terms cancel
        e, h = w / w.norm(), 1e-5
        args = [[t.double() for t in before] for _ in range(2)]
        args[0][which], args[1][which] = args[0][which] + h * e, args[1][which] - h * e
        slope = ((loss(*args[0]) - loss(*args[1])) / (2 * h)).item()
        assert abs(slope - w.norm().item()) < 1e-6 * abs(slope)        # h^2, and 64 bits over 2 h
        off = (b * e.abs()).sum().item()
        assert abs((x * e).sum().item() - slope) < off < 0.9 * slope
