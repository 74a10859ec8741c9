"""Inputs and tolerances the prompt path's tests share."""
import numpy as np
import torch

# Half a step of bf16 relative to the value.
U = torch.finfo(torch.bfloat16).eps / 2
# Everything that is fp32 in the kernels: products of bf16 values are exact and
# summed over at most 128 channels per logit with logits below 2^6, so a logit is
# off by less than 128 x 2^-24 x 2^6 = 2^-11 of one in the worst order of signs,
# and a weight by that share; sums over keys add far less.
FP32 = 2.0 ** -11


def bounded(got, want, abs_sum, what):
    """|got - want| <= (U + FP32) abs_sum + U |want|: one operand of the product that
    formed the value rounded to bf16 (abs_sum: the product over absolute values), the
    fp32 arithmetic, and the result's own rounding of what that gives."""
    live = ~np.isnan(want)
    g, w, s = got[live], want[live], abs_sum[live]
    assert np.isfinite(g).all(), f"{what}: not finite"
    tol = (U + FP32) * s
    tol = tol + U * (np.abs(w) + tol) + 1e-30
    bad = np.abs(g - w) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(g - w) / tol):.2f} of the bound"
    # In the 2-norm: up to three such roundings (two operands, the result), each
    # uniform within its half step, so of rms U / sqrt(3) of what it rounds, together
    # U of abs_sum, which is at most 20 times the result here.
    if s.size and np.linalg.norm(w) > 0.05 * np.linalg.norm(s):
        rel = np.linalg.norm(g - w) / np.linalg.norm(w)
        assert rel <= U * 20, f"{what}: rel {rel}"


def starts(lens, dev=None):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)


def ranges(lens):
    e = np.concatenate([[0], np.cumsum(lens)])
    return [(int(a), int(b)) for a, b in zip(e, e[1:])]


def rand(seed, *shape, unit=False, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * scale
    if unit:
        x = x / x.norm(dim=-1, keepdim=True)
    return x.to(torch.bfloat16)


def rand32(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def f64(t):
    return t.detach().double().cpu().numpy()


def slopes(H):
    return -torch.exp2(-8.0 * (torch.arange(H, dtype=torch.float32) + 1) / H)
