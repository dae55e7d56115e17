"""Plain 64-bit forms of the calibration-pass operators and their error
bounds (test infrastructure only)."""
import math

import torch

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
HALF_BF16 = 2.0 ** -8          # half a step of bf16, relative to the value
U32 = 2.0 ** -24


def kq():
    from second_order_post_b200 import kronq
    return kronq


def act64(z, act):
    """(act(z), act'(z)) in fp64."""
    if act == "relu":
        return z.clamp_min(0), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        v = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        # (1 + tanh v) / 2 = 1 / (1 + exp(-2 v)): where v < -15 the sum on the
        # left keeps fewer than 3 digits even in fp64 (1 + tanh(-15) = 2e-13)
        s = torch.sigmoid(2 * v)
        dv = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
        return z * s, s + z * 2 * s * (1 - s) * dv
    return z, torch.ones_like(z)


def matrix(rows, cols, seed, scale=1.0, pad=0, device="cuda"):
    """A seeded rows x cols bf16 view of a wider buffer whose other elements
    are NaN (row stride: the next multiple of 8, plus 8 * pad)."""
    g = torch.Generator().manual_seed(seed)
    ld = (cols + 7) // 8 * 8 + 8 * pad
    buf = torch.full((rows, ld), math.nan, dtype=torch.bfloat16)
    buf[:, :cols] = (torch.randn(rows, cols, generator=g, dtype=torch.float64) * scale).bfloat16()
    return buf.to(device)[:, :cols]


def out_like(rows, cols, pad=0, device="cuda"):
    """An output view filled with a mark, and the buffer that holds it."""
    ld = (cols + 7) // 8 * 8 + 8 * pad
    buf = torch.full((rows, ld), 77.0, dtype=torch.bfloat16, device=device)
    return buf[:, :cols], buf


def untouched(buf, cols):
    return bool((buf[:, cols:] == 77.0).all())


def acc_bound(a, b):
    """Bound of |fp32 accumulation - exact| for A Bᵀ of bf16 operands (a: M x K,
    b: N x K, fp64): the products are exact; a tensor-core step over 16 of
    them drops less than 2^-23 of the largest magnitude it handles per
    addend (16 + 1 of them), which is at most the running sum of |a b|."""
    k = a.shape[1]
    return (k / 16 + 18) * 2.0 ** -23 * (a.abs() @ b.abs().T)


def close(got, want, tol):
    """Every element within its tolerance (both finite)."""
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (
        f"{int(bad.sum())} of {bad.numel()} off; worst {float((err / tol).max()):.3g} of its bound")
