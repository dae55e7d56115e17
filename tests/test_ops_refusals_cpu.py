"""Calls of the calibration-pass operators that the library refuses before it
touches a device: bad sizes, missing or misaligned matrices, short or odd
strides, overlapping outputs. (n = 0 with nothing to write returns OK.)"""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "second_order_post_b200", "libkronq.so")
MB = 1 << 20


@pytest.fixture(scope="module")
def K():
    if not os.path.exists(LIB):
        from second_order_post_b200 import build
        build.build()
    from second_order_post_b200 import kronq
    return kronq


def _p(v):
    return ctypes.c_void_p(v)


LIN = dict(X=16 * MB, n=8, d_in=64, ldx=64, W=32 * MB, d_out=40, ldw=64, bias=0, act=0, Z=0,
           ldz=40, R=0, ldr=40, Y=48 * MB, ldy=40, info=64)
LINB = dict(dY=16 * MB, lddy=40, Z=20 * MB, ldz=40, act=2, X=24 * MB, ldx=64, W=28 * MB, ldw=64,
            n=8, d_in=64, d_out=40, dZ=32 * MB, lddz=40, db=0, dXr=0, lddxr=64, dX=36 * MB,
            lddx=64, dW=40 * MB, lddw=64, info=64)
GAT = dict(X=16 * MB, n=8, d=64, ldx=64, Wg=20 * MB, Wu=24 * MB, f=40, ldw=64, act=2, A=0, U=0,
           ldau=40, H=28 * MB, ldh=40, info=64)
GATB = dict(dH=16 * MB, lddh=40, A=17 * MB, U=18 * MB, ldau=40, act=2, X=19 * MB, ldx=64,
            Wg=20 * MB, Wu=21 * MB, ldw=64, n=8, d=64, f=40, Gg=22 * MB, Gu=23 * MB, ldg=40,
            dXr=0, lddxr=64, dX=24 * MB, lddx=64, dWg=25 * MB, dWu=26 * MB, lddw=64, info=64)
DFW = dict(Z=16 * MB, zdt=1, n=4, vocab=100, ldz=100, T=20 * MB, tdt=0, idx=21 * MB, k=5, ldt=5,
           tau=1.0, weight=0, loss=22 * MB, lse=23 * MB, info=64)
DBW = dict(Z=16 * MB, zdt=1, n=4, vocab=100, ldz=100, T=20 * MB, tdt=0, idx=21 * MB, k=5, ldt=5,
           tau=1.0, weight=0, lse=23 * MB, dZ=24 * MB, lddz=100, info=64)
DST = dict(Z=16 * MB, zdt=1, n=4, vocab=100, ldz=100, T=20 * MB, tdt=0, idx=21 * MB, k=5, ldt=5,
           tau=1.0, weight=0, loss=22 * MB, lse=23 * MB, dZ=24 * MB, lddz=100, info=64)
BASE = {"kronq_linear": LIN, "kronq_linear_bwd": LINB, "kronq_gated": GAT,
        "kronq_gated_bwd": GATB, "kronq_distill_fwd": DFW, "kronq_distill_bwd": DBW,
        "kronq_distill_step": DST}
INV, UNS = 1, 2

CASES = [
    ("kronq_linear", dict(X=0), INV), ("kronq_linear", dict(W=0), INV),
    ("kronq_linear", dict(Y=0), INV), ("kronq_linear", dict(info=0), INV),
    ("kronq_linear", dict(n=-1), INV), ("kronq_linear", dict(d_in=0), INV),
    ("kronq_linear", dict(d_out=0), INV), ("kronq_linear", dict(act=5), INV),
    ("kronq_linear", dict(act=-1), INV), ("kronq_linear", dict(ldx=56), INV),
    ("kronq_linear", dict(ldy=32), INV), ("kronq_linear", dict(R=60 * MB, ldr=39), INV),
    ("kronq_linear", dict(bias=3), INV),
    ("kronq_linear", dict(ldx=65), UNS), ("kronq_linear", dict(X=16 * MB + 2), UNS),
    ("kronq_linear", dict(W=32 * MB + 8), UNS), ("kronq_linear", dict(ldy=44), UNS),
    ("kronq_linear", dict(Z=60 * MB, ldz=41), UNS), ("kronq_linear", dict(R=60 * MB + 2), UNS),
    ("kronq_linear", dict(n=2 ** 30 + 1), INV),          # rows reach over W and Y
    ("kronq_linear", dict(Y=16 * MB), INV), ("kronq_linear", dict(Y=32 * MB + 128), INV),
    ("kronq_linear", dict(Z=48 * MB), INV), ("kronq_linear", dict(R=48 * MB + 80), INV),
    ("kronq_linear", dict(R=48 * MB, ldr=48), INV), ("kronq_linear", dict(Z=60 * MB, R=60 * MB), INV),
    ("kronq_linear", dict(bias=48 * MB), INV),
    ("kronq_linear_bwd", dict(dY=0), INV), ("kronq_linear_bwd", dict(Z=0), INV),
    ("kronq_linear_bwd", dict(dZ=0), INV), ("kronq_linear_bwd", dict(X=0), INV),
    ("kronq_linear_bwd", dict(W=0), INV), ("kronq_linear_bwd", dict(dX=0, dXr=50 * MB), INV),
    ("kronq_linear_bwd", dict(dW=28 * MB), INV), ("kronq_linear_bwd", dict(dX=24 * MB), INV),
    ("kronq_linear_bwd", dict(dZ=16 * MB + 16), INV), ("kronq_linear_bwd", dict(dX=32 * MB), INV),
    ("kronq_linear_bwd", dict(dXr=36 * MB + 16, lddxr=64), INV),
    ("kronq_linear_bwd", dict(db=40 * MB), INV), ("kronq_linear_bwd", dict(db=42 * MB + 1), INV),
    ("kronq_linear_bwd", dict(lddw=63), INV), ("kronq_linear_bwd", dict(lddw=68), UNS),
    ("kronq_linear_bwd", dict(dZ=32 * MB + 4), UNS),
    ("kronq_gated", dict(Wu=0), INV), ("kronq_gated", dict(A=40 * MB), INV),
    ("kronq_gated", dict(A=40 * MB, U=40 * MB), INV), ("kronq_gated", dict(H=20 * MB), INV),
    ("kronq_gated", dict(ldw=60), INV), ("kronq_gated", dict(ldw=68), UNS),
    ("kronq_gated", dict(A=40 * MB, U=41 * MB, ldau=43), UNS),
    ("kronq_gated", dict(act=9), INV), ("kronq_gated", dict(f=0), INV),
    ("kronq_gated_bwd", dict(A=0), INV), ("kronq_gated_bwd", dict(Gu=0), INV),
    ("kronq_gated_bwd", dict(Gu=22 * MB), INV), ("kronq_gated_bwd", dict(dWu=0), INV),
    ("kronq_gated_bwd", dict(X=0), INV), ("kronq_gated_bwd", dict(Wg=0), INV),
    ("kronq_gated_bwd", dict(Gg=17 * MB, ldg=48), INV), ("kronq_gated_bwd", dict(dX=19 * MB), INV),
    ("kronq_gated_bwd", dict(dWg=26 * MB), INV), ("kronq_gated_bwd", dict(ldg=42), UNS),
    ("kronq_distill_fwd", dict(Z=0), INV), ("kronq_distill_fwd", dict(T=0), INV),
    ("kronq_distill_fwd", dict(idx=0), INV), ("kronq_distill_fwd", dict(loss=0), INV),
    ("kronq_distill_fwd", dict(lse=0), INV), ("kronq_distill_fwd", dict(zdt=2), INV),
    ("kronq_distill_fwd", dict(tdt=-1), INV), ("kronq_distill_fwd", dict(vocab=0), INV),
    ("kronq_distill_fwd", dict(ldz=99), INV), ("kronq_distill_fwd", dict(k=0), INV),
    ("kronq_distill_fwd", dict(ldt=4), INV), ("kronq_distill_fwd", dict(tau=0.0), INV),
    ("kronq_distill_fwd", dict(tau=float("nan")), INV),
    ("kronq_distill_fwd", dict(k=1025, ldt=1025), UNS),
    ("kronq_distill_fwd", dict(Z=16 * MB + 1), INV), ("kronq_distill_fwd", dict(weight=2), INV),
    ("kronq_distill_fwd", dict(loss=23 * MB), INV), ("kronq_distill_fwd", dict(loss=20 * MB), INV),
    ("kronq_distill_bwd", dict(lse=0), INV), ("kronq_distill_bwd", dict(dZ=0), INV),
    ("kronq_distill_bwd", dict(dZ=16 * MB + 2), INV), ("kronq_distill_bwd", dict(dZ=20 * MB), INV),
    ("kronq_distill_bwd", dict(dZ=16 * MB, lddz=104), INV),
    ("kronq_distill_bwd", dict(lddz=90), INV),
    ("kronq_distill_step", dict(loss=0), INV), ("kronq_distill_step", dict(dZ=0), INV),
    ("kronq_distill_step", dict(n=-1), INV), ("kronq_distill_step", dict(lse=24 * MB), INV),
    # nothing to do
    ("kronq_linear", dict(n=0, X=0, Y=0), 0), ("kronq_gated", dict(n=0, X=0, H=0), 0),
]


def _call(K, fn, args):
    lib = K._lib
    kinds = K._SIGS[fn]
    vals = [None] + list(args.values())
    assert len(vals) == len(kinds)
    conv = [_p(v or 0) if t is ctypes.c_void_p else v for v, t in zip(vals, kinds)]
    return getattr(lib, fn)(*conv)


@pytest.mark.parametrize("fn,change,status", CASES)
def test_refused(K, fn, change, status):
    base = BASE[fn]
    assert set(change) <= set(base)
    assert _call(K, fn, {**base, **change}) == status


def test_binding_wants_cuda_tensors(K):
    import torch
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    info = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        K.kronq_linear(x, x, x, info)
    with pytest.raises(ValueError):
        K.kronq_gated(x, x, x, x, info)
    with pytest.raises(ValueError):
        K.kronq_distill_fwd(x, x, x, x, x, info)


@pytest.mark.parametrize("rows,stride", [(1, 1), (1, 129), (1, 1000), (2, 136), (0, 128)])
def test_covariance_of_a_single_row(K, monkeypatch, rows, stride):
    """The stride of one row is not looked at, as in the products before it."""
    import torch
    got = []
    monkeypatch.setattr(K._lib, "kronq_accum_cov", lambda *a: got.append(a[3:6]) or 0)
    monkeypatch.setattr(K, "_stream", lambda s: None)
    A = torch.zeros(1024, dtype=torch.bfloat16).as_strided((rows, 128), (stride, 1))
    info = torch.zeros(1, dtype=torch.int32)
    K.kronq_accum_cov(A, torch.zeros(128, 128), 1.0, 0.0, info)
    assert got == [(rows, 128, stride if rows > 1 else 128)]
