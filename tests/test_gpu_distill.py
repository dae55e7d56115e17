"""kronq_distill_fwd / _bwd / _step against the definition in fp64: padded
and repeated places, rows that do not count, infinities and NaN, odd widths
and strides, both logit types.

Bounds. A row's exponentials are off by (2 + |arg|) 2^-23 relative (the
argument is rounded once, base-2 exponentials are good to 2 ulp), their fp32
sum by the depth of its tree; lse and loss are fp64 from there."""
import math

import pytest
import torch

from ops_helpers import HALF_BF16, U32, close, kq

pytestmark = pytest.mark.gpu

# n, vocab, k
SIZES = [(1, 1, 1), (2, 7, 3), (5, 33, 33), (3, 1000, 16), (2, 4099, 64), (4, 8192, 1),
         (2, 32000, 100), (2, 50257, 17), (1, 65537, 1024), (2, 128256, 64), (1, 300001, 8)]

# rows of every kernel: 64, 128 and 384 threads, clusters, no cluster holds them
FAR_WIDTHS = [600, 9001, 20000, 70003, 300001]


def _case(n, vocab, k, dtype, seed, tdtype=torch.float32, pad=0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(n, vocab, generator=g, dtype=torch.float64) * 3).to(dtype)
    Z = torch.full((n, vocab + pad), math.nan, dtype=dtype)
    Z[:, :vocab] = z
    idx = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(n)])
    T = z.gather(1, idx).float() + torch.randn(n, k, generator=g)
    w = torch.rand(n, generator=g) + 0.1
    return (Z.cuda()[:, :vocab], T.to(tdtype).cuda(), idx.int().cuda(), w.cuda())


def _want(Z, T, idx, tau, w):
    """(loss, lse, dZ, q, p per entry) in fp64 from the definition."""
    z, t, n = Z.double(), T.double(), Z.shape[0]
    kept = (idx >= 0) & (idx < Z.shape[1]) & (t != -math.inf)
    counts = kept.any(1) & (w != 0)
    at = torch.where(kept, idx, 0).long()
    p = torch.softmax(torch.where(kept, t / tau, -math.inf), 1)
    p = torch.where(kept & counts[:, None], p, 0.0)
    m = z.amax(1, keepdim=True)
    lse = m[:, 0] / tau + ((z - m) / tau).exp().sum(1).log()
    logq = z / tau - lse[:, None]
    terms = torch.where(p > 0, p * (p.log() - logq.gather(1, at)), 0.0)
    loss = tau ** 2 * terms.sum(1)
    q = logq.exp()
    dz = w.double()[:, None] * tau * (q.scatter_add(1, at, -p))
    zero = torch.zeros((), dtype=torch.float64, device=Z.device)
    return (torch.where(counts, loss, zero), torch.where(counts, lse, zero),
            torch.where(counts[:, None], dz, zero), q, p, logq, counts)


def _bounds(Z, T, idx, tau, w, want):
    loss, lse, dz, q, p, logq, counts = want
    vocab, k = Z.shape[1], T.shape[1]
    # one exponential; the sum of them adds at most vocab / 256 + 32 roundings
    arg = logq.abs().clamp_max(200) * 1.4427
    e_exp = (3 + arg) * 2.0 ** -23
    e_lse = (q * e_exp).sum(1) + (vocab / 256 + 32) * U32
    b_lse = e_lse + U32 * lse.abs() * 2
    t = T.double()
    tm = torch.where(torch.isfinite(t), t, -1e30).amax(1, keepdim=True)
    e_p = (4 + k / 256 + ((t - tm).abs() / tau).clamp_max(200) * 2) * 2.0 ** -23
    at = idx.clamp(0, vocab - 1).long()
    gap = torch.where(p > 0, p.clamp_min(1e-300).log() - logq.gather(1, at), 0.0).abs()
    b_loss = tau ** 2 * (e_lse + (p * (e_p * (gap + 1))).sum(1) * 2) + U32 * 2 * loss.abs()
    step = HALF_BF16 if Z.dtype == torch.bfloat16 else U32
    # lse is stored in fp32 between the separate calls
    dq = q * (e_exp + e_lse[:, None] + 2 * U32 * lse.abs()[:, None] + 4 * U32)
    dq = dq.scatter_add(1, at, p * (e_p + 2 * U32) * (1 + k * U32))
    b_dz = (w.double() * tau)[:, None].abs() * dq
    # results that underflow (2^-126) may be flushed
    return (b_loss + 1e-37, b_lse + 1e-37,
            b_dz + step * (dz.abs() + b_dz) + 4 * U32 * dz.abs() + 1e-37)


def _run(Z, T, idx, tau, w, fused):
    K = kq()
    n, dev = Z.shape[0], Z.device
    loss, lse = torch.full((n,), 9.0, device=dev), torch.full((n,), 9.0, device=dev)
    buf = torch.full((n, Z.shape[1] + 5), 77.0, dtype=Z.dtype, device=dev)
    dZ = buf[:, :Z.shape[1]]
    info = torch.zeros(1, dtype=torch.int32, device=dev)
    if fused:
        K.kronq_distill_step(Z, T, idx, loss, lse, dZ, info, tau=tau, weight=w)
    else:
        K.kronq_distill_fwd(Z, T, idx, loss, lse, info, tau=tau, weight=w)
        K.kronq_distill_bwd(Z, T, idx, lse, dZ, info, tau=tau, weight=w)
    torch.cuda.synchronize()
    assert bool((buf[:, Z.shape[1]:] == 77).all())
    return loss, lse, dZ, info.item()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fused", [True, False])
def test_distill(cuda_device, size, dtype, fused):
    n, vocab, k = size
    tau = 0.5 + (vocab % 7) * 0.4
    Z, T, idx, w = _case(n, vocab, k, dtype, seed=vocab + k,
                         tdtype=torch.bfloat16 if k % 2 else torch.float32, pad=vocab % 5)
    if k > 4:
        idx[:, k // 2] = -1                      # padding inside the row
        idx[0, -1] = idx[0, 0]                   # the same place twice
    loss, lse, dZ, info = _run(Z, T, idx, tau, w, fused)
    assert info == 0
    want = _want(Z, T, idx, tau, w)
    b_loss, b_lse, b_dz = _bounds(Z, T, idx, tau, w, want)
    close(loss, want[0], b_loss)
    close(lse, want[1], b_lse)
    close(dZ, want[2], b_dz)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [(2500, 37, 5), (1300, 1501, 40), (700, 4500, 9),
                                  (200, 20003, 600)])
def test_forward_of_many_rows(cuda_device, size, dtype):
    """More rows than the chip takes at once, from few to many threads a row, some
    rows without weight; the logits start off 16-byte boundaries."""
    n, vocab, k = size
    Z, T, idx, w = _case(n, vocab, k, dtype, seed=vocab, pad=3)
    w[::7] = 0.0
    K = kq()
    loss, lse = torch.full((n,), 9.0, device="cuda"), torch.full((n,), 9.0, device="cuda")
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kronq_distill_fwd(Z, T, idx, loss, lse, info, tau=1.5, weight=w)
    torch.cuda.synchronize()
    assert info.item() == 0
    want = _want(Z, T, idx, 1.5, w)
    b_loss, b_lse, _ = _bounds(Z, T, idx, 1.5, w, want)
    close(loss, want[0], b_loss)
    close(lse, want[1], b_lse)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [(9, 50, 40), (3, 3000, 700), (2, 40000, 1024)])
def test_places_named_often(cuda_device, size, dtype):
    """Places that one to hundreds of entries name, next to places named once: each
    is written once, with the sum of its entries, and the same way every time."""
    n, vocab, k = size
    Z, T, idx, w = _case(n, vocab, min(k, vocab), dtype, seed=k)
    g = torch.Generator().manual_seed(vocab)
    hot = torch.randint(0, vocab, (n, k), generator=g)
    hot = torch.where(torch.rand(n, k, generator=g) < 0.3, hot % 5 + vocab // 2, hot)
    hot[:, k // 3:k // 3 + 6] = torch.arange(6) // 2 * (vocab // 4)   # pairs
    hot[0, :k // 2] = vocab - 1
    idx = hot.int().cuda()
    T = (Z.double().gather(1, idx.long()) + torch.randn(n, k, generator=g).cuda()).float()
    for fused in (True, False):
        loss, lse, dZ, info = _run(Z, T, idx, 2.0, w, fused)
        assert info == 0
        want = _want(Z, T, idx, 2.0, w)
        b_loss, b_lse, b_dz = _bounds(Z, T, idx, 2.0, w, want)
        close(loss, want[0], b_loss)
        close(lse, want[1], b_lse)
        close(dZ, want[2], b_dz)
        assert torch.equal(dZ, _run(Z, T, idx, 2.0, w, fused)[2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [321, 40000])
def test_rows_that_do_not_count(cuda_device, dtype, vocab):
    """Weight 0 (with NaN logits), nothing kept, teacher logits of -inf, and
    -inf student logits away from the teacher's places."""
    n, k = 6, 9
    Z, T, idx, w = _case(n, vocab, k, dtype, seed=3)
    w[1] = 0
    Z[1] = math.nan
    idx[2] = -1
    T[3] = -math.inf
    T[4, 2:] = -math.inf
    named = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    named[idx[5].long()] = True
    Z[5, ~named & (torch.arange(vocab, device="cuda") % 3 != 0)] = -math.inf
    want = _want(Z, T, idx, 1.5, w)
    b = _bounds(Z, T, idx, 1.5, w, want)
    for fused in (True, False):
        loss, lse, dZ, info = _run(Z, T, idx, 1.5, w, fused)
        assert info == 0
        for r in (1, 2, 3):
            assert loss[r] == 0 and lse[r] == 0 and not dZ[r].any()
        for r in (0, 4, 5):
            close(loss[r], want[0][r], b[0][r])
            close(lse[r], want[1][r], b[1][r])
            close(dZ[r], want[2][r], b[2][r])
        assert not dZ[5][Z[5] == -math.inf].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nonfinite_is_reported(cuda_device, dtype):
    """A NaN logit, a row of -inf, and a student -inf where the teacher has
    weight: reported, and the other rows are as without them."""
    K = kq()
    n, vocab, k = 4, 777, 5
    Z, T, idx, w = _case(n, vocab, k, dtype, seed=8)
    clean = _run(Z, T, idx, 1.0, w, True)
    assert clean[3] == 0
    for kind in ("nan", "row", "place"):
        Z2 = Z.clone()
        if kind == "nan":
            Z2[2, 100] = math.nan
        elif kind == "row":
            Z2[2] = -math.inf
        else:
            Z2[2, idx[2, 1].item()] = -math.inf
        for fused in (True, False):
            loss, lse, dZ, info = _run(Z2, T, idx, 1.0, w, fused)
            assert info == K.KRONQ_ERR_NONFINITE
            assert loss[2] == math.inf if kind == "place" else bool(loss[2].isnan())
            if kind == "place":
                assert bool(dZ[2].isfinite().all())
            else:
                assert bool(dZ[2].isnan().all())
            keep = [0, 1, 3]
            if fused:
                assert torch.equal(loss[keep], clean[0][keep])
                assert torch.equal(dZ[keep], clean[2][keep])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", FAR_WIDTHS)
def test_infinite_logit(cuda_device, dtype, vocab):
    """A logit of +inf, named by the teacher or not: loss (unless it is infinite), lse
    and gradient of its row are NaN and reported, the other rows as without it."""
    K = kq()
    n, k = 4, 5
    Z, T, idx, w = _case(n, vocab, k, dtype, seed=9)
    clean = _run(Z, T, idx, 1.5, w, True)
    for at in (0, vocab - 1, vocab // 2, int(idx[2, 1])):
        Z2 = Z.clone()
        Z2[2, at] = math.inf
        for fused in (True, False):
            loss, lse, dZ, info = _run(Z2, T, idx, 1.5, w, fused)
            assert info == K.KRONQ_ERR_NONFINITE
            assert not bool(loss[2].isfinite())
            assert bool(lse[2].isnan()) and bool(dZ[2].isnan().all())
            keep = [0, 1, 3]
            if fused:
                assert torch.equal(loss[keep], clean[0][keep])
                assert torch.equal(lse[keep], clean[1][keep])
                assert torch.equal(dZ[keep], clean[2][keep])


def test_place_outside_the_vocabulary(cuda_device):
    """Left out like padding, and reported."""
    K = kq()
    n, vocab, k = 3, 500, 6
    Z, T, idx, w = _case(n, vocab, k, torch.float32, seed=4)
    pad = idx.clone()
    idx[1, 2], pad[1, 2] = vocab, -1
    idx[2, 0], pad[2, 0] = 2 ** 31 - 1, -7
    got, want = _run(Z, T, idx, 2.0, w, True), _run(Z, T, pad, 2.0, w, True)
    assert got[3] == K.KRONQ_ERR_INVALID_ARG and want[3] == 0
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1001, 32000, 200000])
def test_in_place_and_without_weights(cuda_device, dtype, vocab):
    K = kq()
    n, k = 3, 12
    Z, T, idx, _ = _case(n, vocab, k, dtype, seed=6)
    ones = torch.ones(n, device="cuda")
    want = _run(Z, T, idx, 1.25, ones, True)
    split = _run(Z, T, idx, 1.25, ones, False)
    loss = torch.empty(n, device="cuda")
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    Z2 = Z.clone()
    K.kronq_distill_step(Z2, T, idx, loss, None, Z2, info, tau=1.25)
    Z3 = Z.clone()
    K.kronq_distill_bwd(Z3, T, idx, split[1], Z3, info, tau=1.25)
    torch.cuda.synchronize()
    assert info.item() == 0
    assert torch.equal(loss, want[0]) and torch.equal(Z2, want[2])
    assert torch.equal(Z3, split[2])


def test_large_logits_and_temperatures(cuda_device):
    """Logits of +-1e4 and the temperatures at the ends: a one-hot or a
    uniform student, no overflow."""
    n, vocab, k = 2, 600, 4
    for tau in (1e-4, 0.02, 1e4):
        Z, T, idx, w = _case(n, vocab, k, torch.float32, seed=2)
        Z = Z * 3000 if tau < 1 else Z
        T = T * 3000 if tau < 1 else T
        loss, lse, dZ, info = _run(Z, T, idx, tau, w, True)
        want = _want(Z, T, idx, tau, w)
        assert info == 0
        # an argument of up to 2^x magnitude is rounded to 2^(x-24) absolute:
        # scale the row's bounds by it (only the largest terms count)
        arg = float((Z.double().abs().max() / tau) * 1.4427)
        slack = 1 + arg * 2.0 ** -20
        b = _bounds(Z, T, idx, tau, w, want)
        close(lse, want[1], b[0] * 0 + b[1] * slack + U32 * 4 * want[1].abs())
        close(loss, want[0], b[0] * slack + 8 * U32 * tau ** 2 * arg)
        close(dZ, want[2], b[2] * slack + 8 * U32 * arg * 1e-3 * float(w.max()) * tau
              + 8 * U32 * float(w.max()) * tau)


def _far(Z, T, idx, tau, w):
    """What _step gives and its bounds, from differences to the row's maximum: lse
    itself may be too large to subtract, even in fp64."""
    z, m = Z.double(), Z.double().amax(1, keepdim=True)
    d = (z - m) / tau
    ls = d.exp().sum(1)
    logq = d - ls.log()[:, None]
    q = logq.exp()
    at = idx.long()
    p = torch.softmax(T.double() / tau, 1)
    terms = torch.where(p > 0, p * (p.log() - logq.gather(1, at)), 0.0)
    loss = tau ** 2 * terms.sum(1)
    lse = m[:, 0] / tau + ls.log()
    dz = w.double()[:, None] * tau * q.scatter_add(1, at, -p)
    none = torch.zeros_like(lse)   # (the step does not go through a stored lse)
    b_loss, b_lse, b_dz = _bounds(Z, T, idx, tau, w, (loss, none, dz, q, p, logq, None))
    return (loss, lse, dz), (b_loss, b_lse + 2 * U32 * lse.abs(), b_dz)


def _check_far(Z, T, idx, tau, w):
    K = kq()
    want, b = _far(Z, T, idx, tau, w)
    loss, lse, dZ, info = _run(Z, T, idx, tau, w, True)
    assert info == 0
    close(loss, want[0], b[0])
    close(lse, want[1], b[1])
    close(dZ, want[2], b[2])
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kronq_distill_fwd(Z, T, idx, loss, lse, info, tau=tau, weight=w)
    torch.cuda.synchronize()
    assert info.item() == 0
    close(loss, want[0], b[0])
    close(lse, want[1], b[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", FAR_WIDTHS)
@pytest.mark.parametrize("mask", [-1e9, -1e10, -1e20, -1e30])
def test_finite_masks(cuda_device, dtype, vocab, mask):
    """Whole slices of a row masked by a large negative logit, at its start, at its end
    and all but a few places: as the definition has it, which gives them nothing."""
    n, k = 4, 6
    Z, T, idx, w = _case(n, vocab, k, dtype, seed=vocab)
    named = torch.zeros(n, vocab, dtype=torch.bool, device="cuda")
    named.scatter_(1, idx.long(), True)
    place = torch.arange(vocab, device="cuda")
    for r, out in enumerate((place < vocab // 2, place > vocab // 3, place != 5, place % 9 > 0)):
        Z[r, out & ~named[r]] = mask
    for tau in (1.0, 2.5, 0.125):
        _check_far(Z, T, idx, tau, w)
        want = _want(Z, T, idx, tau, w)
        b = _bounds(Z, T, idx, tau, w, want)
        loss, lse, dZ, info = _run(Z, T, idx, tau, w, False)
        assert info == 0
        close(loss, want[0], b[0])
        close(lse, want[1], b[1])
        close(dZ, want[2], b[2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", FAR_WIDTHS)
def test_masks_below_the_border(cuda_device, dtype, vocab):
    """A logit below -1e32 is -inf wherever it stands: at a place that the teacher
    names the loss is infinite and reported, and the gradient is that of -inf."""
    K = kq()
    n, k = 4, 5
    Z, T, idx, w = _case(n, vocab, k, dtype, seed=vocab + 1)
    place = torch.arange(vocab, device="cuda")
    for low in (-1.1e32, -1e35, torch.finfo(dtype).min):
        for tau in (0.5, 4.0):
            A, B = Z.clone(), Z.clone()
            named = torch.zeros(n, vocab, dtype=torch.bool, device="cuda")
            named.scatter_(1, idx.long(), True)
            out = (place < vocab // 2)[None, :] & ~named
            out[2, idx[2, 1]] = True
            A[out], B[out] = low, -math.inf
            for fused in (True, False):
                got, want = (_run(t, T, idx, tau, w, fused) for t in (A, B))
                assert got[3] == want[3] == K.KRONQ_ERR_NONFINITE and got[0][2] == math.inf
                assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))


@pytest.mark.parametrize("vocab", FAR_WIDTHS)
def test_logits_at_the_border(cuda_device, vocab):
    """-1e32 itself is a logit: a row of nothing above it has a softmax over the
    places that hold it."""
    n, k = 3, 4
    Z, T, idx, w = _case(n, vocab, k, torch.float32, seed=vocab + 2)
    Z[:] = -1e32
    named = torch.zeros(n, vocab, dtype=torch.bool, device="cuda")
    named.scatter_(1, idx.long(), True)
    Z[1, ~named[1] & (torch.arange(vocab, device="cuda") % 3 == 0)] = -math.inf
    Z[2, ~named[2]] = -2e32
    T = torch.randn(n, k, generator=torch.Generator().manual_seed(vocab)).cuda()
    _check_far(Z, T, idx, 2.0, w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", FAR_WIDTHS)
def test_logits_far_from_zero(cuda_device, dtype, vocab):
    """Rows around a value that is up to 1e10 and more temperatures from zero, of both
    signs: one maximum, several of them, a spread of neighbours, all the same."""
    n, k = 4, 5
    for top, tau in ((3584.0, 1e-4), (1e5, 1e-3), (1e6, 1e-4), (3e9, 1.0), (1e10, 1.0),
                     (1e10, 1e4), (1e20, 1e4), (4e31, 1e-4), (4e31, 1e4)):
        tau = float(torch.tensor(tau, dtype=torch.float32))
        for sign in (1, -1):
            g = torch.Generator().manual_seed(vocab)
            step = torch.finfo(dtype).eps / 2 * top
            Z = torch.full((n, vocab), sign * top, dtype=torch.float64)
            Z[0] -= top * torch.rand(vocab, generator=g)
            Z[0, 77] = (sign + 0.05) * top
            Z[1] -= 0.3 * top * (torch.arange(vocab) % 7 != 3)
            Z[2] -= 2 * step * torch.randint(0, 6, (vocab,), generator=g)
            Z = Z.to(dtype).cuda()
            idx = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(n)]).int()
            idx[:, 1] = 77
            idx[:, 2] = torch.where(idx[:, 2] == 77, 78, idx[:, 2])
            T = torch.randn(n, k, generator=g) * tau
            w = torch.rand(n, generator=g) + 0.1
            _check_far(Z, T.cuda(), idx.cuda(), tau, w.cuda())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", FAR_WIDTHS)
def test_backward_from_a_large_lse(cuda_device, dtype, vocab):
    """The backward pass alone is exp(z / tau - lse) for the lse that it is given, also
    where fp32 holds that no closer than to a few tens.
    Bound: the exponent is (z - m) c + shift with m = tau lse in fp32; z - m and its
    product with c are off by 3 2^-24 of at most |arg| + |shift|, |shift| <= 2^-24 |lse|
    log2(e); fp64 keeps tau lse to 2^-53."""
    K = kq()
    n, k = 4, 5
    for top, tau in ((1e5, 1e-2), (3584.0, 1e-4), (1e5, 1e-3), (2e12, 1e4), (3e4, 1e-4),
                     (1e9, 1.0)):
        tau = float(torch.tensor(tau, dtype=torch.float32))
        for sign in (1, -1):
            g = torch.Generator().manual_seed(vocab)
            Z = torch.full((n, vocab), sign * top, dtype=torch.float64)
            Z -= torch.finfo(dtype).eps * top * torch.randint(0, 4, (n, vocab), generator=g)
            Z[0] -= 0.2 * top * (torch.arange(vocab) % 50 != 3)
            Z = Z.to(dtype).cuda()
            idx = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(n)])
            idx = idx.int().cuda()
            T = (torch.randn(n, k, generator=g) * tau).cuda()
            w = (torch.rand(n, generator=g) + 0.1).cuda()
            z, m = Z.double(), Z.double().amax(1, keepdim=True)
            lse = (m[:, 0] / tau + ((z - m) / tau).exp().sum(1).log()).float()
            dZ, info = torch.empty_like(Z), torch.zeros(1, dtype=torch.int32, device="cuda")
            K.kronq_distill_bwd(Z, T, idx, lse, dZ, info, tau=tau, weight=w)
            torch.cuda.synchronize()
            assert info.item() == 0
            logq = z / tau - lse.double()[:, None]
            q, p = logq.exp(), torch.softmax(T.double() / tau, 1)
            wt = (w.double() * tau)[:, None]
            want = wt * q.scatter_add(1, idx.long(), -p)
            big = lse.double().abs()[:, None]
            arg = (logq.abs() + 2 * 2.0 ** -24 * big) * 1.4427
            e_q = q * ((3 + arg.clamp_max(300)) * 2.0 ** -23 + 2.0 ** -50 * big)
            tm = T.double().amax(1, keepdim=True)
            e_p = p * (4 + (T.double() - tm).abs() / tau * 2) * 2.0 ** -23
            # a q below 2^-126 is flushed to 0 before wt multiplies it: off by at most
            # wt 2^-126 (with tau = 1e4 more than the 1e-37 of the last line)
            e = wt * (e_q.scatter_add(1, idx.long(), e_p) + 2.0 ** -126)
            step = HALF_BF16 if dtype == torch.bfloat16 else U32
            close(dZ, want, e + step * (want.abs() + e) + 4 * U32 * want.abs() + 1e-37)


def test_gradient_against_differences(cuda_device):
    """dZ against central differences of the fp64 loss."""
    n, vocab, k, tau, h = 2, 50, 6, 1.7, 1e-4
    Z, T, idx, w = _case(n, vocab, k, torch.float32, seed=12)
    idx[0, 1] = idx[0, 0]
    dZ = _run(Z, T, idx, tau, w, True)[2].double()

    def total(z):
        return float((w.double() * _want(z, T, idx, tau, w)[0]).sum())

    z = Z.double()
    for r, v in [(0, int(idx[0, 0])), (0, int(idx[0, 3])), (1, int(idx[1, 5])), (1, 0), (0, 49)]:
        p, m = z.clone(), z.clone()
        p[r, v] += h
        m[r, v] -= h
        # differences: O(h^2) and rounding of fp64 losses; dZ: fp32
        assert abs(float(dZ[r, v]) - (total(p) - total(m)) / (2 * h)) <= 1e-6


def test_streams_graphs_and_repeats(cuda_device):
    K = kq()
    n, vocab, k = 40, 9001, 20
    Z, T, idx, w = _case(n, vocab, k, torch.bfloat16, seed=5)
    want = _run(Z, T, idx, 1.0, w, True)
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    dZ = torch.empty_like(Z)
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    K.kronq_distill_step(Z, T, idx, loss, lse, dZ, info, weight=w, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(dZ, want[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kronq_distill_step(Z, T, idx, loss, lse, dZ, info, weight=w)
    dZ.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(dZ, want[2]) and info.item() == 0


def test_no_rows(cuda_device):
    K = kq()
    e = torch.empty(0, 100, device="cuda")
    T, idx = torch.empty(0, 3, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda")
    v, info = torch.empty(0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kronq_distill_step(e, T, idx, v, v, torch.empty(0, 100, device="cuda"), info)
    torch.cuda.synchronize()
    assert info.item() == 0


def test_binding_refuses(cuda_device):
    K = kq()
    Z, T, idx, w = _case(4, 90, 5, torch.float32, seed=1)
    loss, lse = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        K.kronq_distill_fwd(Z, T, idx.long(), loss, lse, info)
    with pytest.raises(TypeError):
        K.kronq_distill_fwd(Z.half(), T, idx, loss, lse, info)
    with pytest.raises(ValueError):
        K.kronq_distill_fwd(Z, T[:, :4], idx, loss, lse, info)
    with pytest.raises(ValueError):
        K.kronq_distill_fwd(Z, T, idx, loss[:3], lse, info)
    for tau in (0.0, -1.0, math.inf, math.nan, 1e-5):
        with pytest.raises(K.KronqError) as err:
            K.kronq_distill_fwd(Z, T, idx, loss, lse, info, tau=tau)
        assert err.value.status == K.KRONQ_ERR_INVALID_ARG
    wide = torch.empty(4, 200, device="cuda")
    with pytest.raises(K.KronqError) as err:     # dZ shifted over Z
        K.kronq_distill_bwd(wide[:, :90], T, idx, lse, wide[:, 10:100], info)
    assert err.value.status == K.KRONQ_ERR_INVALID_ARG
    big = torch.zeros(1, 1025, device="cuda")
    with pytest.raises(K.KronqError) as err:     # k > 1024
        K.kronq_distill_fwd(big, big, big.int(), loss[:1], lse[:1], info)
    assert err.value.status == K.KRONQ_ERR_UNSUPPORTED
