"""The calibration pass of a feed-forward block: products, distillation loss,
backward pass and covariances together, against the same pass in fp64.

Tolerances: every tensor of the chain is rounded to bf16 once (relative error
at most 2^-8 an element, so at most 2^-8 of its norm), and the chain from X to
the last gradient rounds nine (A, U, H, Y, logits, dlogits, dY, dH, G). The
errors of the earlier ones pass through maps whose gains the inputs keep below
2; a gradient is then within 9 * 2 * 2^-8 = 7 % of its norm, and a covariance,
quadratic in its rows, within twice that. Measured errors are about a tenth."""
import pytest
import torch

from ops_helpers import act64, kq, matrix

pytestmark = pytest.mark.gpu
TOL = 9 * 2 * 2.0 ** -8


def _block(d, f, vocab, seed=0):
    Wg, Wu = (matrix(f, d, seed + j, d ** -0.5) for j in (1, 2))
    Wd, Wh = matrix(d, f, seed + 3, f ** -0.5), matrix(vocab, d, seed + 4, 2.0 * d ** -0.5)
    return Wg, Wu, Wd, Wh


def _batch(n, d, vocab, k, seed):
    g = torch.Generator().manual_seed(seed)
    X = matrix(n, d, seed + 50)
    idx = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(n)]).int()
    T = torch.randn(n, k, generator=g) * 2
    idx[::3, -1] = -1
    w = (torch.rand(n, generator=g) < 0.8).float() / n
    w[0] = 1.0 / n
    return X, T.cuda(), idx.cuda(), w.cuda()


def _reference(W, batch, act, tau):
    Wg, Wu, Wd, Wh = (t.double() for t in W)
    X, T, idx, w = batch
    x = X.double()
    a, u = x @ Wg.T, x @ Wu.T
    s, ds = act64(a, act)
    h = s * u
    y = h @ Wd.T + x
    z = y @ Wh.T
    kept = idx >= 0
    at = torch.where(kept, idx, 0).long()
    p = torch.softmax(torch.where(kept, T.double() / tau, -torch.inf), 1)
    logq = torch.log_softmax(z / tau, 1)
    loss = tau ** 2 * torch.where(p > 0, p * (p.log() - logq.gather(1, at)), 0.0).sum(1)
    dz = w.double()[:, None] * tau * logq.exp().scatter_add(1, at, -p)
    dy = dz @ Wh
    dh = dy @ Wd
    gg, gu = dh * u * ds, dh * s
    dx = gg @ Wg + gu @ Wu + dy
    return dict(loss=torch.where(w > 0, loss, 0.0), X=x, H=h, Gg=gg, Gu=gu, dY=dy, dX=dx)


def _near(got, want, tol):
    err = float((got.double() - want).norm() / want.norm())
    assert err <= tol, err


def _covs(refs, total):
    cov = lambda k: sum(r[k].T @ r[k] for r in refs) / total  # noqa: E731
    return {"mlp": cov("X"), "down": cov("H")}, {"gate": cov("Gg"), "up": cov("Gu"),
                                                 "down": cov("dY")}


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_calibration_pass(cuda_device, act):
    """Two batches of unequal size, the second not filling a tile."""
    kq()
    from second_order_post_b200.calib import FeedForwardCalibration
    d, f, vocab, k, tau = 256, 640, 1003, 12, 1.5
    W = _block(d, f, vocab)
    batches = [_batch(300, d, vocab, k, 1), _batch(77, d, vocab, k, 2)]
    cal = FeedForwardCalibration(*W, max_tokens=300, tokens=377, act=act, tau=tau)
    refs = []
    for b in batches:
        loss, dX = cal.step(*b)
        torch.cuda.synchronize()
        cal.check_info()
        ref = _reference(W, b, act, tau)
        refs.append(ref)
        # loss: logits off by 2^-8 relative of |z| <= 16
        assert float((loss.double() - ref["loss"]).abs().max()) <= tau * 16 * 4 * 2.0 ** -8
        _near(dX, ref["dX"], TOL)
    hx, hg = _covs(refs, 377)
    for name, want in hx.items():
        _near(cal.H_X[name], want, 2 * TOL)
    for name, want in hg.items():
        _near(cal.H_G[name], want, 2 * TOL)
    assert torch.equal(cal.H_G["gate"], cal.H_G["gate"].T)


def test_calibrated_block_is_quantized(cuda_device):
    """The covariances feed the quantizer: every sublayer of the block comes out
    finite and near its weights at 4 bits."""
    K = kq()
    from second_order_post_b200.calib import FeedForwardCalibration
    from second_order_post_b200.engine import SublayerEngine
    d, f, vocab, n = 256, 384, 520, 512
    W = _block(d, f, vocab, seed=20)
    cal = FeedForwardCalibration(*W, max_tokens=n, tokens=n)
    cal.step(*_batch(n, d, vocab, 8, 5))
    for sub in ("gate", "up", "down"):
        d_out, d_in = cal.weight(sub).shape
        eng = SublayerEngine(d_out, d_in, bits=4, rot_in=(d_in // 3, 3) if d_in % 3 == 0
                             else (d_in, 1), rot_out=(d_out // 3, 3) if d_out % 3 == 0
                             else (d_out, 1), keep_w_rot=True, damp_rel=0.01)
        res = cal.quantize(sub, eng)
        torch.cuda.synchronize()
        eng.check_info()
        cal.check_info()
        assert bool(res.w_hat.isfinite().all())
        rel = float((res.w_hat - eng.W_ref).norm() / eng.W_ref.norm())
        assert 0 < rel < 0.5
    with pytest.raises(ValueError):
        cal.covariances("q")
    assert K.kronq_kernel_launches() > 0


def test_two_passes_captured(cuda_device):
    """Two calibrations captured into graphs and replayed alternately on new
    tokens give what eager calls give (no state is shared)."""
    kq()
    from second_order_post_b200.calib import FeedForwardCalibration
    d, f, vocab, n = 128, 256, 300, 40
    W = _block(d, f, vocab, seed=40)
    cals = [FeedForwardCalibration(*W, max_tokens=n, tokens=n) for _ in range(3)]
    ins = [list(_batch(n, d, vocab, 6, s)) for s in (1, 2)]
    for c, b in zip(cals, ins):      # kernels are loaded before the capture
        c.step(*b)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, b in zip(cals, ins):
        c._first = True
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.step(*b))
        graphs.append(g)
    new = [_batch(n, d, vocab, 6, s) for s in (7, 8)]
    for b, m in zip(ins, new):
        for t, s in zip(b, m):
            t.copy_(s)
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for c, b, (loss, dX) in zip(cals, new, outs):
        eager = cals[2]
        eager._first = True
        want_loss, want_dX = eager.step(*b)
        torch.cuda.synchronize()
        assert torch.equal(loss, want_loss) and torch.equal(dX, want_dX)
        for k in c.H_X:
            assert torch.equal(c.H_X[k], eager.H_X[k])
        for k in c.H_G:
            assert torch.equal(c.H_G[k], eager.H_G[k])
        c.check_info()


def test_on_another_stream_and_refusals(cuda_device):
    K = kq()
    from second_order_post_b200.calib import FeedForwardCalibration
    d, f, vocab, n = 128, 128, 100, 16
    W = _block(d, f, vocab, seed=60)
    b = _batch(n, d, vocab, 4, 3)
    cal, other = (FeedForwardCalibration(*W, max_tokens=n, tokens=n) for _ in range(2))
    want = [t.clone() for t in cal.step(*b)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = other.step(*b, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    with pytest.raises(ValueError):
        cal.step(torch.empty(n + 1, d, dtype=torch.bfloat16, device="cuda"), *b[1:])
    with pytest.raises(ValueError):
        FeedForwardCalibration(W[0], W[1], W[2], W[3][:, :64], max_tokens=4, tokens=4)
    with pytest.raises(ValueError):
        FeedForwardCalibration(*_block(96, 128, 50), max_tokens=4, tokens=4)
    bad = b[0].clone()
    bad[3, 5] = float("nan")
    cal.step(bad, *b[1:])
    with pytest.raises(K.KronqError) as err:      # the loss of that token
        cal.check_info()
    assert err.value.status == K.KRONQ_ERR_NONFINITE


def test_failure_of_an_early_batch_is_reported(cuda_device, monkeypatch):
    """A covariance's status of the first of two batches is there after the second
    (the library's wait that runs out stands for a pipeline's)."""
    K = kq()
    from second_order_post_b200.calib import FeedForwardCalibration
    d, f, vocab, n = 128, 128, 100, 16
    cal = FeedForwardCalibration(*_block(d, f, vocab, seed=80), max_tokens=n, tokens=2 * n)
    accum, done = K.kronq_accum_cov, []

    def second_fails(A, H, alpha, beta, info, stream=None):
        accum(A, H, alpha, beta, info, stream)
        done.append(1)
        if len(done) == 2:
            K.kronq_selftest_timeout(1000, info, stream)

    monkeypatch.setattr(K, "kronq_accum_cov", second_fails)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for seed in (1, 2):
        cal.step(*_batch(n, d, vocab, 4, seed), stream=side)
    torch.cuda.synchronize()
    assert len(done) == 10
    with pytest.raises(K.KronqError) as err:
        cal.check_info()
    assert err.value.status == K.KRONQ_ERR_TIMEOUT


def test_captured_before_anything_ran(cuda_device):
    """A step captured as the first one adds at every replay, also behind an eager step
    that came between; after a reset the sums start anew."""
    kq()
    from second_order_post_b200.calib import FeedForwardCalibration
    d, f, vocab, n = 128, 256, 300, 40
    W = _block(d, f, vocab, seed=90)
    warm, cal, want = (FeedForwardCalibration(*W, max_tokens=n, tokens=4 * n) for _ in range(3))
    a, b = (_batch(n, d, vocab, 6, s) for s in (1, 2))
    warm.step(*a)                # kernels are loaded before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cal.step(*a)

    def same(batches):
        want.reset()
        for x in batches:
            want.step(*x)
        torch.cuda.synchronize()
        want.check_info()
        cal.check_info()
        for k in want.H_X:
            assert torch.equal(cal.H_X[k], want.H_X[k])
        for k in want.H_G:
            assert torch.equal(cal.H_G[k], want.H_G[k])

    cal.step(*b)
    g.replay()
    g.replay()
    same([b, a, a])
    cal.reset()
    g.replay()
    same([a])
    both = torch.cuda.CUDAGraph()
    with torch.cuda.graph(both):
        cal.reset()
        cal.step(*b)
    both.replay()
    both.replay()
    same([b])


def test_quantized_on_another_stream(cuda_device):
    """The quantizer's calls and the copies around them keep to the stream given."""
    kq()
    from second_order_post_b200.calib import FeedForwardCalibration
    from second_order_post_b200.engine import SublayerEngine
    d, f, vocab, n = 256, 384, 520, 512
    cal = FeedForwardCalibration(*_block(d, f, vocab, seed=20), max_tokens=n, tokens=n)
    cal.step(*_batch(n, d, vocab, 8, 5))
    want, got = (SublayerEngine(d, f, bits=4, rot_in=(128, 3), keep_w_rot=True) for _ in range(2))
    cal.quantize("down", want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    cal.quantize("down", got, stream=side)
    side.synchronize()
    got.check_info()
    assert torch.equal(got.W_ref, want.W_ref) and torch.equal(got.W_rot, want.W_rot)
    assert torch.equal(got.codes, want.codes)


def test_one_token_of_any_stride(cuda_device):
    kq()
    from second_order_post_b200.calib import FeedForwardCalibration
    d, f, vocab = 128, 256, 100
    W = _block(d, f, vocab, seed=70)
    X, *rest = _batch(1, d, vocab, 4, 1)
    cals = [FeedForwardCalibration(*W, max_tokens=2, tokens=1) for _ in range(2)]
    odd = X.reshape(-1).as_strided((1, d), (3, 1))
    for cal, x in zip(cals, (X, odd)):
        cal.step(x, *rest)
    torch.cuda.synchronize()
    for cal in cals:
        cal.check_info()
    for k in cals[0].H_X:
        assert torch.equal(cals[0].H_X[k], cals[1].H_X[k])
    assert float(cals[0].H_X["mlp"].trace()) > 0


def test_status_of_a_pass_still_under_way(cuda_device):
    """check_info right behind a step on another stream that has not started yet."""
    K = kq()
    from second_order_post_b200.calib import FeedForwardCalibration
    d, f, vocab, n = 128, 128, 100, 16
    cal = FeedForwardCalibration(*_block(d, f, vocab, seed=60), max_tokens=n, tokens=n)
    batch = _batch(n, d, vocab, 4, 3)
    side = torch.cuda.Stream()
    cal.step(*batch, stream=side)         # kernels are loaded
    cal.check_info()
    batch[0][2, 7] = float("nan")
    batch[3][2] = 1.0
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(1e8))       # some 50 ms
    cal.step(*batch, stream=side)
    with pytest.raises(K.KronqError) as err:
        cal.check_info()
    assert err.value.status == K.KRONQ_ERR_NONFINITE
