"""What the calibration pass does around the library's calls: status words over
several batches, the start of the sums. The calls themselves are stood in for."""
import pytest
import torch

from ops_helpers import kq


class Calls:
    """Stands in for the library: writes the status words that a test asks for."""

    def __init__(self, K, monkeypatch):
        self.status = {}            # call -> status, by the order of covariance calls
        self.cov, self.others = [], []
        for name in ("kronq_gated", "kronq_linear", "kronq_linear_bwd", "kronq_gated_bwd",
                     "kronq_distill_step"):
            monkeypatch.setattr(K, name, lambda *a, _n=name, **k: self.others.append((_n, a, k)))
        monkeypatch.setattr(K, "kronq_accum_cov", self.accum_cov)

    def accum_cov(self, A, H, alpha, beta, info, stream=None):
        info.fill_(self.status.get(len(self.cov), 0))
        self.cov.append(beta)


def _make(n=8):
    from second_order_post_b200.calib import FeedForwardCalibration
    d, f, vocab = 128, 256, 40
    W = [torch.zeros(*s, dtype=torch.bfloat16) for s in ((f, d), (f, d), (d, f), (vocab, d))]
    batch = (torch.zeros(n, d, dtype=torch.bfloat16), torch.zeros(n, 3),
             torch.zeros(n, 3, dtype=torch.int32))
    return FeedForwardCalibration(*W, max_tokens=n, tokens=n), batch


@pytest.mark.parametrize("call", [0, 3, 4, 7, 14])
def test_failure_of_one_batch_stays(monkeypatch, call):
    """A covariance that fails in one of three batches is reported after the last."""
    K = kq()
    calls = Calls(K, monkeypatch)
    cal, batch = _make()
    calls.status[call] = K.KRONQ_ERR_TIMEOUT
    for _ in range(3):
        cal.step(*batch)
    assert len(calls.cov) == 15
    with pytest.raises(K.KronqError) as err:
        cal.check_info()
    assert err.value.status == K.KRONQ_ERR_TIMEOUT


def test_first_failure_is_kept(monkeypatch):
    K = kq()
    calls = Calls(K, monkeypatch)
    cal, batch = _make()
    cal.step(*batch)
    cal.check_info()
    calls.status.update({6: K.KRONQ_ERR_TIMEOUT, 11: K.KRONQ_ERR_NONFINITE})
    cal.step(*batch)
    cal.step(*batch)
    with pytest.raises(K.KronqError) as err:
        cal.check_info()
    assert err.value.status == K.KRONQ_ERR_TIMEOUT


@pytest.fixture
def fresh_memory_is_nan():
    """torch.empty hands out NaN."""
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(False)


def _sums(cal):
    return [*cal.H_X.values(), *cal.H_G.values()]


def test_sums_start_at_zero(monkeypatch, fresh_memory_is_nan):
    """Before the first step, after a step that was refused on its way, and after a
    reset, whatever was there."""
    K = kq()
    calls = Calls(K, monkeypatch)
    cal, batch = _make()
    assert all(not t.any() for t in _sums(cal))

    def refuses(A, H, alpha, beta, info, stream=None):
        calls.cov.append(beta)
        if len(calls.cov) == 2:
            raise K.KronqError("kronq_accum_cov", K.KRONQ_ERR_CUDA)

    with monkeypatch.context() as m:
        m.setattr(K, "kronq_accum_cov", refuses)
        with pytest.raises(K.KronqError):
            cal.step(*batch)
    cal.step(*batch)
    assert calls.cov == [1.0] * 7
    for t in _sums(cal):
        t.fill_(3.0)
    cal.info.fill_(K.KRONQ_ERR_NONFINITE)
    cal.cov_info.fill_(K.KRONQ_ERR_TIMEOUT)
    cal.reset()
    cal.check_info()
    assert all(not t.any() for t in _sums(cal))
    cal.step(*batch)
    assert calls.cov[7:] == [1.0] * 5
