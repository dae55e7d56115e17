"""What the calibration pass does around the library's calls: status words over
several batches, the start of the sums, the device and the stream. The calls themselves are stood in for."""
import contextlib
import types

import pytest
import torch

from ops_helpers import kq


class Calls:
    """Stands in for the library: writes the status words that a test asks for. And
    for torch's streams, which a machine without a GPU has none of: `stack` holds
    the ones that were made current, `on` what was current at each call."""

    def __init__(self, K, monkeypatch):
        self.status = {}            # call -> status, by the order of covariance calls
        self.cov, self.on = [], []
        for name in ("kronq_gated", "kronq_linear", "kronq_linear_bwd", "kronq_gated_bwd",
                     "kronq_distill_step"):
            monkeypatch.setattr(K, name, lambda *a, **k: self.seen(k.get("stream")))
        monkeypatch.setattr(K, "kronq_accum_cov", self.accum_cov)
        self.stack = ["process"]
        monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: _stream(dev))
        monkeypatch.setattr(torch.cuda, "stream", self.current)
        self.synced = []
        monkeypatch.setattr(torch.cuda, "synchronize", self.synced.append)

    @contextlib.contextmanager
    def current(self, stream):
        self.stack.append(stream)
        yield
        self.stack.pop()

    def seen(self, stream):
        self.on.append(stream or self.stack[-1])

    def accum_cov(self, A, H, alpha, beta, info, stream=None):
        self.seen(stream)
        info.fill_(self.status.get(len(self.cov), 0))
        self.cov.append(beta)


def _stream(dev, name="current"):
    return types.SimpleNamespace(device=dev, name=name)


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


@pytest.mark.parametrize("given", [False, True])
def test_all_calls_go_to_one_stream_of_the_weights_device(monkeypatch, given):
    """Products, covariances and the quantizer's calls, whatever the process has
    current."""
    calls = Calls(kq(), monkeypatch)
    cal, batch = _make()
    dev = cal.Wg.device
    side = _stream(dev, "side") if given else None
    name = "side" if given else "current"
    cal.step(*batch, stream=side)
    assert len(calls.on) == 12
    assert all(s != "process" and s.device == dev and s.name == name for s in calls.on)

    class Engine:
        H_X, H_G = torch.empty(128, 128), torch.empty(256, 256)

        def run_from_covariances(self, W, stream=None):
            assert calls.stack[-1] != "process" and calls.stack[-1].name == name
            assert stream is None or stream is side
            return W

    assert cal.quantize("gate", Engine(), stream=side) is cal.Wg
    assert calls.stack == ["process"]


def test_stream_of_another_device_is_refused(monkeypatch):
    calls = Calls(kq(), monkeypatch)
    cal, batch = _make()
    other = _stream(torch.device("cuda", 1))
    for call in (lambda: cal.step(*batch, stream=other), lambda: cal.reset(stream=other),
                 lambda: cal.quantize("gate", None, stream=other)):
        with pytest.raises(ValueError):
            call()
    assert not calls.on


def test_status_is_read_behind_every_stream(monkeypatch):
    """The pass may have gone to another stream than the reader's."""
    calls = Calls(kq(), monkeypatch)
    cal, batch = _make()
    cal.step(*batch, stream=_stream(cal.Wg.device, "side"))
    cal.check_info()
    assert calls.synced == [cal.Wg.device]
