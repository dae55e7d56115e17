"""The calibration pass of one gated feed-forward block, from its input tokens
to the covariances that the quantizer takes [gptget-en Methodology: H_G from
one backward pass; wmrh §二].

``FeedForwardCalibration`` holds the block's weights (gate, up, down, and the
head that turns its output into logits) and the buffers of one batch of
tokens, and enqueues on one CUDA stream, per batch:

  forward   H = act(X Wgᵀ) * (X Wuᵀ)             kronq_gated
            Y = H Wdᵀ + X                        kronq_linear (residual stream)
            logits = Y Whᵀ                       kronq_linear
  loss      distillation from the teacher's top logits, and its gradient
                                                 kronq_distill_step (in place)
  backward  dY = dlogits Wh                      kronq_linear_bwd
            dH = dY Wd                           kronq_linear_bwd
            Gg, Gu, dX = ... + dY                kronq_gated_bwd
  sums      H_X of gate/up (X) and of down (H), H_G of gate (Gg), up (Gu) and
            down (dY)                            kronq_accum_cov

The block is the model's last: its output goes to the head as it is, without a
norm. A gradient that comes from a later block, or a norm between, takes the same
library calls by hand.

The weights are not updated: no weight gradient is formed. All arithmetic runs
in the library's kernels; this module allocates, passes pointers and keeps the
status words of all batches together.
"""
from __future__ import annotations

import torch

from . import kronq as K

SUBLAYERS = ("gate", "up", "down")


class FeedForwardCalibration:
    def __init__(self, Wg, Wu, Wd, Wh, max_tokens, tokens, act="silu", tau=1.0):
        """bf16 CUDA weights Wg, Wu (f x d), Wd (d x f), Wh (vocab x d), with d
        and f multiples of 128 (the covariances' rule); `max_tokens`: the largest
        batch; `tokens`: how many tokens the covariances are normalised by
        (those of all batches)."""
        f, d = Wg.shape
        if Wu.shape != (f, d) or Wd.shape != (d, f) or Wh.shape[1] != d:
            raise ValueError("the weights do not belong to one block")
        if d % 128 or f % 128:
            raise ValueError("the block's widths must be multiples of 128")
        if max_tokens < 1 or tokens < 1:
            raise ValueError("max_tokens and tokens must be positive")
        self.Wg, self.Wu, self.Wd, self.Wh = Wg, Wu, Wd, Wh
        self.act, self.tau, self.tokens = K.KRONQ_ACTS[act], float(tau), int(tokens)
        self.max_tokens = int(max_tokens)
        dev, n, vocab = Wg.device, self.max_tokens, Wh.shape[0]
        bf = dict(dtype=torch.bfloat16, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        self._act = {name: torch.empty(n, f, **bf) for name in ("A", "U", "H", "dH")}
        self._res = {name: torch.empty(n, d, **bf) for name in ("Y", "dY", "dX")}
        # rows of logits start on 16-byte boundaries, as kronq_linear wants them
        self._logits = torch.empty(n, (vocab + 7) // 8 * 8, **bf)[:, :vocab]
        self._loss = torch.empty(n, **f32)
        # sums over the batches since the last reset
        self.H_X = {"mlp": torch.zeros(d, d, **f32), "down": torch.zeros(f, f, **f32)}
        self.H_G = {"gate": torch.zeros(f, f, **f32), "up": torch.zeros(f, f, **f32),
                    "down": torch.zeros(d, d, **f32)}
        # status words: the block's products and loss (written on failure only,
        # cleared here), then the first failures of the five covariances, whose
        # calls clear the word they are given
        self.info = torch.zeros(1, dtype=torch.int32, device=dev)
        self.cov_info = torch.zeros(5, dtype=torch.int32, device=dev)
        self._batch_info = torch.zeros(5, dtype=torch.int32, device=dev)
        # True: the next step writes over the sums instead of adding to them (if it is
        # captured, so does every replay)
        self._first = False

    def _on(self, stream):
        """The weights' device and the stream of a pass (None: that device's current
        one) as the current ones, which all calls of the pass then go to."""
        dev = self.Wg.device
        if stream is None:
            stream = torch.cuda.current_stream(dev)
        elif stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, not on {dev}")
        return torch.cuda.stream(stream)

    def reset(self, stream=None):
        """Starts anew: the sums and the status words become 0, in stream order (a
        captured step adds its tokens at every replay; a reset captured before it
        starts each replay from 0)."""
        self._first = False
        with self._on(stream):
            for t in (*self.H_X.values(), *self.H_G.values(), self.info, self.cov_info):
                t.zero_()

    def step(self, X, T, idx, weight=None, stream=None):
        """Adds one batch to the sums: X (n x d bf16 tokens), the teacher's top logits T and
        their places idx (n x k), weight (n fp32, None: all 1) of a token's loss.
        Every row of X is a token of H_X, one of weight 0 too, and has to be
        finite: padding is left out of the batch. Returns the tokens' losses and dX,
        the gradient with respect to X (views that the next step overwrites). A step
        that raises may have added a part of its batch: reset()."""
        n = X.shape[0]
        if not 1 <= n <= self.max_tokens:
            raise ValueError(f"a batch has 1 to {self.max_tokens} tokens, not {n}")
        with self._on(stream):
            return self._enqueue(n, X, T, idx, weight)

    def _enqueue(self, n, X, T, idx, weight):
        A, U, H, dH = (self._act[k][:n] for k in ("A", "U", "H", "dH"))
        Y, dY, dX = (self._res[k][:n] for k in ("Y", "dY", "dX"))
        logits, loss, info = self._logits[:n], self._loss[:n], self.info
        K.kronq_gated(X, self.Wg, self.Wu, H, info, act=self.act, A=A, U=U)
        K.kronq_linear(H, self.Wd, Y, info, R=X)
        K.kronq_linear(Y, self.Wh, logits, info)
        K.kronq_distill_step(logits, T, idx, loss, None, logits, info, tau=self.tau,
                             weight=weight)
        K.kronq_linear_bwd(logits, None, self.Wh, info, dX=dY)
        K.kronq_linear_bwd(dY, None, self.Wd, info, dX=dH)
        # Gg and Gu take the place of A and U
        K.kronq_gated_bwd(dH, A, U, None, self.Wg, self.Wu, A, U, info, act=self.act, dX=dX,
                          dXr=dY)
        beta = 0.0 if self._first else 1.0
        sums = ((X, self.H_X["mlp"]), (H, self.H_X["down"]), (A, self.H_G["gate"]),
                (U, self.H_G["up"]), (dY, self.H_G["down"]))
        for i, (rows, cov) in enumerate(sums):
            K.kronq_accum_cov(rows, cov, 1.0 / self.tokens, beta, self._batch_info[i:i + 1])
        self._first = False
        self.cov_info.add_(self._batch_info * (self.cov_info == 0))
        return loss, dX

    def covariances(self, sublayer):
        """(H_X, H_G) of "gate", "up" or "down"."""
        if sublayer not in SUBLAYERS:
            raise ValueError(f"sublayer must be one of {SUBLAYERS}")
        return self.H_X["down" if sublayer == "down" else "mlp"], self.H_G[sublayer]

    def weight(self, sublayer):
        return {"gate": self.Wg, "up": self.Wu, "down": self.Wd}[sublayer]

    def quantize(self, sublayer, engine, stream=None):
        """BiIP, factor and OBS of one sublayer on copies of its covariances, in
        a SublayerEngine of its shape; returns the engine's QuantResult."""
        hx, hg = self.covariances(sublayer)
        with self._on(stream):
            engine.H_X.copy_(hx)
            engine.H_G.copy_(hg)
            return engine.run_from_covariances(self.weight(sublayer))

    def check_info(self):
        """Raises KronqError for a status word that is not 0, once all that is enqueued
        on the weights' device, on whichever stream, has run."""
        torch.cuda.synchronize(self.Wg.device)
        v = int(self.info.item())
        if v:
            raise K.KronqError("kronq calibration pass", v & 0xFF)
        for v in self.cov_info.tolist():
            if v:
                raise K.KronqError("kronq_accum_cov", v & 0xFF)
