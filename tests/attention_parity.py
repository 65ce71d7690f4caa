"""Shared helpers of the attention tests: packed inputs, calls and their comparison.

Tolerances. The probabilities and their gradients are rounded to bf16 as operands (2^-8 of each),
out is rounded where the backward takes its row sums from it (2^-8), and what fp32 loses in scores,
exponentials and sums is below 2^-10 of the same magnitudes for the scores met here: |s| < 64, in
sums of at most 128 products, is off by less than 2^-12, and so is exp(s) relative to itself. So an
output is off by at most SLACK times the magnitudes that these roundings scale with (the oracle's
*_size), and by half a bf16 step of its own. lse: 2^-12 from the scores and as much from the sum.
The gradients of a call of few scores take both operands in two parts (2^-16 of each): what is left
of SLACK is the fp32 part, exp(s - lse) off by 2^-12 from s and 2^-11 from lse, and what is below
2^-13 together.
"""

import itertools

import numpy as np
import torch

from oracle import ops
from rank_bottleneck_online_gb300 import binding as B

from ops_parity import BF, close, f64, guarded

SLACK = 2.0 ** -8 + 2.0 ** -10
FINE = 2.0 ** -10
LSE = 2.0 ** -11
SENTINEL = -7.25                       # a bf16 value that no output takes by chance


def starts(lengths):
    at = [(0, 0)] + lengths
    q, k = (list(itertools.accumulate(n)) for n in zip(*at))
    return (torch.tensor(q, dtype=torch.int32, device="cuda"),
            torch.tensor(k, dtype=torch.int32, device="cuda"))


class Case:
    """Inputs of packed sequences with `tail` rows behind the last, as planes of their own or as
    slices of one projection per side ("packed": heads side by side in a token's row; "heads":
    head by head)."""

    def __init__(self, lengths, hq, hk, dim, *, causal=True, tail=0, layout="planes", seed=0,
                 spread=1.0, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.causal, self.scale, self.tail = lengths, causal, scale, tail
        self.hq, self.hk, self.dim = hq, hk, dim
        self.Tq, self.Tk = (sum(n) + tail for n in zip(*lengths))
        self.q_starts, self.k_starts = starts(lengths)

        def make(T, heads, times=1.0):
            x = (torch.randn(T, heads, dim, generator=g) * times).to(BF).cuda()
            if layout == "packed":
                whole = torch.full((T, heads + 3, dim), 3.0, dtype=BF, device="cuda")
                whole[:, 1:heads + 1] = x
                return whole[:, 1:heads + 1]
            if layout == "heads":
                whole = torch.full((heads, T + 2, dim), 3.0, dtype=BF, device="cuda")
                whole[:, 1:T + 1] = x.transpose(0, 1)
                return whole[:, 1:T + 1].transpose(0, 1)
            return x

        self.q, self.k, self.v = make(self.Tq, hq, spread), make(self.Tk, hk), make(self.Tk, hk)
        self.dout = make(self.Tq, hq)
        self.ws = B.Workspace(B.attention_workspace_bytes(self.Tq, self.Tk, hq, hk, dim, len(lengths)))

    @property
    def args(self):
        return dict(causal=self.causal, scale=self.scale, q_starts=self.q_starts,
                    k_starts=self.k_starts)

    def want(self):
        return ops.attention(f64(self.q), f64(self.k), f64(self.v), self.lengths, self.causal,
                             self.scale, f64(self.dout))

    def outputs(self, heads, T):
        t, whole = guarded((T, heads, self.dim), BF)
        t.fill_(SENTINEL)
        return t, whole

    def forward(self, **kw):
        out, whole_out = self.outputs(self.hq, self.Tq)
        lse, whole_lse = guarded((self.hq, self.Tq), torch.float32)
        lse.fill_(SENTINEL)
        B.attention(self.q, self.k, self.v, self.ws, out=out, lse=lse, **self.args, **kw)
        B.check(self.ws)
        assert whole_out() and whole_lse()
        return out, lse

    def backward(self, out, lse, **kw):
        dq, whole_q = self.outputs(self.hq, self.Tq)
        dk, whole_k = self.outputs(self.hk, self.Tk)
        dv, whole_v = self.outputs(self.hk, self.Tk)
        B.attention_bwd(self.q, self.k, self.v, out, lse, self.dout, self.ws, dq=dq, dk=dk, dv=dv,
                        **self.args, **kw)
        B.check(self.ws)
        assert whole_q() and whole_k() and whole_v()
        return dq, dk, dv

    def rows(self, which):
        """Rows that lie in a sequence, and those behind the last."""
        n = sum(x[which] for x in self.lengths)
        return slice(0, n), slice(n, n + self.tail)

    def check_forward(self, out, lse, want):
        i, behind = self.rows(0)
        close(out[i], want["out"][i], SLACK * want["out_size"][i])
        got, exact = f64(lse[:, i]), want["lse"][:, i]
        empty = np.isinf(exact)
        assert np.array_equal(got[empty], exact[empty])
        assert np.abs(got[~empty] - exact[~empty]).max(initial=0.0) <= LSE
        assert (out[behind] == SENTINEL).all() and (lse[:, behind] == SENTINEL).all()

    def check_backward(self, grads, want, slack=SLACK):
        for name, got, which in zip(("dq", "dk", "dv"), grads, (0, 1, 1)):
            i, behind = self.rows(which)
            close(got[i], want[name][i], slack * want[f"{name}_size"][i])
            assert (got[behind] == SENTINEL).all(), name

    def check(self, slack=SLACK):
        want = self.want()
        out, lse = self.forward()
        self.check_forward(out, lse, want)
        grads = self.backward(out, lse)
        self.check_backward(grads, want, slack)
        return out, lse, grads
