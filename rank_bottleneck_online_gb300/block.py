"""Workloads composed from the C-ABI calls: one block, the LLaMA MLP, the full
layer with or without its attention core, and the SVD-style pair; a block whose forward
multiplies in 8 bits; rotary positions and dropout in the layer; clipping of their gradients.

Each workload owns its device tensors (weights, saved activations, gradients
and one workspace) so that a training step is a fixed sequence of library
calls on one stream with no allocation inside it. Every arithmetic step runs
in the library's CUDA kernels; Python only sequences the calls.
"""

from __future__ import annotations

import math

import torch

from . import binding as B
from .inputs import CONFIGS


def _dev(t, device):
    return None if t is None else t.to(device=device, non_blocking=False).contiguous()


class Block:
    """One bottleneck block: y = B_i . act(s * x @ (gamma A))_i, forward and backward."""

    def __init__(self, T, d, r, k, n, *, S=1, eps=1e-5, act="silu", has_norm=True,
                 weights=None, device="cuda", ws=None):
        self.desc = B.make_desc(T, d, r, k, n, S=S, eps=eps, act=act, has_norm=has_norm)
        self.device = torch.device(device)
        w = weights or {}
        self.gamma = _dev(w.get("gamma"), self.device) if has_norm else None
        self.A = _dev(w.get("A"), self.device)
        self.B = _dev(w.get("B"), self.device)
        need = B.workspace_bytes(self.desc)
        self.ws = ws.ensure(need) if ws is not None else B.Workspace(need, self.device)
        bf = torch.bfloat16
        self.y = torch.empty(k, T, n, dtype=bf, device=self.device)
        self.rstd = torch.empty(T, dtype=torch.float32, device=self.device) if has_norm else None
        self.dx = torch.empty(T, d, dtype=bf, device=self.device)
        self.dA = torch.empty(d, k * r, dtype=bf, device=self.device)
        self.dB = torch.empty(k, r, n, dtype=bf, device=self.device)
        self.dgamma = torch.empty(d, dtype=bf, device=self.device) if has_norm else None

    def forward(self, x, stream=None, residual=None):
        """residual [T, n] (k == 1): y = residual + block(x), added in the epilogue."""
        return B.block_fwd(self.desc, x, self.gamma, self.A, self.B, self.ws, y=self.y,
                           rstd=self.rstd, stream=stream, residual=residual)

    def backward(self, x, dy, stream=None, reuse_rstd=True, dx=None, dx_residual=None):
        """dx: where the input gradient goes (default: this block's own buffer);
        dx_residual [T, d]: added to it in the dx epilogue."""
        return B.block_bwd(self.desc, x, self.gamma, self.A, self.B, dy, self.ws,
                           rstd=self.rstd if reuse_rstd else None,
                           dx=self.dx if dx is None else dx,
                           dgamma=self.dgamma, dA=self.dA, dB=self.dB, stream=stream,
                           dx_residual=dx_residual)

    def weight_grads(self):
        """The gradients of the weights."""
        return [self.dA, self.dB] + ([self.dgamma] if self.dgamma is not None else [])


class Fp8Block(Block):
    """A block whose forward multiplies in 8 bits: e4m3 weights quantised once, with gamma
    folded into A, in square blocks of 128; activations quantised row by row on the way. The
    1/rms scale and the activation stay in the down-projection's epilogue. The backward is the
    bf16 block's on the bf16 weights, which this block keeps (straight-through).

    fused_norm: the norm's statistics and the quantiser from one reading of x, together with the
    addition of a residual to x where one is to be (``add``). The row scales' sums are taken in
    another order than without it."""

    def __init__(self, T, d, r, k, n, *, fused_norm=False, **kw):
        super().__init__(T, d, r, k, n, **kw)
        self.fused_norm = fused_norm and bool(self.desc.has_norm)
        D = self.desc
        f8, bf, dev = torch.float8_e4m3fn, torch.bfloat16, self.device

        def operand(lead, rows, K):
            return (torch.empty(lead + (rows, -(-K // 16) * 16), dtype=f8, device=dev),
                    torch.empty(lead + (B.fp8_scale_bytes(rows, K),), dtype=torch.uint8, device=dev))

        self.A8, self.B8 = operand((), k * r, d), operand((k,), n, r)
        self.x8, self.a8 = operand((), T, d), operand((k,), T, r)
        self.a = torch.empty(T, k * r, dtype=bf, device=dev)
        self.ssq = torch.empty(D.S, T, dtype=torch.float32, device=dev) if D.has_norm else None
        self.ws.ensure(max(B.fp8_matmul_workspace_bytes(T, k * r, d),
                           B.fp8_matmul_workspace_bytes(T, n, r, k)))
        self.act = "silu" if D.act else "identity"
        self.quantize_weights()

    @property
    def ws8(self):
        """The products' workspace: the block's own, so that one check of it sees their errors
        too."""
        return self.ws

    def quantize_weights(self, stream=None):
        """Take the 8-bit weights from A, B and gamma again (after an update of them)."""
        B.fp8_quantize(self.A, way="columns", block_rows=128, gamma=self.gamma, cols_out=self.A8,
                       stream=stream)
        B.fp8_quantize(self.B, way="columns", block_rows=128, cols_out=self.B8, stream=stream)

    def forward(self, x, stream=None, residual=None, add=None):
        """add [T, d] (with ``fused_norm``): x is replaced by x + add, in place, first."""
        D = self.desc
        if residual is not None and D.k != 1:
            raise ValueError("a residual needs one output group")
        if add is not None and not self.fused_norm:
            raise ValueError("the addition in front belongs to the fused norm")
        if self.fused_norm:
            B.norm_quantize(x, residual=add, h=None if add is None else x, eps=D.eps,
                            rstd=self.rstd, rows_out=self.x8, stream=stream)
        else:
            if D.has_norm:
                B.rmsnorm_stats(D, x, self.ssq, self.rstd, stream)
            B.fp8_quantize(x, rows_out=self.x8, stream=stream)
        B.fp8_matmul(*self.x8, *self.A8, D.d, self.ws8, row_scale=self.rstd, act=self.act,
                     out=self.a, stream=stream)
        groups = self.a.view(D.T, D.k, D.r).transpose(0, 1)
        B.fp8_quantize(groups, rows_out=self.a8, stream=stream)
        B.fp8_matmul(*self.a8, *self.B8, D.r, self.ws8, out=self.y, stream=stream)
        if residual is not None:
            B.add(self.y[0], residual, self.y[0], stream=stream)
        return self.y


class Rotary:
    """Rotary positions of q and k for heads of ``dim`` values: base^(-i / pairs) radians a
    position for pair i of ``rot`` / 2 (or ``inv_freq``, any frequencies), shared among the
    position axes by ``sections``."""

    def __init__(self, dim, *, rot=None, base=10000.0, inv_freq=None, sections=None,
                 interleaved=False, device="cuda"):
        pairs = (dim if rot is None else rot) // 2
        if inv_freq is None:
            inv_freq = base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
        self.dim, self.sections, self.interleaved = dim, sections, interleaved
        self.inv_freq = inv_freq.to(device=device, dtype=torch.float64).contiguous()

    def __call__(self, q, k, positions, *, inverse=False, q_out=None, k_out=None, stream=None):
        """Turn q and k [T, heads * dim] or [T, heads, dim] (back, for gradients, when
        ``inverse``): returns (q_out, k_out), new tensors where none are given; k may be None."""
        if positions is None:
            raise ValueError("rotary positions need the tokens' positions")

        def split(t):
            return None if t is None else t.view(
                t.shape[0], math.prod(t.shape[1:]) // self.dim, self.dim)

        turned = B.rope(split(q), split(k), positions, self.inv_freq, sections=self.sections,
                        interleaved=self.interleaved, inverse=inverse, q_out=split(q_out),
                        k_out=split(k_out), stream=stream)
        return tuple(t.view(x.shape) if given is None and x is not None else given
                     for x, given, t in zip((q, k), (q_out, k_out), turned))


class Attention:
    """The layer's attention core: ``heads`` heads of ``dim`` values, causal unless told otherwise,
    over packed sequences (``binding.attention``), with what its backward keeps: a core serves
    one layer, and a second ``Layer`` that is given it makes one of its own (``like``)."""

    def __init__(self, T, heads, dim, *, causal=True, scale=None, sequences=1, device="cuda"):
        """sequences: the most that a call has."""
        self.T, self.heads, self.dim, self.causal, self.scale = T, heads, dim, causal, scale
        self.sequences, self.taken = sequences, False      # taken: by a layer
        self.out = torch.empty(T, heads * dim, dtype=torch.bfloat16, device=device)
        self.lse = torch.empty(heads, T, dtype=torch.float32, device=device)
        # (of fewer sequences, too: they may be cut in more parts)
        self.workspace_bytes = max(B.attention_workspace_bytes(T, T, heads, heads, dim, s)
                                   for s in range(1, sequences + 1))

    def like(self):
        """Another core of this form, with buffers of its own."""
        return Attention(self.T, self.heads, self.dim, causal=self.causal, scale=self.scale,
                         sequences=self.sequences, device=self.out.device)

    def _split(self, t):
        return t.view(self.T, self.heads, self.dim)

    def forward(self, q, k, v, ws, starts=None, stream=None):
        """out [T, heads * dim] of q, k, v of that shape; starts: int32 [sequences + 1]."""
        B.attention(self._split(q), self._split(k), self._split(v), ws, causal=self.causal,
                    scale=self.scale, q_starts=starts, k_starts=starts, out=self._split(self.out),
                    lse=self.lse, stream=stream)
        return self.out

    def backward(self, q, k, v, dout, ws, dq, dk, dv, starts=None, stream=None):
        """The last forward's gradients, into dq, dk and dv."""
        s = self._split
        B.attention_bwd(s(q), s(k), s(v), s(self.out), self.lse, s(dout), ws, causal=self.causal,
                        scale=self.scale, q_starts=starts, k_starts=starts, dq=s(dq), dk=s(dk),
                        dv=s(dv), stream=stream)
        return dq, dk, dv


class MLP:
    """LLaMA MLP of two bottlenecks: gate/up (normed, k=2) -> SwiGLU -> down (k=1)."""

    def __init__(self, T, d, r, ffn, *, S=1, eps=1e-5, act="silu", weights=None,
                 device="cuda", ws=None, fused_glu=True, checkpoint="input", fp8=False,
                 fused_norm=False):
        w = weights or {}
        self.T, self.d, self.r, self.ffn = T, d, r, ffn
        # SwiGLU forward in the gate/up up-projection's epilogue, and its backward in the
        # down block's dgrad epilogue (False: separate SwiGLU passes)
        self.fused_glu = fused_glu
        # What the backward starts from. "input": each block's input (x, and h with the
        # gate/up values it was formed from) is kept from the forward, and each block
        # regenerates its own bottleneck activation. "bottleneck": only the gate/up
        # block's r-wide bottleneck activation is kept; the backward regenerates gate,
        # up and h from it (the cut at the tensor-parallel block boundary of §2.1).
        if checkpoint not in ("input", "bottleneck"):
            raise ValueError("checkpoint is 'input' or 'bottleneck'")
        if checkpoint == "bottleneck" and not fused_glu:
            raise ValueError("the bottleneck cut regenerates gate, up and h with the fused kernel")
        self.checkpoint = checkpoint
        # fp8: both blocks' forward in 8 bits (with a separate SwiGLU pass between them)
        if fp8 and checkpoint != "input":
            raise ValueError("the bottleneck cut regenerates the bf16 block's activations")
        self.fp8 = fp8
        if fused_norm and not fp8:
            raise ValueError("the fused norm gives 8-bit values")
        block = Fp8Block if fp8 else Block
        self.gu = block(T, d, r, 2, ffn, S=S, eps=eps, act=act, has_norm=True,
                        weights={"gamma": w.get("gamma"), "A": w.get("A1"), "B": w.get("B1")},
                        device=device, ws=ws, **({"fused_norm": fused_norm} if fp8 else {}))
        self.dn = block(T, ffn, r, 1, d, S=1, eps=eps, act=act, has_norm=False,
                        weights={"A": w.get("A2"), "B": w.get("B2")}, device=device,
                        ws=self.gu.ws if checkpoint == "input" else None)
        if checkpoint == "input":
            self.gu.ws = self.dn.ws   # one workspace sized for both blocks
        # (bottleneck cut: the gate/up block keeps its own workspace, whose a survives
        # the down block's forward)
        dev = self.gu.device
        self.h = torch.empty(T, ffn, dtype=torch.bfloat16, device=dev)
        self.dy1 = torch.empty(2, T, ffn, dtype=torch.bfloat16, device=dev)

    @property
    def out(self):
        return self.dn.y[0]

    def forward(self, x, stream=None, residual=None, add=None):
        """residual [T, d]: out = residual + MLP(x), added in the down block's epilogue. add
        [T, d] (with ``fused_norm``): x is replaced by x + add, in place, first (so that residual
        may be x itself)."""
        if add is not None and not self.fp8:
            raise ValueError("the addition in front belongs to the fused norm")
        if self.fused_glu and not self.fp8:
            gu = self.gu
            B.block_fwd_swiglu(gu.desc, x, gu.gamma, gu.A, gu.B, gu.ws, y=gu.y, h=self.h,
                               rstd=gu.rstd, stream=stream)
        else:
            y1 = self.gu.forward(x, stream, **({} if add is None else {"add": add}))
            B.swiglu_fwd(y1[0], y1[1], self.h, stream=stream)
        return self.dn.forward(self.h, stream, residual=residual)[0]

    def saved_bytes(self):
        """Bytes of activations the backward needs from the forward beyond the input x
        and the row scale: gate, up and h for the input cut, the gate/up block's
        bottleneck activation for the bottleneck cut."""
        if self.checkpoint == "input":
            return 3 * self.T * self.ffn * 2
        return self.T * 2 * self.r * 2

    def backward(self, x, dout, stream=None, dx_residual=None):
        """dx_residual [T, d]: added to the MLP's input gradient in the dx epilogue."""
        dy2 = dout.view(1, self.T, self.d)
        if self.checkpoint == "bottleneck":
            gu = self.gu
            a1 = B.ws_view(gu.ws, B.ws_layout(gu.desc)["a"], (self.T, 2 * self.r),
                           torch.bfloat16)
            B.block_up(gu.desc, a1, gu.B, gu.ws, y=gu.y, h=self.h, stream=stream)
        if self.fused_glu:
            B.block_bwd_swiglu(self.dn.desc, self.h, self.dn.A, self.dn.B, dy2, self.gu.y[0],
                               self.gu.y[1], self.dn.ws, dgate=self.dy1[0], dup=self.dy1[1],
                               dA=self.dn.dA, dB=self.dn.dB, stream=stream)
        else:
            dh = self.dn.backward(self.h, dy2, stream)[0]
            B.swiglu_bwd(self.gu.y[0], self.gu.y[1], dh, self.dy1[0], self.dy1[1],
                         stream=stream)
        return self.gu.backward(x, self.dy1, stream, dx_residual=dx_residual)

    def grads(self):
        return {"dx": self.gu.dx, "dgamma": self.gu.dgamma, "dA1": self.gu.dA, "dB1": self.gu.dB,
                "dA2": self.dn.dA, "dB2": self.dn.dB}

    def weight_grads(self):
        """The gradients of the weights."""
        return self.gu.weight_grads() + self.dn.weight_grads()


class Layer:
    """QKV (normed, k=3) -> O (k=1) on V -> residual -> MLP -> residual.

    attention (an ``Attention``): O works on the attention of q, k and v, and the backward forms
    their gradients; without it O works on V, and the gradients of q and k are given. The
    layer's own is its ``attention``: the one given, or one like it where that is another layer's.

    Both residual adds run in GEMM epilogues: x1 = x + O(v) in the O block's
    up-projection, out = x1 + MLP(x1) in the MLP's down up-projection; in the backward,
    dx1 = dout + (MLP input gradient) in the MLP's dx epilogue and dx = dx1 + (QKV input
    gradient) in the QKV block's.

    rotary (a ``Rotary``): q and k are turned in place in the QKV block's output, and the
    attention core's gradients of the turned q and k back on their way into the QKV block's
    upstream gradient. dropout (p > 0): x1 = x + dropout(O(v)), out = x1 + dropout(MLP(x1)),
    with the masks of (``seed``, ``mask`` of the call) and none stored. Give the layers of a
    model different seeds, any ones: branches share a mask only where seed, mask and branch are
    the same. fp8: the blocks' forward in 8 bits (``Fp8Block``); fused_norm: theirs."""

    def __init__(self, T, d, r, ffn, *, S=1, eps=1e-5, act="silu", weights=None, device="cuda",
                 rotary=None, dropout=0.0, seed=0, fp8=False, attention=None, fused_norm=False):
        p = weights or {}
        self.T, self.d = T, d
        self.rotary, self.dropout, self.seed = rotary, dropout, seed
        if attention is not None and (attention.T, attention.heads * attention.dim) != (T, d):
            raise ValueError(f"the attention core is of {attention.T} tokens and {attention.heads} "
                             f"heads of {attention.dim}, the layer of {T} x {d}")
        if fused_norm and not fp8:
            raise ValueError("the fused norm gives 8-bit values")
        if attention is not None:
            if attention.taken:
                attention = attention.like()
            attention.taken = True
        self.attention, self.fused_norm = attention, fused_norm
        block = Fp8Block if fp8 else Block
        self.qkv = block(T, d, r, 3, d, S=S, eps=eps, act=act, has_norm=True,
                         weights={"gamma": p.get("gamma1"), "A": p.get("A_qkv"),
                                  "B": p.get("B_qkv")}, device=device,
                         **({"fused_norm": fused_norm} if fp8 else {}))
        ws = self.qkv.ws
        self.o = block(T, d, r, 1, d, S=1, eps=eps, act=act, has_norm=False,
                       weights={"A": p.get("A_o"), "B": p.get("B_o")}, device=device, ws=ws)
        self.mlp = MLP(T, d, r, ffn, S=S, eps=eps, act=act,
                       weights={"gamma": p.get("gamma2"), "A1": p.get("A_gu"), "B1": p.get("B_gu"),
                                "A2": p.get("A_dn"), "B2": p.get("B_dn")}, device=device, ws=ws,
                       fp8=fp8, fused_norm=fused_norm)
        ws = self.mlp.gu.ws
        for blk in (self.qkv, self.o):
            blk.ws = ws
        dev = self.qkv.device
        self.dqkv = torch.empty(3, T, d, dtype=torch.bfloat16, device=dev)
        if attention is not None:
            ws.ensure(attention.workspace_bytes)
            self.dattention = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
        # gradient of a branch behind its dropout
        self.dbranch = torch.empty(T, d, dtype=torch.bfloat16, device=dev) if dropout else None

    @property
    def x1(self):
        """x + O(v): the MLP's input (the O block's output buffer)."""
        return self.o.y[0]

    @property
    def out(self):
        """x1 + MLP(x1) (the MLP's output buffer)."""
        return self.mlp.out

    @property
    def dx1(self):
        """Gradient at x1: dout + the MLP's input gradient (the MLP's dx buffer)."""
        return self.mlp.gu.dx

    @property
    def dx(self):
        """Gradient at x: dx1 + the QKV block's input gradient (its dx buffer)."""
        return self.qkv.dx

    def _words(self, which, mask):
        """The generator's seed and offset of branch ``which``: seed + which, so layers with
        neighbouring seeds meet in one of them, and odd and even seeds therefore have offsets
        of their own, below and from 2^63."""
        if not 0 <= mask < 1 << 63:
            raise ValueError("mask must be an unsigned 63-bit value")
        return (self.seed + which) % (1 << 64), mask + ((self.seed + 1) % 2 << 63)

    def _join(self, branch, residual, which, mask, counter, stream):
        """residual + dropout(branch), in the branch's buffer."""
        return B.dropout_add(branch, self.dropout, *self._words(which, mask), residual=residual,
                             out=branch, counter=counter, stream=stream)

    def _split(self, grad, which, mask, counter, stream):
        """Gradient of the branch whose dropout joined it to the residual."""
        if not self.dropout:
            return grad
        return B.dropout_bwd(grad, self.dropout, *self._words(which, mask), dx=self.dbranch,
                             counter=counter, stream=stream)

    def forward(self, x, stream=None, positions=None, mask=0, counter=None, starts=None):
        """positions ([T] or [axes, T]): those of the tokens, with ``rotary``. mask: which
        dropout masks (plus ``counter``, a device value, as in ``binding.dropout_add``), below
        2^63 together. starts: where the packed sequences begin (int32 [sequences + 1], on the
        device; from 0 to T, so that every row has an output), with ``attention``."""
        if starts is not None and self.attention is None:
            raise ValueError("sequences without an attention core")
        qkv = self.qkv.forward(x, stream)
        if self.rotary is not None:
            self.rotary(qkv[0], qkv[1], positions, q_out=qkv[0], k_out=qkv[1], stream=stream)
        v = qkv[2]
        if self.attention is not None:
            v = self.attention.forward(qkv[0], qkv[1], v, self.qkv.ws, starts, stream)
        if not self.dropout:
            if self.fused_norm:
                x1 = self.o.forward(v, stream)[0]
                return self.mlp.forward(x1, stream, residual=x1, add=x)
            x1 = self.o.forward(v, stream, residual=x)[0]
            return self.mlp.forward(x1, stream, residual=x1)
        x1 = self._join(self.o.forward(v, stream)[0], x, 0, mask, counter, stream)
        return self._join(self.mlp.forward(x1, stream), x1, 1, mask, counter, stream)

    def backward(self, x, dout, dq=None, dk=None, stream=None, positions=None, mask=0,
                 counter=None, starts=None):
        """With ``attention`` its gradients of q, k and v are formed here (starts: the forward's).
        Else dq, dk: the attention core's gradients of q and k (the turned ones, with
        ``rotary``). The QKV block's upstream gradient is the stacked [dq, dk, dv]; dq and
        dk are turned back or copied into it (copied unless they are already its first two
        planes, `dqkv[0]`, `dqkv[1]`), and the O block writes dv straight into the third.
        positions, mask, counter: those of the forward."""
        dm = self._split(dout, 1, mask, counter, stream)
        dx1 = self.mlp.backward(self.x1, dm, stream, dx_residual=dout)[0]
        if self.attention is not None:
            if dq is not None or dk is not None:
                raise ValueError("the attention core forms the gradients of q and k")
            do = self._split(dx1, 0, mask, counter, stream)
            att, (dq, dk, dv) = self.attention, self.dqkv
            self.o.backward(att.out, do.view(1, self.T, self.d), stream, dx=self.dattention)
            att.backward(*self.qkv.y, self.dattention, self.qkv.ws, dq, dk, dv, starts, stream)
            if self.rotary is not None:
                self.rotary(dq, dk, positions, inverse=True, q_out=dq, k_out=dk, stream=stream)
            return self.qkv.backward(x, self.dqkv, stream, dx_residual=dx1)[0]
        if dq is None or dk is None or starts is not None:
            raise ValueError("without an attention core its gradients of q and k are needed, and "
                             "there are no sequences")
        if self.rotary is not None:
            self.rotary(dq, dk, positions, inverse=True, q_out=self.dqkv[0], k_out=self.dqkv[1],
                        stream=stream)
        else:
            s = torch.cuda.current_stream() if stream is None else stream
            with torch.cuda.stream(s):
                for i, g in enumerate((dq, dk)):
                    if g.data_ptr() != self.dqkv[i].data_ptr():
                        self.dqkv[i].copy_(g)
        do = self._split(dx1, 0, mask, counter, stream)
        self.o.backward(self.qkv.y[2], do.view(1, self.T, self.d), stream, dx=self.dqkv[2])
        return self.qkv.backward(x, self.dqkv, stream, dx_residual=dx1)[0]

    def weight_grads(self):
        """The gradients of the weights."""
        return self.qkv.weight_grads() + self.o.weight_grads() + self.mlp.weight_grads()


class SVDPair:
    """Two normed SVD-style bottlenecks (identity act) on one x: QKV and gate/up. The
    input gradient is the sum of the two blocks', added in the gate/up block's dx
    epilogue."""

    def __init__(self, T, d, r, ffn, *, S=1, eps=1e-5, weights=None, device="cuda"):
        p = weights or {}
        self.qkv = Block(T, d, r, 3, d, S=S, eps=eps, act="identity", has_norm=True,
                         weights={"gamma": p.get("gamma_qkv"), "A": p.get("A_qkv"),
                                  "B": p.get("B_qkv")}, device=device)
        self.gu = Block(T, d, r, 2, ffn, S=S, eps=eps, act="identity", has_norm=True,
                        weights={"gamma": p.get("gamma_gu"), "A": p.get("A_gu"),
                                 "B": p.get("B_gu")}, device=device, ws=self.qkv.ws)
        self.qkv.ws = self.gu.ws

    @property
    def dx(self):
        """Gradient at x: the QKV block's plus the gate/up block's (the latter's dx buffer)."""
        return self.gu.dx

    def forward(self, x, stream=None):
        return self.qkv.forward(x, stream), self.gu.forward(x, stream)

    def backward(self, x, dy_qkv, dy_gu, stream=None):
        dxq = self.qkv.backward(x, dy_qkv, stream)[0]
        return self.gu.backward(x, dy_gu, stream, dx_residual=dxq)[0]

    def weight_grads(self):
        """The gradients of the weights."""
        return self.qkv.weight_grads() + self.gu.weight_grads()


def clip_gradients(workloads, max_norm, ws, *, norm=None, stream=None):
    """The weight gradients of these blocks, MLPs, layers or pairs scaled in place to a norm over
    all of them of ``max_norm`` at most (None: left as they are). Returns the norm (float32 [1], on
    the device). ws: a workspace of ``binding.grad_clip_workspace_bytes()``, a block's own for
    instance."""
    return B.grad_clip([g for w in workloads for g in w.weight_grads()], max_norm, ws, norm=norm,
                       stream=stream)


def build_workload(name, tensors, device="cuda", T=None):
    """Instantiate a named workload with its (CPU) input tensors moved to ``device``."""
    c = dict(CONFIGS[name])
    if T is not None:
        c["T"] = T
    eps = 1e-5
    if c["kind"] == "block":
        return Block(c["T"], c["d"], c["r"], c["k"], c["n"], S=c["S"], eps=eps, act=c["act"],
                     weights=tensors, device=device)
    if c["kind"] == "mlp":
        return MLP(c["T"], c["d"], c["r"], c["ffn"], S=c["S"], eps=eps, act=c["act"],
                   weights=tensors, device=device)
    if c["kind"] == "layer":
        return Layer(c["T"], c["d"], c["r"], c["ffn"], S=c["S"], eps=eps, act=c["act"],
                     weights=tensors["p"], device=device)
    if c["kind"] == "svd_pair":
        return SVDPair(c["T"], c["d"], c["r"], c["ffn"], S=c["S"], eps=eps,
                       weights=tensors["p"], device=device)
    raise KeyError(name)
