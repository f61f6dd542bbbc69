"""A feed-forward layer on MXFP8 weights: the training step and the decoding step that the
operators of :mod:`.layer` are made for, on weights that :mod:`.writeback` keeps.

    y = down(swiglu(gate(n), up(n))),  n = layer norm of x

The three weights are MXFP8 storage (row-wise and column-wise copies): forward products read the
row-wise copies, the gradients of the inputs the column-wise ones.  Between the operators
activations are 8-bit matrices in blocks of 128: row-wise for the next product, column-wise as
the checkpoint that the weight gradients read; the gate's inputs are kept in 8 bits for its
backward pass.  For a step of T tokens, C features and F hidden features the backward pass so reads
T (C + 3 F) bytes of checkpoints beside x, where BF16 would take 2 T (C + 3 F).

Everything is planned once for a number of tokens: buffers, workspaces and calls.  A layer owns
all of them, also those that hold nothing from the forward pass to the backward: beside the
checkpoints and their scales that is T (7 C + 5 F) bytes of x, y, the norm's and the products'
outputs and the 8-bit inputs of products, for training T (12 C + 6 F) more, and the products'
workspaces.
"""
from __future__ import annotations

import torch

from . import layer as L
from . import writeback as W


def _mat8(rows, cols, by_cols, device):
    shape = (L._blocks(rows, L.BLOCK), cols) if by_cols else (rows, L._blocks(cols, L.BLOCK))
    return (torch.empty(rows, cols, dtype=torch.uint8, device=device),
            torch.empty(shape, dtype=torch.uint8, device=device))


def weight_specs(features: int, hidden: int) -> list:
    """The batch of weights, in buffer order: gate and up [hidden, features], down
    [features, hidden]."""
    return [W.WeightSpec(hidden, features, True), W.WeightSpec(hidden, features, True),
            W.WeightSpec(features, hidden, True)]


class FeedForward:
    """The layer for steps of ``tokens`` tokens.  ``writeback`` is a ``Writeback`` of
    ``weight_specs(features, hidden)`` with full-size storage; later updates of it change the
    weights this layer reads.  ``gamma`` and ``beta`` are float32 vectors.

    ``backward`` adds to ``grads`` (float32): gate, up, down; and fills dgamma and dbeta.  The layer
    is no node of autograd: it takes the values of tensors that require gradients, and its outputs
    require none."""

    def __init__(self, writeback: W.Writeback, gamma, beta, tokens: int, *, eps: float = 1e-5,
                 training: bool = True):
        features, device = gamma.numel(), gamma.device
        hidden = writeback.storage[0].spec.rows
        bf16 = torch.bfloat16

        def buffer(cols, dtype=bf16):
            return torch.empty(tokens, cols, dtype=dtype, device=device)

        def rowwise(st):  # [out, in], summed along the columns
            return L.make_operand(st.data_row.view(st.spec.rows, st.spec.cols), st.scale_row, block=32)

        def colwise(st):  # [out, in], summed down the rows
            return L.make_operand(st.data_col.view(st.spec.rows, st.spec.cols), st.scale_col,
                                  along="rows", block=32)

        def by_rows(m):
            return L.make_operand(*m)

        def by_cols(m):
            return L.make_operand(*m, along="rows")

        gate, up, down = writeback.storage
        self.x, self.y = buffer(features), buffer(features)
        normed, g, u = buffer(features), buffer(hidden), buffer(hidden)
        mean, rstd = (torch.empty(tokens, device=device) for _ in range(2))
        n_row, a_row = (_mat8(tokens, c, False, device) for c in (features, hidden))
        n_col, a_col = (_mat8(tokens, c, True, device) for c in (features, hidden))
        saved = [_mat8(tokens, hidden, False, device) for _ in range(2)]
        if not training:
            n_col = a_col = saved = None
        self._forward = [
            (L.mxfp8_layernorm_forward, L.make_layernorm(self.x, gamma, beta, mean=mean, rstd=rstd,
                                                         y=normed, eps=eps)),
            (L.mxfp8_act_forward, L.make_act("none", inputs=[normed], row=[n_row], col=[n_col])),
            (L.mxfp8_matmul, L.make_product(by_rows(n_row), rowwise(gate), g)),
            (L.mxfp8_matmul, L.make_product(by_rows(n_row), rowwise(up), u)),
            (L.mxfp8_act_forward, L.make_act("swiglu", inputs=[g, u], saved=saved or [], row=[a_row],
                                             col=[a_col])),
            (L.mxfp8_matmul, L.make_product(by_rows(a_row), rowwise(down), self.y)),
        ]
        self._backward = None
        if not training:
            return
        self.dy, self.dx = buffer(features), buffer(features)
        self.dgamma, self.dbeta = torch.empty_like(gamma), torch.empty_like(gamma)
        self.grads = [torch.zeros(st.spec.rows, st.spec.cols, device=device) for st in writeback.storage]
        da, dn_part, dn = buffer(hidden), buffer(features, torch.float32), buffer(features)
        dy_row, dy_col = _mat8(tokens, features, False, device), _mat8(tokens, features, True, device)
        d_row = [_mat8(tokens, hidden, False, device) for _ in range(2)]
        d_col = [_mat8(tokens, hidden, True, device) for _ in range(2)]

        def gradient(d, inputs, into):  # into += d^T inputs, over the tokens
            return L.mxfp8_matmul, L.make_product(by_cols(d), by_cols(inputs), into, addend=into)

        self._backward = [
            (L.mxfp8_act_forward, L.make_act("none", inputs=[self.dy], row=[dy_row], col=[dy_col])),
            (L.mxfp8_matmul, L.make_product(by_rows(dy_row), colwise(down), da)),
            gradient(dy_col, a_col, self.grads[2]),
            (L.mxfp8_act_backward, L.make_act("swiglu", grad=da, saved=saved, row=d_row, col=d_col)),
            gradient(d_col[0], n_col, self.grads[0]),
            gradient(d_col[1], n_col, self.grads[1]),
            (L.mxfp8_matmul, L.make_product(by_rows(d_row[0]), colwise(gate), dn_part)),
            (L.mxfp8_matmul, L.make_product(by_rows(d_row[1]), colwise(up), dn, addend=dn_part)),
            (L.mxfp8_layernorm_backward, L.make_layernorm(
                self.x, gamma, mean=mean, rstd=rstd, dy=dn, dx=self.dx, dgamma=self.dgamma,
                dbeta=self.dbeta, eps=eps)),
        ]

    def _take(self, buffer, values, what):
        """Copies a step's values into the layer's buffer, which a broadcast would fill with others and
        a copy of a tensor with a graph would hang on that graph."""
        if values.shape != buffer.shape:
            raise ValueError(f"{what} must be {list(buffer.shape)}, got {list(values.shape)}")
        buffer.copy_(values.detach())

    def forward(self, x) -> torch.Tensor:
        """y [tokens, features] bfloat16 (the layer's own buffer) of x [tokens, features]."""
        self._take(self.x, x, "x")
        for call, plan in self._forward:
            call(plan)
        return self.y

    def backward(self, dy) -> torch.Tensor:
        """The gradient of x (the layer's own buffer) for the last forward pass."""
        if self._backward is None:
            raise ValueError("the layer was planned without training")
        self._take(self.dy, dy, "dy")
        for call, plan in self._backward:
            call(plan)
        return self.dx
