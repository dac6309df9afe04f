"""PyTorch autograd bridge: the fused forward and adjoint passes as a differentiable op.

The pages wrap their fused kernels in a differentiable PyTorch module (hugo-pages
summary, section 3.3).  This module plays that role over the C ABI: the forward
runs ``hqml_forward`` (keeping the fused-pass outputs), the backward runs
``hqml_backward`` with the incoming dL/dE, so any loss built from the
expectation values gets its gradient from the fused adjoint kernels.  Gradients
flow to theta only; the encoding angles x are data.  DenseLayer and GroupNormLayer do the
same for the layers around the circuits, and DenseInt8Layer serves a trained dense layer in 8-bit
integers.  Marshalling only: no arithmetic of the method runs here.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.forward_ad import unpack_dual

from . import Context, Dense, DenseInt8, GroupNorm, quantise_rows


class HEAExpectation(torch.autograd.Function):
    """E_b = <O> for a batch, differentiable in theta through the fused adjoint pass."""

    @staticmethod
    def forward(ctx, theta, x, hq_ctx):
        e = hq_ctx.forward(x, theta, save_for_backward=True)
        ctx.hq = hq_ctx
        ctx.fwd_id = hq_ctx.fwd_id
        return e

    @staticmethod
    def backward(ctx, grad_e):
        if ctx.hq.fwd_id != ctx.fwd_id:
            raise RuntimeError("this layer ran another forward after the one being differentiated; "
                               "a layer keeps the saved states of its latest forward only")
        return ctx.hq.backward(grad_e.contiguous()), None, None


class HEALayer(torch.nn.Module):
    """Hardware-efficient ansatz layer: angle encoding Ry(x_q), n_layers of Rx, Ry, Rz on
    every qubit plus the CZ chain (or the CNOT chain, entangler="cnot"), output <O> per
    sample (O = Z_0 unless obs_mask / obs_x_mask say otherwise).  theta
    [n_layers][n_qubits][3] is the trainable parameter.
    The remaining arguments are those of the C ABI's hqml_config; storage defaults to
    the compute type's (complex128 states with compute="fp64")."""

    def __init__(self, n_qubits, n_layers, max_batch, storage=None, ckpt_block=0, compute="fp32",
                 obs_mask=0, obs_x_mask=0, theta=None, device=None, entangler="cz"):
        super().__init__()
        if storage is None:
            storage = "fp64" if compute == "fp64" else "fp32"
        dtype = torch.float64 if compute == "fp64" else torch.float32
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else int(device))
        if theta is None:
            theta = torch.rand(n_layers, n_qubits, 3, dtype=torch.float64) * (2.0 * math.pi)
        self.theta = torch.nn.Parameter(torch.as_tensor(theta).to(dev, dtype).contiguous())
        self.hq = Context(n_qubits, n_layers, max_batch, storage=storage, ckpt_block=ckpt_block,
                          device=dev.index, compute=compute, obs_mask=obs_mask, obs_x_mask=obs_x_mask,
                          entangler=entangler)

    def forward(self, x):
        return HEAExpectation.apply(self.theta, x, self.hq)


class DenseFunction(torch.autograd.Function):
    """y = alpha act(x w^T + bias) + residual, differentiable in all four."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, dense, gradients):
        ctx.dense = dense
        if not gradients or not any(ctx.needs_input_grad[:3]):   # the residual's needs nothing kept
            return dense.forward(x, weight, bias, residual)
        y, z = dense.forward_train(x, weight, bias, residual)
        ctx.save_for_backward(x, weight, z)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        need = ctx.needs_input_grad
        dx = dw = db = None
        if any(need[:3]):
            x, weight, z = ctx.saved_tensors
            dx, dw, db = ctx.dense.backward(dy, x, weight, z, input=need[0], weight=need[1], bias=need[2])
        return dx, dw, db, dy if need[3] else None, None, None


class DenseLayer(torch.nn.Module):
    """Dense layer y = alpha act(x weight^T + bias) + residual over the last axis of x, with
    weight [out_features][in_features] and bias [out_features] as trainable parameters
    (initialised uniformly within 1/sqrt(in_features)).  max_batch bounds the product of x's
    other axes.  activation="sigmoid" with alpha=pi maps features to encoding angles."""

    def __init__(self, in_features, out_features, max_batch, dtype="fp32", activation="none", alpha=1.0, bias=True,
                 device=None):
        super().__init__()
        self.dense = Dense(in_features, out_features, max_batch, dtype=dtype, activation=activation, alpha=alpha,
                           device=device)
        bound = 1.0 / math.sqrt(in_features)

        def parameter(*shape):
            v = (torch.rand(*shape, dtype=torch.float64) * 2.0 - 1.0) * bound
            return torch.nn.Parameter(v.to(self.dense.device, self.dense.dtype))

        self.weight = parameter(out_features, in_features)
        self.bias = parameter(out_features) if bias else None

    def forward(self, x, residual=None):
        lead = x.shape[:-1]
        x = x.reshape(-1, x.shape[-1])
        if residual is not None:
            residual = residual.reshape(-1, residual.shape[-1])
        # through the function whether or not a gradient is wanted: it refuses a tangent that it would lose, and a trace
        # shows it
        y = DenseFunction.apply(x, self.weight, self.bias, residual, self.dense, torch.is_grad_enabled())
        return y.reshape(*lead, y.shape[-1])


class DenseInt8Layer(torch.nn.Module):
    """A dense layer served in 8-bit integers: y = alpha act(x w^T + bias) + residual over the last axis of x, with the
    weights held as int8 codes [out_features][in_features] and a scale for each output channel.  `of` makes one of a
    trained DenseLayer; codes, scales and bias are buffers.  There is no gradient: an input that wants one, or has a tangent, is
    refused."""

    def __init__(self, in_features, out_features, max_batch, dtype="fp32", activation="none", alpha=1.0, bias=True,
                 device=None):
        super().__init__()
        self.dense = DenseInt8(in_features, out_features, max_batch, dtype=dtype, activation=activation, alpha=alpha,
                               device=device)
        weight = torch.zeros(out_features, in_features, device=self.dense.device)
        codes, scales = quantise_rows(weight)
        self.register_buffer("codes", codes)
        self.register_buffer("scales", scales)
        self.register_buffer("bias", torch.zeros(out_features, dtype=self.dense.dtype, device=self.dense.device)
                             if bias else None)

    @classmethod
    def of(cls, layer):
        """The DenseLayer `layer` in 8-bit integers."""
        c = layer.dense.cfg
        made = cls(c.in_features, c.out_features, c.max_batch, dtype=c.dtype, activation=c.activation, alpha=c.alpha,
                   bias=layer.bias is not None, device=c.device)
        with torch.no_grad():
            made.codes, made.scales = quantise_rows(layer.weight)
            if layer.bias is not None:
                made.bias.copy_(layer.bias)
        return made

    def forward(self, x, residual=None):
        given = [t for t in (x, residual, self.scales, self.bias) if t is not None]
        if torch.is_grad_enabled() and any(t.requires_grad for t in given):
            raise RuntimeError("a dense layer in 8-bit integers has no gradient: call it under torch.no_grad()")
        if any(unpack_dual(t).tangent is not None for t in given):
            raise RuntimeError("a dense layer in 8-bit integers has no forward-mode derivative")
        lead = x.shape[:-1]
        x = x.reshape(-1, x.shape[-1])
        if residual is not None:
            residual = residual.reshape(-1, residual.shape[-1])
        y = self.dense.forward(x, self.codes, self.scales, self.bias, residual)
        return y.reshape(*lead, y.shape[-1])


class GroupNormFunction(torch.autograd.Function):
    """y = act(weight xhat + bias), differentiable in all three."""

    @staticmethod
    def forward(ctx, x, weight, bias, norm, gradients):
        ctx.norm = norm
        if not gradients or not any(ctx.needs_input_grad[:3]):
            return norm.forward(x, weight, bias)
        y, mean, rstd = norm.forward_train(x, weight, bias)
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        need = ctx.needs_input_grad
        dx = dw = db = None
        if any(need[:3]):
            x, weight, bias, mean, rstd = ctx.saved_tensors
            dx, dw, db = ctx.norm.backward(dy, x, weight, bias, mean, rstd, input=need[0], parameters=need[1] or need[2])
        return dx, dw if need[1] else None, db if need[2] else None, None, None


class GroupNormLayer(torch.nn.Module):
    """Group norm with an activation over channels-last arrays [samples][...positions][channels], with weight (1 at
    first) and bias (0) [channels] as trainable parameters.  max_rows bounds samples times positions."""

    def __init__(self, channels, groups, max_rows, dtype="fp32", activation="none", eps=1e-5, affine=True, device=None):
        super().__init__()
        self.norm = GroupNorm(channels, groups, max_rows, dtype=dtype, activation=activation, eps=eps, device=device)

        def parameter(value):
            return torch.nn.Parameter(torch.full((channels,), value, dtype=self.norm.dtype, device=self.norm.device))

        self.weight = parameter(1.0) if affine else None
        self.bias = parameter(0.0) if affine else None

    def forward(self, x):
        return GroupNormFunction.apply(x, self.weight, self.bias, self.norm, torch.is_grad_enabled())
