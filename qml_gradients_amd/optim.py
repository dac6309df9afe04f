"""AdamW over all of a model's tensors in one launch: circuit angles and dense weights alike.

Marshalling only: the step runs in ``hqml_adamw_step``.  The moments are torch tensors in the
optimiser's state, held in 32 bits (64 for 64-bit parameters) or in 8 bits: e4m3 codes and one
32-bit scale per 256 elements, the second moment as its square root.
"""
from __future__ import annotations

import copy
import ctypes

import torch

from . import (HQML_ADAMW_BLOCK, HQML_DTYPE_BF16, HQML_DTYPE_FP32, HQML_DTYPE_FP64, HQML_MOMENTS_8, HQML_MOMENTS_32,
               hqml_adamw_config, hqml_adamw_step)

_DTYPES = {torch.float32: HQML_DTYPE_FP32, torch.bfloat16: HQML_DTYPE_BF16, torch.float64: HQML_DTYPE_FP64}
_current_stream = torch._C._cuda_getCurrentRawStream


class AdamW(torch.optim.Optimizer):
    """AdamW with decoupled weight decay.  Parameters: contiguous CUDA tensors in fp32, bf16 or
    (state_bits=32 only) fp64; a gradient may be bf16 for an fp32 parameter and the other way
    round.  state[p] holds "step" and, with state_bits=32, "exp_avg" and "exp_avg_sq"; with
    state_bits=8, "exp_avg" and "exp_avg_sq_root" (torch.float8_e4m3fn) and their scales under
    the same names with "_scale" appended: value = code * scale of its 256 elements.
    The step runs on each device's current stream, which must not be under graph capture."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, state_bits=32):
        if not lr >= 0.0 or not eps >= 0.0 or not weight_decay >= 0.0:
            raise ValueError("lr, eps and weight_decay must be >= 0")
        if not all(0.0 <= b < 1.0 for b in betas):
            raise ValueError("betas must be in [0, 1)")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps, weight_decay=weight_decay,
                                      state_bits=state_bits))

    def add_param_group(self, param_group):
        super().add_param_group(param_group)
        group = self.param_groups[-1]
        for p in group["params"]:
            if not p.is_cuda or p.dtype not in _DTYPES or not p.is_contiguous():
                raise ValueError("parameters must be contiguous CUDA tensors in fp32, bf16 or fp64")
            if p.dtype is torch.float64 and group["state_bits"] == 8:
                raise ValueError("8-bit moments are for fp32 and bf16 parameters")

    def _begin(self, p, bits):
        """The moments before the first step."""
        if bits == 32:
            dtype = torch.float64 if p.dtype is torch.float64 else torch.float32
            return {"step": 0, "exp_avg": torch.zeros_like(p, dtype=dtype),
                    "exp_avg_sq": torch.zeros_like(p, dtype=dtype)}
        blocks = -(-p.numel() // HQML_ADAMW_BLOCK)
        state = {"step": 0}
        for name in ("exp_avg", "exp_avg_sq_root"):
            state[name] = torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(torch.float8_e4m3fn)
            state[name + "_scale"] = torch.zeros(blocks, dtype=torch.float32, device=p.device)
        return state

    def step(self, closure=None):
        for hook in tuple(self._optimizer_step_pre_hooks.values()):
            hook(self, (), {})
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        state = self.state
        for group in self.param_groups:
            eight = group["state_bits"] == 8
            calls = {}   # tensors that one call can take
            for p in group["params"]:
                g = p.grad
                if g is None:
                    continue
                if g.layout is not torch.strided or g.dtype not in _DTYPES:
                    raise ValueError("gradients must be dense, in fp32, bf16 or fp64")
                if not p.is_contiguous():
                    raise ValueError("parameters must be contiguous")
                if not g.is_contiguous():
                    g = g.detach().contiguous()
                s = state[p]
                if not s:
                    s.update(self._begin(p, group["state_bits"]))
                key = (p.dtype, g.dtype, p.get_device(), s["step"])
                call = calls.get(key)
                if call is None:
                    call = calls[key] = ([], [], [], [])
                words, params, grads, states = call
                if eight:
                    words += (p.data_ptr(), g.data_ptr(), s["exp_avg"].data_ptr(), s["exp_avg_sq_root"].data_ptr(),
                              s["exp_avg_scale"].data_ptr(), s["exp_avg_sq_root_scale"].data_ptr(), p.numel())
                else:
                    words += (p.data_ptr(), g.data_ptr(), s["exp_avg"].data_ptr(), s["exp_avg_sq"].data_ptr(), 0, 0,
                              p.numel())
                params.append(p)
                grads.append(g)    # kept until its kernel is queued
                states.append(s)
            for (pd, gd, device, before), (words, params, grads, states) in calls.items():
                cfg = hqml_adamw_config(_DTYPES[pd], _DTYPES[gd], HQML_MOMENTS_8 if eight else HQML_MOMENTS_32,
                                        before + 1, group["lr"], *group["betas"], group["eps"], group["weight_decay"],
                                        device, _current_stream(device))
                hqml_adamw_step(cfg, len(params), (ctypes.c_longlong * len(words))(*words))
                for s in states:
                    s["step"] = before + 1
                # a backward pass that saved a parameter from before this step has to refuse it
                torch.autograd.graph.increment_version(params)
        for hook in tuple(self._optimizer_step_post_hooks.values()):
            hook(self, (), {})
        return loss

    # torch wraps a step that does not say this in a profiler range and the hooks, which cost four times the
    # launch; the optimiser's own hooks run above
    step.hooked = True

    def load_state_dict(self, state_dict):
        """As torch's, but the moments keep the types they were saved in."""
        super().load_state_dict(state_dict)
        saved = state_dict["state"]
        ids = [i for g in state_dict["param_groups"] for i in g["params"]]
        params = [p for g in self.param_groups for p in g["params"]]
        for i, p in zip(ids, params):
            if i in saved:
                self.state[p] = {k: v.detach().to(p.device, copy=True).contiguous() if isinstance(v, torch.Tensor)
                                 else copy.deepcopy(v) for k, v in saved[i].items()}
