"""The optimisers of a model around circuits.

AdamW takes all of its tensors in one launch, circuit angles and dense weights alike; Muon takes weight matrices, whose
updates it orthogonalises.  Marshalling only: the steps run in ``hqml_adamw_step`` and ``hqml_muon_step``.  AdamW's moments
are torch tensors in the optimiser's state, held in 32 bits (64 for 64-bit parameters) or in 8 bits: e4m3 codes and one
32-bit scale per 256 elements, the second moment as its square root.  Muon's momentum is held in 32 bits.
"""
from __future__ import annotations

import copy
import ctypes
import math
import struct

import torch
from torch.optim.optimizer import _global_optimizer_post_hooks, _global_optimizer_pre_hooks

from . import (HQML_ADAMW_BLOCK, HQML_DTYPE_BF16, HQML_DTYPE_FP32, HQML_DTYPE_FP64, HQML_MOMENTS_8, HQML_MOMENTS_32,
               HQML_MUON_MAX_SIDE, HQML_MUON_MAX_STEPS, hqml_adamw_config, hqml_adamw_step, hqml_muon_config,
               hqml_muon_step, hqml_muon_workspace_bytes)

_DTYPES = {torch.float32: HQML_DTYPE_FP32, torch.bfloat16: HQML_DTYPE_BF16, torch.float64: HQML_DTYPE_FP64}
_WIDE = {torch.float32: torch.float32, torch.bfloat16: torch.float32, torch.float64: torch.float64}
_CODES = torch.float8_e4m3fn
_MATRIX = (torch.float32, torch.bfloat16)   # Muon's types
_TENSOR = "QQQiid"   # hqml_muon_tensor: three addresses, rows, columns, its factor of lr
_current_stream = torch._C._cuda_getCurrentRawStream


class AdamW(torch.optim.Optimizer):
    """AdamW with decoupled weight decay.  Parameters: contiguous CUDA tensors in fp32, bf16 or
    (state_bits=32 only) fp64; a gradient may be bf16 for an fp32 parameter and the other way
    round.  state[p] holds "step" and, with state_bits=32, "exp_avg" and "exp_avg_sq"; with
    state_bits=8, "exp_avg" and "exp_avg_sq_root" (torch.float8_e4m3fn) and their scales under
    the same names with "_scale" appended: value = code * scale of its 256 elements.  A root in 8
    bits falls only with its block's largest (its decay in a step is less than half a code):
    elements whose gradients fade while others' of the same 256 do not keep too small a step, and
    are for 32 bits.
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

    def _fit(self, p, s, bits):
        """Moments in 32 or 64 bits take p's type; what else of a state s of p is not of the type and size that the
        step takes is refused."""
        wide = torch.float64 if p.dtype is torch.float64 else torch.float32
        if bits == 32:
            need = (("exp_avg", wide, p.shape), ("exp_avg_sq", wide, p.shape))
        else:
            codes, blocks = torch.float8_e4m3fn, (-(-p.numel() // HQML_ADAMW_BLOCK),)
            need = (("exp_avg", codes, p.shape), ("exp_avg_sq_root", codes, p.shape),
                    ("exp_avg_scale", torch.float32, blocks), ("exp_avg_sq_root_scale", torch.float32, blocks))
        for name, dtype, shape in need:
            t = s.get(name)
            if t is None or t.shape != shape or t.device != p.device or not t.is_contiguous():
                raise ValueError(f"{name} of a parameter {tuple(p.shape)} on {p.device} must be a contiguous tensor "
                                 f"{tuple(shape)} there")
            if t.dtype is not dtype:
                if bits != 32 or t.dtype not in (torch.float32, torch.float64):
                    raise ValueError(f"{name} of a parameter in {p.dtype} must be {dtype}, not {t.dtype}")
                s[name] = t.to(dtype)

    def _step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        state = self.state
        for group in self.param_groups:
            bits = group["state_bits"]
            calls = {}   # tensors that one call can take
            for p in group["params"]:
                g = p.grad
                if g is None:
                    continue
                if g.layout is not torch.strided or g.dtype not in _DTYPES:
                    raise ValueError("gradients must be dense, in fp32, bf16 or fp64")
                n, dtype = p.numel(), p.dtype
                if not p.is_contiguous() or dtype not in _DTYPES:
                    raise ValueError("parameters must be contiguous, in fp32, bf16 or fp64")
                if g.numel() != n:
                    raise ValueError(f"a parameter of {n} elements has a gradient of {g.numel()}")
                if not g.is_contiguous():
                    g = g.detach().contiguous()
                s = state[p]
                if not s:
                    s.update(self._begin(p, bits))
                # the kernel walks a state by its parameter's type and size, and nothing behind the addresses says
                # how large it is; that it is on the device is the entry point's to check
                m, v = s.get("exp_avg"), s.get("exp_avg_sq_root" if bits == 8 else "exp_avg_sq")
                fits = (m is not None and v is not None and m.dtype is v.dtype is (_CODES if bits == 8 else _WIDE[dtype])
                        and m.numel() == n == v.numel() and m.is_contiguous() and v.is_contiguous())
                if bits == 8 and fits:
                    ms, vs, blocks = s.get("exp_avg_scale"), s.get("exp_avg_sq_root_scale"), -(-n // HQML_ADAMW_BLOCK)
                    fits = (ms is not None and vs is not None and ms.dtype is vs.dtype is torch.float32
                            and ms.numel() == blocks == vs.numel() and ms.is_contiguous() and vs.is_contiguous())
                if not fits:
                    self._fit(p, s, bits)   # or an error; with 8 bits always one
                    m, v = s["exp_avg"], s["exp_avg_sq"]
                key = (dtype, g.dtype, p.get_device(), s["step"])
                call = calls.get(key)
                if call is None:
                    call = calls[key] = ([], [], [], [])
                words, params, grads, states = call
                words += (p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(), ms.data_ptr() if bits == 8 else 0,
                          vs.data_ptr() if bits == 8 else 0, n)
                params.append(p)
                grads.append(g)    # kept until its kernel is queued
                states.append(s)
            for (pd, gd, device, before), (words, params, grads, states) in calls.items():
                cfg = hqml_adamw_config(_DTYPES[pd], _DTYPES[gd], HQML_MOMENTS_8 if bits == 8 else HQML_MOMENTS_32,
                                        before + 1, group["lr"], *group["betas"], group["eps"], group["weight_decay"],
                                        device, _current_stream(device))
                hqml_adamw_step(cfg, len(params), (ctypes.c_longlong * len(words))(*words))
                for s in states:
                    s["step"] = before + 1
                # a backward pass that saved a parameter from before this step has to refuse it
                torch.autograd.graph.increment_version(params)
        return loss

    _hooked_step = torch.optim.Optimizer.profile_hook_step(_step)

    def step(self, closure=None):
        """One step of every parameter that has a gradient; what `closure` returns, called first with gradients on."""
        # torch's hooks and profiler range cost four times the launch: taken where somebody asked for one
        if (_global_optimizer_pre_hooks or _global_optimizer_post_hooks or self._optimizer_step_pre_hooks
                or self._optimizer_step_post_hooks or torch.autograd._profiler_enabled()):
            return self._hooked_step() if closure is None else self._hooked_step(closure)
        return self._step(closure)

    step.hooked = True   # torch wraps a step that does not say so itself

    def load_state_dict(self, state_dict):
        """As torch's, but the moments keep the precision they were saved in (32 and 64 bits follow the parameter's
        type).  A state that does not fit its parameter is refused before anything is taken over."""
        # as the last hook before the load, it sees what the others made of state_dict
        last = self.register_load_state_dict_pre_hook(AdamW._keep)
        try:
            super().load_state_dict(state_dict)
        finally:
            last.remove()
            self._kept = ()

    _kept = ()

    def _keep(self, state_dict):
        """The states to load, as they were saved and checked: torch casts its own copies to the parameters' types."""
        saved, kept = state_dict["state"], []
        for own, group in zip(self.param_groups, state_dict["param_groups"]):
            bits = group.get("state_bits")
            if bits not in (8, 32):
                raise ValueError("state_bits must be 8 or 32")
            for i, p in zip(group["params"], own["params"]):
                if p.dtype is torch.float64 and bits == 8:
                    raise ValueError("8-bit moments are for fp32 and bf16 parameters")
                if not saved.get(i):
                    continue
                s = {k: v.detach().to(p.device, copy=True).contiguous() if isinstance(v, torch.Tensor)
                     else copy.deepcopy(v) for k, v in saved[i].items()}
                self._fit(p, s, bits)
                kept.append((p, s))
        self._kept = kept

    def __setstate__(self, state):   # during a load: before the hooks that follow it
        super().__setstate__(state)
        for p, s in self._kept:
            self.state[p] = s


def _rms(rows, cols):
    return 0.2 * math.sqrt(max(rows, cols))


def _spectral(rows, cols):
    return math.sqrt(max(1.0, rows / cols))


class Muon(torch.optim.Optimizer):
    """Momentum and orthogonalised updates (K. Jordan et al., 2024) for weight matrices:
      m = momentum m + (1 - momentum) g,  u = momentum m + (1 - momentum) g (nesterov) or m,
      X = u / max(|u|, eps);  `steps` times, with A = X X^T:  X = a X + (b A + c A^2) X,
      p = p (1 - lr weight_decay) - lr f X
    with (a, b, c) = coefficients.  f by `adjust`: "spectral", sqrt(max(1, rows / cols)); "rms", 0.2 sqrt(max(rows,
    cols)), which gives updates the size of AdamW's; "none", 1.  Parameters: contiguous CUDA matrices in fp32 or bf16
    (vectors, angles and the like are AdamW's); a gradient may be bf16 for an fp32 parameter and the other way round.
    state[p]["momentum"] is m, in fp32.  X is as exact as 32 bits make it: off by some 2e-6 of its size, by 3e-5 where a gradient
    has few directions (a small batch's).  half=True: the products of bf16 parameters take operands of 11 bits instead of 22, in a
    third of the time; X is then off by 1.5e-3 and 4e-2.  Matrices of up to 64 on one side take 24 bits or more either way, long
    ones of them with up to six steps of these coefficients.  The step runs on each device's current stream and can be captured
    into a graph, which then repeats it with the lr it was captured with."""

    def __init__(self, params, lr=0.02, momentum=0.95, weight_decay=0.0, nesterov=True,
                 coefficients=(3.4445, -4.7750, 2.0315), steps=5, eps=1e-7, adjust="spectral", half=False):
        super().__init__(params, dict(lr=lr, momentum=momentum, weight_decay=weight_decay, nesterov=nesterov,
                                      coefficients=tuple(coefficients), steps=steps, eps=eps, adjust=adjust, half=half))

    _adjust = {"spectral": _spectral, "rms": _rms, "none": lambda rows, cols: 1.0}

    def add_param_group(self, param_group):
        super().add_param_group(param_group)
        group = self.param_groups[-1]
        if not group["lr"] >= 0.0 or not group["weight_decay"] >= 0.0:
            raise ValueError("lr and weight_decay must be >= 0")
        if not 0.0 <= group["momentum"] < 1.0 or not group["eps"] > 0.0:
            raise ValueError("momentum must be in [0, 1), eps > 0")
        if len(group["coefficients"]) != 3 or not 1 <= group["steps"] <= HQML_MUON_MAX_STEPS:
            raise ValueError(f"there are three coefficients and 1 to {HQML_MUON_MAX_STEPS} steps")
        if group["adjust"] not in self._adjust:
            raise ValueError(f"adjust must be one of {', '.join(self._adjust)}")
        for p in group["params"]:
            self._accept(p)

    @staticmethod
    def _accept(p):
        if not p.is_cuda:
            raise ValueError("parameters must be CUDA tensors")
        Muon._fits(p)

    @staticmethod
    def _fits(p):
        if p.dim() != 2 or p.dtype not in _MATRIX or not p.is_contiguous() or max(p.shape) > HQML_MUON_MAX_SIDE:
            raise ValueError("parameters must be contiguous matrices in fp32 or bf16, of up to 2^16 rows and columns")

    @staticmethod
    def _momentum(p, s):
        """The momentum of a state s of p, checked: the kernel walks it by its parameter's size."""
        m = s.get("momentum")
        if m is None:
            m = s["momentum"] = torch.zeros_like(p, dtype=torch.float32)
        elif m.shape != p.shape or m.dtype is not torch.float32 or m.device != p.device or not m.is_contiguous():
            raise ValueError(f"the momentum of a parameter {tuple(p.shape)} on {p.device} must be a contiguous fp32 "
                             "tensor of its shape there")
        return m

    def _step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            size_of = self._adjust[group["adjust"]]
            calls = {}   # matrices that one call can take
            state = self.state
            for p in group["params"]:
                g = p.grad
                if g is None:
                    continue
                self._fits(p)
                shape, dtype = p.shape, g.dtype
                if dtype not in _MATRIX or g.layout is not torch.strided:
                    raise ValueError("gradients must be dense, in fp32 or bf16")
                if g.shape != shape:
                    raise ValueError(f"a parameter {tuple(shape)} has a gradient {tuple(g.shape)}")
                if not g.is_contiguous():
                    g = g.detach().contiguous()
                m = self._momentum(p, state[p])
                key = (p.dtype, dtype, p.get_device())
                call = calls.get(key)
                if call is None:
                    call = calls[key] = ([], [], [])
                words, params, kept = call
                rows, cols = shape
                words += (p.data_ptr(), g.data_ptr(), m.data_ptr(), rows, cols, size_of(rows, cols) if rows and cols else 0.0)
                params.append(p)
                kept.append(g)    # until its kernels are queued
            for (pd, gd, device), (words, params, kept) in calls.items():
                cfg = hqml_muon_config(_DTYPES[pd], _DTYPES[gd], bool(group["nesterov"]), group["steps"], group["lr"],
                                       group["momentum"], group["weight_decay"], group["eps"], *group["coefficients"],
                                       device, _current_stream(device), not group["half"])
                n = len(params)
                tensors = struct.pack(_TENSOR * n, *words)   # n hqml_muon_tensor
                need = hqml_muon_workspace_bytes(cfg, n, tensors)
                # torch's memory: freed at once, it is handed out again only to what the stream runs later
                work = torch.empty(need, dtype=torch.uint8, device=params[0].device) if need else None
                hqml_muon_step(cfg, n, tensors, work.data_ptr() if need else None, need)
                # a backward pass that saved a parameter from before this step has to refuse it
                torch.autograd.graph.increment_version(params)
        return loss

    _hooked_step = torch.optim.Optimizer.profile_hook_step(_step)

    def step(self, closure=None):
        """One step of every parameter that has a gradient; what `closure` returns, called first with gradients on."""
        # torch's hooks and profiler range cost time: taken where somebody asked for one
        if (_global_optimizer_post_hooks or _global_optimizer_pre_hooks or self._optimizer_step_pre_hooks
                or self._optimizer_step_post_hooks or torch.autograd._profiler_enabled()):
            return self._hooked_step() if closure is None else self._hooked_step(closure)
        return self._step(closure)

    step.hooked = True   # torch wraps a step that does not say so itself

    def load_state_dict(self, state_dict):
        """As torch's, but the momentum stays in fp32.  A state that does not fit its parameter is refused before anything
        is taken over."""
        # as the last hook before the load, it sees what the others made of state_dict
        last = self.register_load_state_dict_pre_hook(Muon._keep)
        try:
            super().load_state_dict(state_dict)
        finally:
            last.remove()
            self._kept = ()

    _kept = ()

    def _keep(self, state_dict):
        """The states to load, as they were saved and checked: torch casts its own copies to the parameters' types."""
        saved, kept = state_dict["state"], []
        for own, group in zip(self.param_groups, state_dict["param_groups"]):
            for i, p in zip(group["params"], own["params"]):
                if not saved.get(i):
                    continue
                s = {k: v.detach().to(p.device, copy=True).contiguous() if isinstance(v, torch.Tensor)
                     else copy.deepcopy(v) for k, v in saved[i].items()}
                self._momentum(p, s)
                kept.append((p, s))
        self._kept = kept

    def __setstate__(self, state):   # during a load: before the hooks that follow it
        super().__setstate__(state)
        for group in self.param_groups:
            group.setdefault("half", False)   # a state saved by an earlier version has none
        for p, s in self._kept:
            self.state[p] = s
