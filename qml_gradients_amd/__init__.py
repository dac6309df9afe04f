"""qml_gradients_amd -- Python binding of the hqml C-ABI library (libhqml.so).

The library runs the whole training step (fused forward passes, the fused
adjoint backward passes and every reduction) in its own gfx950 kernels.  This
module only marshals arguments: it passes device pointers of torch tensors to
the C entry points of ``include/hqml.h``, whose names it keeps.  PyTorch is used
for device memory and streams only.  There is no fallback: if ``libhqml.so`` is
missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhqml.so")

HQML_OK = 0
HQML_ERR_ARG = -1
HQML_ERR_OOM = -2
HQML_ERR_HIP = -3
HQML_ERR_STATE = -4
HQML_ERR_UNSUPPORTED = -5
HQML_STORE_FP32 = 0
HQML_STORE_BF16 = 1
HQML_STORE_FP64 = 2
HQML_COMPUTE_FP32 = 0
HQML_COMPUTE_FP64 = 1
HQML_FUSED = 0
HQML_GATE_BY_GATE = 1
HQML_ENT_CZ = 0
HQML_ENT_CNOT = 1
HQML_DTYPE_FP32, HQML_DTYPE_BF16, HQML_DTYPE_FP64 = range(3)
HQML_ACT_NONE, HQML_ACT_RELU, HQML_ACT_GELU, HQML_ACT_SILU, HQML_ACT_TANH, HQML_ACT_SIGMOID = range(6)
HQML_DENSE_MAX_FEATURES = 1 << 20
HQML_DENSE_MAX_BATCH = 1 << 24
HQML_MOMENTS_32 = 0
HQML_MOMENTS_8 = 1
HQML_ADAMW_BLOCK = 256
HQML_DENSE8_MAX_IN = 1 << 17
HQML_NORM_MAX_CHANNELS = 4096
HQML_NORM_MAX_ROWS = 1 << 30
HQML_MUON_MAX_SIDE = 1 << 16
HQML_MUON_MAX_STEPS = 100
HQML_K_FWD_PASS, HQML_K_BWD_PASS, HQML_K_SMALL, HQML_K_OTHER, HQML_K_GATE, HQML_K_COUNT = range(6)


class hqml_config(ctypes.Structure):
    _fields_ = [
        ("n_qubits", ctypes.c_int),
        ("n_layers", ctypes.c_int),
        ("max_batch", ctypes.c_int),
        ("storage", ctypes.c_int),
        ("ckpt_block", ctypes.c_int),
        ("device", ctypes.c_int),
        ("stream", ctypes.c_void_p),
        ("fusion", ctypes.c_int),
        ("compute", ctypes.c_int),
        ("obs_mask", ctypes.c_int),
        ("obs_x_mask", ctypes.c_int),
        ("entangler", ctypes.c_int),
    ]


class hqml_dense_config(ctypes.Structure):
    _fields_ = [
        ("in_features", ctypes.c_int),
        ("out_features", ctypes.c_int),
        ("max_batch", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("activation", ctypes.c_int),
        ("alpha", ctypes.c_float),
        ("device", ctypes.c_int),
        ("stream", ctypes.c_void_p),
    ]


class hqml_adamw_tensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("m", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("m_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("numel", ctypes.c_longlong),
    ]


class hqml_adamw_config(ctypes.Structure):
    _fields_ = [
        ("param_dtype", ctypes.c_int),
        ("grad_dtype", ctypes.c_int),
        ("moments", ctypes.c_int),
        ("step", ctypes.c_longlong),
        ("lr", ctypes.c_double),
        ("beta1", ctypes.c_double),
        ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double),
        ("weight_decay", ctypes.c_double),
        ("device", ctypes.c_int),
        ("stream", ctypes.c_void_p),
    ]


class hqml_norm_config(ctypes.Structure):
    _fields_ = [
        ("channels", ctypes.c_int),
        ("groups", ctypes.c_int),
        ("max_rows", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("activation", ctypes.c_int),
        ("eps", ctypes.c_float),
        ("device", ctypes.c_int),
        ("stream", ctypes.c_void_p),
    ]


class hqml_muon_tensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("momentum", ctypes.c_void_p),
        ("rows", ctypes.c_int),
        ("cols", ctypes.c_int),
        ("scale", ctypes.c_double),
    ]


class hqml_muon_config(ctypes.Structure):
    _fields_ = [
        ("param_dtype", ctypes.c_int),
        ("grad_dtype", ctypes.c_int),
        ("nesterov", ctypes.c_int),
        ("steps", ctypes.c_int),
        ("lr", ctypes.c_double),
        ("momentum", ctypes.c_double),
        ("weight_decay", ctypes.c_double),
        ("eps", ctypes.c_double),
        ("a", ctypes.c_double),
        ("b", ctypes.c_double),
        ("c", ctypes.c_double),
        ("device", ctypes.c_int),
        ("stream", ctypes.c_void_p),
        ("precise", ctypes.c_int),
    ]


class HqmlError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"hqml status {status}: {message}")
        self.status = status


_lib = None


def load() -> ctypes.CDLL:
    """Load libhqml.so (built by ``python -m qml_gradients_amd.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"hqml library not built: {LIB_PATH} is missing "
                           "(run `python -m qml_gradients_amd.build`)")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    i = ctypes.c_int
    ll = ctypes.c_longlong
    cfgp = ctypes.POINTER(hqml_config)
    densep = ctypes.POINTER(hqml_dense_config)
    normp = ctypes.POINTER(hqml_norm_config)
    muonp = ctypes.POINTER(hqml_muon_config)
    sig = {
        "hqml_workspace_bytes": (ctypes.c_size_t, [cfgp]),
        "hqml_create": (i, [cfgp, ctypes.POINTER(P)]),
        "hqml_destroy": (i, [P]),
        "hqml_forward": (i, [P, i, P, P, P, i]),
        "hqml_backward": (i, [P, P, P]),
        "hqml_train_step": (i, [P, i, P, P, P, P, P, P]),
        "hqml_forward_f64": (i, [P, i, P, P, P, i]),
        "hqml_backward_f64": (i, [P, P, P]),
        "hqml_train_step_f64": (i, [P, i, P, P, P, P, P, P]),
        "hqml_status_str": (ctypes.c_char_p, [i]),
        "hqml_last_error": (ctypes.c_char_p, [P]),
        "hqml_set_timing": (i, [P, i]),
        "hqml_set_overlap": (i, [P, i]),
        "hqml_kernel_times": (i, [P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_longlong), i]),
        "hqml_plan_info": (i, [P, ctypes.POINTER(i), ctypes.POINTER(i), ctypes.POINTER(i),
                              ctypes.POINTER(ctypes.c_size_t)]),
        "hqml_describe_plan": (ctypes.c_longlong, [cfgp, ctypes.c_char_p, ctypes.c_size_t]),
        "hqml_train_step_noalloc": (i, [cfgp, i, P, P, P, P, P, P]),
        "hqml_dense_workspace_bytes": (ctypes.c_size_t, [densep]),
        "hqml_dense_create": (i, [densep, ctypes.POINTER(P)]),
        "hqml_dense_destroy": (i, [P]),
        "hqml_dense_last_error": (ctypes.c_char_p, [P]),
        "hqml_dense_forward": (i, [P, i, P, ll, P, ll, P, P, ll, P, ll, P]),
        "hqml_dense_backward": (i, [P, i, P, ll, P, ll, P, ll, P, P, ll, P, P]),
        "hqml_adamw_step": (i, [ctypes.POINTER(hqml_adamw_config), i, P]),
        "hqml_quantise_rows": (i, [i, P, i, ll, i, P, ll, P, ll, P]),
        "hqml_dense8_workspace_bytes": (ctypes.c_size_t, [densep]),
        "hqml_dense8_create": (i, [densep, ctypes.POINTER(P)]),
        "hqml_dense8_destroy": (i, [P]),
        "hqml_dense8_last_error": (ctypes.c_char_p, [P]),
        "hqml_dense8_forward": (i, [P, i, P, ll, P, ll, P, P, P, ll, P, ll]),
        "hqml_norm_workspace_bytes": (ctypes.c_size_t, [normp]),
        "hqml_norm_create": (i, [normp, ctypes.POINTER(P)]),
        "hqml_norm_destroy": (i, [P]),
        "hqml_norm_last_error": (ctypes.c_char_p, [P]),
        "hqml_norm_forward": (i, [P, i, i, P, ll, P, P, P, ll, P, P]),
        "hqml_norm_backward": (i, [P, i, i, P, ll, P, ll, P, P, P, P, P, ll, P, P]),
        "hqml_muon_workspace_bytes": (ctypes.c_size_t, [muonp, i, P]),
        "hqml_muon_step": (i, [muonp, i, P, P, ctypes.c_size_t]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


EXPORTED = ("hqml_workspace_bytes", "hqml_create", "hqml_destroy", "hqml_forward", "hqml_backward",
            "hqml_train_step", "hqml_forward_f64", "hqml_backward_f64", "hqml_train_step_f64", "hqml_status_str", "hqml_last_error", "hqml_set_timing",
            "hqml_set_overlap", "hqml_kernel_times", "hqml_plan_info", "hqml_describe_plan",
            "hqml_train_step_noalloc", "hqml_dense_workspace_bytes", "hqml_dense_create", "hqml_dense_destroy",
            "hqml_dense_last_error", "hqml_dense_forward", "hqml_dense_backward", "hqml_adamw_step",
            "hqml_quantise_rows", "hqml_dense8_workspace_bytes", "hqml_dense8_create", "hqml_dense8_destroy",
            "hqml_dense8_last_error", "hqml_dense8_forward", "hqml_norm_workspace_bytes", "hqml_norm_create",
            "hqml_norm_destroy", "hqml_norm_last_error", "hqml_norm_forward", "hqml_norm_backward",
            "hqml_muon_workspace_bytes", "hqml_muon_step")


def make_config(n_qubits, n_layers, max_batch, storage="fp32", ckpt_block=0, device=0, stream=None,
                fusion="fused", obs_mask=0, compute="fp32", obs_x_mask=0, entangler="cz"):
    st = {"fp32": HQML_STORE_FP32, "bf16": HQML_STORE_BF16, "fp64": HQML_STORE_FP64}.get(storage, storage)
    fu = {"fused": HQML_FUSED, "gate_by_gate": HQML_GATE_BY_GATE}.get(fusion, fusion)
    co = {"fp32": HQML_COMPUTE_FP32, "fp64": HQML_COMPUTE_FP64}.get(compute, compute)
    en = {"cz": HQML_ENT_CZ, "cnot": HQML_ENT_CNOT}.get(entangler, entangler)
    return hqml_config(int(n_qubits), int(n_layers), int(max_batch), int(st), int(ckpt_block),
                       int(device), ctypes.c_void_p(stream or 0), int(fu), int(co), int(obs_mask),
                       int(obs_x_mask), int(en))


DENSE_DTYPES = {"fp32": HQML_DTYPE_FP32, "bf16": HQML_DTYPE_BF16}
ACTIVATIONS = {"none": HQML_ACT_NONE, "relu": HQML_ACT_RELU, "gelu": HQML_ACT_GELU, "silu": HQML_ACT_SILU,
               "tanh": HQML_ACT_TANH, "sigmoid": HQML_ACT_SIGMOID}


def make_dense_config(in_features, out_features, max_batch, dtype="fp32", activation="none", alpha=1.0, device=0,
                      stream=None):
    return hqml_dense_config(int(in_features), int(out_features), int(max_batch), int(DENSE_DTYPES.get(dtype, dtype)),
                             int(ACTIVATIONS.get(activation, activation)), float(alpha), int(device),
                             ctypes.c_void_p(stream or 0))


def make_norm_config(channels, groups, max_rows, dtype="fp32", activation="none", eps=1e-5, device=0, stream=None):
    return hqml_norm_config(int(channels), int(groups), int(max_rows), int(DENSE_DTYPES.get(dtype, dtype)),
                            int(ACTIVATIONS.get(activation, activation)), float(eps), int(device),
                            ctypes.c_void_p(stream or 0))


# ---- the C entry points, same names, argument marshalling only ----

def hqml_workspace_bytes(cfg: hqml_config) -> int:
    return int(load().hqml_workspace_bytes(ctypes.byref(cfg)))


def hqml_describe_plan(cfg: hqml_config) -> str:
    lib = load()
    need = lib.hqml_describe_plan(ctypes.byref(cfg), None, 0)
    if need < 0:
        raise HqmlError(int(need), "invalid configuration")
    buf = ctypes.create_string_buffer(int(need) + 1)
    lib.hqml_describe_plan(ctypes.byref(cfg), buf, len(buf))
    return buf.value.decode()


def hqml_create(cfg: hqml_config) -> ctypes.c_void_p:
    lib = load()
    h = ctypes.c_void_p()
    rc = lib.hqml_create(ctypes.byref(cfg), ctypes.byref(h))
    if rc != HQML_OK:
        raise HqmlError(rc, lib.hqml_last_error(None).decode())
    return h


def _check(ctx, rc):
    if rc != HQML_OK:
        raise HqmlError(rc, load().hqml_last_error(ctx).decode())


def hqml_destroy(ctx) -> None:
    load().hqml_destroy(ctx)


def hqml_forward(ctx, B, x_ptr, theta_ptr, expz_ptr, save_for_backward) -> None:
    _check(ctx, load().hqml_forward(ctx, int(B), x_ptr, theta_ptr, expz_ptr, int(save_for_backward)))


def hqml_backward(ctx, dlde_ptr, grad_ptr) -> None:
    _check(ctx, load().hqml_backward(ctx, dlde_ptr, grad_ptr))


def hqml_train_step(ctx, B, x_ptr, theta_ptr, y_ptr, expz_ptr, loss_ptr, grad_ptr) -> None:
    _check(ctx, load().hqml_train_step(ctx, int(B), x_ptr, theta_ptr, y_ptr, expz_ptr, loss_ptr, grad_ptr))


def hqml_forward_f64(ctx, B, x_ptr, theta_ptr, expz_ptr, save_for_backward) -> None:
    _check(ctx, load().hqml_forward_f64(ctx, int(B), x_ptr, theta_ptr, expz_ptr, int(save_for_backward)))


def hqml_backward_f64(ctx, dlde_ptr, grad_ptr) -> None:
    _check(ctx, load().hqml_backward_f64(ctx, dlde_ptr, grad_ptr))


def hqml_train_step_f64(ctx, B, x_ptr, theta_ptr, y_ptr, expz_ptr, loss_ptr, grad_ptr) -> None:
    _check(ctx, load().hqml_train_step_f64(ctx, int(B), x_ptr, theta_ptr, y_ptr, expz_ptr, loss_ptr, grad_ptr))


def hqml_train_step_noalloc(cfg: hqml_config, B, x_ptr, theta_ptr, y_ptr, expz_ptr, loss_ptr, grad_ptr) -> None:
    lib = load()
    rc = lib.hqml_train_step_noalloc(ctypes.byref(cfg), int(B), x_ptr, theta_ptr, y_ptr, expz_ptr, loss_ptr, grad_ptr)
    if rc != HQML_OK:
        raise HqmlError(rc, lib.hqml_last_error(None).decode())


def hqml_dense_workspace_bytes(cfg: hqml_dense_config) -> int:
    return int(load().hqml_dense_workspace_bytes(ctypes.byref(cfg)))


def hqml_dense_create(cfg: hqml_dense_config) -> ctypes.c_void_p:
    lib = load()
    h = ctypes.c_void_p()
    rc = lib.hqml_dense_create(ctypes.byref(cfg), ctypes.byref(h))
    if rc != HQML_OK:
        raise HqmlError(rc, lib.hqml_last_error(None).decode())
    return h


def hqml_dense_destroy(h) -> None:
    load().hqml_dense_destroy(h)


def hqml_dense_last_error(h) -> str:
    return load().hqml_dense_last_error(h).decode()


def hqml_dense_forward(h, M, x_ptr, ldx, w_ptr, ldw, bias_ptr, residual_ptr, ldr, y_ptr, ldy, z_ptr) -> None:
    rc = load().hqml_dense_forward(h, M, x_ptr, ldx, w_ptr, ldw, bias_ptr, residual_ptr, ldr, y_ptr, ldy, z_ptr)
    if rc != HQML_OK:
        raise HqmlError(rc, hqml_dense_last_error(h))


def hqml_dense_backward(h, M, dy_ptr, lddy, x_ptr, ldx, w_ptr, ldw, z_ptr, dx_ptr, lddx, dw_ptr, db_ptr) -> None:
    rc = load().hqml_dense_backward(h, M, dy_ptr, lddy, x_ptr, ldx, w_ptr, ldw, z_ptr, dx_ptr, lddx, dw_ptr, db_ptr)
    if rc != HQML_OK:
        raise HqmlError(rc, hqml_dense_last_error(h))


def hqml_adamw_step(cfg: hqml_adamw_config, n_tensors, tensors) -> None:
    """tensors: a ctypes array of hqml_adamw_tensor, or of as many 64-bit words."""
    lib = load()
    rc = lib.hqml_adamw_step(ctypes.byref(cfg), int(n_tensors), tensors)
    if rc != HQML_OK:
        raise HqmlError(rc, lib.hqml_last_error(None).decode())


def hqml_quantise_rows(device, stream, dtype, rows, K, x_ptr, ldx, codes_ptr, ldc, scales_ptr) -> None:
    lib = load()
    rc = lib.hqml_quantise_rows(device, stream, dtype, rows, K, x_ptr, ldx, codes_ptr, ldc, scales_ptr)
    if rc != HQML_OK:
        raise HqmlError(rc, lib.hqml_last_error(None).decode())


def _created(create, cfg) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    rc = create(ctypes.byref(cfg), ctypes.byref(h))
    if rc != HQML_OK:
        raise HqmlError(rc, load().hqml_last_error(None).decode())
    return h


def hqml_dense8_workspace_bytes(cfg: hqml_dense_config) -> int:
    return int(load().hqml_dense8_workspace_bytes(ctypes.byref(cfg)))


def hqml_dense8_create(cfg: hqml_dense_config) -> ctypes.c_void_p:
    return _created(load().hqml_dense8_create, cfg)


def hqml_dense8_destroy(h) -> None:
    load().hqml_dense8_destroy(h)


def hqml_dense8_last_error(h) -> str:
    return load().hqml_dense8_last_error(h).decode()


def hqml_dense8_forward(h, M, x_ptr, ldx, codes_ptr, ldw, scales_ptr, bias_ptr, residual_ptr, ldr, y_ptr, ldy) -> None:
    rc = load().hqml_dense8_forward(h, M, x_ptr, ldx, codes_ptr, ldw, scales_ptr, bias_ptr, residual_ptr, ldr, y_ptr, ldy)
    if rc != HQML_OK:
        raise HqmlError(rc, hqml_dense8_last_error(h))


def hqml_norm_workspace_bytes(cfg: hqml_norm_config) -> int:
    return int(load().hqml_norm_workspace_bytes(ctypes.byref(cfg)))


def hqml_norm_create(cfg: hqml_norm_config) -> ctypes.c_void_p:
    return _created(load().hqml_norm_create, cfg)


def hqml_norm_destroy(h) -> None:
    load().hqml_norm_destroy(h)


def hqml_norm_last_error(h) -> str:
    return load().hqml_norm_last_error(h).decode()


def hqml_norm_forward(h, B, S, x_ptr, ldx, gamma_ptr, beta_ptr, y_ptr, ldy, mean_ptr, rstd_ptr) -> None:
    rc = load().hqml_norm_forward(h, B, S, x_ptr, ldx, gamma_ptr, beta_ptr, y_ptr, ldy, mean_ptr, rstd_ptr)
    if rc != HQML_OK:
        raise HqmlError(rc, hqml_norm_last_error(h))


def hqml_norm_backward(h, B, S, dy_ptr, lddy, x_ptr, ldx, gamma_ptr, beta_ptr, mean_ptr, rstd_ptr, dx_ptr, lddx, dgamma_ptr,
                       dbeta_ptr) -> None:
    rc = load().hqml_norm_backward(h, B, S, dy_ptr, lddy, x_ptr, ldx, gamma_ptr, beta_ptr, mean_ptr, rstd_ptr, dx_ptr, lddx,
                                   dgamma_ptr, dbeta_ptr)
    if rc != HQML_OK:
        raise HqmlError(rc, hqml_norm_last_error(h))


def hqml_muon_workspace_bytes(cfg: hqml_muon_config, n_tensors, tensors) -> int:
    """tensors: a ctypes array of hqml_muon_tensor, or their bytes."""
    return int(load().hqml_muon_workspace_bytes(ctypes.byref(cfg), int(n_tensors), tensors))


def hqml_muon_step(cfg: hqml_muon_config, n_tensors, tensors, workspace_ptr, workspace_bytes) -> None:
    lib = load()
    rc = lib.hqml_muon_step(ctypes.byref(cfg), int(n_tensors), tensors, workspace_ptr, int(workspace_bytes))
    if rc != HQML_OK:
        raise HqmlError(rc, lib.hqml_last_error(None).decode())


def hqml_set_timing(ctx, enable: bool) -> None:
    _check(ctx, load().hqml_set_timing(ctx, int(bool(enable))))


def hqml_set_overlap(ctx, chunks: int) -> None:
    _check(ctx, load().hqml_set_overlap(ctx, int(chunks)))


def hqml_kernel_times(ctx, reset: bool = True):
    ms = (ctypes.c_double * HQML_K_COUNT)()
    cnt = (ctypes.c_longlong * HQML_K_COUNT)()
    _check(ctx, load().hqml_kernel_times(ctx, ms, cnt, int(bool(reset))))
    return list(ms), list(cnt)


def hqml_plan_info(ctx):
    f, b, t = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    sb = ctypes.c_size_t()
    _check(ctx, load().hqml_plan_info(ctx, ctypes.byref(f), ctypes.byref(b), ctypes.byref(t), ctypes.byref(sb)))
    return {"fwd_passes": f.value, "bwd_passes": b.value, "tiles_per_sample": t.value,
            "state_bytes": sb.value}


# ---- convenience wrapper over torch tensors ----

class Context:
    """One hqml context on the current torch device and stream.

    Inputs and outputs are torch CUDA tensors (float32; float64 for a context with
    compute="fp64", through the *_f64 entry points); the library reads and writes
    them in place through their device pointers.
    """

    def __init__(self, n_qubits, n_layers, max_batch, storage="fp32", ckpt_block=0, device=None,
                 stream=None, fusion="fused", obs_mask=0, compute="fp32", obs_x_mask=0, entangler="cz"):
        import torch
        if not torch.cuda.is_available():
            raise RuntimeError("hqml needs a GPU (torch.cuda.is_available() is False)")
        dev = torch.cuda.current_device() if device is None else int(device)
        if stream is None:
            stream = torch.cuda.current_stream(dev).cuda_stream
        self.torch = torch
        self.device = torch.device("cuda", dev)
        self.n, self.L, self.max_batch = int(n_qubits), int(n_layers), int(max_batch)
        self.cfg = make_config(n_qubits, n_layers, max_batch, storage, ckpt_block, dev, stream, fusion,
                               obs_mask, compute, obs_x_mask, entangler)
        self.f64 = compute == "fp64" or compute == HQML_COMPUTE_FP64
        self.dtype = torch.float64 if self.f64 else torch.float32
        self.handle = hqml_create(self.cfg)
        self.fwd_id = 0          # counts forwards (the saved states belong to the latest one)

    def close(self):
        if self.handle is not None:
            hqml_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _dev(self, a, shape):
        t = self.torch
        a = t.as_tensor(a, dtype=self.dtype, device=self.device).contiguous()
        if tuple(a.shape) != tuple(shape):
            raise ValueError(f"expected shape {tuple(shape)}, got {tuple(a.shape)}")
        return a

    def forward(self, x, theta, save_for_backward=True):
        B = int(x.shape[0])
        x = self._dev(x, (B, self.n))
        theta = self._dev(theta, (self.L, self.n, 3))
        expz = self.torch.empty(B, dtype=self.dtype, device=self.device)
        fwd = hqml_forward_f64 if self.f64 else hqml_forward
        fwd(self.handle, B, x.data_ptr(), theta.data_ptr(), expz.data_ptr(), save_for_backward)
        self.fwd_id += 1
        self._keep = (x, theta)
        return expz

    def backward(self, dlde):
        dlde = self._dev(dlde, (int(dlde.shape[0]),))
        grad = self.torch.empty((self.L, self.n, 3), dtype=self.dtype, device=self.device)
        bwd = hqml_backward_f64 if self.f64 else hqml_backward
        bwd(self.handle, dlde.data_ptr(), grad.data_ptr())
        self._keep_b = dlde
        return grad

    def train_step(self, x, theta, y):
        B = int(x.shape[0])
        x = self._dev(x, (B, self.n))
        theta = self._dev(theta, (self.L, self.n, 3))
        y = self._dev(y, (B,))
        t = self.torch
        expz = t.empty(B, dtype=self.dtype, device=self.device)
        loss = t.empty(1, dtype=self.dtype, device=self.device)
        grad = t.empty((self.L, self.n, 3), dtype=self.dtype, device=self.device)
        step = hqml_train_step_f64 if self.f64 else hqml_train_step
        step(self.handle, B, x.data_ptr(), theta.data_ptr(), y.data_ptr(), expz.data_ptr(), loss.data_ptr(),
             grad.data_ptr())
        self.fwd_id += 1
        self._keep = (x, theta, y)
        return expz, loss, grad

    def set_timing(self, enable=True):
        hqml_set_timing(self.handle, enable)

    def set_overlap(self, chunks):
        hqml_set_overlap(self.handle, chunks)

    def kernel_times(self, reset=True):
        return hqml_kernel_times(self.handle, reset)

    def plan_info(self):
        return hqml_plan_info(self.handle)


class _Layer:
    """What the handles of dense layers and norms share: the device, the stream, the call's queueing and its arrays."""

    def _open(self, device, stream):
        """The handle's device, and the stream it is made on."""
        import torch
        if not torch.cuda.is_available():
            raise RuntimeError("hqml needs a GPU (torch.cuda.is_available() is False)")
        dev = torch.cuda.current_device() if device is None else int(device)
        self.torch = torch
        self.device = torch.device("cuda", dev)
        self.stream = torch.cuda.current_stream(dev).cuda_stream if stream is None else int(stream)
        self._index, self._lib = dev, load()
        self._current_stream = torch._C._cuda_getCurrentRawStream
        self.handle = None
        return dev

    def _make(self, create):
        self.dtype = self.torch.bfloat16 if self.cfg.dtype == HQML_DTYPE_BF16 else self.torch.float32
        try:
            self.handle = create(self.cfg)
        except HqmlError as e:
            if e.status != HQML_ERR_OOM:
                raise
            self.torch.cuda.empty_cache()   # torch may hold what the workspace needs, unused
            self.handle = create(self.cfg)

    def close(self):
        if self.handle is not None:
            self._destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, t, shape, name, dtype):
        if t.dtype is not dtype or t.get_device() != self._index:
            raise TypeError(f"{name} must be {dtype} on {self.device}, got {t.dtype} on {t.device}")
        if t.shape != shape:
            raise ValueError(f"expected shape {shape} for {name}, got {tuple(t.shape)}")

    def _rows(self, t, rows, length, name):
        """t, with rows the kernels can walk, and its row stride."""
        if t.dtype is not self.dtype or t.get_device() != self._index or t.shape != (rows, length):
            self._check(t, (rows, length), name, self.dtype)
        if not t.is_contiguous():
            ld = t.stride(0)
            if (length == 1 or t.stride(1) == 1) and (rows == 1 or length <= ld <= HQML_DENSE_MAX_FEATURES):
                return t, ld if rows > 1 else length
            t = t.contiguous()
        return t, length

    def _new(self, rows, length, like, ld):
        """An array [rows][length]; `like`, if its rows have no gaps, is the quicker way to one."""
        if ld == length:
            return self.torch.empty_like(like)
        return self.torch.empty((rows, length), dtype=self.dtype, device=self.device)

    def _queue(self, call, *args):
        if self._current_stream(self._index) == self.stream:
            rc = call(self.handle, *args)
        else:
            cuda = self.torch.cuda
            if not self.stream and cuda.is_current_stream_capturing():
                # the default stream takes no part in a capture, and must not wait for a stream that does
                raise RuntimeError("a handle made on the default stream cannot be captured: make it on the stream of "
                                   "the capture, or on any but the default one")
            here = cuda.current_stream(self.device)
            own = (cuda.ExternalStream(self.stream, device=self.device) if self.stream
                   else cuda.default_stream(self.device))
            own.wait_stream(here)
            rc = call(self.handle, *args)
            here.wait_stream(own)
        if rc != HQML_OK:
            raise HqmlError(rc, self._error(self.handle))


class Dense(_Layer):
    """One dense layer's handle: y = alpha act(x w^T + bias) + residual and its gradients.

    Tensors are torch CUDA tensors of the handle's device and dtype ("fp32" or "bf16"):
    x [M][in_features], w [out_features][in_features], bias [out_features], residual and y
    [M][out_features], M <= max_batch.  Rows may be strided (a slice of columns is used in
    place); other layouts are copied.  Work is queued on the stream the handle was made on (or
    `stream`); a call from another current stream waits for that one and is waited for by it.
    A graph can capture calls of a handle made on any stream but the default one.
    """

    _destroy, _error = staticmethod(hqml_dense_destroy), staticmethod(hqml_dense_last_error)

    def __init__(self, in_features, out_features, max_batch, dtype="fp32", activation="none", alpha=1.0,
                 device=None, stream=None):
        dev = self._open(device, stream)
        self.K, self.N, self.max_batch = int(in_features), int(out_features), int(max_batch)
        self.cfg = make_dense_config(in_features, out_features, max_batch, dtype, activation, alpha, dev, self.stream)
        self.plain = self.cfg.activation == HQML_ACT_NONE   # the gradient needs no z
        self._make(hqml_dense_create)

    def _forward(self, x, w, bias, residual, out, keep):
        M = x.shape[0]
        x, ldx = self._rows(x, M, self.K, "x")
        w, ldw = self._rows(w, self.N, self.K, "w")
        if bias is not None:
            self._check(bias, (self.N,), "bias", self.dtype)
            bias = bias.contiguous()
        ldr = 0
        if residual is not None:
            residual, ldr = self._rows(residual, M, self.N, "residual")
        if out is None:
            y, ldy = self._new(M, self.N, residual, ldr), self.N
        else:
            y, ldy = self._rows(out, M, self.N, "out")
            if y is not out:
                raise ValueError("out must have rows without gaps between their elements")
            if M and y.data_ptr() in (x.data_ptr(), w.data_ptr()):
                raise ValueError("out must not overlap x or w")
        z = None
        if keep and not self.plain:
            z = self.torch.empty((M, self.N), dtype=self.torch.float32, device=self.device)
        self._queue(self._lib.hqml_dense_forward, M, x.data_ptr(), ldx, w.data_ptr(), ldw,
                    None if bias is None else bias.data_ptr(), None if residual is None else residual.data_ptr(), ldr,
                    y.data_ptr(), ldy, None if z is None else z.data_ptr())
        if out is not None:   # a backward pass that saved it from before has to refuse it
            self.torch.autograd.graph.increment_version(out)
        return y, z

    def forward(self, x, w, bias=None, residual=None, out=None):
        """y.  `out` may be the residual itself; it must not overlap another argument."""
        return self._forward(x, w, bias, residual, out, False)[0]

    def forward_train(self, x, w, bias=None, residual=None, out=None):
        """(y, z): z, in fp32, is what backward needs (None without an activation)."""
        return self._forward(x, w, bias, residual, out, True)

    def backward(self, dy, x, w, z=None, input=True, weight=True, bias=True):
        """(dx, dw, db) for dy = dL/dy and the arguments and z of a forward call; those not
        asked for are None.  The residual's gradient is dy."""
        M = dy.shape[0]
        dy, lddy = self._rows(dy, M, self.N, "dy")
        x, ldx = self._rows(x, M, self.K, "x")
        w, ldw = self._rows(w, self.N, self.K, "w")
        if not self.plain:
            if z is None:
                raise ValueError("the gradient of an activation needs the forward call's z")
            self._check(z, (M, self.N), "z", self.torch.float32)
            z = z.contiguous()
        dx = self._new(M, self.K, x, ldx) if input else None
        dw = self._new(self.N, self.K, w, ldw) if weight else None
        db = self.torch.empty(self.N, dtype=self.dtype, device=self.device) if bias else None
        self._queue(self._lib.hqml_dense_backward, M, dy.data_ptr(), lddy, x.data_ptr(), ldx, w.data_ptr(), ldw,
                    None if self.plain else z.data_ptr(), dx.data_ptr() if input else None, self.K,
                    dw.data_ptr() if weight else None, db.data_ptr() if bias else None)
        return dx, dw, db


def quantise_rows(x):
    """(codes, scales) of the rows of x, a CUDA tensor [rows][K] in fp32 or bf16: x ~ codes * scales[:, None], codes of
    -127..127 in int8, scales in fp32.  The codes' rows are a multiple of 16 apart, as DenseInt8 takes them.  Runs on the
    current stream of x's device."""
    import torch
    if x.dim() != 2 or x.dtype not in (torch.float32, torch.bfloat16) or not x.is_cuda:
        raise TypeError(f"x must be a CUDA matrix in fp32 or bf16, got {x.dtype} {tuple(x.shape)} on {x.device}")
    rows, K = x.shape
    if K < 1:
        raise ValueError("rows must not be empty")
    x = x.detach()
    ldx = x.stride(0)
    if (K > 1 and x.stride(1) != 1) or (rows > 1 and not K <= ldx <= HQML_DENSE_MAX_FEATURES):
        x = x.contiguous()
        ldx = K
    Kp = -(-K // 16) * 16
    codes = torch.empty((rows, Kp), dtype=torch.int8, device=x.device)
    scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    dtype = HQML_DTYPE_BF16 if x.dtype is torch.bfloat16 else HQML_DTYPE_FP32
    device = x.get_device()
    hqml_quantise_rows(device, torch._C._cuda_getCurrentRawStream(device), dtype, rows, K, x.data_ptr(),
                       ldx if rows > 1 else K, codes.data_ptr(), Kp, scales.data_ptr())
    return codes[:, :K], scales


class DenseInt8(_Layer):
    """A dense layer served in 8-bit integers: y = alpha act(x w^T + bias) + residual with w given as codes and scales
    (quantise_rows) and x rounded to codes within the call, a scale for each of its rows.

    x, bias, residual and y as Dense's, in fp32 or bf16; codes [out_features][in_features] in int8, rows a multiple
    of 16 apart (others are copied), scales [out_features] in fp32.  Streams and graphs as Dense's.  There is no gradient."""

    _destroy, _error = staticmethod(hqml_dense8_destroy), staticmethod(hqml_dense8_last_error)

    def __init__(self, in_features, out_features, max_batch, dtype="fp32", activation="none", alpha=1.0,
                 device=None, stream=None):
        dev = self._open(device, stream)
        self.K, self.N, self.max_batch = int(in_features), int(out_features), int(max_batch)
        self.cfg = make_dense_config(in_features, out_features, max_batch, dtype, activation, alpha, dev, self.stream)
        self._make(hqml_dense8_create)

    def _codes(self, codes):
        """codes in rows that the kernels can load sixteen at a time, and the rows' distance."""
        N, K, Kp = self.N, self.K, -(-self.K // 16) * 16
        self._check(codes, (N, K), "codes", self.torch.int8)
        ld = codes.stride(0) if N > 1 else Kp
        if ((K == 1 or codes.stride(1) == 1) and ld % 16 == 0 and Kp <= ld <= HQML_DENSE_MAX_FEATURES
                and codes.data_ptr() % 16 == 0
                and codes.storage_offset() + (N - 1) * ld + Kp <= codes.untyped_storage().nbytes()):
            return codes, ld
        held = self.torch.zeros((N, Kp), dtype=self.torch.int8, device=self.device)
        held[:, :K] = codes
        return held, Kp

    def forward(self, x, codes, scales, bias=None, residual=None, out=None):
        """y.  `out` may be the residual itself; it must not overlap another argument."""
        M = x.shape[0]
        x, ldx = self._rows(x, M, self.K, "x")
        codes, ldw = self._codes(codes)
        self._check(scales, (self.N,), "scales", self.torch.float32)
        scales = scales.contiguous()
        if bias is not None:
            self._check(bias, (self.N,), "bias", self.dtype)
            bias = bias.contiguous()
        ldr = 0
        if residual is not None:
            residual, ldr = self._rows(residual, M, self.N, "residual")
        if out is None:
            y, ldy = self._new(M, self.N, residual, ldr), self.N
        else:
            y, ldy = self._rows(out, M, self.N, "out")
            if y is not out:
                raise ValueError("out must have rows without gaps between their elements")
        self._queue(self._lib.hqml_dense8_forward, M, x.data_ptr(), ldx, codes.data_ptr(), ldw, scales.data_ptr(),
                    None if bias is None else bias.data_ptr(), None if residual is None else residual.data_ptr(), ldr,
                    y.data_ptr(), ldy)
        if out is not None:   # a backward pass that saved it from before has to refuse it
            self.torch.autograd.graph.increment_version(out)
        return y


class GroupNorm(_Layer):
    """Group norm with an activation, channels last: y = act(weight xhat + bias), xhat = (x - mean) rstd over a sample's
    group of channels / groups neighbouring channels and all its positions.

    x [samples][...positions][channels] in fp32 or bf16 (the handle's dtype), samples times positions up to max_rows;
    weight and bias [channels] or None.  Positions may be strided evenly (a slice of channels is used in place); other
    layouts are copied.  Streams and graphs as Dense's."""

    _destroy, _error = staticmethod(hqml_norm_destroy), staticmethod(hqml_norm_last_error)

    def __init__(self, channels, groups, max_rows, dtype="fp32", activation="none", eps=1e-5, device=None, stream=None):
        dev = self._open(device, stream)
        self.C, self.G, self.max_rows = int(channels), int(groups), int(max_rows)
        self.cfg = make_norm_config(channels, groups, max_rows, dtype, activation, eps, dev, self.stream)
        self._make(hqml_norm_create)

    def _positions(self, t, shape, name):
        """t with positions the kernels can walk, and their distance."""
        if t.dtype is not self.dtype or t.get_device() != self._index or t.shape != shape:
            self._check(t, tuple(shape), name, self.dtype)
        if not t.is_contiguous():
            rows = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n > 1]   # from the outermost in
            ld = rows[-1][1] if rows else self.C
            even = all(a[1] == b[0] * b[1] for a, b in zip(rows, rows[1:]))
            if (self.C == 1 or t.stride(-1) == 1) and even and self.C <= ld <= HQML_DENSE_MAX_FEATURES:
                return t, ld
            t = t.contiguous()
        return t, self.C

    def _sizes(self, x):
        if x.dim() < 2:
            raise ValueError(f"expected [samples][...][{self.C}], got {tuple(x.shape)}")
        shape, S = x.shape, 1
        for n in shape[1:-1]:
            S *= n
        if shape[-1] != self.C:
            raise ValueError(f"expected {self.C} channels, got {tuple(shape)}")
        return shape, shape[0], S

    def _like(self, x, shape):
        """An array without gaps; `x`, if it has none, is the quicker way to one."""
        if x.is_contiguous():
            return self.torch.empty_like(x)
        return self.torch.empty(shape, dtype=self.dtype, device=self.device)

    def _parameter(self, t, name):
        if t is None:
            return None
        self._check(t, (self.C,), name, self.dtype)
        return t.contiguous()

    def _forward(self, x, weight, bias, out, keep):
        shape, B, S = self._sizes(x)
        x, ldx = self._positions(x, shape, "x")
        weight, bias = self._parameter(weight, "weight"), self._parameter(bias, "bias")
        if out is None:
            y, ldy = self._like(x, shape), self.C
        else:
            y, ldy = self._positions(out, shape, "out")
            if y is not out:
                raise ValueError("out must have evenly strided positions")
        mean = rstd = None
        if keep:
            mean, rstd = self.torch.empty((2, B, self.G), dtype=self.torch.float32, device=self.device).unbind()
        self._queue(self._lib.hqml_norm_forward, B, S, x.data_ptr(), ldx, None if weight is None else weight.data_ptr(),
                    None if bias is None else bias.data_ptr(), y.data_ptr(), ldy, mean.data_ptr() if keep else None,
                    rstd.data_ptr() if keep else None)
        if out is not None:   # a backward pass that saved it from before has to refuse it
            self.torch.autograd.graph.increment_version(out)
        return y, mean, rstd

    def forward(self, x, weight=None, bias=None, out=None):
        """y.  `out` may be x itself; it must not overlap another argument."""
        return self._forward(x, weight, bias, out, False)[0]

    def forward_train(self, x, weight=None, bias=None):
        """(y, mean, rstd): mean and rstd [samples][groups], in fp32, are what backward needs."""
        return self._forward(x, weight, bias, None, True)

    def backward(self, dy, x, weight, bias, mean, rstd, input=True, parameters=True):
        """(dx, dweight, dbias) for dy = dL/dy and the arguments and statistics of a forward_train call; those not asked
        for are None."""
        shape, B, S = self._sizes(x)
        x, ldx = self._positions(x, shape, "x")
        dy, lddy = self._positions(dy, shape, "dy")
        weight, bias = self._parameter(weight, "weight"), self._parameter(bias, "bias")
        for t, name in ((mean, "mean"), (rstd, "rstd")):
            self._check(t, (B, self.G), name, self.torch.float32)
        mean, rstd = mean.contiguous(), rstd.contiguous()
        dx = self._like(x, shape) if input else None
        dw = db = None
        if parameters:
            dw, db = self.torch.empty((2, self.C), dtype=self.dtype, device=self.device).unbind()
        self._queue(self._lib.hqml_norm_backward, B, S, dy.data_ptr(), lddy, x.data_ptr(), ldx,
                    None if weight is None else weight.data_ptr(), None if bias is None else bias.data_ptr(),
                    mean.data_ptr(), rstd.data_ptr(), dx.data_ptr() if input else None, self.C,
                    dw.data_ptr() if parameters else None, db.data_ptr() if parameters else None)
        return dx, dw, db
