"""The dense layer in 64 bits, with a bound on what 32-bit sums may be off by.

With e = 2^-24 the rounding unit of the sums and u that of the arrays' type (2^-24 fp32, 2^-8 bf16), elementwise:
  z:   (K + 8) e (|x| |w|^T + |bias|): K products and a bias in any order; a product of planes rounds its sum six times
       a step and leaves out 2 e.  z is held in 32 bits with either type
  y:   |alpha| (1.2 err(z) + 32 e (1 + |z|)): slopes are below 1.13, the activations good to that; 2 e for the
       residual's sum; u for the rounding
  dz:  |alpha dy| (0.8 err(z) + 32 e (1 + |z|)) as |act''| < 0.8; where z's sign is open, relu's slope is too. bf16
       gradients that are not small: u |dz|, as dz goes through memory; never in db, whose sums take it before
  dx, dw, db: err(dz) through the product's magnitudes, (terms + 8) e times the magnitudes, u for the rounding.
"""
import math

import torch

E = 2.0 ** -24
TYPES = {"fp32": (torch.float32, 2.0 ** -24), "bf16": (torch.bfloat16, 2.0 ** -8)}


def make(M, K, N, dtype, seed, device="cuda", offset=0, gap=0, bias=True, residual=True):
    """Arguments of a training step; rows begin `offset` elements into a wider array and are `gap` elements apart, NaN
    between them."""
    g = torch.Generator(device=device).manual_seed(seed)

    def rows(n, length, scale=1.0):
        wide = torch.full((n * (length + gap) + offset,), float("nan"), dtype=TYPES[dtype][0], device=device)
        t = wide[offset:].view(n, length + gap)[:, :length]
        t.copy_(torch.randn(n, length, generator=g, device=device) * scale)
        return t

    return dict(x=rows(M, K), w=rows(N, K, 1.0 / math.sqrt(K)),
                bias=(torch.randn(N, generator=g, device=device) * 0.3).to(TYPES[dtype][0]) if bias else None,
                residual=rows(M, N) if residual else None, dy=rows(M, N, 1.0 / math.sqrt(M)))


def act64(z, act):
    f = {"none": lambda t: t, "relu": torch.nn.functional.relu, "gelu": torch.nn.functional.gelu,
         "silu": torch.nn.functional.silu, "tanh": torch.tanh, "sigmoid": torch.sigmoid}[act]
    z = z.detach().requires_grad_(True)
    a = f(z) * 1.0
    s, = torch.autograd.grad(a.sum(), z)
    return a.detach(), s


def expect(d, dtype, act, alpha, small, held=lambda z: z):
    """(value, bound) of y, z, dx, dw, db.  small: gradients of a small layer, whose dz is never rounded.  held: what z
    becomes between the passes (a planted mistake)."""
    u = TYPES[dtype][1]
    x, w, dy = (d[k].detach().double().contiguous() for k in ("x", "w", "dy"))
    (M, K), N = x.shape, w.shape[0]
    b = torch.zeros(N, dtype=torch.float64, device=x.device) if d["bias"] is None else d["bias"].double()
    wt = w.t().contiguous()
    z = x @ wt + b
    ez = (K + 8) * E * (x.abs() @ wt.abs() + b.abs())
    a, _ = act64(z, act)
    y = alpha * a
    ey = abs(alpha) * (1.2 * ez + 32 * E * (1 + z.abs()))
    if d["residual"] is not None:
        ey = ey + 2 * E * y.abs()
        y = y + d["residual"].double()
        ey = ey + 2 * E * y.abs()
    ey = ey + u * (y.abs() + ey)
    _, s = act64(held(z), act)
    dz = alpha * s * dy
    if act == "none":
        edz = 2 * E * dz.abs()
    else:
        edz = (alpha * dy).abs() * (0.8 * ez + 32 * E * (1 + z.abs()))
        if act == "relu":
            edz = torch.where(z.abs() <= ez, (alpha * dy).abs(), edz)
    ein = edz if small or dtype == "fp32" else edz + u * (dz.abs() + edz)

    def product(A, eA, B, terms):
        m = A.abs() @ B.abs()
        err = eA @ B.abs()
        v, err = A @ B, err + (terms + 8) * E * (m + err)
        return v, err + u * (v.abs() + err)

    dzt = dz.t().contiguous()
    ones = torch.ones(M, 1, dtype=torch.float64, device=x.device)
    db, edb = product(dzt, edz.t().contiguous(), ones, M)
    return {"y": (y, ey), "z": (z, ez), "dx": product(dz, ein, w, N), "dw": product(dzt, ein.t().contiguous(), x, M),
            "db": (db[:, 0], edb[:, 0])}


def excess(got, want):
    """How far the worst value is above its bound (not above 0 if all are within)."""
    value, bound = want
    return float(((got.double() - value).abs() - bound).max())


def run(d, dtype, act, alpha, layer=None):
    """A training step of the library."""
    import qml_gradients_amd as hq
    (M, K), N = d["x"].shape, d["w"].shape[0]
    layer = layer or hq.Dense(K, N, M, dtype=dtype, activation=act, alpha=alpha)
    y, z = layer.forward_train(d["x"], d["w"], d["bias"], d["residual"])
    dx, dw, db = layer.backward(d["dy"], d["x"], d["w"], z)
    return {"y": y, "z": z, "dx": dx, "dw": dw, "db": db}
