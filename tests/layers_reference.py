"""The 8-bit dense layer, group norm and Muon in 64 bits, with bounds on what the library's results may be off by.

E = 2^-24 is the rounding unit of 32-bit arithmetic, u that of an array's type (half a step: 2^-24 fp32, 2^-8 bf16)."""
import math

import torch

E = 2.0 ** -24
TYPES = {"fp32": (torch.float32, 2.0 ** -24), "bf16": (torch.bfloat16, 2.0 ** -8)}
ACTS = ("none", "relu", "gelu", "silu", "tanh", "sigmoid")


def act64(z, act):
    """The activation and its slope."""
    f = {"none": lambda t: t, "relu": torch.nn.functional.relu, "gelu": torch.nn.functional.gelu,
         "silu": torch.nn.functional.silu, "tanh": torch.tanh, "sigmoid": torch.sigmoid}[act]
    z = z.detach().requires_grad_(True)
    a = f(z) * 1.0
    s, = torch.autograd.grad(a.sum(), z)
    return a.detach(), s


def excess(got, want):
    """How far the worst value is above its bound (not above 0 if all are within); a NaN is."""
    value, bound = want
    d = (got.double() - value).abs() - bound
    return float("inf") if bool(torch.isnan(d).any()) else float(d.max()) if d.numel() else 0.0


# ---- 8-bit integers ----

def codes64(x):
    """(codes, scales) of the rows of x by their definition, with whole numbers and fractions only.

    With scale = size / 127 the code is the nearest integer to 127 x / size, ties to even: 254 |x| and (2 n + 1) size are exact
    in 64 bits for x in 32, so comparing them decides the side."""
    x = x.double()
    size = x.abs().amax(1, keepdim=True)
    num = torch.where(size > 127 * 2.0 ** -100, torch.full_like(size, 127.0), torch.full_like(size, 2.0 ** 100))
    den = torch.where(size > 127 * 2.0 ** -100, size, torch.ones_like(size))
    a = x.abs() * num
    n = torch.floor(a / den)
    n = torch.where(n * den > a, n - 1, n)
    n = torch.where((n + 1) * den <= a, n + 1, n)
    above = 2 * a - (2 * n + 1) * den
    n = n + torch.where(above > 0, 1.0, torch.where(above < 0, 0.0, torch.remainder(n, 2.0)))
    finite = torch.isfinite(size)
    codes = torch.where(finite, torch.sign(x) * n, torch.zeros_like(n))
    scales = torch.where(finite, torch.clamp(size / 127, min=2.0 ** -100), torch.full_like(size, math.nan))
    return torch.where(torch.isnan(codes), torch.zeros_like(codes), codes).to(torch.int8), scales.float()[:, 0]


def dense8(x, codes, scales, bias, residual, act, alpha, dtype):
    """(y, bound).  Sums of codes are exact, so z is off by the conversion of a sum to fp32, the scales' product, its
    product with the sum and the bias: 3 E |z0| and E |z|.  y: |alpha| (1.2 err(z) + 32 E (1 + |z|)): slopes are below 1.13, the
    activations good to that; 2 E for alpha and the residual; u for the rounding."""
    u = TYPES[dtype][1]
    cx, sx = codes64(x)
    z = (cx.double() @ codes.double().t()) * sx.double()[:, None] * scales.double()
    ez = 4 * E * z.abs()
    if bias is not None:
        z = z + bias.double()
    ez = ez + E * z.abs()
    a, _ = act64(z, act)
    y = alpha * a
    ey = abs(alpha) * (1.2 * ez + (32 * E * (1 + z.abs()) if act != "none" else 0)) + E * y.abs()
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2 * E * y.abs()
    return y, ey + u * (y.abs() + ey)


# ---- group norm ----

def norm(x, gamma, beta, dy, G, act, eps, dtype):
    """{name: (value, bound)} of y, mean, rstd and, if dy is given, dx, dgamma, dbeta.

    A sum of n values in 32 bits is off by at most E times the longest chain of additions times the sum of magnitudes.
    Chains here: 16 positions of a thread, up to 512 threads, 32 channels, or the partial sums of up to 32 workgroups
    after each other: below 700; no more than n.  Beyond one workgroup, chunks are joined by means, which adds a few.
      mean: D E mean|x|          var: the mean's error squared, and (D + 4) E var
      rstd: half of var's relative error, and 4 E for the root and quotient
      xhat, z, y, dz and the sums: errors through the formulas, D E of the magnitudes for each sum."""
    u = TYPES[dtype][1]
    x = x.double()
    C = x.shape[-1]
    B, per = x.shape[0], C // G
    X = x.reshape(B, -1, G, per)
    N = X.shape[1] * per
    D = min(N, 700) + 8
    mean = X.mean((1, 3), keepdim=True)
    emean = D * E * X.abs().mean((1, 3), keepdim=True)
    var = ((X - mean) ** 2).mean((1, 3), keepdim=True)
    evar = emean ** 2 + (D + 4) * E * (var + emean ** 2)
    rstd = 1 / torch.sqrt(var + eps)
    rel = 0.5 * evar / (var + eps) * 1.01 + 4 * E
    hat = (X - mean) * rstd
    ehat = (emean + E * (X - mean).abs()) * rstd * (1 + rel) + hat.abs() * (rel + 3 * E)
    ones = torch.ones(C, dtype=torch.float64, device=x.device)
    g = (ones if gamma is None else gamma.double()).view(G, per)
    b = (0 * ones if beta is None else beta.double()).view(G, per)
    z = hat * g + b
    ez = g.abs() * ehat + 3 * E * ((hat * g).abs() + b.abs())
    a, s = act64(z, act)
    ey = 1.2 * ez + (32 * E * (1 + z.abs()) if act != "none" else 0)
    shape = x.shape
    out = {"y": (a.view(shape), (ey + u * (a.abs() + ey)).view(shape)),
           "mean": (mean[:, 0, :, 0], emean[:, 0, :, 0] + E * mean[:, 0, :, 0].abs()),
           "rstd": (rstd[:, 0, :, 0], (rel * rstd)[:, 0, :, 0])}
    if dy is None:
        return out
    d = dy.double().view_as(X)
    dz = d * s
    edz = d.abs() * (0.8 * ez + 32 * E * (1 + z.abs())) if act != "none" else torch.zeros_like(d)
    if act == "relu":
        edz = torch.where(z.abs() <= ez, d.abs(), edz)
    edz = edz + E * dz.abs()
    D2 = min(B * X.shape[1], 1500) + 8
    h, eh = hat, ehat
    db, edb = dz.sum((0, 1)), (edz + D2 * E * (dz.abs() + edz)).sum((0, 1))
    p, ep = dz * h, edz * (h.abs() + eh) + dz.abs() * eh
    dg, edg = p.sum((0, 1)), (ep + D2 * E * (p.abs() + ep)).sum((0, 1))
    out["dbeta"] = (db.reshape(C), (edb + u * (db.abs() + edb)).reshape(C))
    out["dgamma"] = (dg.reshape(C), (edg + u * (dg.abs() + edg)).reshape(C))
    q, eq = g * dz, g.abs() * edz
    m1 = q.mean((1, 3), keepdim=True)
    em1 = (eq + (D + 4) * E * (q.abs() + eq)).mean((1, 3), keepdim=True)
    r, er = g * p, g.abs() * ep
    m2 = r.mean((1, 3), keepdim=True)
    em2 = (er + (D + 4) * E * (r.abs() + er)).mean((1, 3), keepdim=True)
    inner = q - m1 - h * m2
    einner = eq + em1 + eh * (m2.abs() + em2) + h.abs() * em2 + 4 * E * (q.abs() + m1.abs() + (h * m2).abs())
    dx = rstd * inner
    edx = rstd * (1 + rel) * einner + dx.abs() * (rel + 2 * E)
    out["dx"] = (dx.reshape(shape), (edx + u * (dx.abs() + edx)).reshape(shape))
    return out


# ---- Muon ----

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonal(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7, noise=None):
    """The polynomial steps of a matrix in 64 bits.  noise(t): what a held operand becomes."""
    keep = noise or (lambda t: t)
    a, b, c = coefficients
    x = u.double() / max(float(torch.linalg.vector_norm(u.double())), eps)
    tall = x.shape[0] > x.shape[1]
    x = keep(x.t().contiguous() if tall else x)
    for step in range(steps):
        A = keep(x @ x.t())
        B = keep(b * A + c * (A @ A))
        x = a * x + B @ x
        if step + 1 < steps:
            x = keep(x)
    return x.t().contiguous() if tall else x


def orthogonal_bound(u, dtype, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    """(X, bound on the error's norm, and on its largest value).

    Every held operand is off by a rounding: up to 2^-11 of each value for one fp16 value, 2^-22 for two, whose products also
    leave out one of that size; 32-bit sums of K terms add sqrt(K) 2^-24 or so to a value of their size, 2^-21 of it at
    these sizes.  Two 64-bit runs tell what roundings of that size make of X, one with operands off by random parts of 2^-11
    (bf16 parameters) or 2^-20 (fp32) of their values, one without.  The bound is four times their difference: the
    library's errors are another draw of the same size; its largest value at most eight times the mean size."""
    eta = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -20
    g = torch.Generator(device=u.device).manual_seed(5)

    def noise(t):
        r = torch.rand(t.shape, generator=g, device=t.device, dtype=torch.float64) * 2 - 1
        return t * (1 + eta * r)

    x = orthogonal(u, steps, coefficients, eps)
    d = orthogonal(u, steps, coefficients, eps, noise) - x
    norm_of = float(torch.linalg.vector_norm(d))
    return x, 4 * norm_of, 8 * 4 * norm_of / math.sqrt(x.numel())


def muon(p, g, m, lr, mu, decay, nesterov, f, bits=False):
    """(m, u) of a step in 64 bits, before it is orthogonalised."""
    g, m = g.double(), m.double()
    m = mu * m + (1 - mu) * g
    return m, mu * m + (1 - mu) * g if nesterov else m
