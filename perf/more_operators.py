"""Three more operators of the layers around the circuits, and what to measure of them.

In their plain form (elementary torch operations) and as the library's calls:

  * dense8: a dense layer served in 8-bit integers, y = alpha act(x w^T + bias) + residual.
    The weights are held as codes times a scale for each output channel; x is rounded to codes
    times a scale for each of its rows (tokens, samples) within the call.
    scale = max(largest magnitude of the row / 127, 2^-100), code = the nearest integer to
    x / scale, ties to even.
  * muon: one step of momentum and orthogonalised updates over a model's weight matrices.
    m = MOMENTUM m + (1 - MOMENTUM) g, u = MOMENTUM m + (1 - MOMENTUM) g (Nesterov) or m;
    X = u / max(|u|, EPS) goes five times through X <- a X + (b A + c A^2) X, A = X X^T, which
    brings its singular values near 1; p = p (1 - lr decay) - lr sqrt(max(1, rows / columns)) X.
  * norm, norm_train: group norm over channels-last arrays [batch][positions][channels] with an
    activation, y = act(gamma xhat + beta); norm_train is the forward pass and the gradients
    dx, dgamma and dbeta for a given dy.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu", "tanh", "sigmoid")
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "bf16": 2}
SCALE_MIN = 2.0 ** -100
LR, MOMENTUM, DECAY, EPS = 0.02, 0.95, 0.01, 1e-7
STEPS, COEFFICIENTS = 5, (3.4445, -4.7750, 2.0315)
NORM_EPS = 1e-5
PRODUCT_MOST = 8192 * 4096 * 4096        # multiply-adds of the largest dense8 case
NORM_MOST = 32 * 4096 * 512              # elements of the largest norm case


def dense8_case(name, M, K, N, dtype, act, alpha=1.0, bias=True, residual=False):
    return {"name": name, "op": "dense8", "M": M, "K": K, "N": N, "dtype": dtype, "act": act, "alpha": alpha,
            "bias": bias, "residual": residual}


def muon_case(name, tensors, rows, cols, dtype, nesterov=True):
    return {"name": name, "op": "muon", "tensors": tensors, "rows": rows, "cols": cols, "dtype": dtype,
            "nesterov": nesterov}


def norm_case(name, op, B, S, C, G, dtype, act):
    return {"name": name, "op": op, "B": B, "S": S, "C": C, "G": G, "dtype": dtype, "act": act}


def listed():
    return [
        # one 28 x 28 image becomes the angles of a 20-qubit circuit: pure latency
        dense8_case("serve8_sample", 1, 784, 20, "fp32", "sigmoid", math.pi),
        # one sample through a wide residual layer: every code is read once
        dense8_case("serve8_one", 1, 4096, 4096, "bf16", "gelu", residual=True),
        # a small batch of no round size anywhere
        dense8_case("serve8_ragged", 45, 1531, 803, "fp32", "silu", residual=True),
        # the largest forward pass: a big batch through a wide residual layer
        dense8_case("serve8_large", 8192, 4096, 4096, "bf16", "gelu", residual=True),
        # a readout's three small matrices: pure latency
        muon_case("muon_readout", 3, 64, 32, "fp32"),
        # four matrices of no round size anywhere
        muon_case("muon_ragged", 4, 803, 517, "fp32", nesterov=False),
        # an ordinary 32-bit encoder: wide matrices
        muon_case("muon_encoder", 2, 1024, 4096, "fp32"),
        # two wide residual layers' weights
        muon_case("muon_wide", 2, 4096, 4096, "bf16"),
        # one 28 x 28 image of 32 channels: pure latency
        norm_case("norm_sample", "norm", 1, 784, 32, 8, "fp32", "silu"),
        # feature vectors without positions in front of a dense layer
        norm_case("norm_features", "norm_train", 1000, 1, 784, 16, "fp32", "tanh"),
        # training over 7 x 7 positions, three channels a group
        norm_case("norm_ragged", "norm_train", 61, 49, 123, 41, "bf16", "gelu"),
        # the largest: 64 x 64 positions of 512 channels
        norm_case("norm_large", "norm_train", 32, 4096, 512, 32, "bf16", "silu"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("dense8", "muon", "norm", "norm_train"))
    dtype = rng.choice(("fp32", "bf16"))
    while op == "dense8":
        M, K, N = spread(1, 16384), spread(12, 8192), spread(4, 8192)
        if rng.random() < 0.5:
            M, K, N = (v if v < 16 else v // 16 * 16 for v in (M, K, N))
        if M * K * N <= PRODUCT_MOST:
            act = rng.choice(ACTS)
            return {"op": op, "M": M, "K": K, "N": N, "dtype": dtype, "act": act,
                    "alpha": math.pi if act == "sigmoid" else 1.0, "bias": rng.random() < 0.8,
                    "residual": rng.random() < 0.5}
    while op == "muon":
        case = {"op": op, "tensors": rng.randint(1, 8), "rows": spread(4, 6000), "cols": spread(4, 6000), "dtype": dtype,
                "nesterov": rng.random() < 0.7}
        if rng.random() < 0.4:
            case["rows"], case["cols"] = (v if v < 16 else v // 16 * 16 for v in (case["rows"], case["cols"]))
        if plain_cost(case) <= plain_cost({"tensors": 2, "rows": 4096, "cols": 4096}):
            return case
    while True:
        B, S, G, per = spread(1, 2000), spread(1, 16384), spread(1, 64), spread(1, 64)
        if B * S * G * per <= NORM_MOST and G * per <= 2048 and S * per >= 4:
            # relu's slope jumps at 0: the last bit of one z would decide a whole term of the sums
            act = rng.choice(ACTS if op == "norm" else [a for a in ACTS if a != "relu"])
            return {"op": op, "B": B, "S": S, "C": G * per, "G": G, "dtype": dtype, "act": act}


def plain_cost(case):
    n, m = sorted((case["rows"], case["cols"]))
    return case["tensors"] * n * n * (4 * m + 2 * n)


def shapes(case):
    """(rows, columns) of each matrix of a muon case: every other one lies the other way round."""
    r, c = case["rows"], case["cols"]
    return [(c, r) if i % 2 else (r, c) for i in range(case["tensors"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = dict(case)
    dt = TYPES[case["dtype"]]
    if case["op"] == "muon":
        s["p"], s["g"], s["m"] = [], [], []
        for r, c in shapes(case):
            s["p"].append(normal(r, c, scale=0.05, dtype=dt))

            def gradient():   # a few directions stand out of the noise
                few = normal(r, 8) @ normal(8, c)
                return (few + normal(r, c)) * 1e-3
            s["g"].append(gradient().to(dt))
            s["m"].append(gradient())
        if own:
            from qml_gradients_amd.optim import Muon
            params = [torch.nn.Parameter(p) for p in s["p"]]
            opt = Muon(params, lr=LR, momentum=MOMENTUM, weight_decay=DECAY, nesterov=case["nesterov"],
                       coefficients=COEFFICIENTS, steps=STEPS, eps=EPS)
            for p, grad, m in zip(params, s["g"], s["m"]):
                p.grad = grad
                opt.state[p]["momentum"] = m
            s["opt"] = opt
        return s
    if case["op"] == "dense8":
        M, K, N = case["M"], case["K"], case["N"]
        # rows of unlike sizes
        s["x"] = (normal(M, K) * torch.exp(normal(M, 1))).to(dt)
        w = (torch.rand(N, K, generator=g, device="cuda") * 2 - 1) / math.sqrt(K) * 1.7
        w = (w * torch.exp(0.3 * normal(N, 1))).to(dt)
        s["b"] = normal(N, scale=0.1, dtype=dt) if case["bias"] else None
        s["r"] = normal(M, N, dtype=dt) if case["residual"] else None
        if own:
            import qml_gradients_amd as hq
            s["codes"], s["scales"] = hq.quantise_rows(w)
            s["layer"] = hq.DenseInt8(K, N, M, dtype=case["dtype"], activation=case["act"], alpha=case["alpha"])
        else:
            s["codes"], s["scales"] = quantise(w)
        return s
    B, S, C = case["B"], case["S"], case["C"]
    # channels of unlike sizes and means
    s["x"] = (normal(B, S, C) * torch.exp(0.5 * normal(C)) + 2 * normal(C)).to(dt)
    s["gamma"] = (1 + 0.3 * normal(C)).to(dt)
    s["beta"] = normal(C, scale=0.3, dtype=dt)
    if case["op"] == "norm_train":
        s["dy"] = normal(B, S, C, scale=1.0 / math.sqrt(B * S), dtype=dt)
    if own:
        import qml_gradients_amd as hq
        s["layer"] = hq.GroupNorm(C, case["G"], B * S, dtype=case["dtype"], activation=case["act"], eps=NORM_EPS)
    return s


# ---- the plain forms ----

def activate(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "tanh":
        return torch.tanh(z)
    return 1 / (1 + torch.exp(-z))


def slope(z, act):
    """d act / dz"""
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi)
    if act == "tanh":
        t = torch.tanh(z)
        return 1 - t * t
    f = 1 / (1 + torch.exp(-z))
    return f * (1 - f) if act == "sigmoid" else f * (1 + z * (1 - f))


def quantise(x):
    """(codes, scales) of x's rows.  In 64 bits, where a quotient next to the middle of two codes goes to its own."""
    size = x.abs().amax(1, keepdim=True).double()
    scale = torch.clamp(size / 127, min=SCALE_MIN)
    codes = torch.where(size / 127 > SCALE_MIN, x.double() * 127 / size, x.double() / scale)
    return torch.round(codes).to(torch.int8), scale.float()[:, 0]


def plain_dense8(s):
    codes, scales = quantise(s["x"])
    # sums of products of codes: whole numbers, exact in 32 bits up to 2^24
    z = (codes.float() @ s["codes"].float().t()) * (scales[:, None] * s["scales"])
    if s["b"] is not None:
        z = z + s["b"].float()
    y = activate(z, s["act"]) * s["alpha"]
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(s["x"].dtype)}


def plain_muon(p, g, m, nesterov):
    """One matrix's step, in place."""
    G = g.float()
    M = m * MOMENTUM + G * (1 - MOMENTUM)
    X = M * MOMENTUM + G * (1 - MOMENTUM) if nesterov else M
    X = X / torch.sqrt((X.double() * X.double()).sum()).clamp_min(EPS).float()
    tall = X.shape[0] > X.shape[1]
    if tall:
        X = X.t()
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    if tall:
        X = X.t()
    size = LR * math.sqrt(max(1.0, p.shape[0] / p.shape[1]))
    p.copy_(p.float() * (1 - LR * DECAY) - size * X)
    m.copy_(M)


def plain_norm(s):
    B, S, C, G = s["B"], s["S"], s["C"], s["G"]
    dt = s["x"].dtype
    x = s["x"].float().view(B, S, G, C // G)
    gamma, beta = s["gamma"].float(), s["beta"].float()
    centred = x - x.mean((1, 3), keepdim=True)
    r = 1 / torch.sqrt((centred * centred).mean((1, 3), keepdim=True) + NORM_EPS)
    xhat = (centred * r).view(B, S, C)
    z = xhat * gamma + beta
    out = {"y": activate(z, s["act"]).to(dt)}
    if s["op"] == "norm_train":
        dz = s["dy"].float() * slope(z, s["act"])
        out["dgamma"], out["dbeta"] = (dz * xhat).sum((0, 1)).to(dt), dz.sum((0, 1)).to(dt)
        d, h = (dz * gamma).view(B, S, G, C // G), xhat.view(B, S, G, C // G)
        dx = r * (d - d.mean((1, 3), keepdim=True) - h * (d * h).mean((1, 3), keepdim=True))
        out["dx"] = dx.view(B, S, C).to(dt)
    return out


def run(state):
    s = state
    if s["op"] == "muon":
        if own:
            s["opt"].step()
        else:
            for p, g, m in zip(s["p"], s["g"], s["m"]):
                plain_muon(p, g, m, s["nesterov"])
        return {"p": s["p"], "m": s["m"]}
    if s["op"] == "dense8":
        if own:
            return {"y": s["layer"].forward(s["x"], s["codes"], s["scales"], s["b"], s["r"])}
        return plain_dense8(s)
    if not own:
        return plain_norm(s)
    layer = s["layer"]
    if s["op"] == "norm":
        return {"y": layer.forward(s["x"], s["gamma"], s["beta"])}
    y, mean, rstd = layer.forward_train(s["x"], s["gamma"], s["beta"])
    dx, dgamma, dbeta = layer.backward(s["dy"], s["x"], s["gamma"], s["beta"], mean, rstd)
    return {"y": y, "dgamma": dgamma, "dbeta": dbeta, "dx": dx}


# ---- what a pass cannot do without ----

def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "muon":
        values = sum(r * c for r, c in shapes(case))
        n, m = sorted((case["rows"], case["cols"]))
        # gradient read, parameter and momentum read and written; X X^T and A^2 are symmetric
        return {"bytes": values * (3 * b + 8),
                "flops": case["tensors"] * STEPS * (n * (n + 1) * m + n * n * (n + 1) + 2 * n * n * m)}
    if case["op"] == "dense8":
        M, K, N = case["M"], case["K"], case["N"]
        values = M * K + (N if case["bias"] else 0) + (M * N if case["residual"] else 0) + M * N
        return {"bytes": b * values + N * K + 4 * N, "flops": 2 * M * N * K}
    values, C = case["B"] * case["S"] * case["C"], case["C"]
    if case["op"] == "norm":
        return {"bytes": b * (2 * values + 2 * C), "flops": 12 * values}
    return {"bytes": b * (4 * values + 4 * C), "flops": 30 * values}


# ---- the same from the definitions, in 64 bits ----

def exact_rows(x):
    """Rows of x as the values that codes and scales of 64 bits stand for, the scale rounded to 32."""
    x = x.double()
    largest = x.abs().max(1).values
    step = torch.maximum(largest / 127.0, torch.full_like(largest, SCALE_MIN))
    below = torch.floor(x / step[:, None])
    # the nearer of two neighbours by comparing products, which are exact: x 254 with (2 n + 1) largest
    if bool((largest / 127.0 <= SCALE_MIN).any()):
        lean = x / step[:, None] - below - 0.5
    else:
        below = torch.where(x * 127.0 < below * largest[:, None], below - 1, below)
        below = torch.where(x * 127.0 >= (below + 1) * largest[:, None], below + 1, below)
        lean = x * 254.0 - (2 * below + 1) * largest[:, None]
    odd = torch.remainder(below, 2.0)
    code = below + torch.where(lean > 0, 1.0, torch.where(lean < 0, 0.0, odd))
    return code, step.float().double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "muon":
        out = {"p": [], "m": []}
        a, b, c = COEFFICIENTS
        for p, g, m in zip(s["p"], s["g"], s["m"]):
            p, g, m = p.double(), g.double(), m.double()
            m = m + (1 - MOMENTUM) * (g - m)
            u = g + MOMENTUM * (m - g) if case["nesterov"] else m
            o = u / max(float(torch.linalg.vector_norm(u)), EPS)
            tall = o.shape[0] > o.shape[1]
            for _ in range(STEPS):
                # the same polynomial from whichever side is smaller
                gram = torch.matmul(o.t(), o) if tall else torch.matmul(o, o.t())
                poly = torch.matmul(gram, c * gram)
                poly += b * gram
                poly.diagonal().add_(a)
                o = torch.matmul(o, poly) if tall else torch.matmul(poly, o)
            rows, cols = p.shape
            out["p"].append(p - LR * DECAY * p - LR * max(1.0, rows / cols) ** 0.5 * o)
            out["m"].append(m)
        return out
    act = {"none": lambda t: t * 1.0, "relu": torch.nn.functional.relu, "gelu": torch.nn.functional.gelu,
           "silu": torch.nn.functional.silu, "tanh": torch.tanh, "sigmoid": torch.sigmoid}[case["act"]]
    if case["op"] == "dense8":
        code, step = exact_rows(s["x"])
        z = torch.matmul(code, s["codes"].double().t())
        z *= step[:, None]
        z *= s["scales"].double()
        if s["b"] is not None:
            z += s["b"].double()
        y = case["alpha"] * act(z)
        return {"y": y if s["r"] is None else y + s["r"].double()}
    B, S, C, G = case["B"], case["S"], case["C"], case["G"]
    x = s["x"].double().view(B, S, G, C // G)
    var, mean = torch.var_mean(x, (1, 3), correction=0, keepdim=True)
    hat = x.sub_(mean)
    hat /= torch.sqrt(var + NORM_EPS)
    hat = hat.view(B, S, C)
    z = torch.addcmul(s["beta"].double(), hat, s["gamma"].double()).requires_grad_(case["op"] == "norm_train")
    y = act(z)
    out = {"y": y.detach()}
    if case["op"] == "norm_train":
        dz, = torch.autograd.grad(y, z, s["dy"].double())
        del z, y
        out["dgamma"], out["dbeta"] = (dz * hat).sum((0, 1)), dz.sum((0, 1))
        d, h = (dz * s["gamma"].double()).view(B, S, G, C // G), hat.view(B, S, G, C // G)
        n = S * (C // G)
        first, second = d.sum((1, 3), keepdim=True) / n, (d * h).sum((1, 3), keepdim=True) / n
        out["dx"] = ((d - first - h * second) / torch.sqrt(var + NORM_EPS)).view(B, S, C)
    return out
