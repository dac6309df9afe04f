"""The operators of a trained layer around the circuits, and what to measure of them.

Two operators, in their plain form (elementary torch operations) and as the library's calls:

  * dense: y = alpha * act(x w^T + bias) + residual for a batch x [M][K], weights w [N][K].
    In front of a circuit it maps a sample's features to encoding angles
    (alpha = pi, act = sigmoid: angles in (0, pi)); behind the circuits it reads their
    expectation values out.  "dense" is the forward pass, "dense_train" the forward pass and
    the gradients dx, dw and dbias for a given dy (dresidual is dy itself).
  * adamw: one AdamW step over all of a model's tensors (circuit angles and dense weights),
    with the moments held in 32 bits (64 for 64-bit parameters) or in 8.
    In 8 bits a moment is an OCP e4m3 value times a 32-bit scale shared by 256 elements;
    the second moment is held as its square root.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu", "tanh", "sigmoid")
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp64": torch.float64}
BYTES = {"fp32": 4, "bf16": 2, "fp64": 8}
BLOCK = 256            # elements that share a scale of the 8-bit moments
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01
STEP0 = 37             # steps that the moments have behind them
LARGEST = 3 * 8192 * 4096 * 4096   # multiply-adds of the largest dense case


def dense_case(name, op, M, K, N, dtype, act, alpha=1.0, bias=True, residual=False):
    return {"name": name, "op": op, "M": M, "K": K, "N": N, "dtype": dtype, "act": act, "alpha": alpha,
            "bias": bias, "residual": residual}


def adamw_case(name, tensors, numel, dtype, bits, even=False):
    return {"name": name, "op": "adamw", "tensors": tensors, "numel": numel, "dtype": dtype, "bits": bits,
            "even": even}


def listed():
    return [
        # one sample's 64 features become the angles of the 4-qubit circuit: pure latency
        dense_case("encode_sample", "dense", 1, 64, 4, "fp32", "sigmoid", math.pi),
        # a 1,000-sample epoch of 28 x 28 images becomes angles for 20 qubits
        dense_case("encode_epoch", "dense", 1000, 784, 20, "fp32", "sigmoid", math.pi),
        # one sample through a wide residual layer: every weight is read once
        dense_case("serve_one", "dense", 1, 4096, 4096, "bf16", "gelu", residual=True),
        # a batch of no round size anywhere
        dense_case("forward_ragged", "dense", 333, 1021, 517, "bf16", "silu", residual=True),
        # the largest forward pass: a big batch through a wide residual layer
        dense_case("forward_large", "dense", 8192, 4096, 4096, "bf16", "gelu", residual=True),
        # a readout's training step: 64 samples, 12 expectation values, 64 hidden values
        dense_case("train_readout", "dense_train", 64, 12, 64, "fp32", "tanh"),
        # training at no round size anywhere
        dense_case("train_ragged", "dense_train", 997, 1531, 803, "fp32", "gelu", residual=True),
        # an ordinary 32-bit training step
        dense_case("train_fp32", "dense_train", 2048, 2048, 2048, "fp32", "silu", residual=True),
        # the largest training step
        dense_case("train_large", "dense_train", 8192, 4096, 4096, "bf16", "gelu", residual=True),
        # the 60,000 angles of the 1000-layer, 20-qubit circuit and a readout's small tensors
        adamw_case("adamw_angles", 4, 62000, "fp32", 32),
        # a model of a dozen tensors of odd sizes
        adamw_case("adamw_model", 12, 20000003, "fp32", 32),
        # eight wide layers' weights, moments in 8 bits
        adamw_case("adamw_wide_8bit", 8, 8 * 4096 * 4096, "bf16", 8, even=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    if rng.random() < 0.3:
        dtype = rng.choice(("fp32", "fp32", "bf16", "bf16", "fp64"))
        bits = 32 if dtype == "fp64" else rng.choice((32, 8))
        numel = spread(24, 2e6 if dtype == "fp64" else 8 * 4096 * 4096)
        return {"op": "adamw", "tensors": rng.randint(1, 12), "numel": max(12, numel), "dtype": dtype,
                "bits": bits, "even": rng.random() < 0.3}
    op = rng.choice(("dense", "dense_train"))
    products = 3 if op == "dense_train" else 1
    while True:
        M, K, N = spread(1, 16384), spread(12, 8192), spread(4, 8192)
        if rng.random() < 0.5:
            M, K, N = (v if v < 8 else v // 8 * 8 for v in (M, K, N))
        if products * M * K * N <= LARGEST and K != 3072 and N != 3072 and M != 3072:
            break
    dtype, act = rng.choice(("fp32", "bf16")), rng.choice(ACTS)
    if op == "dense_train" and dtype == "fp32" and act == "relu":
        act = "tanh"   # relu's slope jumps at 0: the last bit of one z would decide a whole term of the sums
    return {"op": op, "M": M, "K": K, "N": N, "dtype": dtype, "act": act,
            "alpha": math.pi if act == "sigmoid" else 1.0, "bias": rng.random() < 0.8,
            "residual": rng.random() < 0.5}


def sizes(case):
    """Elements of each tensor of an adamw case."""
    n, total = case["tensors"], case["numel"]
    if case["even"]:
        return [max(1, total // n)] * n
    weights = [(i + 1) ** 2 for i in range(n)]
    return [max(1, total * w // sum(weights)) for w in weights]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = dict(case)
    dt = TYPES[case["dtype"]]
    if case["op"] == "adamw":
        s["p"], s["g"], s["m"], s["v"], s["step"] = [], [], [], [], STEP0
        for n in sizes(case):
            s["p"].append(normal(n, scale=0.05, dtype=dt))
            # gradients of one tensor spread over several orders of magnitude
            size = torch.exp(normal(n, scale=1.5) - 7.0)
            s["g"].append((normal(n) * size).to(dt))
            m, r = normal(n) * size * 0.3, size * (0.5 + torch.rand(n, generator=g, device="cuda"))
            if case["bits"] == 8:
                s["m"].append(quantise(m))
                s["v"].append(quantise(r))
            else:
                s["m"].append(m.double() if dt == torch.float64 else m)
                s["v"].append((r * r).double() if dt == torch.float64 else r * r)
            del size, m, r
        if own:
            from qml_gradients_amd.optim import AdamW
            params = [torch.nn.Parameter(p) for p in s["p"]]
            opt = AdamW(params, lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, state_bits=case["bits"])
            for p, grad, m, v in zip(params, s["g"], s["m"], s["v"]):
                p.grad = grad
                if case["bits"] == 8:
                    opt.state[p].update(step=STEP0, exp_avg=m[0], exp_avg_scale=m[1],
                                        exp_avg_sq_root=v[0], exp_avg_sq_root_scale=v[1])
                else:
                    opt.state[p].update(step=STEP0, exp_avg=m, exp_avg_sq=v)
            s["opt"] = opt
        return s
    M, K, N = case["M"], case["K"], case["N"]
    s["x"] = normal(M, K, dtype=dt)
    s["w"] = ((torch.rand(N, K, generator=g, device="cuda") * 2 - 1) / math.sqrt(K) * 1.7).to(dt)
    s["b"] = normal(N, scale=0.1, dtype=dt) if case["bias"] else None
    s["r"] = normal(M, N, dtype=dt) if case["residual"] else None
    if case["op"] == "dense_train":
        s["dy"] = normal(M, N, scale=1.0 / math.sqrt(M), dtype=dt)
    if own:
        import qml_gradients_amd as hq
        s["layer"] = hq.Dense(K, N, M, dtype=case["dtype"], activation=case["act"], alpha=case["alpha"])
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


def plain_dense(s):
    dt = s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = activate(z, s["act"]) * s["alpha"]
    if s["r"] is not None:
        y = y + s["r"].float()
    out = {"y": y.to(dt)}
    if s["op"] == "dense_train":
        dz = s["dy"].float() * (slope(z, s["act"]) * s["alpha"])
        out.update(dx=(dz @ w).to(dt), dw=(dz.t() @ x).to(dt))
        if s["b"] is not None:
            out["db"] = dz.sum(0).to(dt)
    return out


def blocks(x):
    """[n] as [blocks][256], the last block filled up with zeros."""
    pad = -x.numel() % BLOCK
    return torch.cat([x, x.new_zeros(pad)]).view(-1, BLOCK) if pad else x.view(-1, BLOCK)


def quantise(x):
    """(e4m3 values, one 32-bit scale per 256 elements) that stand for x: x ~ value * scale.
    A value that is not zero does not become zero: it is held as the smallest code at least."""
    rows = blocks(x)
    scale = (rows.abs().amax(1, keepdim=True) * (1.0 / E4M3_MAX)).clamp_min(SCALE_MIN)
    u = rows * (1.0 / scale)
    u = torch.where(u > 0, u.clamp_min(2.0 ** -9), u)
    u = torch.where(u < 0, u.clamp_max(-(2.0 ** -9)), u)
    return u.to(torch.float8_e4m3fn).view(-1)[: x.numel()].contiguous(), scale.view(-1)


def values(q):
    return (blocks(q[0].float()) * q[1][:, None]).view(-1)[: q[0].numel()]


def plain_adamw(p, g, m, v, step, bits):
    """One tensor's step, in place."""
    wide = torch.float64 if p.dtype == torch.float64 else torch.float32
    root1, root2 = 1 - BETA1 ** step, math.sqrt(1 - BETA2 ** step)
    P, G = p.to(wide), g.to(wide)
    if bits == 8:
        r = values(v)
        M, V = values(m) * BETA1 + G * (1 - BETA1), (r * r) * BETA2 + (G * G) * (1 - BETA2)
    else:
        M, V = m * BETA1 + G * (1 - BETA1), v * BETA2 + (G * G) * (1 - BETA2)
    R = torch.sqrt(V)
    P = P * (1 - LR * DECAY) - (M / (R * (1 / root2) + EPS)) * (LR / root1)
    p.copy_(P)
    if bits == 8:
        for held, new in ((m, quantise(M)), (v, quantise(R))):
            held[0].copy_(new[0])
            held[1].copy_(new[1])
    else:
        m.copy_(M)
        v.copy_(V)


def run(state):
    s = state
    if s["op"] == "adamw":
        if own:
            s["opt"].step()
        else:
            s["step"] += 1
            [plain_adamw(p, g, m, v, s["step"], s["bits"]) for p, g, m, v in zip(s["p"], s["g"], s["m"], s["v"])]
        return {"p": s["p"], "m": s["m"], "v": s["v"]}
    if not own:
        return plain_dense(s)
    if s["op"] == "dense":
        return {"y": s["layer"].forward(s["x"], s["w"], s["b"], s["r"])}
    y, z = s["layer"].forward_train(s["x"], s["w"], s["b"], s["r"])
    dx, dw, db = s["layer"].backward(s["dy"], s["x"], s["w"], z, bias=s["b"] is not None)
    out = {"y": y, "dx": dx, "dw": dw}
    if db is not None:
        out["db"] = db
    return out


# ---- what a pass cannot do without ----

def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "adamw":
        n = sum(sizes(case))
        # gradient read, parameter and both moments read and written
        held = 2 * 2 * (1 + 4.0 / BLOCK) if case["bits"] == 8 else 2 * 2 * max(4, b)
        return {"bytes": n * (3 * b + held), "flops": 15 * n}
    M, K, N = case["M"], case["K"], case["N"]
    read = M * K + N * K + (N if case["bias"] else 0) + (M * N if case["residual"] else 0)
    if case["op"] == "dense":
        return {"bytes": b * (read + M * N), "flops": 2 * M * N * K}
    written = M * N + M * K + N * K + (N if case["bias"] else 0)
    return {"bytes": b * (read + M * N + written), "flops": 6 * M * N * K}


# ---- the same from the definitions, in 64 bits ----

def exact_e4m3(x):
    """Nearest value code * scale in 64 bits: (codes' values, scales)."""
    n = x.numel()
    rows = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    rows[:n] = x
    rows = rows.view(-1, BLOCK)
    scale = torch.clamp(rows.abs().max(1, keepdim=True).values / E4M3_MAX, min=SCALE_MIN)
    size = (rows / scale).abs()
    exponent = torch.floor(torch.log2(size.clamp_min(2.0 ** -6)))
    step = torch.exp2(exponent - 3)
    code = torch.round(size / step) * step
    code = torch.where((size > 0) & (code == 0), torch.full_like(code, 2.0 ** -9), code)
    return (torch.sign(rows) * code).view(-1)[:n], scale.view(-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        out = {"p": [], "m": [], "v": []}
        t = STEP0 + 1
        for p, g, m, v in zip(s["p"], s["g"], s["m"], s["v"]):
            p, g = p.double(), g.double()
            if case["bits"] == 8:
                at = torch.arange(p.numel(), device=p.device) // BLOCK
                m, r = m[0].double() * m[1].double()[at], v[0].double() * v[1].double()[at]
                v = r ** 2
                del at, r
            m = BETA1 * m.double() + (1 - BETA1) * g
            v = BETA2 * v.double() + (1 - BETA2) * g ** 2
            mean, var = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
            out["p"].append(p - LR * DECAY * p - LR * mean / (var.sqrt() + EPS))
            del mean, var, p, g
            out["m"].append(exact_e4m3(m) if case["bits"] == 8 else m)
            out["v"].append(exact_e4m3(v.sqrt()) if case["bits"] == 8 else v)
        return out
    x, w = s["x"].double(), s["w"].double()
    z = torch.matmul(x, w.t())
    if s["b"] is not None:
        z += s["b"].double()
    z.requires_grad_(True)
    act = {"none": lambda t: t * 1.0, "relu": torch.nn.functional.relu, "gelu": torch.nn.functional.gelu,
           "silu": torch.nn.functional.silu, "tanh": torch.tanh, "sigmoid": torch.sigmoid}[case["act"]]
    a = case["alpha"] * act(z)
    y = a.detach()
    if s["r"] is not None:
        y = y + s["r"].double()
    out = {"y": y}
    if case["op"] == "dense_train":
        dz, = torch.autograd.grad(a, z, s["dy"].double())
        out.update(dx=torch.matmul(dz, w), dw=torch.matmul(dz.t(), x))
        if s["b"] is not None:
            out["db"] = dz.sum(0)
    return out
