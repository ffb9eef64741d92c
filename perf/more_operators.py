"""Cases for the training operators around the compressors' fp32 gradients, with
their plain forms: layer norm behind a block's dropout and residual sum, and
its gradient; the orthogonalised update of weight matrices by Newton-Schulz
products, alone and as a whole optimiser step that reads the reduced gradient.
Sizes come from the BERT-Base, ResNet-50 and VGG-16 parameter lists (hidden
768; 3x3 convolutions of 64 channels as 64 x 576; 25088 x 4096 of the first
fully connected layer), or are generic."""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
LN_EPS = 1e-5
NS_EPS = 1e-7
# one step of the iteration: x <- a x + b (x x') x + c (x x')^2 x
QUINTIC = (3.4445, -4.7750, 2.0315)  # grows small singular values fast, ends near 1
EXACT3 = (1.5, -0.5, 0.0)            # converges to 1
SERIES = {"quintic": (QUINTIC,) * 5, "mixed": (QUINTIC, QUINTIC, QUINTIC, EXACT3), "cubic": (EXACT3,) * 3}

# The largest drawn sizes: values of one activation, and of an update.
MAX_VALUES = 16384 * 4096
LARGEST = (1, 25088, 4096)


def listed():
    return [
        # a handful of tokens between two blocks: latency
        {"name": "layer norm few rows", "op": "layer_norm", "rows": 16, "d": 768, "dtype": "bf16", "p": 0.0, "sub": False},
        # 512 x 16 tokens of hidden 768 behind a block's dropout, added to the stream
        {"name": "layer norm block", "op": "layer_norm", "rows": 8192, "d": 768, "dtype": "bf16", "p": 0.1, "sub": True},
        # a large batch of a wide model, the norm alone
        {"name": "layer norm wide", "op": "layer_norm", "rows": 16384, "d": 4096, "dtype": "bf16", "p": 0.0, "sub": False},
        # an fp32 model's gradient through dropout, odd numbers of rows and channels
        {"name": "layer norm grad odd f32", "op": "layer_norm_grad", "rows": 4095, "d": 1001, "dtype": "f32", "p": 0.1,
         "sub": True},
        # the wide model's gradient
        {"name": "layer norm grad wide", "op": "layer_norm_grad", "rows": 16384, "d": 4096, "dtype": "bf16", "p": 0.0,
         "sub": False},
        # one early convolution: latency
        {"name": "orthogonalize 64 x 576", "op": "orthogonalize", "count": 1, "m": 64, "n": 576, "dtype": "f32",
         "out": "bf16", "series": "quintic"},
        # an fp32 update of odd sizes, kept in fp32
        {"name": "orthogonalize odd f32", "op": "orthogonalize", "count": 3, "m": 1001, "n": 2500, "dtype": "f32",
         "out": "f32", "series": "quintic"},
        # a large square matrix of a wide model
        {"name": "orthogonalize 4096 x 4096", "op": "orthogonalize", "count": 1, "m": 4096, "n": 4096, "dtype": "bf16",
         "out": "bf16", "series": "quintic"},
        # the first fully connected layer of VGG-16, tall
        {"name": "orthogonalize 25088 x 4096", "op": "orthogonalize", "count": LARGEST[0], "m": LARGEST[1], "n": LARGEST[2],
         "dtype": "f32", "out": "bf16", "series": "quintic"},
        # one attention matrix of BERT-Base from the reduced gradient: latency
        {"name": "step one matrix", "op": "muon_step", "count": 1, "m": 768, "n": 768, "dtype": "bf16", "series": "quintic"},
        # the 48 attention matrices of BERT-Base, fp32 weights
        {"name": "step 48 matrices f32", "op": "muon_step", "count": 48, "m": 768, "n": 768, "dtype": "f32",
         "series": "quintic"},
        # four large matrices of a wide model
        {"name": "step wide", "op": "muon_step", "count": 4, "m": 2048, "n": 8192, "dtype": "bf16", "series": "quintic"},
    ]


def _log_size(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _products(count, m, n):
    """Multiply-adds of one step: x x' and its square, half of each as they
    are symmetric, and what they multiply x by."""
    r, c = min(m, n), max(m, n)
    return count * (r * r * c // 2 + r * r * r // 2 + r * r * c)


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_grad", "orthogonalize", "muon_step"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op.startswith("layer"):
        d = _log_size(rng, 64, 8192)
        if rng.random() < 0.6:
            d = -(-d // 64) * 64
        sub = rng.random() < 0.5
        return {"op": op, "rows": _log_size(rng, 1, min(16384, MAX_VALUES // d // 2)), "d": d, "dtype": dtype,
                "p": rng.choice([0.0, 0.1, 0.3]) if sub else 0.0, "sub": sub}
    m, n = _log_size(rng, 16, 8192), _log_size(rng, 16, 16384)
    if rng.random() < 0.6:
        m, n = -(-m // 64) * 64, -(-n // 64) * 64
    out = dtype if op == "muon_step" else rng.choice(["f32", "bf16", "f16"])
    # more than one product stands behind a value that is kept to more than 8 bits
    most = _products(*LARGEST) // (4 if out != "bf16" else 1)
    while _products(1, m, n) > most:
        m, n = max(16, m // 2), max(16, n // 2)
    count = _log_size(rng, 1, max(1, min(48, most // _products(1, m, n), 2 * MAX_VALUES // (m * n))))
    case = {"op": op, "count": count, "m": m, "n": n, "dtype": dtype}
    return case | ({"out": out} if op == "orthogonalize" else {}) | {"series": rng.choice(["quintic", "mixed", "cubic"])}


# ---- inputs ---------------------------------------------------------------

def prepare(case, seed):
    op, t = case["op"], DTYPES[case["dtype"]]
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE)

    s = dict(case, t=t, seed=seed * 1_000_003 + 12345, worker=seed % 8)
    if op.startswith("layer"):
        rows, d = case["rows"], case["d"]
        # a stream with some channels much larger than the others, off zero
        wide = 1.0 + 4.0 * (torch.rand(d, generator=g, device=DEVICE) < 0.02)
        s["x"] = (normal(rows, d) * wide + 0.3 * normal(d)).to(t)
        s["y"] = (normal(rows, d) * 0.7).to(t) if case["sub"] else None
        s["gain"], s["bias"] = 1.0 + 0.1 * normal(d), 0.1 * normal(d)
        if op == "layer_norm":
            s["z"] = torch.empty_like(s["x"]) if case["sub"] else None
            s["h"] = torch.empty_like(s["x"])
            s["mean"], s["rstd"] = (torch.empty(rows, device=DEVICE) for _ in range(2))
            return s
        # the forward pass kept the sum and its statistics
        z, _, s["mean"], s["rstd"] = _plain_norm(s)
        s["z"] = s["x"] if z is None else z
        del s["x"], s["y"]
        s["dh"] = (normal(rows, d) * 0.01).to(t)
        s["dz"] = (normal(rows, d) * 0.01).to(t) if case["sub"] else None
        s["dx"] = torch.empty_like(s["z"])
        s["dy"] = torch.empty_like(s["z"]) if case["sub"] else None
        s["dgain"], s["dbias"] = torch.empty(d, device=DEVICE), torch.empty(d, device=DEVICE)
        return s
    count, m, n = case["count"], case["m"], case["n"]

    def gradient(scale):
        # a few strong directions over many weak ones, as gradients of weights have
        k = min(8, m, n)
        strong = (normal(count, m, k) * (2.0 ** -torch.arange(k, device=DEVICE))) @ normal(count, k, n)
        return (strong + 0.5 * normal(count, m, n)) * scale

    if op == "orthogonalize":
        s["x"] = gradient(1e-3).to(t)
        s["o"] = torch.empty(count, m, n, dtype=DTYPES[case["out"]], device=DEVICE)
        return s
    # the sum of eight workers' gradients, as the reducer leaves it
    s["g"], s["m0"] = gradient(8e-3), gradient(1e-3)
    s["w"] = (normal(count, m, n) / math.sqrt(n)).to(t)
    s["m1"], s["w1"] = torch.empty_like(s["m0"]), torch.empty_like(s["w"])
    s["kw"] = dict(momentum=0.95, grad_scale=1.0 / 8, lr=0.02, weight_decay=0.01,
                   update_scale=math.sqrt(max(1.0, m / n)), nesterov=True)
    return s


# ---- plain forms ----------------------------------------------------------

def _plain_factor(s, rows, d):
    """What dropout multiplies a row's values by: 24 bits of each value's word
    of Philox4x32-10 against p. Words are held in int64, whose products wrap
    modulo 2^64."""
    if s["p"] == 0.0:
        return 1.0
    low, n = 0xFFFFFFFF, rows * d
    slot = torch.arange(-(-n // 4), device=DEVICE)
    c0, c1 = slot & low, slot >> 32
    c2, c3 = torch.full_like(slot, s["worker"]), torch.full_like(slot, 2)
    k0, k1 = s["seed"] & low, (s["seed"] >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    r = torch.stack([c0, c1, c2, c3], dim=1).reshape(-1)[:n].reshape(rows, d)
    return ((r >> 8) >= math.ceil(s["p"] * 2.0 ** 24)).float() * (1.0 / (1.0 - s["p"]))


def _plain_norm(s):
    z = s["x"].float()
    if s["sub"]:
        z = z + s["y"].float() * _plain_factor(s, *z.shape)
    mean = z.mean(dim=1)
    c = z - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(dim=1) + LN_EPS)
    h = c * rstd[:, None] * s["gain"] + s["bias"]
    return z.to(s["t"]) if s["sub"] else None, h.to(s["t"]), mean, rstd


def _plain_norm_grad(s):
    z, dh = s["z"].float(), s["dh"].float()
    zn = (z - s["mean"][:, None]) * s["rstd"][:, None]
    g = dh * s["gain"]
    dx = s["rstd"][:, None] * (g - g.mean(dim=1, keepdim=True) - zn * (g * zn).mean(dim=1, keepdim=True))
    dgain, dbias = (dh * zn).sum(dim=0), dh.sum(dim=0)
    if not s["sub"]:
        return dx.to(s["t"]), dgain, dbias
    dx = dx + s["dz"].float()
    return dx.to(s["t"]), (dx * _plain_factor(s, *z.shape)).to(s["t"]), dgain, dbias


def _plain_orthogonal(x, series):
    """fp32 [count, m, n]"""
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + NS_EPS)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    for a, b, c in SERIES[series]:
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(1, 2).contiguous() if tall else x


def _plain_step(s):
    k = s["kw"]
    g = s["g"] * k["grad_scale"]
    m1 = k["momentum"] * s["m0"] + (1.0 - k["momentum"]) * g
    o = _plain_orthogonal(k["momentum"] * m1 + (1.0 - k["momentum"]) * g, s["series"])
    w1 = (1.0 - k["lr"] * k["weight_decay"]) * s["w"].float() - (k["lr"] * k["update_scale"]) * o
    return w1.to(s["t"]), m1


# ---- one pass -------------------------------------------------------------

def run(state):
    s, op = state, state["op"]
    if own:
        return _own(s, op)
    if op == "layer_norm":
        return _plain_norm(s)
    if op == "layer_norm_grad":
        return _plain_norm_grad(s)
    if op == "orthogonalize":
        return _plain_orthogonal(s["x"].float(), s["series"]).to(s["o"].dtype)
    return _plain_step(s)


def _own(s, op):
    import gradient_compression_quantize_amd as gcq
    if op == "layer_norm":
        gcq.layer_norm(s["x"], s["h"], y=s["y"], z=s["z"], gain=s["gain"], bias=s["bias"], eps=LN_EPS, p=s["p"],
                       seed=s["seed"], worker=s["worker"], mean=s["mean"], rstd=s["rstd"])
        return s["z"], s["h"], s["mean"], s["rstd"]
    if op == "layer_norm_grad":
        if "ws" not in s:  # kept by the caller from step to step
            size = gcq.layer_norm_grad_ws_bytes(*s["z"].shape)
            s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEVICE)
        gcq.layer_norm_grad(s["z"], s["dh"], s["dx"], s["ws"], dz=s["dz"], dy=s["dy"], gain=s["gain"], p=s["p"],
                            seed=s["seed"], worker=s["worker"], mean=s["mean"], rstd=s["rstd"], dgain=s["dgain"],
                            dbias=s["dbias"])
        return (s["dx"], s["dy"], s["dgain"], s["dbias"]) if s["sub"] else (s["dx"], s["dgain"], s["dbias"])
    count, m, n = s["count"], s["m"], s["n"]
    if "ws" not in s:
        size = (gcq.orthogonalize_ws_bytes(count, m, n, s["o"].dtype) if op == "orthogonalize" else
                gcq.muon_step_ws_bytes(count, m, n, s["t"]))
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEVICE)
    if op == "orthogonalize":
        gcq.orthogonalize(s["x"].unbind(), s["o"].unbind(), s["ws"], coefficients=SERIES[s["series"]], eps=NS_EPS)
        return s["o"]
    gcq.muon_step(s["g"].unbind(), s["m0"].unbind(), s["w"].unbind(), s["ws"], coefficients=SERIES[s["series"]],
                  eps=NS_EPS, new_momenta=s["m1"].unbind(), new_weights=s["w1"].unbind(), **s["kw"])
    return s["w1"], s["m1"]


# ---- work and exact values ------------------------------------------------

def work(case):
    op, b = case["op"], SIZE[case["dtype"]]
    if op.startswith("layer"):
        values, d, rows = case["rows"] * case["d"], case["d"], case["rows"]
        if op == "layer_norm":
            return {"bytes": values * b * (4 if case["sub"] else 2) + 8 * d + 8 * rows, "flops": 9 * values}
        return {"bytes": values * b * (5 if case["sub"] else 3) + 12 * d + 8 * rows, "flops": 14 * values}
    count, m, n = case["count"], case["m"], case["n"]
    values, r, c = count * m * n, min(m, n), max(m, n)
    flops = 0
    for _, _, last in SERIES[case["series"]]:
        flops += 2 * _products(count, m, n) - (0 if last else count * r * r * r)
    if op == "orthogonalize":
        return {"bytes": values * (b + SIZE[case["out"]]), "flops": flops}
    return {"bytes": values * (12 + 2 * b), "flops": flops}


def _exact_factor(s, rows, d):
    """The dropout factors once more, in numpy's unsigned 64-bit words, a block
    of counters at a time."""
    n, p = rows * d, s["p"]
    out = np.empty(-(-n // 4) * 4, dtype=bool)
    mask, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for lo in range(0, out.size // 4, 1 << 16):
        i = np.arange(lo, min(lo + (1 << 16), out.size // 4), dtype=np.uint64)
        x, y, z, w = i & mask, i >> sh, np.full_like(i, s["worker"]), np.full_like(i, 2)
        key = [s["seed"] & 0xFFFFFFFF, (s["seed"] >> 32) & 0xFFFFFFFF]
        for _ in range(10):
            p0, p1 = x * np.uint64(0xD2511F53), z * np.uint64(0xCD9E8D57)
            x, y, z, w = ((p1 >> sh) ^ y ^ np.uint64(key[0]), p1 & mask, (p0 >> sh) ^ w ^ np.uint64(key[1]), p0 & mask)
            key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
        u = np.stack([x, y, z, w], axis=1) >> np.uint64(8)
        out[lo * 4:(lo + i.size) * 4] = (u.astype(np.float64) * 2.0 ** -24 >= p).reshape(-1)
    return torch.from_numpy(out[:n].reshape(rows, d)).to(DEVICE).double() / (1.0 - p)


def _exact_orthogonal(x, series):
    """float64 [m, n]: a polynomial of the smaller Gram matrix, nested, on its
    side of x."""
    x = x / ((x * x).sum() ** 0.5 + NS_EPS)
    left = x.shape[0] <= x.shape[1]
    for a, b, c in SERIES[series]:
        gram = torch.mm(x, x.t()) if left else torch.mm(x.t(), x)
        inner = c * gram
        inner.diagonal().add_(b)
        poly = torch.mm(gram, inner)
        poly.diagonal().add_(a)
        x = torch.mm(poly, x) if left else torch.mm(x, poly)
    return x


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op.startswith("layer"):
        rows, d = case["rows"], case["d"]
        gain = s["gain"].double()
        f = _exact_factor(s, rows, d) if case["p"] > 0.0 else 1.0
        if op == "layer_norm":
            z = s["x"].double() + (s["y"].double() * f if case["sub"] else 0.0)
            mean = z.sum(1) / d
            rstd = (((z - mean[:, None]) ** 2).sum(1) / d + LN_EPS) ** -0.5
            h = s["bias"].double() + gain * rstd[:, None] * (z - mean[:, None])
            return z if case["sub"] else None, h, mean, rstd
        # h = bias + gain rstd (z - mean); rstd and mean are functions of z
        rstd, c = s["rstd"].double()[:, None], s["z"].double() - s["mean"].double()[:, None]
        dh = s["dh"].double()
        e = rstd * gain * dh
        e = e - e.sum(1, keepdim=True) / d - rstd ** 3 * c * ((gain * dh * c).sum(1, keepdim=True) / d)
        dgain, dbias = (dh * rstd * c).sum(0), dh.sum(0)
        if not case["sub"]:
            return e, dgain, dbias
        e = e + s["dz"].double()
        return e, e * f, dgain, dbias
    count = case["count"]
    if op == "orthogonalize":
        return torch.stack([_exact_orthogonal(s["x"][k].double(), case["series"]) for k in range(count)])
    k = s["kw"]
    g, m0 = s["g"].double() * k["grad_scale"], s["m0"].double()
    m1 = m0 + (1.0 - k["momentum"]) * (g - m0)
    u = g + k["momentum"] * (m1 - g)
    o = torch.stack([_exact_orthogonal(u[i], case["series"]) for i in range(count)])
    w = s["w"].double()
    return w - k["lr"] * (k["weight_decay"] * w + k["update_scale"] * o), m1
