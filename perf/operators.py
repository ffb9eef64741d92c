"""Cases for the training operators that feed the gradient compressors, with
their plain forms: counter-based dropout, the norms around a block with its
gate and residual scale, and softmax cross entropy over a vocabulary taken in
pieces. Sizes come from the BERT-Base parameter list (hidden 768, vocabulary
30522), or are generic."""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
IGNORE = -100
EPS = 1e-6

# The largest drawn sizes: values of one activation, and multiply-adds of one
# product with the vocabulary matrix.
MAX_VALUES = 16384 * 4096
MAX_PRODUCT = 8192 * 64000 * 4096


def listed():
    return [
        # one token's hidden state on its way through a small fine-tuning step: latency
        {"name": "dropout one token", "op": "dropout", "n": 768, "dtype": "f32", "p": 0.1, "residual": False},
        # 512 x 16 tokens of hidden 768, added to the residual stream, and a ragged end
        {"name": "dropout add bf16", "op": "dropout", "n": 8192 * 768 + 5, "dtype": "bf16", "p": 0.1, "residual": True},
        # the gradient through the dropout of a large batch's activations
        {"name": "dropout backward large", "op": "dropout_backward", "n": MAX_VALUES, "dtype": "bf16", "p": 0.1,
         "residual": False},
        # a handful of tokens between two blocks
        {"name": "norm few rows", "op": "norm_residual", "rows": 16, "d": 768, "groups": 1, "dtype": "bf16", "p": 0.0,
         "scale": 1.0},
        # a large batch, one gate a sequence, dropout inside
        {"name": "norm large", "op": "norm_residual", "rows": 16384, "d": 4096, "groups": 16, "dtype": "bf16", "p": 0.1,
         "scale": 0.5},
        # an fp32 model's gradient, odd numbers of rows and channels
        {"name": "norm grad odd f32", "op": "norm_residual_grad", "rows": 4095, "d": 1001, "groups": 1, "dtype": "f32",
         "p": 0.1, "scale": 1.0},
        # the large batch's gradient
        {"name": "norm grad large", "op": "norm_residual_grad", "rows": 16384, "d": 4096, "groups": 16, "dtype": "bf16",
         "p": 0.1, "scale": 0.5},
        # scoring one token against the BERT-Base vocabulary: reading the matrix is all there is
        {"name": "loss one token", "op": "linear_xent_loss", "tokens": 1, "vocab": 30522, "d": 768, "dtype": "bf16"},
        # a fine-tuning batch's loss
        {"name": "loss batch", "op": "linear_xent_loss", "tokens": 8192, "vocab": 30522, "d": 768, "dtype": "bf16"},
        # odd sizes throughout, an fp32 model
        {"name": "loss odd f32", "op": "linear_xent_loss", "tokens": 1001, "vocab": 33333, "d": 1001, "dtype": "f32"},
        # the BERT-Base vocabulary's gradient in fp32, as the compressors take it
        {"name": "grad batch f32 out", "op": "linear_xent_grad", "tokens": 8192, "vocab": 30522, "d": 768, "dtype": "bf16",
         "dweight": "f32"},
        # a wide model with a large vocabulary, gradients in the model's own type
        {"name": "grad wide", "op": "linear_xent_grad", "tokens": 8192, "vocab": 64000, "d": 4096, "dtype": "bf16",
         "dweight": "bf16"},
    ]


def _log_size(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["dropout", "dropout_backward", "norm_residual", "norm_residual_grad", "linear_xent_loss",
                     "linear_xent_grad"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op.startswith("dropout"):
        n = _log_size(rng, 1000, MAX_VALUES if dtype != "f32" else MAX_VALUES // 2)
        return {"op": op, "n": n, "dtype": dtype, "p": rng.choice([0.05, 0.1, 0.3, 0.5]),
                "residual": op == "dropout" and rng.random() < 0.5}
    if op.startswith("norm"):
        d = _log_size(rng, 64, 8192)
        if rng.random() < 0.6:
            d = -(-d // 64) * 64
        rows = _log_size(rng, 1, min(16384, MAX_VALUES // d // 2))
        groups = 1
        if rows >= 48 and rng.random() < 0.3:  # one gate for every three rows
            rows, groups = rows // 3 * 3, rows // 3
        return {"op": op, "rows": rows, "d": d, "groups": groups, "dtype": dtype, "p": rng.choice([0.0, 0.1]),
                "scale": rng.choice([1.0, 0.5])}
    d = _log_size(rng, 64, 4096)
    if rng.random() < 0.6:
        d = -(-d // 64) * 64
    vocab = _log_size(rng, 1000, 64000)
    # inputs of 32 bits have three times the products behind them
    most = MAX_PRODUCT // (4 if dtype == "bf16" else 12)
    tokens = _log_size(rng, 1, max(1, min(8192, most // vocab // d)))
    case = {"op": op, "tokens": tokens, "vocab": vocab, "d": d, "dtype": dtype}
    return case | {"dweight": rng.choice([dtype, "f32"])} if op.endswith("grad") else case


# ---- inputs ---------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    op, t = case["op"], DTYPES[case["dtype"]]
    g = _generator(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE)

    s = dict(case, t=t, seed=seed * 1_000_003 + 12345, worker=seed % 8)
    if op.startswith("dropout"):
        s["x"] = normal(case["n"]).to(t)
        s["r"] = normal(case["n"]).to(t) if case["residual"] else None
        s["out"] = torch.empty_like(s["x"])
        return s
    if op.startswith("norm"):
        rows, d, groups = case["rows"], case["d"], case["groups"]
        # a residual stream with some channels much larger than the others
        wide = 1.0 + 4.0 * (torch.rand(d, generator=g, device=DEVICE) < 0.02)
        s["x"] = (normal(rows, d) * wide).to(t)
        s["y"] = (normal(rows, d) * 0.7).to(t)
        s["post"] = 1.0 + 0.1 * normal(d)
        s["pre"] = 1.0 + 0.1 * normal(d)
        s["gate"] = 0.5 + 0.5 * normal(groups, d)
        s["z"], s["h"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        s["rstd_post"], s["rstd_pre"] = (torch.empty(rows, device=DEVICE) for _ in range(2))
        if op == "norm_residual_grad":
            z, _, s["rstd_post"], s["rstd_pre"] = _plain_norm(s)
            s["z"] = z
            s["dz"], s["dh"] = (normal(rows, d) * 0.01).to(t), (normal(rows, d) * 0.01).to(t)
            s["dx"], s["dy"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
            s["dpost"], s["dpre"], s["dgate"] = (torch.empty_like(s[k]) for k in ("post", "pre", "gate"))
            del s["x"], s["h"]
        return s
    n, v, d = case["tokens"], case["vocab"], case["d"]
    s["hidden"] = normal(n, d).to(t)
    # logits of a spread of about 2, as those of a model that has begun to learn
    s["weight"] = (normal(v, d) * (2.0 / math.sqrt(d))).to(t)
    s["target"] = torch.randint(0, v, (n,), generator=g, device=DEVICE)
    # an eighth of the tokens have no target, as padding; one token alone has one
    if n > 1:
        s["target"][torch.rand(n, generator=g, device=DEVICE) < 0.125] = IGNORE
    s["loss"], s["lse"] = torch.empty(n, device=DEVICE), torch.empty(n, device=DEVICE)
    if op == "linear_xent_grad":
        s["lse"] = _plain_loss(s)[1]
        s["dloss"] = (1.0 + 0.1 * normal(n)) / n
        s["dhidden"] = torch.empty_like(s["hidden"])
        s["dweight"] = torch.empty(v, d, dtype=DTYPES[case["dweight"]], device=DEVICE)
    return s


# ---- plain forms ----------------------------------------------------------

def _plain_keep(n, p, seed, worker):
    """Whether each of n values is kept: 24 bits of its word of Philox4x32-10
    against p. Words are held in int64, whose products wrap modulo 2^64."""
    low = 0xFFFFFFFF
    slot = torch.arange(-(-n // 4), device=DEVICE)
    c0, c1 = slot & low, slot >> 32
    c2, c3 = torch.full_like(slot, worker), torch.full_like(slot, 2)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    r = torch.stack([c0, c1, c2, c3], dim=1).reshape(-1)[:n]
    return (r >> 8) >= math.ceil(p * 2.0 ** 24)


def _plain_dropout(s):
    keep = _plain_keep(s["n"], s["p"], s["seed"], s["worker"])
    out = torch.where(keep, s["x"].float() * (1.0 / (1.0 - s["p"])), 0.0)
    if s["r"] is not None:
        out = out + s["r"].float()
    return out.to(s["t"])


def _plain_mask(s):
    rows, d = s["y"].shape
    if s["p"] == 0.0:
        return 1.0
    keep = _plain_keep(rows * d, s["p"], s["seed"], s["worker"]).reshape(rows, d)
    return keep.float() * (1.0 / (1.0 - s["p"]))


def _plain_norm(s):
    x, y = s["x"].float(), s["y"].float()
    rows, d = y.shape
    gate = s["gate"].repeat_interleave(rows // s["gate"].shape[0], dim=0)
    rstd_post = torch.rsqrt(y.square().mean(dim=1) + EPS)
    u = y * rstd_post[:, None] * s["post"]
    z = s["scale"] * x + gate * (u * _plain_mask(s))
    rstd_pre = torch.rsqrt(z.square().mean(dim=1) + EPS)
    h = z * rstd_pre[:, None] * s["pre"]
    return z.to(s["t"]), h.to(s["t"]), rstd_post, rstd_pre


def _plain_norm_grad(s):
    y, z, dz, dh = (s[k].float() for k in ("y", "z", "dz", "dh"))
    rows, d = y.shape
    groups = s["gate"].shape[0]
    gate = s["gate"].repeat_interleave(rows // groups, dim=0)
    zn = z * s["rstd_pre"][:, None]
    g = dh * s["pre"]
    total = dz + s["rstd_pre"][:, None] * (g - zn * (g * zn).mean(dim=1, keepdim=True))
    mask = _plain_mask(s)
    yn = y * s["rstd_post"][:, None]
    dgate = (total * (yn * s["post"] * mask)).reshape(groups, rows // groups, d).sum(dim=1)
    du = total * gate * mask
    g = du * s["post"]
    dy = s["rstd_post"][:, None] * (g - yn * (g * yn).mean(dim=1, keepdim=True))
    return ((s["scale"] * total).to(s["t"]), dy.to(s["t"]), (du * yn).sum(dim=0), dgate, (dh * zn).sum(dim=0))


def _plain_loss(s):
    logits = s["hidden"].float() @ s["weight"].float().t()
    top = logits.max(dim=1, keepdim=True).values
    lse = (top + (logits - top).exp().sum(dim=1, keepdim=True).log()).squeeze(1)
    has = s["target"] != IGNORE
    at = torch.where(has, s["target"], 0)
    loss = torch.where(has, lse - logits.gather(1, at[:, None]).squeeze(1), 0.0)
    return loss, lse


def _plain_loss_grad(s):
    hidden, weight = s["hidden"].float(), s["weight"].float()
    has = s["target"] != IGNORE
    at = torch.where(has, s["target"], 0)
    p = ((hidden @ weight.t()) - s["lse"][:, None]).exp_()
    rows = torch.arange(p.shape[0], device=p.device)
    p[rows, at] -= 1.0
    p *= torch.where(has, s["dloss"], 0.0)[:, None]
    return (p @ weight).to(s["dhidden"].dtype), (p.t() @ hidden).to(s["dweight"].dtype)


# ---- one pass -------------------------------------------------------------

def run(state):
    s, op = state, state["op"]
    if own:
        return _own(s, op)
    if op.startswith("dropout"):
        return _plain_dropout(s)
    if op == "norm_residual":
        return _plain_norm(s)
    if op == "norm_residual_grad":
        return _plain_norm_grad(s)
    return _plain_loss(s) if op == "linear_xent_loss" else _plain_loss_grad(s)


def _own(s, op):
    import gradient_compression_quantize_amd as gcq
    if op == "dropout":
        gcq.dropout(s["x"], s["p"], s["seed"], s["worker"], s["out"], residual=s["r"])
        return s["out"]
    if op == "dropout_backward":
        gcq.dropout_backward(s["x"], s["p"], s["seed"], s["worker"], s["out"])
        return s["out"]
    if op == "norm_residual":
        gcq.norm_residual(s["x"], s["y"], s["z"], h=s["h"], post_gain=s["post"], gate=s["gate"], pre_gain=s["pre"],
                          residual_scale=s["scale"], eps=EPS, p=s["p"], seed=s["seed"], worker=s["worker"],
                          rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"])
        return s["z"], s["h"], s["rstd_post"], s["rstd_pre"]
    if op == "norm_residual_grad":
        if "ws" not in s:  # kept by the caller from step to step
            rows, d = s["y"].shape
            size = gcq.norm_residual_grad_ws_bytes(rows, d, s["groups"])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEVICE)
        gcq.norm_residual_grad(s["z"], s["y"], s["dx"], s["dy"], s["ws"], dz=s["dz"], dh=s["dh"], post_gain=s["post"],
                               gate=s["gate"], pre_gain=s["pre"], residual_scale=s["scale"], p=s["p"], seed=s["seed"],
                               worker=s["worker"], rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"],
                               dpost_gain=s["dpost"], dgate=s["dgate"], dpre_gain=s["dpre"])
        return s["dx"], s["dy"], s["dpost"], s["dgate"], s["dpre"]
    if "ws" not in s:
        n, d = s["hidden"].shape
        v = s["weight"].shape[0]
        size = (gcq.linear_xent_loss_ws_bytes(n, v, d, s["t"]) if op == "linear_xent_loss" else
                gcq.linear_xent_grad_ws_bytes(n, v, d, s["t"], s["dhidden"].dtype, s["dweight"].dtype))
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEVICE)
    if op == "linear_xent_loss":
        gcq.linear_xent_loss(s["hidden"], s["weight"], s["target"], s["loss"], s["lse"], s["ws"], ignore_index=IGNORE)
        return s["loss"], s["lse"]
    gcq.linear_xent_grad(s["hidden"], s["weight"], s["target"], s["lse"], s["dloss"], s["dhidden"], s["dweight"],
                         s["ws"], ignore_index=IGNORE)
    return s["dhidden"], s["dweight"]


# ---- work and exact values ------------------------------------------------

def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    b, op = size[case["dtype"]], case["op"]
    if op.startswith("dropout"):
        return {"bytes": case["n"] * b * (3 if case["residual"] else 2), "flops": 2 * case["n"]}
    if op.startswith("norm"):
        values, d, rows = case["rows"] * case["d"], case["d"], case["rows"]
        small = 4 * (d * (2 + case["groups"]) + 2 * rows)
        if op == "norm_residual":
            return {"bytes": 4 * values * b + small, "flops": 10 * values}
        return {"bytes": 6 * values * b + small + 4 * d * (2 + case["groups"]), "flops": 24 * values}
    n, v, d = case["tokens"], case["vocab"], case["d"]
    if op == "linear_xent_loss":
        return {"bytes": (n + v) * d * b + 16 * n, "flops": 2 * n * v * d}
    return {"bytes": (n + v) * d * b + n * d * b + v * d * size[case["dweight"]] + 16 * n, "flops": 6 * n * v * d}


def _exact_keep(n, p, seed, worker):
    """The kept values once more, in numpy's unsigned 64-bit words, a block of
    counters at a time."""
    out = np.empty(-(-n // 4) * 4, dtype=bool)
    mask, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for lo in range(0, out.size // 4, 1 << 16):
        i = np.arange(lo, min(lo + (1 << 16), out.size // 4), dtype=np.uint64)
        x, y = i & mask, i >> sh
        z, w = np.full_like(i, worker), np.full_like(i, 2)
        key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
        for _ in range(10):
            p0, p1 = x * np.uint64(0xD2511F53), z * np.uint64(0xCD9E8D57)
            x, y, z, w = ((p1 >> sh) ^ y ^ np.uint64(key[0]), p1 & mask, (p0 >> sh) ^ w ^ np.uint64(key[1]), p0 & mask)
            key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
        u = np.stack([x, y, z, w], axis=1) >> np.uint64(8)
        out[lo * 4:(lo + i.size) * 4] = (u.astype(np.float64) * 2.0 ** -24 >= p).reshape(-1)
    return out[:n]


def _exact_factor(n, s):
    if s["p"] == 0.0:
        return torch.ones(n, dtype=torch.float64, device=DEVICE)
    return torch.from_numpy(_exact_keep(n, s["p"], s["seed"], s["worker"])).to(DEVICE).double() / (1.0 - s["p"])


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op.startswith("dropout"):
        out = s["x"].double() * _exact_factor(case["n"], s)
        return out if s["r"] is None else out + s["r"].double()
    if op.startswith("norm"):
        rows, d, groups = case["rows"], case["d"], case["groups"]
        f = _exact_factor(rows * d, s).reshape(groups, rows // groups, d)
        y = s["y"].double().reshape(f.shape)
        gate, post, pre = s["gate"].double()[:, None, :], s["post"].double(), s["pre"].double()
        if op == "norm_residual":
            a = ((y ** 2).sum(-1) / d + EPS) ** -0.5
            z = case["scale"] * s["x"].double().reshape(f.shape) + gate * (f * (a[..., None] * y * post))
            b = ((z ** 2).sum(-1) / d + EPS) ** -0.5
            return z.reshape(rows, d), (b[..., None] * z * pre).reshape(rows, d), a.reshape(rows), b.reshape(rows)
        a, b = (s[k].double().reshape(groups, -1, 1) for k in ("rstd_post", "rstd_pre"))
        z, dz, dh = (s[k].double().reshape(f.shape) for k in ("z", "dz", "dh"))
        # z b pre through its own norm: b is a function of z
        e = dz + b * dh * pre - b ** 3 * z * ((dh * pre * z).sum(-1, keepdim=True) / d)
        du = e * gate * f
        dy = a * du * post - a ** 3 * y * ((du * post * y).sum(-1, keepdim=True) / d)
        return ((case["scale"] * e).reshape(rows, d), dy.reshape(rows, d), (du * a * y).sum((0, 1)),
                (e * f * a * y * post).sum(1), (dh * b * z).sum((0, 1)))
    hidden, weight = s["hidden"].double(), s["weight"].double()
    n = case["tokens"]
    has = s["target"] != IGNORE
    if op == "linear_xent_loss":
        logits = hidden @ weight.t()
        lse = torch.logsumexp(logits, dim=1)
        rows = torch.arange(n, device=DEVICE)[has]
        loss = torch.zeros(n, dtype=torch.float64, device=DEVICE)
        loss[rows] = lse[rows] - logits[rows, s["target"][rows]]
        return loss, lse
    g = torch.exp(hidden @ weight.t() - s["lse"].double()[:, None])
    g[~has] = 0.0
    rows = torch.arange(n, device=DEVICE)[has]
    g[rows, s["target"][rows]] -= 1.0
    g *= s["dloss"].double()[:, None]
    return g @ weight, g.t() @ hidden
