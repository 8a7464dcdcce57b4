"""Measurement cases of the training operators beside the MXFP8 casts.

Three groups of operators of a mixture-of-experts layer's training step that
stay in 16 or 32 bits:

- layer norm, forward (with the row statistics) and backward (with the
  reductions of the weight's and the bias's gradients);
- the experts' bf16 matrix products over ragged token groups: forward
  y = x W_g^T, input gradient dx = dy W_g, weight gradient dW_g = dy_g^T x_g;
- orthogonalising weight updates by five quintic Newton-Schulz steps.

`own` False computes each operator in its plain form (elementary torch
operations in fp32, rounded once at the end); True calls the framework.
"""
import math

import torch

own = False

NS_COEFFS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7
LN_EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
def listed():
    def ln(op, name, rows, width, dtype):
        return {"name": name, "op": op, "rows": rows, "width": width, "dtype": dtype}

    def experts(op, name, tokens, groups, n, k, skew, out):
        return {"name": name, "op": op, "tokens": tokens, "experts": groups, "n": n, "k": k, "skew": skew, "out": out}

    def ortho(name, batch, rows, cols, dtype):
        return {"name": name, "op": "ortho", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype}

    return [
        # the norm of a handful of tokens: the call's own latency counts
        ln("ln_fwd", "ln_fwd_8x5120_bf16", 8, 5120, "bf16"),
        # the norm in front of a layer, at a training step's token count
        ln("ln_fwd", "ln_fwd_16384x8192_bf16", 16384, 8192, "bf16"),
        # its backward pass, at the layer's other width
        ln("ln_bwd", "ln_bwd_16384x5120_bf16", 16384, 5120, "bf16"),
        # a ragged batch in fp32, whose rows start at odd multiples of 4 bytes
        ln("ln_bwd", "ln_bwd_1021x2049_f32", 1021, 2049, "f32"),
        # a few tokens over many experts: the weights' bytes are the time
        experts("experts_fwd", "experts_fwd_24t_16e", 24, 16, 4096, 2048, 0.0, "bf16"),
        # the training step of a mixture-of-experts layer, each product
        experts("experts_fwd", "experts_fwd_16640t_4e", 16640, 4, 8192, 5120, 0.3, "bf16"),
        experts("experts_dgrad", "experts_dgrad_16640t_4e", 16640, 4, 8192, 5120, 0.3, "bf16"),
        experts("experts_wgrad", "experts_wgrad_16640t_4e", 16640, 4, 8192, 5120, 0.3, "f32"),
        # many small experts with uneven loads and sizes off the tile grid
        experts("experts_wgrad", "experts_wgrad_5003t_32e", 5003, 32, 1432, 1096, 0.5, "bf16"),
        # one small projection's update
        ortho("ortho_1x256x512_f32", 1, 256, 512, "f32"),
        # a stack of experts' updates, tall, in bf16
        ortho("ortho_8x2048x1024_bf16", 8, 2048, 1024, "bf16"),
        # one full-size weight's update in fp32
        ortho("ortho_1x8192x5120_f32", 1, 8192, 5120, "f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "experts_fwd", "experts_dgrad", "experts_wgrad", "ortho"])
    dtype = rng.choice(["bf16", "f32"])
    if op in ("ln_fwd", "ln_bwd"):
        width = _log_int(rng, 64, 8192)
        if rng.random() < 0.5:  # half of them whole vectors, half any width
            width = (width + 7) // 8 * 8
        return {"op": op, "rows": _log_int(rng, 1, 16384), "width": width, "dtype": dtype}
    if op == "ortho":
        while True:
            case = {"op": op, "batch": _log_int(rng, 1, 16), "rows": _log_int(rng, 32, 8192),
                    "cols": _log_int(rng, 32, 8192), "dtype": dtype}
            if work(case)["flops"] <= work({"op": op, "batch": 1, "rows": 8192, "cols": 5120, "dtype": "f32"})["flops"]:
                return case
    while True:
        case = {"op": op, "tokens": _log_int(rng, 1, 16640), "experts": _log_int(rng, 1, 64),
                "n": 8 * _log_int(rng, 32, 1024), "k": 8 * _log_int(rng, 32, 640),
                "skew": rng.choice([0.0, 0.3, 0.6]), "out": dtype}
        if case["experts"] * case["n"] * case["k"] <= 4 * 8192 * 5120:
            return case


# ----------------------------------------------------------------- inputs
def _generator(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _group_ends(tokens, experts, skew, seed):
    """Cumulative group ends of `tokens` routed to `experts` with log-normal popularity."""
    g = _generator(seed, "cpu")
    p = torch.softmax(skew * torch.randn(experts, generator=g), 0)
    counts = torch.bincount(torch.multinomial(p, tokens, replacement=True, generator=g), minlength=experts)
    return torch.cumsum(counts, 0).to(torch.int32), int(counts.max())


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _generator(seed, dev)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = dict(case)
    if case["op"] in ("ln_fwd", "ln_bwd"):
        dt, (M, N) = DTYPES[case["dtype"]], (case["rows"], case["width"])
        # a residual stream: channels of unequal scale, a few of them large, off centre
        scale = torch.exp(0.5 * randn(N)) * (1 + 20 * (torch.rand(N, generator=g, device=dev) < 0.002))
        s["x"] = (randn(M, N) * scale + 0.2 * randn(N)).to(dt)
        s["w"] = (1 + 0.1 * randn(N)).to(dt)
        s["b"] = (0.1 * randn(N)).to(dt)
        if case["op"] == "ln_bwd":
            s["dy"] = (1e-3 * randn(M, N)).to(dt)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + LN_EPS)
        return s
    if case["op"] == "ortho":
        B, m, n = case["batch"], case["rows"], case["cols"]
        # a momentum buffer: a few strong directions over a floor of noise
        r = min(32, m, n)
        sv = torch.exp(-0.15 * torch.arange(r, device=dev))
        u, v = randn(B, m, r) * (sv / math.sqrt(m)), randn(B, r, n) / math.sqrt(n)
        s["g"] = (1e-2 * (torch.matmul(u, v) + 0.3 * randn(B, m, n) / math.sqrt(m * n) * math.sqrt(r))).to(DTYPES[case["dtype"]])
        return s
    T, G, N, K = case["tokens"], case["experts"], case["n"], case["k"]
    ends, cap = _group_ends(T, G, case["skew"], seed)
    s["ends"], s["capacity"] = ends.to(dev), max(cap, 1)
    if case["op"] != "experts_dgrad":
        s["x"] = randn(T, K).to(torch.bfloat16)
    if case["op"] != "experts_fwd":
        s["dy"] = (1e-2 * randn(T, N)).to(torch.bfloat16)
    if case["op"] != "experts_wgrad":
        s["w"] = (randn(G, N, K) / math.sqrt(K)).to(torch.bfloat16)
    return s


# ------------------------------------------------------------- plain forms
def _plain_ln_fwd(x, w, b):
    x32 = x.float()
    mean = x32.mean(1, keepdim=True)
    d = x32 - mean
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + LN_EPS)
    return (d * rstd * w.float() + b.float()).to(x.dtype), mean[:, 0], rstd[:, 0]


def _plain_ln_bwd(dy, x, mean, rstd, w):
    dy32 = dy.float()
    xhat = (x.float() - mean[:, None]) * rstd[:, None]
    wdy = dy32 * w.float()
    c1 = wdy.mean(1, keepdim=True)
    c2 = (wdy * xhat).mean(1, keepdim=True)
    dx = (wdy - c1 - xhat * c2) * rstd[:, None]
    return dx.to(x.dtype), (dy32 * xhat).sum(0), dy32.sum(0)


def _pad_groups(t, ends, capacity):
    """t [T, C] as fp32 [G, capacity, C], each group's rows padded with zeros."""
    starts = torch.cat([torch.zeros_like(ends[:1]), ends[:-1]]).long()
    pos = starts[:, None] + torch.arange(capacity, device=t.device)
    inside = pos < ends[:, None]
    return t.float()[pos.clamp(max=t.shape[0] - 1)] * inside[:, :, None]


def _unpad_groups(p, ends, tokens):
    """The rows [T, C] of the padded groups p [G, capacity, C]."""
    rows = torch.arange(tokens, device=p.device, dtype=torch.int32)
    group = torch.searchsorted(ends, rows, right=True)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends[:-1]])
    return p[group, (rows - starts[group]).long()]


def _plain_step(x):
    a, b, c = NS_COEFFS
    s = torch.matmul(x, x.transpose(1, 2))
    return a * x + torch.matmul(b * s + c * torch.matmul(s, s), x)


def _plain_ortho(g):
    x = g.float()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    x = _plain_step(_plain_step(_plain_step(_plain_step(_plain_step(x)))))
    return (x.transpose(1, 2) if tall else x).to(g.dtype).contiguous()


def run(s):
    op = s["op"]
    if own:
        import swiglu_activation_cast_amd as mx

        if op == "ln_fwd":
            return mx.mxtrain_layer_norm_fwd(s["x"], s["w"], s["b"], eps=LN_EPS)
        if op == "ln_bwd":
            return mx.mxtrain_layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
        if op == "experts_fwd":
            return mx.mxtrain_grouped_gemm(s["x"], s["w"], s["ends"], out_dtype=DTYPES[s["out"]])
        if op == "experts_dgrad":
            return mx.mxtrain_grouped_gemm(s["dy"], s["w"], s["ends"], transpose_b=False, out_dtype=DTYPES[s["out"]])
        if op == "experts_wgrad":
            return mx.mxtrain_grouped_gemm_k(s["dy"], s["x"], s["ends"], out_dtype=DTYPES[s["out"]])
        return mx.mxtrain_newton_schulz(s["g"], steps=5, coeffs=NS_COEFFS, eps=NS_EPS)
    if op == "ln_fwd":
        return _plain_ln_fwd(s["x"], s["w"], s["b"])
    if op == "ln_bwd":
        return _plain_ln_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    if op == "ortho":
        return _plain_ortho(s["g"])
    ends, cap = s["ends"], s["capacity"]
    if op == "experts_fwd":
        y = torch.matmul(_pad_groups(s["x"], ends, cap), s["w"].float().transpose(1, 2))
        return _unpad_groups(y, ends, s["tokens"]).to(DTYPES[s["out"]])
    if op == "experts_dgrad":
        y = torch.matmul(_pad_groups(s["dy"], ends, cap), s["w"].float())
        return _unpad_groups(y, ends, s["tokens"]).to(DTYPES[s["out"]])
    dw = torch.matmul(_pad_groups(s["dy"], ends, cap).transpose(1, 2), _pad_groups(s["x"], ends, cap))
    return dw.to(DTYPES[s["out"]])


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        M, N, e = case["rows"], case["width"], SIZE[case["dtype"]]
        if op == "ln_fwd":  # x and the parameters in, y and the statistics out
            return {"bytes": 2 * M * N * e + 2 * N * e + 8 * M, "flops": 8 * M * N}
        return {"bytes": 3 * M * N * e + N * e + 8 * M + 8 * N, "flops": 14 * M * N}
    if op == "ortho":
        B, short, long_ = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        # a step: half of X X^T (it is symmetric), half of its square, and the product with X
        step = short * short * long_ + short ** 3 + 2 * short * short * long_
        return {"bytes": 2 * B * short * long_ * SIZE[case["dtype"]], "flops": 5 * B * step}
    T, G, N, K = case["tokens"], case["experts"], case["n"], case["k"]
    flops = 2 * T * N * K
    if op == "experts_wgrad":
        return {"bytes": 2 * T * (N + K) + G * N * K * SIZE[case["out"]] + 4 * G, "flops": flops}
    active = G * (1 - (1 - 1 / G) ** T)  # experts that get a token, in the mean over even routings
    rows_in, rows_out = (K, N) if op == "experts_fwd" else (N, K)
    return {"bytes": 2 * T * rows_in + SIZE[case["out"]] * T * rows_out + 2 * active * N * K + 4 * G, "flops": flops}


# ------------------------------------------------------------ 64-bit values
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "ln_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + LN_EPS)
        y = torch.addcmul(s["b"].double(), (x - mean[:, None]) * rstd[:, None], s["w"].double())
        return y, mean, rstd
    if op == "ln_bwd":
        dy, w, r = s["dy"].double(), s["w"].double(), s["rstd"].double()[:, None]
        xh = (s["x"].double() - s["mean"].double()[:, None]) * r
        n = case["width"]
        dxh = dy * w
        dx = r / n * (n * dxh - dxh.sum(1, keepdim=True) - xh * (dxh * xh).sum(1, keepdim=True))
        return dx, torch.einsum("mn,mn->n", dy, xh), dy.sum(0)
    if op == "ortho":
        a, b, c = NS_COEFFS
        out = []
        for g in s["g"]:
            x = g.double()
            x = x / (torch.linalg.norm(x) + NS_EPS)
            for _ in range(5):
                if x.shape[0] > x.shape[1]:
                    m = x.T @ x
                    x = a * x + b * (x @ m) + c * ((x @ m) @ m)
                else:
                    m = x @ x.T
                    x = a * x + b * (m @ x) + c * (m @ (m @ x))
            out.append(x)
        return torch.stack(out)
    ends = [0] + s["ends"].tolist()
    parts = []
    for g, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        if op == "experts_fwd":
            parts.append(s["x"][lo:hi].double() @ s["w"][g].double().T)
        elif op == "experts_dgrad":
            parts.append(s["dy"][lo:hi].double() @ s["w"][g].double())
        else:
            parts.append((s["dy"][lo:hi].double().T @ s["x"][lo:hi].double())[None])
    return torch.cat(parts)
