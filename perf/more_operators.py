"""Measurement cases of the operators that bring tokens to the experts and back.

Three groups, all in 16 or 32 bits, around the products and norms of a
mixture-of-experts layer's training step:

- tokens sorted by expert (stable), their rows moved into that order, the
  experts' results weighted and summed back, and the gradients of both;
- embedding lookup with a scale, and its dense gradient;
- dropout whose mask is recomputed from a counter (Philox4x32-10, 16 bits an
  element), with the residual added.

`own` False computes each operator in its plain form (elementary torch
operations in fp32, rounded once at the end); True calls the framework.
"""
import functools
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
IDS = {"i64": torch.int64, "i32": torch.int32}
ROUTED = ("dispatch", "dispatch_bwd", "combine", "combine_bwd")


# ------------------------------------------------------------------ cases
def listed():
    def routed(op, name, tokens, k, experts, width, dtype, shards=1, residual=False):
        return {"name": name, "op": op, "tokens": tokens, "k": k, "experts": experts, "width": width, "dtype": dtype,
                "shards": shards, "residual": residual, "ids": "i64"}

    def embed(op, name, tokens, vocab, width, dtype, out):
        return {"name": name, "op": op, "tokens": tokens, "vocab": vocab, "width": width, "dtype": dtype, "out": out,
                "ids": "i64"}

    def dropout(name, rows, width, dtype, p, residual):
        return {"name": name, "op": "dropout", "rows": rows, "width": width, "dtype": dtype, "p": p, "residual": residual}

    return [
        # a handful of tokens to their experts: the call's own latency counts
        routed("dispatch", "dispatch_8t_k2_16e_5120", 8, 2, 16, 5120, "bf16"),
        # a training step's tokens, each to eight of many small experts
        routed("dispatch", "dispatch_16384t_k8_64e_2048", 16384, 8, 64, 2048, "bf16"),
        # the experts' results back, weighted, with the layer's residual
        routed("combine", "combine_16384t_k8_64e_2048", 16384, 8, 64, 2048, "bf16", residual=True),
        # the gradient of moving, at odd sizes in fp32, on one of two shards of the experts
        routed("dispatch_bwd", "dispatch_bwd_5003t_k3_32e_1433", 5003, 3, 32, 1433, "f32", shards=2),
        # the gradient of weighting: rows for the experts, numbers for the router
        routed("combine_bwd", "combine_bwd_16384t_k8_64e_2048", 16384, 8, 64, 2048, "bf16"),
        # the same for a ragged batch in fp32
        routed("combine_bwd", "combine_bwd_1021t_k2_16e_2049", 1021, 2, 16, 2049, "f32"),
        # lookups of a few new tokens
        embed("embed", "embed_16t_65536v_8192", 16, 65536, 8192, "bf16", "bf16"),
        # and of a training step's
        embed("embed", "embed_16640t_65536v_5120", 16640, 65536, 5120, "bf16", "bf16"),
        # the dense gradient of a large vocabulary: most rows are zero
        embed("embed_bwd", "embed_bwd_16384t_65536v_5120", 16384, 65536, 5120, "bf16", "f32"),
        # many tokens on a small vocabulary with odd sizes: most of the work is sums
        embed("embed_bwd", "embed_bwd_65537t_4099v_2050", 65537, 4099, 2050, "bf16", "bf16"),
        # a layer's output on its way into the residual stream
        dropout("dropout_16384x8192_bf16", 16384, 8192, "bf16", 0.1, True),
        # the gradient through it (the same mask on dy) for a ragged batch in fp32
        dropout("dropout_1021x2049_f32", 1021, 2049, "f32", 0.25, False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    n = _log_int(rng, lo, hi)
    return (n + 7) // 8 * 8 if rng.random() < 0.5 else n  # half of them whole vectors, half any width


def draw(rng):
    op = rng.choice([*ROUTED, "embed", "embed_bwd", "dropout", "dropout"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "dropout":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "width": _width(rng, 64, 4096), "dtype": dtype,
                "p": rng.choice([0.05, 0.1, 0.3, 0.5]), "residual": rng.random() < 0.5}
    ids = rng.choice(["i64", "i32"])
    if op in ROUTED:
        experts = _log_int(rng, 1, 512)
        while True:
            case = {"op": op, "tokens": _log_int(rng, 1, 16640), "k": min(rng.randint(1, 8), experts), "experts": experts,
                    "width": _width(rng, 64, 8192), "dtype": dtype, "shards": rng.choice([1, 1, min(2, experts), min(8, experts)]),
                    "residual": op == "combine" and rng.random() < 0.5, "ids": ids}
            if case["tokens"] * case["k"] < 64 * case["shards"]:
                case["shards"] = 1  # too few pairs for a shard to be sure of some
            if case["tokens"] * case["k"] * case["width"] * SIZE[dtype] <= 16384 * 8 * 2048 * 2:
                return case
    while True:
        case = {"op": op, "tokens": _log_int(rng, 1, 65537), "vocab": _log_int(rng, 64, 131072), "width": _width(rng, 64, 8192),
                "dtype": dtype, "out": rng.choice(["bf16", "f32"]), "ids": ids}
        if max(case["vocab"], case["tokens"]) * case["width"] <= 65536 * 2560:
            return case


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = dict(case)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "dropout":
        M, N = case["rows"], case["width"]
        s["x"] = randn(M, N).to(dt)
        s["res"] = (2 * randn(M, N)).to(dt) if case["residual"] else None
        # a run's seed and the number of this call in it, past 32 bits each
        s["seed"], s["offset"] = 0x1234567890 + 977 * seed, (seed << 33) + 5
        return s
    T, H = case["tokens"], case["width"]
    if case["op"] in ROUTED:
        E, k, n = case["experts"], case["k"], T * case["k"]
        # a router's choice: experts of unequal popularity, weights that add up to one
        top = torch.topk(randn(T, E) + 0.5 * randn(E), k, dim=1)
        s["e"] = top.indices.to(IDS[case["ids"]])
        s["w"] = torch.softmax(top.values, 1)
        s["local"] = E // case["shards"]  # the experts held here: a contiguous range of all
        s["first"] = s["local"] * (seed % case["shards"])
        if case["op"] == "dispatch":
            s["x"] = randn(T, H).to(dt)
            # where other shards hold experts, part of the rows stays unused: a buffer kept between steps
            s["rows"] = torch.zeros((n, H), dtype=dt, device=dev) if case["shards"] > 1 else None
            return s
        s["rank"], s["order"], _ = _plain_sort(s["e"], s["local"], s["first"])
        if case["op"] in ("dispatch_bwd", "combine"):
            s["rows"] = randn(n, H).to(dt)
            s["res"] = randn(T, H).to(dt) if case["residual"] else None
        else:
            s["dy"] = (1e-2 * randn(T, H)).to(dt)
            s["ys"] = randn(n, H).to(dt)
            s["rows"] = torch.zeros((n, H), dtype=dt, device=dev) if case["shards"] > 1 else None
        return s
    V = case["vocab"]
    # words by falling frequency (Zipf), spread over the vocabulary.  Drawn by whole numbers, whose running sums are
    # the same every time: those of floating-point numbers are not on a GPU, and would move words from run to run
    shares = (2.0 ** 40 / (torch.arange(V, dtype=torch.float64, device=dev) + 2.7)).long()
    sums = torch.cumsum(shares, 0)
    words = torch.searchsorted(sums, torch.randint(int(sums[-1]), (T,), generator=g, device=dev), right=True)
    s["t"] = torch.randperm(V, generator=g, device=dev)[words].to(IDS[case["ids"]])
    s["scale"] = math.sqrt(H)
    if case["op"] == "embed":
        s["table"] = (randn(V, H) / math.sqrt(H)).to(dt)
    else:
        s["dy"] = (1e-3 * randn(T, H)).to(dt)
    return s


# ------------------------------------------------------------- plain forms
def _plain_sort(ids, experts, first):
    key = ids.reshape(-1).long() - first
    kept = (key >= 0) & (key < experts)
    key = torch.where(kept, key, experts)
    order = torch.argsort(key, stable=True)
    place = torch.arange(order.numel(), device=order.device)
    rank = torch.empty_like(order).scatter_(0, order, place)
    ends = torch.searchsorted(key[order], torch.arange(experts, device=key.device), right=True)
    rank = torch.where(kept, rank, -1).reshape(ids.shape)
    return rank.to(torch.int32), torch.where(kept[order], order, -1).to(torch.int32), ends.to(torch.int32)


def _plain_rows(rows, rank):
    """The rows [T, k, H] of each token in fp32, zero where a pair is dropped."""
    return torch.where((rank >= 0)[:, :, None], rows[rank.clamp(min=0).long()].float(), 0.0)


def _plain_moved(x, order, k):
    """x's row (or x's entry of the pair) for each sorted row, zero past the last."""
    return torch.where((order >= 0)[:, None], x[torch.div(order.clamp(min=0), k, rounding_mode="floor").long()], 0)


def _mul_hi_lo(a, b):
    p = a * b  # modulo 2^64, of which both halves are wanted
    return (p >> 32) & 0xFFFFFFFF, p & 0xFFFFFFFF


def _plain_round(state, r):
    c0, c1, c2, c3, k0, k1 = state
    h0, l0 = _mul_hi_lo(c0, 0xD2511F53)
    h1, l1 = _mul_hi_lo(c2, 0xCD9E8D57)
    return h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0, (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF


def _plain_bits(M, N, seed, offset, device):
    """16 random bits for each element of [M, N]."""
    C = (N + 7) // 8
    zero = torch.zeros((M, C), dtype=torch.int64, device=device)
    row = torch.arange(M, device=device)[:, None] + zero
    col = torch.arange(C, device=device) + zero
    state = (col, row, zero + (offset & 0xFFFFFFFF), zero + (offset >> 32), seed & 0xFFFFFFFF, seed >> 32)
    words = torch.stack(functools.reduce(_plain_round, range(10), state)[:4], 2)
    return torch.stack((words & 0xFFFF, words >> 16), 3).reshape(M, 8 * C)[:, :N]


def _plain_dropout(x, p, seed, offset, res):
    border = round(p * 65536)
    kept = _plain_bits(*x.shape, seed, offset, x.device) >= border
    y = torch.where(kept, x.float() * (65536 / (65536 - border)), 0.0)
    return (y if res is None else res.float() + y).to(x.dtype)


def run(s):
    op = s["op"]
    if own:
        import swiglu_activation_cast_amd as mx

        if op == "dispatch":
            return mx.mxtrain_sort_dispatch(s["x"], s["e"], s["local"], first=s["first"], out=s["rows"])
        if op == "dispatch_bwd":
            return mx.mxtrain_dispatch_bwd(s["rows"], s["rank"])
        if op == "combine":
            return mx.mxtrain_combine_fwd(s["rows"], s["rank"], s["w"], residual=s["res"])
        if op == "combine_bwd":
            return mx.mxtrain_combine_bwd(s["dy"], s["ys"], s["rank"], s["w"], out=s["rows"])
        if op == "embed":
            return mx.mxtrain_embedding_fwd(s["table"], s["t"], scale=s["scale"], out_dtype=DTYPES[s["out"]])
        if op == "embed_bwd":
            return mx.mxtrain_embedding_bwd(s["dy"], s["t"], s["vocab"], scale=s["scale"], out_dtype=DTYPES[s["out"]])
        return mx.mxtrain_dropout_fwd(s["x"], s["p"], s["seed"], s["offset"], residual=s["res"])
    if op == "dispatch":
        rank, order, ends = _plain_sort(s["e"], s["local"], s["first"])
        return _plain_moved(s["x"], order, s["k"]), rank, ends, order
    if op == "dispatch_bwd":
        return _plain_rows(s["rows"], s["rank"]).sum(1).to(s["rows"].dtype)
    if op == "combine":
        y = (_plain_rows(s["rows"], s["rank"]) * s["w"][:, :, None]).sum(1)
        return (y if s["res"] is None else y + s["res"].float()).to(s["rows"].dtype)
    if op == "combine_bwd":
        weight = _plain_moved(s["w"].reshape(-1, 1), s["order"], 1)
        dys = (weight * _plain_moved(s["dy"].float(), s["order"], s["k"])).to(s["dy"].dtype)
        return dys, (_plain_rows(s["ys"], s["rank"]) * s["dy"].float()[:, None, :]).sum(2)
    if op == "embed":
        return (s["table"][s["t"].long()].float() * s["scale"]).to(DTYPES[s["out"]])
    if op == "embed_bwd":
        dw = torch.zeros((s["vocab"], s["width"]), device=s["dy"].device)
        return (dw.index_add_(0, s["t"].long(), s["dy"].float()) * s["scale"]).to(DTYPES[s["out"]])
    return _plain_dropout(s["x"], s["p"], s["seed"], s["offset"], s["res"])


# ------------------------------------------------------------------- work
def work(case):
    op, H, e = case["op"], case["width"], SIZE[case["dtype"]]
    if op == "dropout":
        n = case["rows"] * H
        return {"bytes": n * e * (3 if case["residual"] else 2), "flops": 3 * n}
    T, i = case["tokens"], 8 if case["ids"] == "i64" else 4
    if op in ROUTED:
        n = T * case["k"]
        kept = n * (case["experts"] // case["shards"]) / case["experts"]  # rows of this shard's experts, in the mean
        if op == "dispatch":
            return {"bytes": (T + kept) * H * e + n * (i + 8), "flops": 0}
        if op == "combine_bwd":
            return {"bytes": (T + 2 * kept) * H * e + 12 * n, "flops": 3 * kept * H}
        rows = T * (2 if case["residual"] else 1) + kept
        return {"bytes": rows * H * e + n * (8 if op == "combine" else 4), "flops": 2 * kept * H}
    V, o = case["vocab"], SIZE[case["out"]]
    if op == "embed":
        p = 1.0 / (np.arange(V) + 2.7)
        rows = float((1 - (1 - p / p.sum()) ** T).sum())  # distinct words, in the mean
        return {"bytes": rows * H * e + T * H * o + T * i, "flops": T * H}
    return {"bytes": T * H * e + V * H * o + T * i, "flops": T * H + V * H}


# ------------------------------------------------------------ 64-bit values
def _exact_bits(rows, N, seed, offset):
    """The generator's 16 bits for the given rows of N elements, in numpy."""
    u = np.uint64
    low, sh = u(0xFFFFFFFF), u(32)
    row, col = np.meshgrid(rows.astype(u), np.arange((N + 7) // 8, dtype=u), indexing="ij")
    x = [col, row, np.full_like(row, offset & 0xFFFFFFFF), np.full_like(row, offset >> 32)]
    for r in range(10):
        a, b = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        k0 = u((seed + r * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = u(((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
        x = [(b >> sh) ^ x[1] ^ k0, b & low, (a >> sh) ^ x[3] ^ k1, a & low]
    words = np.stack(x, -1).astype("<u4").view("<u2")
    return words.reshape(len(rows), -1)[:, :N]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "dropout":
        N, border = case["width"], round(case["p"] * 65536)
        parts = []
        for lo in range(0, case["rows"], 64):
            rows = np.arange(lo, min(lo + 64, case["rows"]))
            parts.append(torch.from_numpy(_exact_bits(rows, N, s["seed"], s["offset"]) >= border))
        y = s["x"].double() * torch.cat(parts).to(s["x"].device) * 65536 / (65536 - border)
        return y if s["res"] is None else y + s["res"].double()
    T, H = case["tokens"], case["width"]
    if op in ROUTED:
        k, n = case["k"], T * case["k"]
        if op == "dispatch":
            out = torch.zeros((n, H), dtype=torch.float64, device=s["x"].device)
            key = s["e"].reshape(-1) - s["first"]
            at = 0
            for e in range(s["local"]):
                pairs = torch.nonzero(key == e)[:, 0]
                out[at:at + len(pairs)] = s["x"][pairs // k].double()
                at += len(pairs)
            return out, None, None, None
        rank = s["rank"].long()
        if op == "combine_bwd":
            dys = torch.zeros((n, H), dtype=torch.float64, device=s["dy"].device)
            dw = torch.zeros((T, k), dtype=torch.float64, device=s["dy"].device)
        else:
            y = torch.zeros((T, H), dtype=torch.float64, device=s["rows"].device)
            if s["res"] is not None:
                y += s["res"].double()
        for j in range(k):
            t = torch.nonzero(rank[:, j] >= 0)[:, 0]
            r = rank[t, j]
            if op == "combine_bwd":
                d = s["dy"][t].double()
                dys[r] = d * s["w"][t, j, None].double()
                dw[t, j] = torch.linalg.vecdot(d, s["ys"][r].double())
            elif op == "combine":
                y[t] = torch.addcmul(y[t], s["rows"][r].double(), s["w"][t, j, None].double())
            else:
                y[t] += s["rows"][r].double()
        return (dys, dw) if op == "combine_bwd" else y
    if op == "embed":
        return torch.index_select(s["table"], 0, s["t"].long()).double() * s["scale"]
    # the sums of each word's rows, taken in sorted order from running sums of each part of the columns
    V = case["vocab"]
    order = torch.argsort(s["t"])
    ends = torch.cumsum(torch.bincount(s["t"].long(), minlength=V), 0)
    dw = torch.empty((V, H), dtype=torch.float64, device=s["dy"].device)
    for c in range(0, H, 512):
        run_ = torch.cumsum(s["dy"][:, c:c + 512][order].double(), 0)
        run_ = torch.cat([torch.zeros_like(run_[:1]), run_])
        dw[:, c:c + 512] = torch.diff(run_[ends], dim=0, prepend=torch.zeros_like(run_[:1])) * s["scale"]
    return dw
