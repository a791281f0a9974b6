"""Measured cases of the 8-bit boundary, the 8-bit product that reads its output, and the router's balance loss.

A case names its operator ("op") and sizes. ``run`` computes it either in plain torch operations or, where ``own`` is
true, through the calls of ``sandwich_norm_residual_gb300``.
"""
import math

import torch

own = False

EPS = 1e-6
ALPHA = 1e-3
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the dense boundary of one decode step of four requests: latency
        {"name": "dense_decode", "op": "dense", "T": 4, "D": 5120, "n": 2},
        # a hidden size that fills no launch shape evenly, an odd number of tokens
        {"name": "dense_odd", "op": "dense", "T": 1003, "D": 4104, "n": 104},
        # the dense boundary of a prefill chunk of eight prompts of 2048 tokens
        {"name": "dense_prefill", "op": "dense", "T": 16384, "D": 5120, "n": 7},
        # the expert combine of a decode batch of 64 requests
        {"name": "moe_decode", "op": "moe", "T": 64, "D": 5120, "n": 20},
        # the expert combine of a prefill chunk
        {"name": "moe_prefill", "op": "moe", "T": 16384, "D": 5120, "n": 20},
        # the query projection (48 heads of 128) of a single token
        {"name": "matmul_token", "op": "matmul", "M": 1, "N": 6144, "K": 5120, "out": "bf16"},
        # the feed-forward down projection of a decode batch
        {"name": "matmul_decode", "op": "matmul", "M": 64, "N": 5120, "K": 20480, "out": "bf16"},
        # ragged everywhere: a short chunk, an odd number of channels, FP32 for a reader that wants it
        {"name": "matmul_odd", "op": "matmul", "M": 517, "N": 2565, "K": 2576, "out": "fp32"},
        # the feed-forward up projection of a prefill chunk
        {"name": "matmul_prefill", "op": "matmul", "M": 16384, "N": 20480, "K": 5120, "out": "bf16"},
        # router statistics of a small micro-batch: latency
        {"name": "balance_small", "op": "balance", "T": 128, "E": 256, "topk": 8, "S": 1, "pad": 0},
        # eight training sequences of one batch, some rows of padding behind the last
        {"name": "balance_batch", "op": "balance", "T": 16384, "E": 256, "topk": 8, "S": 8, "pad": 100},
        # a long packed batch of ragged documents
        {"name": "balance_packed", "op": "balance", "T": 131072, "E": 256, "topk": 8, "S": 61, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dense", "moe", "matmul", "matmul", "balance"])
    if op in ("dense", "moe"):
        T, D = _log_int(rng, 1, 16384), 8 * _log_int(rng, 16, 1024)
        T = max(1, min(T, 16384 * 5120 // D))
        return {"op": op, "T": T, "D": D, "n": rng.randint(1, 105)}
    if op == "matmul":
        M, N, K = _log_int(rng, 1, 16384), _log_int(rng, 64, 20480), 16 * _log_int(rng, 8, 1280)
        M = max(1, min(M, 16384 * 20480 * 5120 // (N * K)))
        return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "fp32"])}
    T = _log_int(rng, 16, 131072)
    E = 4 * rng.randint(4, 64)
    S = min(T, _log_int(rng, 1, 64))
    return {"op": op, "T": T, "E": E, "topk": rng.randint(1, 8), "S": S, "pad": rng.randint(0, T // 8)}


# ---------------------------------------------------------------- inputs

def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _int8_rows(g, rows, cols):
    """Rows of normal values in 8 bits with one scale each, as the boundary writes them."""
    v = _normal(g, rows, cols)
    amax = v.abs().amax(1)
    return torch.round(v * (127.0 / amax)[:, None]).to(torch.int8), amax / 127.0


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] in ("dense", "moe"):
        T, D = case["T"], case["D"]
        s["h"] = _normal(g, T, D, dtype=torch.bfloat16)
        s["post_w"] = (1 + 0.1 * _normal(g, D)).to(torch.bfloat16)
        s["pre_w"] = (1 + 0.1 * _normal(g, D)).to(torch.bfloat16)
        if case["op"] == "dense":
            s["x"] = _normal(g, T, D, dtype=torch.bfloat16)
        else:
            e = torch.empty((T, 8, D), dtype=torch.bfloat16, device=DEV)
            for k in range(8):
                e[:, k] = _normal(g, T, D, dtype=torch.bfloat16)
            s["expert_out"] = e
            w = torch.sigmoid(_normal(g, T, 8))
            s["topk_w"] = w / w.sum(1, keepdim=True) * 2.5
    elif case["op"] == "matmul":
        s["a"], s["a_scale"] = _int8_rows(g, case["M"], case["K"])
        s["w"], w_scale = _int8_rows(g, case["N"], case["K"])
        s["w_scale"] = w_scale / math.sqrt(case["K"])
        s["dtype"] = torch.float32 if case["out"] == "fp32" else torch.bfloat16
    else:
        T, E, S = case["T"], case["E"], case["S"]
        s["logits"] = 2 * _normal(g, T, E) + 0.5 * _normal(g, E)
        score = torch.sigmoid(s["logits"]) + 0.05 * _normal(g, E)
        s["idx"] = torch.topk(score, case["topk"], dim=1).indices.to(torch.int32)
        # ragged sequences over the first T - pad tokens (a sequence may be empty)
        cuts = torch.randint(0, T - case["pad"] + 1, (S - 1,), generator=g, device=DEV).sort().values
        ends = torch.tensor([T - case["pad"]], device=DEV)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), cuts, ends]).to(torch.int32)
        s["dloss"] = torch.rand(S, generator=g, device=DEV) + 0.5
    return s


# ---------------------------------------------------------------- plain forms

def _rms_factor(v):
    """1 / sqrt(mean(v^2) + eps): the sum in 64 bits, every later step in 32."""
    total = v.double().square().sum(1, keepdim=True).float()
    mean = torch.div(total, torch.full_like(total, float(v.shape[1])))
    return torch.div(torch.ones_like(mean), torch.sqrt(mean + EPS))


def _bf16(v):
    """Rounded to BF16, held in 32 bits."""
    return v.to(torch.bfloat16).float()


def _plain_boundary(s):
    # the codes are whole numbers and are returned as they are, beside their scales
    if s["op"] == "moe":
        # one multiply-add rounded to 32 bits for each expert, in order: the product is exact in 64 bits
        x = torch.zeros_like(s["h"], dtype=torch.float32)
        for k in range(8):
            x = (s["topk_w"][:, k, None].double() * s["expert_out"][:, k].double() + x.double()).float()
        x = _bf16(x)
    else:
        x = s["x"].float()
    n = s["n"]
    c1, c2 = math.sqrt((n - 1) / n), 1.0 / math.sqrt(n)
    xn = _bf16(x * _rms_factor(x) * s["post_w"].float())
    h = _bf16(_bf16(s["h"].float() * c1) + _bf16(xn * c2))
    y = _bf16(h * _rms_factor(h) * s["pre_w"].float())
    amax = y.abs().amax(1, keepdim=True)
    scale = torch.div(amax, torch.full_like(amax, 127.0))
    inv = torch.where(amax > 0, torch.div(torch.full_like(amax, 127.0), amax), torch.zeros_like(amax))
    q = torch.round(y * inv).to(torch.int8)
    s["h"].copy_(h)
    return s["h"], q, scale[:, 0]


def _plain_matmul(s):
    acc = s["a"].float() @ s["w"].float().t()
    return (acc * s["a_scale"][:, None] * s["w_scale"][None, :]).to(s["dtype"])


def _segments(offsets, T):
    """The sequence of every token (S for none), and the sequences' lengths."""
    t = torch.arange(T, device=offsets.device, dtype=torch.int32)
    return torch.searchsorted(offsets[1:].contiguous(), t, right=True), offsets[1:] - offsets[:-1]


def _plain_balance(s, dtype=torch.float32):
    z, idx, off, K = s["logits"].to(dtype), s["idx"].long(), s["offsets"], s["topk"]
    T, E = z.shape
    S = off.shape[0] - 1
    seg, length = _segments(off, T)
    sig = 1 / (1 + torch.exp(-z))
    total = sig.sum(1, keepdim=True)
    p = sig / total
    # one row more than there are sequences: the padding's
    Q = torch.zeros((S + 1, E), dtype=torch.float64, device=z.device).index_add_(0, seg, p.double())
    c = torch.zeros((S + 1) * E, dtype=torch.int32, device=z.device)
    c = c.index_add_(0, (seg[:, None] * E + idx).reshape(-1), torch.ones_like(s["idx"]).reshape(-1)).view(S + 1, E)
    c[S] = 0
    n = length.double()
    factor = torch.where(n > 0, ALPHA * E / (K * n.clamp(min=1).square()), torch.zeros_like(n))
    loss = (factor * (c[:S].double() * Q[:S]).sum(1)).to(dtype)
    g = torch.cat([factor * s["dloss"].double(), torch.zeros(1, dtype=torch.float64, device=z.device)]).to(dtype)
    ct = c.to(dtype)[seg]
    dz = g[seg][:, None] * sig * (1 - sig) / total * (ct - (ct * p).sum(1, keepdim=True))
    return loss, c[:S], dz


def run(state):
    s = state
    if own:
        import sandwich_norm_residual_gb300 as snr
        if s["op"] == "dense":
            q, scale = snr.boundary_fused_int8(s["h"], s["x"], s["post_w"], s["pre_w"], s["n"], EPS)
            return s["h"], q, scale
        if s["op"] == "moe":
            q, scale = snr.moe_combine_boundary_int8(s["h"], s["expert_out"], s["topk_w"], s["post_w"], s["pre_w"],
                                                     s["n"], EPS)
            return s["h"], q, scale
        if s["op"] == "matmul":
            return snr.matmul_int8(s["a"], s["a_scale"], s["w"], s["w_scale"], out_dtype=s["dtype"])
        loss, counts = snr.moe_balance_loss(s["logits"], s["idx"], ALPHA, seq_offsets=s["offsets"])
        dz = snr.moe_balance_loss_backward(s["dloss"], s["logits"], counts, s["topk"], ALPHA, seq_offsets=s["offsets"])
        return loss, counts, dz
    if s["op"] in ("dense", "moe"):
        return _plain_boundary(s)
    return _plain_matmul(s) if s["op"] == "matmul" else _plain_balance(s)


# ---------------------------------------------------------------- floors and 64-bit values

def work(case):
    if case["op"] in ("dense", "moe"):
        T, D = case["T"], case["D"]
        # read h and the branch, write h', the codes and the scale; the norms' squares and products
        branch, extra = (2 * D, 0) if case["op"] == "dense" else (16 * D + 32, 16 * D)
        return {"bytes": T * (2 * D + branch + 2 * D + D + 4) + 4 * D, "flops": T * (16 * D + extra)}
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        out = 4 if case["out"] == "fp32" else 2
        return {"bytes": (M + N) * (K + 4) + M * N * out, "flops": 2 * M * N * K}
    T, E, S, live = case["T"], case["E"], case["S"], case["T"] - case["pad"]
    # forward: logits and choices; backward: the logits again, and the gradient of every row
    return {"bytes": live * (8 * E + 4 * case["topk"]) + T * 4 * E + 8 * S * E + 8 * S, "flops": live * 20 * E}


def _to32(v):
    """64-bit values rounded to FP32, held in 64 bits."""
    return v.float().double()


def _to16(v):
    """64-bit values rounded to FP32 and then to BF16 (nearest even), held in 64 bits."""
    m, e = torch.frexp(_to32(v))
    return torch.ldexp(torch.round(torch.ldexp(m, torch.full_like(e, 8))), e - 8)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("dense", "moe"):
        # the definition rounds at fixed places (FP32 steps, BF16 tensors): 64-bit arithmetic between them
        n, D = case["n"], case["D"]
        if case["op"] == "dense":
            x = s["x"].double()
        else:
            x = torch.zeros((case["T"], D), dtype=torch.float64, device=DEV)
            for k in range(8):
                x = _to32(torch.addcmul(x, s["topk_w"][:, k, None].double(), s["expert_out"][:, k].double()))
            x = _to16(x)

        def norm(v, w):
            mean = _to32(_to32(torch.einsum("td,td->t", v, v)) / D)
            r = _to32(1 / _to32((_to32(mean + float(torch.tensor(EPS)))).sqrt()))
            return _to16(_to32(v * r[:, None]) * w.double())

        xn = norm(x, s["post_w"])
        c1, c2 = (float(torch.tensor(v, dtype=torch.float32)) for v in (((n - 1) / n) ** 0.5, n ** -0.5))
        h = _to16(_to16(c1 * s["h"].double()) + _to16(c2 * xn))
        y = norm(h, s["pre_w"])
        top = y.abs().max(1).values
        codes = torch.round(_to32(y * _to32(127 / top)[:, None]))
        return h, codes.to(torch.int8), _to32(top / 127)
    if case["op"] == "matmul":
        a, w = s["a"].double() * s["a_scale"].double()[:, None], s["w"].double() * s["w_scale"].double()[:, None]
        return torch.cat([part @ w.t() for part in a.split(4096)])
    z, off = s["logits"].double(), s["offsets"].tolist()
    sig = torch.sigmoid(z)
    p = sig / sig.sum(1, keepdim=True)
    losses, counts, dz = [], [], torch.zeros_like(z)
    for i in range(case["S"]):
        lo, hi = off[i], off[i + 1]
        c = torch.bincount(s["idx"][lo:hi].reshape(-1).long(), minlength=case["E"])
        counts.append(c)
        if hi == lo:
            losses.append(torch.zeros((), dtype=torch.float64, device=DEV))
            continue
        f = c.double() * case["E"] / (case["topk"] * (hi - lo))
        losses.append(ALPHA * (f * p[lo:hi].mean(0)).sum())
        # d p_j / d z_e = s_e (1 - s_e) / sum(s) (delta_je - p_j)
        mixed = f[None, :] - (p[lo:hi] * f).sum(1, keepdim=True)
        dz[lo:hi] = (s["dloss"][i].double() * ALPHA / (hi - lo)) * mixed * (
            sig[lo:hi] * (1 - sig[lo:hi]) / sig[lo:hi].sum(1, keepdim=True))
    return torch.stack(losses), torch.stack(counts).to(torch.int32), dz
