"""Measured cases of the expert layer: tokens sorted by expert and back, the 8-bit floating-point products between, and
the kernels that write their operands.

A case names its operator ("op") and sizes. ``run`` computes it either in plain torch operations or, where ``own`` is
true, through the calls of ``sandwich_norm_residual_gb300``.
"""
import math

import torch

own = False

EPS = 1e-6
DEV = "cuda"
BLOCK = 128  # values, or values by values, that share a scale
TOP = 448.0  # the largest E4M3 number
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of four requests, 8-bit rows with their scales to the experts: latency
        {"name": "dispatch_decode", "op": "dispatch", "T": 4, "E": 256, "topk": 8, "D": 5120, "kind": "fp8", "pad": 0},
        # a training batch of eight sequences of 2048, 100 rows of padding that no expert takes; with the gradient
        {"name": "dispatch_train", "op": "dispatch", "T": 16384, "E": 256, "topk": 8, "D": 5120, "kind": "bf16", "pad": 100},
        # the experts' outputs of 64 decoding requests added up
        {"name": "combine_decode", "op": "combine", "T": 64, "E": 256, "topk": 8, "D": 5120, "train": False, "pad": 0},
        # the same for a training batch, with the gradients of the rows and of the routing weights
        {"name": "combine_train", "op": "combine", "T": 16384, "E": 256, "topk": 8, "D": 5120, "train": True, "pad": 100},
        # the query projection (48 heads of 128) of a single token
        {"name": "matmul_token", "op": "matmul", "M": 1, "N": 6144, "K": 5120, "out": "bf16"},
        # ragged everywhere: a short chunk, an odd number of channels, a last block that is not whole
        {"name": "matmul_odd", "op": "matmul", "M": 517, "N": 2565, "K": 2576, "out": "fp32"},
        # gate and up projections of 256 experts for 64 decoding requests: nearly all weights for two rows each
        {"name": "experts_decode", "op": "experts", "T": 64, "E": 256, "topk": 8, "N": 5120, "K": 5120, "out": "bf16"},
        # the same for a prefill chunk of eight prompts of 2048 tokens
        {"name": "experts_prefill", "op": "experts", "T": 16384, "E": 256, "topk": 8, "N": 5120, "K": 5120, "out": "bf16"},
        # the dense boundary at a hidden size whose last block is not whole, an odd number of tokens
        {"name": "boundary_odd", "op": "boundary", "T": 1003, "D": 4104, "n": 104, "moe": False},
        # the boundary behind the experts, for a prefill chunk
        {"name": "boundary_moe", "op": "boundary", "T": 16384, "D": 5120, "n": 20, "moe": True},
        # the experts' activation for 64 decoding requests
        {"name": "swiglu_decode", "op": "swiglu", "R": 512, "F": 2560},
        # the same for a prefill chunk
        {"name": "swiglu_prefill", "op": "swiglu", "R": 131072, "F": 2560},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "matmul", "experts", "boundary", "swiglu"])
    if op in ("dispatch", "combine"):
        D, topk = 16 * _log_int(rng, 8, 512), rng.randint(1, 8)
        T = _log_int(rng, 1, max(1, min(65536, 16384 * 8 * 5120 // (topk * D))))
        c = {"op": op, "T": T, "E": rng.randint(topk, 256), "topk": topk, "D": D}
        c.update({"kind": rng.choice(["fp8", "bf16"])} if op == "dispatch" else {"train": rng.choice([True, False])})
        return {**c, "pad": rng.randint(0, T // 8)}
    if op == "matmul":
        M, N, K = _log_int(rng, 1, 16384), _log_int(rng, 64, 20480), 16 * _log_int(rng, 8, 1280)
        M = max(1, min(M, 16384 * 20480 * 5120 // (N * K)))
        return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "fp32"])}
    if op == "experts":
        topk, N, K = rng.randint(1, 8), _log_int(rng, 256, 5120), 16 * _log_int(rng, 16, 320)
        E = _log_int(rng, max(4, topk), 256)
        T = _log_int(rng, 1, max(1, min(65536, 16384 * 8 * 5120 * 5120 // (topk * N * K))))
        return {"op": op, "T": T, "E": E, "topk": topk, "N": N, "K": K, "out": rng.choice(["bf16", "fp32"])}
    if op == "boundary":
        T, D = _log_int(rng, 1, 16384), 8 * _log_int(rng, 16, 1024)
        T = max(1, min(T, 16384 * 5120 // D))
        return {"op": op, "T": T, "D": D, "n": rng.randint(1, 105), "moe": rng.choice([True, False])}
    F = 16 * _log_int(rng, 8, 1280)
    return {"op": op, "R": _log_int(rng, 1, 131072 * 2560 // F), "F": F}


# ---------------------------------------------------------------- inputs

def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _fp8_rows(g, rows, cols):
    """Rows of normal values as E4M3 with one scale for each 128, as a boundary writes them."""
    blocks = -(-cols // BLOCK)
    v = torch.nn.functional.pad(_normal(g, rows, cols), (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    scale = v.abs().amax(2) / TOP
    q = (v / scale[:, :, None]).clamp_(-TOP, TOP).to(FP8).view(rows, blocks * BLOCK)
    return q[:, :cols].contiguous(), scale


def _fp8_channels(g, n, k):
    """A weight matrix as E4M3 with one scale for each 128 by 128."""
    bn, bk = -(-n // BLOCK), -(-k // BLOCK)
    v = torch.nn.functional.pad(_normal(g, n, k), (0, bk * BLOCK - k, 0, bn * BLOCK - n)).view(bn, BLOCK, bk, BLOCK)
    scale = v.abs().amax((1, 3)) / TOP
    q = (v / scale[:, None, :, None]).clamp_(-TOP, TOP).to(FP8).view(bn * BLOCK, bk * BLOCK)
    return q[:n, :k].contiguous(), scale / math.sqrt(k)


def _choices(g, T, E, topk, pad):
    """The experts of every token, none for the last `pad`: some experts are liked more than others."""
    score = torch.sigmoid(2 * _normal(g, T, E) + 0.5 * _normal(g, E))
    idx = torch.topk(score, topk, dim=1).indices.to(torch.int32)
    if pad:
        idx[T - pad:] = -1
    return idx


def _places(idx, E):
    """offsets [E + 1] of the experts' rows and the row of every choice (-1 for none), in the choices' order."""
    flat = idx.reshape(-1)
    key = torch.where(flat < 0, E, flat).long()
    place = torch.empty_like(key)
    place[torch.sort(key, stable=True).indices] = torch.arange(key.numel(), device=key.device)
    ends = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=key.device), ends]).to(torch.int32)
    return offsets, torch.where(flat < 0, -1, place).to(torch.int32).view(idx.shape)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op in ("dispatch", "combine"):
        T, E, topk, D = case["T"], case["E"], case["topk"], case["D"]
        s["idx"] = _choices(g, T, E, topk, case["pad"])
        R = T * topk
        # the program's own buffers: rows behind the last expert's stay as they are
        if op == "dispatch":
            if case["kind"] == "fp8":
                s["x"], s["scale"] = _fp8_rows(g, T, D)
                s["out"] = torch.zeros((R, D), dtype=torch.uint8, device=DEV).view(FP8)
                s["out_scale"] = torch.zeros((R, s["scale"].shape[1]), device=DEV)
            else:
                s["x"] = _normal(g, T, D, dtype=torch.bfloat16)
                s["out"] = torch.zeros((R, D), dtype=torch.bfloat16, device=DEV)
                s["drows"] = _normal(g, R, D, dtype=torch.bfloat16)
        else:
            s["offsets"], s["slots"] = _places(s["idx"], E)
            s["rows"] = _normal(g, R, D, dtype=torch.bfloat16)
            w = torch.sigmoid(_normal(g, T, topk))
            s["topk_w"] = w / w.sum(1, keepdim=True) * 2.5
            if case["train"]:
                s["dx"] = _normal(g, T, D, dtype=torch.bfloat16)
                s["drows"] = torch.zeros((R, D), dtype=torch.bfloat16, device=DEV)
    elif op == "matmul":
        s["a"], s["a_scale"] = _fp8_rows(g, case["M"], case["K"])
        s["w"], s["w_scale"] = _fp8_channels(g, case["N"], case["K"])
        s["dtype"] = torch.float32 if case["out"] == "fp32" else torch.bfloat16
    elif op == "experts":
        E, N, K = case["E"], case["N"], case["K"]
        s["offsets"], _ = _places(_choices(g, case["T"], E, case["topk"], 0), E)
        s["bounds"] = s["offsets"].tolist()  # the router's counts, as a program that logs them has them
        s["a"], s["a_scale"] = _fp8_rows(g, case["T"] * case["topk"], K)
        s["w"] = torch.empty((E, N, K), dtype=FP8, device=DEV)
        s["w_scale"] = torch.empty((E, -(-N // BLOCK), -(-K // BLOCK)), device=DEV)
        for e in range(E):
            s["w"][e], s["w_scale"][e] = _fp8_channels(g, N, K)
        s["dtype"] = torch.float32 if case["out"] == "fp32" else torch.bfloat16
    elif op == "boundary":
        T, D = case["T"], case["D"]
        s["h"] = _normal(g, T, D, dtype=torch.bfloat16)
        s["post_w"] = (1 + 0.1 * _normal(g, D)).to(torch.bfloat16)
        s["pre_w"] = (1 + 0.1 * _normal(g, D)).to(torch.bfloat16)
        if case["moe"]:
            e = torch.empty((T, 8, D), dtype=torch.bfloat16, device=DEV)
            for k in range(8):
                e[:, k] = _normal(g, T, D, dtype=torch.bfloat16)
            s["expert_out"] = e
            w = torch.sigmoid(_normal(g, T, 8))
            s["topk_w"] = w / w.sum(1, keepdim=True) * 2.5
        else:
            s["x"] = _normal(g, T, D, dtype=torch.bfloat16)
    else:
        s["gate_up"] = _normal(g, case["R"], 2 * case["F"], dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------- plain forms

def _row_of(slots, R):
    """The rows' index of every choice; R, one behind the last, for none."""
    return torch.where(slots < 0, R, slots).long()


def _plain_dispatch(s):
    idx, E = s["idx"], s["E"]
    T, K = idx.shape
    R = T * K
    offsets, slots = _places(idx, E)
    at = _row_of(slots, R)
    held = slots >= 0

    def rows(x, out):
        live = torch.zeros(R + 1, dtype=torch.bool, device=x.device)
        live[at.reshape(-1)] = held.reshape(-1)
        token = torch.zeros(R + 1, dtype=torch.int64, device=x.device)
        token[at.reshape(-1)] = torch.arange(R, device=x.device) // K
        live, moved = live[:R, None], x[token[:R]]
        out.copy_(torch.where(live, moved, out))
        return out

    if s["kind"] == "fp8":
        codes = rows(s["x"].view(torch.uint8), s["out"].view(torch.uint8)).view(FP8)
        return offsets, slots, codes, rows(s["scale"], s["out_scale"])
    out = rows(s["x"], s["out"])
    parts = s["drows"].float()[at.clamp(max=R - 1)]
    dx = torch.where(held[:, :, None], parts, torch.zeros_like(parts)).sum(1).to(torch.bfloat16)
    return offsets, slots, out, dx


def _plain_combine(s):
    rows, slots, w = s["rows"], s["slots"], s["topk_w"]
    R = rows.shape[0]
    at, held = _row_of(slots, R), slots >= 0
    parts = rows.float()[at.clamp(max=R - 1)]
    w = torch.where(held, w, torch.zeros_like(w))
    x = (parts * w[:, :, None]).sum(1).to(torch.bfloat16)
    if not s["train"]:
        return x
    dx = s["dx"].float()
    dw = torch.where(held, (parts * dx[:, None, :]).sum(2), torch.zeros_like(w))
    token = torch.zeros(R + 1, dtype=torch.int64, device=rows.device)
    token[at.reshape(-1)] = torch.arange(R, device=rows.device) // slots.shape[1]
    weight = torch.zeros(R + 1, device=rows.device)
    weight[at.reshape(-1)] = w.reshape(-1)
    live = torch.zeros(R + 1, dtype=torch.bool, device=rows.device)
    live[at.reshape(-1)] = held.reshape(-1)
    moved = (weight[:R, None] * dx[token[:R]]).to(torch.bfloat16)
    s["drows"].copy_(torch.where(live[:R, None], moved, s["drows"]))
    return x, s["drows"], dw


def _rows32(q, scale):
    return q.float() * scale.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _channels32(q, scale):
    s = scale.repeat_interleave(BLOCK, 0)[:q.shape[0]].repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    return q.float() * s


def _plain_experts(s):
    a, b = _rows32(s["a"], s["a_scale"]), s["bounds"]
    out = torch.empty((a.shape[0], s["w"].shape[1]), dtype=s["dtype"], device=a.device)
    for e, (lo, hi) in enumerate(zip(b, b[1:])):
        if hi > lo:
            out[lo:hi] = (a[lo:hi] @ _channels32(s["w"][e], s["w_scale"][e]).t()).to(s["dtype"])
    return out


def _to_fp8(y):
    """E4M3 codes of FP32 rows and one scale for each 128 of them."""
    R, D = y.shape
    blocks = -(-D // BLOCK)
    v = torch.nn.functional.pad(y, (0, blocks * BLOCK - D)).view(R, blocks, BLOCK)
    amax = v.abs().amax(2)
    scale = torch.div(amax, torch.full_like(amax, TOP))
    inv = torch.where(amax > 0, torch.div(torch.full_like(amax, TOP), amax), torch.zeros_like(amax))
    q = (v * inv[:, :, None]).clamp(-TOP, TOP).to(FP8).view(R, blocks * BLOCK)
    return q[:, :D].contiguous(), scale


def _rms_factor(v):
    """1 / sqrt(mean(v^2) + eps): the sum in 64 bits, every later step in 32."""
    total = v.double().square().sum(1, keepdim=True).float()
    mean = torch.div(total, torch.full_like(total, float(v.shape[1])))
    return torch.div(torch.ones_like(mean), torch.sqrt(mean + EPS))


def _bf16(v):
    """Rounded to BF16, held in 32 bits."""
    return v.to(torch.bfloat16).float()


def _plain_boundary(s):
    if s["moe"]:
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
    q, scale = _to_fp8(_bf16(h * _rms_factor(h) * s["pre_w"].float()))
    s["h"].copy_(h)
    return s["h"], q, scale


def _plain_swiglu(s):
    gate, up = s["gate_up"].float().split(s["F"], 1)
    return _to_fp8(gate / (1 + torch.exp(-gate)) * up)


def run(state):
    s, op = state, state["op"]
    if own:
        import sandwich_norm_residual_gb300 as snr
        if op == "dispatch":
            offsets, slots = snr.moe_sort(s["idx"], s["E"])
            if s["kind"] == "fp8":
                codes, scale = snr.moe_gather(s["x"], slots, scale=s["scale"], out=s["out"], out_scale=s["out_scale"])
                return offsets, slots, codes, scale
            out = snr.moe_gather(s["x"], slots, out=s["out"])
            return offsets, slots, out, snr.moe_gather_backward(s["drows"], slots)
        if op == "combine":
            x = snr.moe_combine(s["rows"], s["slots"], s["topk_w"])
            if not s["train"]:
                return x
            drows, dw = snr.moe_combine_backward(s["dx"], s["rows"], s["slots"], s["topk_w"], drows=s["drows"])
            return x, drows, dw
        if op == "matmul":
            return snr.matmul_fp8(s["a"], s["a_scale"], s["w"], s["w_scale"], out_dtype=s["dtype"])
        if op == "experts":
            return snr.matmul_fp8_experts(s["a"], s["a_scale"], s["offsets"], s["w"], s["w_scale"], out_dtype=s["dtype"])
        if op == "boundary":
            if s["moe"]:
                q, scale = snr.moe_combine_boundary_fp8(s["h"], s["expert_out"], s["topk_w"], s["post_w"], s["pre_w"],
                                                        s["n"], EPS)
            else:
                q, scale = snr.boundary_fused_fp8(s["h"], s["x"], s["post_w"], s["pre_w"], s["n"], EPS)
            return s["h"], q, scale
        return snr.swiglu_fp8(s["gate_up"])
    if op == "dispatch":
        return _plain_dispatch(s)
    if op == "combine":
        return _plain_combine(s)
    if op == "matmul":
        return (_rows32(s["a"], s["a_scale"]) @ _channels32(s["w"], s["w_scale"]).t()).to(s["dtype"])
    if op == "experts":
        return _plain_experts(s)
    return _plain_boundary(s) if op == "boundary" else _plain_swiglu(s)


# ---------------------------------------------------------------- floors and 64-bit values

def work(case):
    op = case["op"]
    if op in ("dispatch", "combine"):
        T, E, topk, D = case["T"], case["E"], case["topk"], case["D"]
        live = T - case["pad"]
        R = live * topk
        if op == "dispatch":
            row = D + 4 * -(-D // BLOCK) if case["kind"] == "fp8" else 2 * D
            # choices in, places and offsets out, each live token's row once, a copy for each choice
            moved = 8 * T * topk + 4 * (E + 1) + (live + R) * row
            if case["kind"] == "fp8":
                return {"bytes": moved, "flops": 0}
            # the gradient: the copies' rows added up for every token
            return {"bytes": moved + 4 * T * topk + (R + T) * 2 * D, "flops": R * D}
        moved, flops = R * 2 * D + 8 * T * topk + T * 2 * D, 2 * R * D
        if case["train"]:
            # backward: the rows and weights again, the gradient of x in, those of rows and weights out
            moved, flops = moved + (live + 2 * R) * 2 * D + 12 * T * topk, flops + 3 * R * D
        return {"bytes": moved, "flops": flops}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        bn, bk = -(-N // BLOCK), -(-K // BLOCK)
        out = 4 if case["out"] == "fp32" else 2
        return {"bytes": (M + N) * K + 4 * (M + bn) * bk + M * N * out, "flops": 2 * M * N * K}
    if op == "experts":
        R, E, N, K = case["T"] * case["topk"], case["E"], case["N"], case["K"]
        bn, bk = -(-N // BLOCK), -(-K // BLOCK)
        out = 4 if case["out"] == "fp32" else 2
        # the experts that are taken, were all liked alike: a few more than in earnest where there are few rows
        taken = E * (1 - (1 - case["topk"] / E) ** case["T"])
        return {"bytes": R * K + 4 * R * bk + taken * (N * K + 4 * bn * bk) + R * N * out, "flops": 2 * R * N * K}
    if op == "boundary":
        T, D = case["T"], case["D"]
        # read h and the branch, write h', the codes and the scales; the norms' squares and products
        branch, extra = (16 * D + 32, 16 * D) if case["moe"] else (2 * D, 0)
        return {"bytes": T * (2 * D + branch + 2 * D + D + 4 * -(-D // BLOCK)) + 4 * D, "flops": T * (16 * D + extra)}
    R, F = case["R"], case["F"]
    return {"bytes": R * (4 * F + F + 4 * -(-F // BLOCK)), "flops": R * 8 * F}


def _to32(v):
    """64-bit values rounded to FP32, held in 64 bits."""
    return v.float().double()


def _to16(v):
    """64-bit values rounded to FP32 and then to BF16 (nearest even), held in 64 bits."""
    m, e = torch.frexp(_to32(v))
    return torch.ldexp(torch.round(torch.ldexp(m, torch.full_like(e, 8))), e - 8)


def _blocks64(v):
    """64-bit rows as E4M3 numbers (nearest even) with a scale for each 128, the scale in 64 bits."""
    codes, scales = [], []
    for part in v.split(BLOCK, 1):
        top = part.abs().max(1, keepdim=True).values
        u = torch.where(top > 0, part * (TOP / top), torch.zeros_like(part))
        # the step of E4M3: eight to a binade, 2^-9 below 2^-6
        e = torch.frexp(u).exponent.clamp(min=-5)
        step = torch.ldexp(torch.ones_like(u), e - 4)
        codes.append((torch.round(u / step) * step).clamp(-TOP, TOP))
        scales.append(top[:, 0] / TOP)
    return torch.cat(codes, 1), torch.stack(scales, 1)


def _dequantised64(q, scale, per_row):
    rows, cols = torch.arange(q.shape[0], device=DEV), torch.arange(q.shape[1], device=DEV) // BLOCK
    return q.double() * scale.double()[(rows if per_row else rows // BLOCK)[:, None], cols[None, :]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        idx = s["idx"].tolist()
        lists = [[] for _ in range(case["E"])]
        for t, chosen in enumerate(idx):
            for k, e in enumerate(chosen):
                if e >= 0:
                    lists[e].append((t, k))
        offsets, slots, source, at = [0], [[-1] * case["topk"] for _ in idx], [], 0
        for members in lists:
            for t, k in members:
                slots[t][k] = at
                source.append(t)
                at += 1
            offsets.append(at)
        source = torch.tensor(source, dtype=torch.int64, device=DEV)
        offsets = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        slots = torch.tensor(slots, dtype=torch.int32, device=DEV)
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        out[:at] = s["x"].double()[source]
        if case["kind"] == "fp8":
            scale = torch.zeros(s["out_scale"].shape, dtype=torch.float64, device=DEV)
            scale[:at] = s["scale"].double()[source]
            return offsets, slots, out, scale
        dx = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
        dx.index_add_(0, source, s["drows"][:at].double())
        return offsets, slots, out, dx
    if op == "combine":
        x = torch.zeros((case["T"], case["D"]), dtype=torch.float64, device=DEV)
        drows = torch.zeros((case["T"] * case["topk"], case["D"]), dtype=torch.float64, device=DEV) if case["train"] else None
        dw = torch.zeros((case["T"], case["topk"]), dtype=torch.float64, device=DEV)
        for k in range(case["topk"]):
            t = torch.nonzero(s["slots"][:, k] >= 0)[:, 0]
            p = s["slots"][t, k].long()
            row, w = s["rows"][p].double(), s["topk_w"][t, k, None].double()
            x[t] += w * row
            if case["train"]:
                d = s["dx"][t].double()
                drows[p] = w * d
                dw[t, k] = torch.einsum("td,td->t", row, d)
        return (x, drows, dw) if case["train"] else x
    if op == "matmul":
        if 2 * case["M"] * case["N"] * case["K"] > 4e12:
            return None
        a, w = _dequantised64(s["a"], s["a_scale"], True), _dequantised64(s["w"], s["w_scale"], False)
        return torch.cat([part @ w.t() for part in a.split(4096)])
    if op == "experts":
        if 2 * case["T"] * case["topk"] * case["N"] * case["K"] > 4e12:
            return None
        out = []
        for e in range(case["E"]):
            lo, hi = s["bounds"][e], s["bounds"][e + 1]
            if hi > lo:
                a = _dequantised64(s["a"][lo:hi], s["a_scale"][lo:hi], True)
                out.append(a @ _dequantised64(s["w"][e], s["w_scale"][e], False).t())
        return torch.cat(out)
    if op == "swiglu":
        codes, scales = [], []
        for part in s["gate_up"].split(16384):
            gate, up = part[:, :case["F"]].double(), part[:, case["F"]:].double()
            q, scale = _blocks64(gate * torch.sigmoid(gate) * up)
            codes.append(q.float())
            scales.append(scale)
        return torch.cat(codes), torch.cat(scales)
    # the definition rounds at fixed places (FP32 steps, BF16 tensors): 64-bit arithmetic between them
    n, D = case["n"], case["D"]
    if case["moe"]:
        x = torch.zeros((case["T"], D), dtype=torch.float64, device=DEV)
        for k in range(8):
            x = _to32(torch.addcmul(x, s["topk_w"][:, k, None].double(), s["expert_out"][:, k].double()))
        x = _to16(x)
    else:
        x = s["x"].double()

    def norm(v, w):
        mean = _to32(_to32(torch.einsum("td,td->t", v, v)) / D)
        r = _to32(1 / _to32((_to32(mean + float(torch.tensor(EPS)))).sqrt()))
        return _to16(_to32(v * r[:, None]) * w.double())

    xn = norm(x, s["post_w"])
    c1, c2 = (float(torch.tensor(v, dtype=torch.float32)) for v in (((n - 1) / n) ** 0.5, n ** -0.5))
    h = _to16(_to16(c1 * s["h"].double()) + _to16(c2 * xn))
    codes, scales = _blocks64(norm(h, s["pre_w"]))
    return h, codes, scales
