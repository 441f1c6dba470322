"""Cases of the operators around the W8A8 Linear of a transformer block: what is measured, and in what form.

* norm_train: layer norm forward and backward (the gradient of the input, of the weight and of the bias);
* norm_quant: layer norm whose rows leave as E4M3 codes with one scale per token, the input of a W8A8 Linear;
* rope: rotary positions with several axes (time, height, width) on the queries and keys of a fused projection;
* lora: the scaled FP8 Linear with low-rank adapters of many requests beside it.

With ``own`` false ``run`` computes the plain form in elementary torch operations (32 bits, rounded once at the
end); with ``own`` true it calls this package's entry points.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


def listed():
    return [
        # A video transformer's hidden states (32760 tokens, 5120 channels) through a norm with weight and bias,
        # as a fine-tuning step runs it.
        {"name": "norm_train_video", "op": "norm_train", "M": 32760, "K": 5120, "dtype": "bf16", "wdtype": "bf16",
         "groups": 1, "affine": "both", "offset": 0.0, "pad": 0},
        # Adaptive norm of four images: one scale and shift per image, fp32 modulation of fp16 states.
        {"name": "norm_train_adaptive", "op": "norm_train", "M": 16384, "K": 1536, "dtype": "fp16", "wdtype": "fp32",
         "groups": 4, "affine": "both", "offset": 1.0, "pad": 0},
        # A text encoder's short ragged batch in fp32, rows of odd length inside wider ones, no bias.
        {"name": "norm_train_text", "op": "norm_train", "M": 517, "K": 1001, "dtype": "fp32", "wdtype": "fp32",
         "groups": 1, "affine": "weight", "offset": 0.0, "pad": 3},
        # The video block's norm and modulation in front of Q, K and V: 75600 tokens straight to FP8 codes.
        {"name": "norm_quant_video", "op": "norm_quant", "M": 75600, "K": 5120, "dtype": "bf16", "wdtype": "bf16",
         "groups": 1, "affine": "both", "offset": 1.0, "pad": 0, "qmax": 448.0},
        # Serving, eight single tokens: latency of one small launch.
        {"name": "norm_quant_tokens", "op": "norm_quant", "M": 8, "K": 5120, "dtype": "bf16", "wdtype": "fp32",
         "groups": 1, "affine": "both", "offset": 0.0, "pad": 0, "qmax": 448.0},
        # Video queries and keys (21 x 45 x 80 grid, 40 heads of 128) read out of the fused Q/K/V projection,
        # adjacent pairs, channels split 44/42/42 over time, height and width.
        {"name": "rope_video", "op": "rope", "M": 75600, "heads": 40, "kv_heads": 40, "D": 128, "dims": "44,42,42",
         "freqs": "axis", "pairing": "interleaved", "dtype": "bf16", "positions": "grid", "inverse": False},
        # Image and text tokens of a vision-language prompt: grouped keys, halves pairing, one frequency ladder
        # shared out over the axes, far positions.
        {"name": "rope_image", "op": "rope", "M": 6889, "heads": 28, "kv_heads": 4, "D": 128, "dims": "32,48,48",
         "freqs": "ladder", "pairing": "halves", "dtype": "fp16", "positions": "far", "inverse": False},
        # One decoding step of seven sequences in fp32, part of each head rotated.
        {"name": "rope_tokens", "op": "rope", "M": 7, "heads": 16, "kv_heads": 2, "D": 80, "dims": "16,24,24",
         "freqs": "axis", "pairing": "halves", "dtype": "fp32", "positions": "far", "inverse": False},
        # Five requests' prompts packed one after the other, four adapters of rank 64 and rows without one.
        {"name": "lora_prompts", "op": "lora", "M": 32760, "K": 5120, "N": 5120, "R": 64, "adapters": 4,
         "order": "runs", "bias": True},
        # A ragged batch whose rows go to adapters in any order (tokens of many users interleaved).
        {"name": "lora_mixed", "op": "lora", "M": 1777, "K": 5120, "N": 13824, "R": 24, "adapters": 12,
         "order": "any", "bias": False},
        # One decoding step of 64 users, each with an adapter of its own.
        {"name": "lora_users", "op": "lora", "M": 64, "K": 5120, "N": 5120, "R": 16, "adapters": 64,
         "order": "any", "bias": True},
        # A single token with one adapter: latency.
        {"name": "lora_token", "op": "lora", "M": 1, "K": 5120, "N": 5120, "R": 32, "adapters": 3,
         "order": "any", "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_train", "norm_quant", "rope", "lora"])
    if op in ("norm_train", "norm_quant"):
        groups = rng.choice([1, 1, 1, 2, 3, 4, 7])
        M = _log(rng, 1, 33000)
        K = _log(rng, 16, 9000)
        if op == "norm_quant" or rng.random() < 0.6:
            K = -(-K // 16) * 16
        M = min(M, 32000 * 5120 // K)
        M = -(-M // groups) * groups
        c = {"op": op, "M": M, "K": K, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
             "wdtype": "", "groups": groups, "affine": rng.choice(["both", "both", "weight", "none"]),
             "offset": rng.choice([0.0, 1.0]), "pad": rng.choice([0, 0, 5, 64])}
        c["wdtype"] = rng.choice([c["dtype"], "fp32"])
        if op == "norm_quant":
            c["qmax"] = rng.choice([448.0, 448.0, 14.0, 7.0])
        return c
    if op == "rope":
        D = rng.choice([32, 64, 80, 96, 128, 128, 256])
        n = rng.choice([1, 2, 3, 3, 4])
        rot = D if rng.random() < 0.7 else D // 4 * 2
        dims = [rot // n // 2 * 2] * n
        dims[0] += rot - sum(dims)
        heads = rng.choice([1, 3, 8, 16, 40])
        kv = rng.choice([h for h in (1, 3, 4, 8, 16, 40) if heads % h == 0])
        M = min(_log(rng, 1, 40000), 75600 * 40 * 128 // ((heads + kv) * D))
        return {"op": op, "M": M, "heads": heads, "kv_heads": kv, "D": D, "dims": ",".join(map(str, dims)),
                "freqs": rng.choice(["axis", "ladder"]), "pairing": rng.choice(["interleaved", "halves"]),
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "positions": rng.choice(["grid", "far"]),
                "inverse": rng.random() < 0.4}
    K = -(-_log(rng, 64, 14000) // 16) * 16
    N = -(-_log(rng, 64, 14000) // 8) * 8
    R = rng.choice([8, 16, 24, 32, 64, 64, 128])
    M = max(1, min(_log(rng, 1, 32000), 32760 * 5120 * 5000 // (K * N)))
    return {"op": op, "M": M, "K": K, "N": N, "R": R, "adapters": rng.randint(1, max(1, min(64, 2048 // R))),
            "order": rng.choice(["runs", "runs", "any"]), "bias": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _frequencies(c):
    """(inverse frequencies, axis) of every rotated pair, as a model's configuration gives them."""
    dims = [int(d) for d in c["dims"].split(",")]
    pairs = [(a, j, d) for a, d in enumerate(dims) for j in range(d // 2)]
    if c["freqs"] == "axis":  # every axis with a ladder of its own
        inv = [10000.0 ** (-2.0 * j / d) for _, j, d in pairs]
    else:  # one ladder over all rotated channels, shared out over the axes
        inv = [10000.0 ** (-2.0 * i / sum(dims)) for i in range(len(pairs))]
    return torch.tensor(inv, dtype=torch.float64), torch.tensor([a for a, _, _ in pairs], dtype=torch.int32)


def _states(M, K, g, pad=0, dtype=torch.bfloat16):
    """Hidden states: unit normal, an offset per channel, 1 % of the channels thirty times larger."""
    gain = torch.ones(K, device="cuda")
    gain[torch.rand(K, generator=g, device="cuda") < 0.01] = 30.0
    x = torch.empty((M, K + pad), dtype=dtype, device="cuda")
    x.normal_(generator=g)
    x[:, :K].mul_(gain.to(dtype)).add_((0.5 * torch.randn(K, generator=g, device="cuda")).to(dtype))
    return x[:, :K]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if c["op"] in ("norm_train", "norm_quant"):
        M, K, G, dt, wdt = c["M"], c["K"], c["groups"], DTYPES[c["dtype"]], DTYPES[c["wdtype"]]
        s = {"case": c, "x": _states(M, K, g, c["pad"], dt), "w": None, "b": None}
        shape = (G, K) if G > 1 else (K,)
        if c["affine"] != "none":
            s["w"] = (1.0 - c["offset"] + 0.2 * randn(*shape)).to(wdt)
        if c["affine"] == "both":
            s["b"] = (0.2 * randn(*shape)).to(wdt)
        if c["op"] == "norm_train":
            s["dy"] = (0.01 * randn(M, K)).to(dt)
        return s
    if c["op"] == "rope":
        M, H, Hk, D, dt = c["M"], c["heads"], c["kv_heads"], c["D"], DTYPES[c["dtype"]]
        qkv = torch.empty((M, H + 2 * Hk, D), dtype=dt, device="cuda").normal_(generator=g)
        inv, axis = _frequencies(c)
        n = len(c["dims"].split(","))
        if c["positions"] == "grid":  # raster order over the axes, the first one slowest
            side = [1] * n
            while math.prod(side) < M:
                i = min(range(n), key=lambda a: side[a] * (2 if a == 0 else 1))
                side[i] += 1
            pos, rest = [], torch.arange(M, device="cuda")
            for d in reversed(side):
                pos.append(rest % d)
                rest = rest // d
            pos = torch.stack(pos[::-1], 1)
        else:
            pos = torch.randint(-100, 1 << 20, (M, n), generator=g, device="cuda")
        return {"case": c, "q": qkv[:, :H], "k": qkv[:, H:H + Hk], "pos": pos.to(torch.int32), "inv": inv,
                "axis": axis, "inv_gpu": inv.cuda(), "axis_gpu": axis.cuda().long()}
    M, K, N, R, n = c["M"], c["K"], c["N"], c["R"], c["adapters"]
    x = _states(M, K, g)
    s_a = x.float().abs().amax(1).clamp_min(1e-12) / 448.0
    A_q = (x.float() / s_a[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    w = 0.02 * randn(N, K)
    s_w = w.abs().amax(1).clamp_min(1e-12) / 448.0
    W_q = (w / s_w[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    lora_A = (randn(n, R, K) / math.sqrt(K)).bfloat16()
    lora_B = (0.3 * randn(n, N, R) / math.sqrt(R)).bfloat16()
    scaling = 0.5 + torch.rand(n, generator=g, device="cuda")
    if c["order"] == "runs":  # requests one after the other, one in five without an adapter
        cuts = torch.sort(torch.randint(0, M, (n,), generator=g, device="cuda")).values
        which = torch.randint(-1, n, (n + 1,), generator=g, device="cuda")
        idx = which[torch.searchsorted(cuts, torch.arange(M, device="cuda"), right=True)]
    else:
        idx = torch.randint(-1 if M > 1 else 0, n, (M,), generator=g, device="cuda")
    return {"case": c, "x": x, "A_q": A_q, "s_a": s_a, "W_q": W_q, "s_w": s_w, "lora_A": lora_A, "lora_B": lora_B,
            "scaling": scaling, "idx": idx.to(torch.int32), "bias": randn(N).bfloat16() if c["bias"] else None,
            # the adapter's second factor as a server keeps it beside this weight: scaled, in units of s_w
            "lora_Bs": (lora_B.float() * scaling[:, None, None] / s_w[None, :, None]).bfloat16()}


# -------------------------------------------------------------- plain forms
def _rows(v, M, K, offset):
    """A weight or bias per row: [K] or [G, K] spread over the G groups of equally many rows."""
    v = v.float().reshape(-1, K) + offset
    return v if v.shape[0] == 1 else v.repeat_interleave(M // v.shape[0], 0)


def _norm(s):
    x = s["x"].float()
    M, K = x.shape
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    xhat = xc * rstd
    y = xhat
    if s["w"] is not None:
        y = y * _rows(s["w"], M, K, s["case"]["offset"])
    if s["b"] is not None:
        y = y + _rows(s["b"], M, K, 0.0)
    return y, xhat, rstd


def _plain_norm_train(s):
    x, w, b = s["x"], s["w"], s["b"]
    M, K = x.shape
    y, xhat, rstd = _norm(s)
    y = y.to(x.dtype)
    dy = s["dy"].float()
    wdy = dy if w is None else dy * _rows(w, M, K, s["case"]["offset"])
    dx = (wdy - wdy.mean(1, keepdim=True) - xhat * (wdy * xhat).mean(1, keepdim=True)) * rstd
    out = {"y": y, "dx": dx.to(x.dtype)}
    G = s["case"]["groups"]
    if w is not None:
        out["dw"] = (dy * xhat).view(G, M // G, K).sum(1).reshape(w.shape).to(w.dtype)
    if b is not None:
        out["db"] = dy.view(G, M // G, K).sum(1).reshape(b.shape).to(b.dtype)
    return out


def _plain_norm_quant(s):
    y, _, _ = _norm(s)
    qmax = s["case"]["qmax"]
    scale = y.abs().amax(1).clamp_min(1e-12) / qmax
    q = (y / scale[:, None]).clamp(-qmax, qmax).to(torch.float8_e4m3fn)
    return {"q": q, "s": scale}


def _plain_rope(s):
    c = s["case"]
    angle = s["pos"].double()[:, s["axis_gpu"]] * s["inv_gpu"]  # 64 bits: positions up to a million
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if c["inverse"]:
        sin = -sin
    P = angle.shape[1]

    def rotate(v):
        f = v.float()
        if c["pairing"] == "interleaved":
            a, b = f[..., 0:2 * P:2], f[..., 1:2 * P:2]
            r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = f[..., :P], f[..., P:2 * P]
            r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((r, f[..., 2 * P:]), -1).to(v.dtype)

    return {"q": rotate(s["q"]), "k": rotate(s["k"])}


def _plain_lora(s):
    x, A, B, idx = s["x"], s["lora_A"], s["lora_B"], s["idx"]
    n, R, K = A.shape
    N = B.shape[1]
    y = s["A_q"].view(torch.float8_e4m3fn).float() @ s["W_q"].view(torch.float8_e4m3fn).float().t()
    y = y * s["s_a"][:, None] * s["s_w"][None, :]
    # every adapter's product, the rows' own kept
    t = (x.float() @ A.float().view(n * R, K).t()).view(-1, n, R)
    mine = (idx[:, None] == torch.arange(n, device=idx.device)[None, :]).float() * s["scaling"][None, :]
    t = t * mine[:, :, None]
    y = y + t.view(-1, n * R) @ B.float().transpose(1, 2).reshape(n * R, N)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return {"y": y.bfloat16()}


# ------------------------------------------------------------------- calls
def run(state):
    s, c = state, state["case"]
    if own:
        import int8_w8a8_quantized_b200 as tfq
        if c["op"] == "norm_train":
            y, mean, rstd = tfq.tfq_layer_norm(s["x"], s["w"], s["b"], eps=EPS, weight_offset=c["offset"], stats=True)
            dx, dw, db = tfq.tfq_layer_norm_backward(s["dy"], s["x"], s["w"], mean, rstd, weight_offset=c["offset"],
                                                     need_bias=s["b"] is not None)
            out = {"y": y, "dx": dx}
            if dw is not None:
                out["dw"] = dw
            if db is not None:
                out["db"] = db
            return out
        if c["op"] == "norm_quant":
            q, scale = tfq.tfq_layer_norm_quant_fp8(s["x"], s["w"], s["b"], eps=EPS, weight_offset=c["offset"],
                                                    qmax=c["qmax"])
            return {"q": q.view(torch.float8_e4m3fn), "s": scale}
        if c["op"] == "rope":
            q, k = tfq.tfq_rope_axes(s["q"], s["k"], s["pos"], s["inv"], s["axis"], pairing=c["pairing"],
                                     inverse=c["inverse"])
            return {"q": q, "k": k}
        return {"y": tfq.tfq_scaled_fp8_linear_lora(s["A_q"], s["s_a"], s["W_q"], s["s_w"], s["x"], s["lora_A"],
                                                    s["lora_Bs"], s["idx"], bias=s["bias"])}
    plain = {"norm_train": _plain_norm_train, "norm_quant": _plain_norm_quant, "rope": _plain_rope,
             "lora": _plain_lora}
    return plain[c["op"]](s)


def work(case):
    c = case
    if c["op"] in ("norm_train", "norm_quant"):
        M, K, e, we = c["M"], c["K"], SIZE[c["dtype"]], SIZE[c["wdtype"]]
        vecs = {"none": 0, "weight": 1, "both": 2}[c["affine"]] * c["groups"] * K * we
        if c["op"] == "norm_quant":
            return {"bytes": M * K * (e + 1) + 4 * M + vecs, "flops": 9 * M * K}
        return {"bytes": 4 * M * K * e + 2 * vecs, "flops": 20 * M * K}
    if c["op"] == "rope":
        n = c["M"] * (c["heads"] + c["kv_heads"]) * c["D"]
        axes = len(c["dims"].split(","))
        return {"bytes": 2 * n * SIZE[c["dtype"]] + 4 * c["M"] * axes, "flops": 3 * n}
    M, K, N, R = c["M"], c["K"], c["N"], c["R"]
    used = min(c["adapters"], M)
    return {"bytes": 3 * M * K + 8 * M + N * (K + 4) + 2 * M * N + 2 * used * R * (K + N) + 2 * N * c["bias"],
            "flops": 2 * M * N * K + 2 * M * R * (K + N)}


# -------------------------------------------- the definitions in 64 bits
def _e4m3(v):
    """The E4M3 value nearest to v (|v| <= 448, ties to the even code), in 64 bits."""
    _, e = torch.frexp(v)  # |v| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp_min(-9))
    return torch.round(v / step) * step


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] in ("norm_train", "norm_quant"):
        x = s["x"].to(f64)
        M, K = x.shape
        G = c["groups"]
        x = x.view(G, M // G, K)
        var, mean = torch.var_mean(x, dim=2, unbiased=False, keepdim=True)
        r = torch.rsqrt(var + EPS)
        xh = (x - mean).mul_(r)
        del x
        w = None if s["w"] is None else s["w"].to(f64).view(G, 1, K) + c["offset"]
        y = xh if w is None else xh * w
        if s["b"] is not None:
            y = y + s["b"].to(f64).view(G, 1, K)
        y = y.reshape(M, K)
        if c["op"] == "norm_quant":
            sc = y.abs().amax(1).clamp_min(1e-12) / c["qmax"]
            return {"q": _e4m3((y / sc[:, None]).clamp(-c["qmax"], c["qmax"])), "s": sc}
        dy = s["dy"].to(f64).view(G, M // G, K)
        out = {"y": y}
        if s["w"] is not None:
            out["dw"] = torch.einsum("gmk,gmk->gk", dy, xh).reshape(s["w"].shape)
        if s["b"] is not None:
            out["db"] = torch.einsum("gmk->gk", dy).reshape(s["b"].shape)
        h = dy if w is None else dy * w
        c1 = torch.einsum("gmk->gm", h)[..., None] / K
        c2 = torch.einsum("gmk,gmk->gm", h, xh)[..., None] / K
        out["dx"] = (r * (h - c1 - xh * c2)).reshape(M, K)
        return {k: out[k] for k in ("y", "dx", "dw", "db") if k in out}
    if c["op"] == "rope":
        turn = torch.complex(torch.zeros(1, dtype=f64, device="cuda"),
                             s["pos"].to(f64)[:, s["axis_gpu"]] * s["inv_gpu"] * (-1.0 if c["inverse"] else 1.0))
        turn = torch.exp(turn)[:, None]
        P = turn.shape[-1]

        def rotated(v):
            f = v.to(f64)
            r = f.clone()
            first, second = ((slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if c["pairing"] == "interleaved" else
                             (slice(0, P), slice(P, 2 * P)))
            z = torch.complex(f[..., first], f[..., second]) * turn
            r[..., first], r[..., second] = z.real, z.imag
            return r

        return {"q": rotated(s["q"]), "k": rotated(s["k"])}
    y = s["A_q"].view(torch.float8_e4m3fn).to(f64).mul_(s["s_a"].to(f64)[:, None]) @ \
        s["W_q"].view(torch.float8_e4m3fn).to(f64).mul_(s["s_w"].to(f64)[:, None]).T
    for a in range(c["adapters"]):  # the rows of one adapter at a time
        rows = torch.nonzero(s["idx"] == a).flatten()
        if rows.numel():
            t = s["x"][rows].to(f64) @ s["lora_A"][a].to(f64).T
            y[rows] += (t @ s["lora_B"][a].to(f64).T) * s["scaling"][a].to(f64)
    if s["bias"] is not None:
        y += s["bias"].to(f64)
    return {"y": y}
