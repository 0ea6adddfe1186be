"""Cases that measure the expert FFN's 8-bit products with a scale for each block of 128 and what feeds them:
the root-mean-square norm that hands its rows on in 8 bits, the router's balance loss, the quantizers of
rows, tokens and weights, and linear layers grouped by expert on 8-bit operands.

`run` computes a case either in plain torch operations (`own` false) or with the library's entry points
(`own` true); `exact` gives the same outputs from the operators' definitions in 64 bits.

8 bits: E4M3 codes with one float32 scale per block, amax / 448, and codes of value * (448 / amax).  A block is
128 consecutive values of a row ("rows"), 128 rows of one column ("tokens"), or 128 rows of 128 columns
("tiles").  Blocks of rows start anew with every expert, whose rows are laid out on multiples of 128.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 128
TINY = 2.0 ** -100                                                      # the smallest magnitude a scale is made for


# ---- cases --------------------------------------------------------------------------------------
def listed():
    return [
        # one token of a served model: the residual added, rows for the router (bf16) and for the 8-bit product
        dict(name="rms_fwd_T1_H4096_fp8", op="rms", rows=1, H=4096, f32=False, residual=True, save8=True, step=False),
        # the fine-grained workload's tokens in training
        dict(name="rms_step_T32768_H2048_fp8", op="rms", rows=32768, H=2048, f32=False, residual=True, save8=True, step=True),
        # odd rows of a float32 stream that no wide load fits
        dict(name="rms_step_T1237_H1001_f32", op="rms", rows=1237, H=1001, f32=True, residual=False, save8=False, step=True),
        # a small fine-tuning batch on eight experts: latency
        dict(name="balance_T64_E8_k2", op="balance", rows=64, E=8, k=2, masked=False),
        # the fine-grained workload's routing, with padded tokens
        dict(name="balance_T32768_E64_k6_masked", op="balance", rows=32768, E=64, k=6, masked=True),
        # a gradient on its way to the input's and the weights' gradients: along rows and along tokens
        dict(name="quant_R65536_C2048_E64", op="quant", rows=65536, cols=2048, E=64, skew=2.0, f32=False, tiles=False),
        # the uneven workload's gate_up weights
        dict(name="quant_weights_N5632_K1024_E8", op="weights", N=5632, K=1024, E=8, f32=False),
        # one token through a dense projection of a Mixtral-shaped model: latency and the weights
        dict(name="linear8_fwd_R1_K14336_N4096_E1", op="linear8", rows=1, K=14336, N=4096, E=1, skew=0.0, step=False),
        # eight tokens of a served Mixtral-shaped model: bound by reading the experts' weights once
        dict(name="linear8_fwd_R16_K4096_N28672_E8", op="linear8", rows=16, K=4096, N=28672, E=8, skew=0.5, step=False),
        # the Mixtral-shaped workload's gate_up product
        dict(name="linear8_fwd_R32768_K4096_N28672_E8", op="linear8", rows=32768, K=4096, N=28672, E=8, skew=0.2, step=False),
        # the fine-grained workload's gate_up layer, forward and both gradients, skewed loads with empty experts
        dict(name="linear8_step_R196608_K2048_N2816_E64", op="linear8", rows=196608, K=2048, N=2816, E=64, skew=2.0, step=True),
        # ragged in every size
        dict(name="linear8_step_R777_K208_N144_E5", op="linear8", rows=777, K=208, N=144, E=5, skew=1.0, step=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rms", "balance", "quant", "weights", "linear8", "linear8"])
    if op == "rms":
        H = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            H = (H + 7) // 8 * 8
        return dict(op=op, rows=_log(rng, 1, min(65536, 60_000_000 // H)), H=H, f32=rng.random() < 0.3,
                    residual=rng.random() < 0.5, save8=rng.random() < 0.7, step=rng.random() < 0.6)
    if op == "balance":
        E = _log(rng, 2, 256)
        return dict(op=op, rows=_log(rng, 1, min(65536, 4_000_000 // E)), E=E, k=rng.randint(1, min(8, E)),
                    masked=rng.random() < 0.5)
    if op == "quant":
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            cols = (cols + 15) // 16 * 16
        return dict(op=op, rows=_log(rng, 1, min(65536, 100_000_000 // cols)), cols=cols, E=_log(rng, 1, 64),
                    skew=round(rng.uniform(0.0, 2.0), 2), f32=rng.random() < 0.3, tiles=rng.random() < 0.4)
    E = _log(rng, 1, 64)
    K, N = 16 * _log(rng, 4, 256), 16 * _log(rng, 4, 512)
    while E * K * N > (100_000_000 if op == "weights" else 500_000_000):
        E, N = max(1, E // 2), N if E > 1 else max(16, N // 32 * 16)
    if op == "weights":
        return dict(op=op, N=N, K=K, E=E, f32=rng.random() < 0.4)
    rows = _log(rng, 1, max(2, min(65536, int(6e11 / (K * N)))))
    return dict(op=op, rows=rows, K=K, N=N, E=E, skew=round(rng.uniform(0.0, 2.0), 2), step=rng.random() < 0.5)


# ---- 8 bits in plain operations -------------------------------------------------------------------
def _codes(v, amax):
    """E4M3 codes of v (float32) and their scale, of blocks whose largest magnitudes are amax (broadcast over v)."""
    amax = amax.clamp(min=TINY)
    return (v * (448.0 / amax)).to(torch.float8_e4m3fn), amax / 448.0


def _blocks(v, dim):
    """v with dimension `dim` cut into blocks of 128, the last one filled up with zeros."""
    fill = -v.shape[dim] % BLOCK
    if fill:
        v = torch.cat([v, v.new_zeros([fill if d == dim else n for d, n in enumerate(v.shape)])], dim)
    return v.unflatten(dim, (-1, BLOCK))


def _rows8(v):
    """Codes [R][C] and scales [ceil(C/128)][R] of float32 rows."""
    b = _blocks(v, 1)
    c, s = _codes(b, b.abs().amax(2, keepdim=True))
    return c.flatten(1)[:, : v.shape[1]], s.squeeze(2).t().contiguous()


def _rows8_back(c, s):
    return _blocks(c.float(), 1).mul_(s.t()[:, :, None]).flatten(1)[:, : c.shape[1]]


def _tokens8(v, tiles):
    """Codes [B*128][C] and scales, [B][C] or (tiles) [B][ceil(C/128)], of float32 rows laid out on blocks of 128."""
    b = v.unflatten(0, (-1, BLOCK))
    if not tiles:
        c, s = _codes(b, b.abs().amax(1, keepdim=True))
        return c.flatten(0, 1), s.squeeze(1)
    b = _blocks(b, 2)                                                   # [B][128][ceil][128]
    c, s = _codes(b, b.abs().amax((1, 3), keepdim=True))
    return c.flatten(0, 1).flatten(1)[:, : v.shape[1]], s[:, 0, :, 0]


def _tokens8_back(c, s, tiles):
    if not tiles:
        return c.float().unflatten(0, (-1, BLOCK)).mul_(s[:, None, :]).flatten(0, 1)
    b = _blocks(c.float(), 1).unflatten(0, (-1, BLOCK))
    return b.mul_(s[:, None, :, None]).flatten(0, 1).flatten(1)[:, : c.shape[1]]


def _weight8(w):
    """Codes [N][K] and scales [ceil(N/128)][ceil(K/128)] of one float32 matrix."""
    c, s = _tokens8(_blocks(w, 0).flatten(0, 1), True)
    return c[: w.shape[0]], s


def _weight8_back(c, s):
    return _tokens8_back(_blocks(c.float(), 0).flatten(0, 1), s, True)[: c.shape[0]]


# ---- inputs -------------------------------------------------------------------------------------
def _counts(case, g):
    """Rows of each expert: a multinomial over softmax(skew * normal), the last of several experts empty."""
    E = case["E"]
    p = torch.softmax(case["skew"] * torch.randn(E, generator=g, dtype=torch.float64), 0)
    if E > 2:
        p[E - 1] = 0.0
    pick = torch.multinomial(p, case["rows"], replacement=True, generator=g)
    return torch.bincount(pick, minlength=E).tolist()


def _places(counts, dev):
    """The row of every row in the layout on blocks of 128, and that layout's blocks (as many as any split of the rows takes)."""
    n = torch.tensor(counts, dtype=torch.int64)
    blocks = (n + BLOCK - 1) // BLOCK
    first = (torch.cumsum(blocks, 0) - blocks) * BLOCK
    at = torch.repeat_interleave(first - (torch.cumsum(n, 0) - n), n) + torch.arange(int(n.sum()))
    return at.to(dev), int(n.sum()) // BLOCK + len(counts)


def _spread(v, places, blocks):
    return v.new_zeros(blocks * BLOCK, v.shape[1]).index_copy_(0, places, v)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    op, u8, f32, bf16 = case["op"], torch.uint8, torch.float32, torch.bfloat16

    def normal(*shape, dtype=bf16, std=1.0, mean=0.0):
        t = torch.randn(*shape, generator=g, device=dev, dtype=bf16 if dtype == bf16 else f32)
        return t.mul_(std).add_(mean).to(dtype)

    def empty(*shape, dtype=bf16):
        return torch.zeros(*shape, device=dev, dtype=dtype)

    def channels(n):
        return normal(n, dtype=f32, std=0.5).exp_()                     # a few channels carry more than the others

    s = {"case": dict(case)}
    if op == "rms":
        R, H, t = case["rows"], case["H"], f32 if case["f32"] else bf16
        s["x"] = (normal(R, H, dtype=f32) * channels(H)).to(t)
        s["residual"] = normal(R, H, dtype=t, std=0.3) if case["residual"] else None
        s["gamma"] = normal(H, dtype=t, std=0.1, mean=1.0)
        s["h"] = empty(R, H, dtype=t) if case["residual"] else None
        s["y"], s["rstd"] = empty(R, H, dtype=t), empty(R, dtype=f32)
        if case["save8"]:
            s["codes"], s["scales"] = empty(R, H, dtype=u8), empty((H + 127) // BLOCK, R, dtype=f32)
            s["y8"] = empty(R, H)
        if case["step"]:
            s["dy"] = normal(R, H, dtype=t, std=0.01)
            s["dres"] = normal(R, H, dtype=t, std=0.01) if case["residual"] else None
            s["dx"], s["dgamma"] = empty(R, H, dtype=t), empty(H, dtype=t)
    elif op == "balance":
        T, E, k = case["rows"], case["E"], case["k"]
        s["logits"] = normal(T, E, dtype=f32) + normal(E, dtype=f32)    # some experts are liked more than others
        s["idx"] = s["logits"].topk(k, 1).indices.to(torch.int32)
        s["mask"] = None
        if case["masked"]:                                              # padding behind sequences of all lengths
            s["mask"] = (torch.rand(T, generator=g, device=dev) < 0.8).to(u8)
        s["alpha"], s["beta"] = 0.01, 0.001
        s["grad"] = torch.rand(1, generator=g, device=dev) + 0.5        # what the loss is multiplied by behind it
        s["counts"], s["prob"], s["loss"] = empty(E + 1, dtype=torch.int32), empty(E, dtype=f32), empty(3, dtype=f32)
        s["dlogits"] = empty(T, E, dtype=f32)
    elif op == "quant":
        R, C, E = case["rows"], case["cols"], case["E"]
        s["src"] = (normal(R, C, dtype=f32, std=0.01) * channels(C)).to(f32 if case["f32"] else bf16)
        s["counts"] = _counts(case, host)
        s["split_sizes"] = torch.tensor(s["counts"], dtype=torch.int32, device=dev)
        s["places"], blocks = _places(s["counts"], dev)
        s["blocks"] = blocks
        s["codes"], s["scales"] = empty(R, C, dtype=u8), empty((C + 127) // BLOCK, R, dtype=f32)
        s["tcodes"] = empty(blocks * BLOCK, C, dtype=u8)
        s["tscales"] = empty(blocks, (C + 127) // BLOCK if case["tiles"] else C, dtype=f32)
        s["back"], s["tback"] = empty(R, C), empty(blocks * BLOCK, C)
    elif op == "weights":
        E, N, K = case["E"], case["N"], case["K"]
        s["w"] = normal(E, N, K, dtype=f32 if case["f32"] else bf16, std=0.02)
        s["codes"] = empty(E, N, K, dtype=u8)
        s["scales"] = empty(E, (N + 127) // BLOCK, (K + 127) // BLOCK, dtype=f32)
        s["back"] = empty(E, N, K)
    else:
        R, K, N, E = case["rows"], case["K"], case["N"], case["E"]
        s["counts"] = _counts(case, host)
        s["split_sizes"] = torch.tensor(s["counts"], dtype=torch.int32, device=dev)
        wq = [_weight8(normal(N, K, dtype=f32, std=0.02)) for _ in range(E)]
        s["w"], s["w_scales"] = torch.stack([c for c, _ in wq]).view(u8), torch.stack([q for _, q in wq])
        x = normal(R, K, dtype=f32) * channels(K)
        c, s["x_scales"] = _rows8(x)
        s["x"] = c.contiguous().view(u8)
        s["y"] = empty(R, N)
        if case["step"]:
            places, blocks = _places(s["counts"], dev)
            dy = normal(R, N, dtype=f32, std=0.01) * torch.rand(R, 1, generator=g, device=dev)
            c, s["dy_scales"] = _rows8(dy)
            s["dy"] = c.contiguous().view(u8)
            c, s["xt_scales"] = _tokens8(_spread(x, places, blocks), True)
            s["xt"] = c.contiguous().view(u8)
            c, s["dyt_scales"] = _tokens8(_spread(dy, places, blocks), False)
            s["dyt"] = c.contiguous().view(u8)
            s["xt_scales"], s["dyt_scales"] = s["xt_scales"].contiguous(), s["dyt_scales"].contiguous()
            s["dx"], s["dw"] = empty(R, K), empty(E, N, K)
    return s


# ---- plain forms --------------------------------------------------------------------------------
def _plain_rms(s):
    c = s["case"]
    t = s["x"].dtype
    h = s["x"].float()
    if c["residual"]:
        h = h + s["residual"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    gamma = s["gamma"].float()
    y = h * rstd * gamma
    out = {"y": y.to(t)}
    if c["residual"]:
        out["h"] = h.to(t)
    if c["save8"]:
        out["y8"] = _rows8_back(*_rows8(y)).to(torch.bfloat16)
    if c["step"]:
        n = h.to(t).float() * rstd                                      # what is kept is the rounded sum
        dy = s["dy"].float()
        d = dy * gamma
        dx = rstd * (d - n * (d * n).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dres"].float()
        out["dx"], out["dgamma"] = dx.to(t), (dy * n).sum(0).to(t)
    return out


def _plain_balance(s):
    c = s["case"]
    T, E, k = c["rows"], c["E"], c["k"]
    live = torch.ones(T, dtype=torch.bool, device=s["logits"].device) if s["mask"] is None else s["mask"] != 0
    tokens = live.sum()
    chosen = torch.zeros(T, E, dtype=torch.int32, device=live.device).scatter_(1, s["idx"].long(), 1)
    counts = (chosen * live[:, None]).sum(0, dtype=torch.int32)
    top = s["logits"].amax(1, keepdim=True)
    e = torch.exp(s["logits"] - top)
    z = e.sum(1, keepdim=True)
    soft, lse = e / z, (top + torch.log(z)).squeeze(1)
    zero = torch.zeros((), device=live.device)
    soft, lse = torch.where(live[:, None], soft, zero), torch.where(live, lse, zero)
    n = tokens.clamp(min=1).double()
    prob = (soft.double().sum(0) / n).float()                           # long sums
    load = E * counts.double() / (k * n)
    balance, zl = (load * prob).sum(), (lse.double() ** 2).sum() / n
    loss = torch.stack([s["alpha"] * balance + s["beta"] * zl, balance, zl]).float()
    # the loads less their mean, so that even loads do not cancel (the softmax sums to one)
    f = (load - 1.0).float()
    scale = s["grad"] / n.float()
    d = s["alpha"] * soft * (f - (soft * f).sum(1, keepdim=True)) + 2.0 * s["beta"] * lse[:, None] * soft
    return {"counts": torch.cat([counts, tokens[None].to(torch.int32)]), "prob": prob, "loss": loss, "dlogits": d * scale}


def _plain_linear(s):
    c = s["case"]
    u = torch.float8_e4m3fn
    y = torch.empty_like(s["y"])
    out = {"y": y}
    x = _rows8_back(s["x"].view(u), s["x_scales"])
    if c["step"]:
        out["dx"], out["dw"] = torch.empty_like(s["dx"]), torch.zeros_like(s["dw"])
        dy = _rows8_back(s["dy"].view(u), s["dy_scales"])
        xt = _tokens8_back(s["xt"].view(u), s["xt_scales"], True)
        dyt = _tokens8_back(s["dyt"].view(u), s["dyt_scales"], False)
    r0 = b0 = 0
    for e, n in enumerate(s["counts"]):
        if n == 0:
            continue
        rows, padded = slice(r0, r0 + n), slice(b0, b0 + n)
        w = _weight8_back(s["w"][e].view(u), s["w_scales"][e])
        y[rows] = x[rows] @ w.t()
        if c["step"]:
            out["dx"][rows] = dy[rows] @ w
            out["dw"][e] = dyt[padded].t() @ xt[padded]
        r0 += n
        b0 += (n + BLOCK - 1) // BLOCK * BLOCK
    return out


def _plain_quant(s):
    v = s["src"].float()
    tiles = s["case"]["tiles"]
    t = _tokens8(_spread(v, s["places"], s["blocks"]), tiles)
    return {"rows": _rows8_back(*_rows8(v)).to(torch.bfloat16), "tokens": _tokens8_back(*t, tiles).to(torch.bfloat16)}


def _plain_weights(s):
    w = s["w"]
    N = w.shape[1]
    b = _blocks(w.float(), 1).flatten(1, 2)                             # every expert's rows on blocks of 128
    back = _tokens8_back(*_tokens8(b.flatten(0, 1), True), True)
    return {"back": back.view(b.shape)[:, :N].to(torch.bfloat16)}


# ---- the library's entry points -------------------------------------------------------------------
def _workspace(s, size):
    if "ws" not in s:
        dev = torch.device("cuda")
        s["ws"] = torch.zeros(max(256, size), dtype=torch.uint8, device=dev)
    return s["ws"]


def _own_rms(s):
    from moe_expert_ffn_03_gb300 import binding as B
    c = s["case"]
    n = B.norm(c["rows"], c["H"], x_f32=c["f32"], w_f32=c["f32"], eps=EPS)
    codes, scales = s.get("codes"), s.get("scales")
    B.moe_rmsnorm_fwd(n, s["x"], s["residual"], s["gamma"], s["h"], s["y"], s["rstd"], codes, scales)
    out = {"y": s["y"]}
    if c["residual"]:
        out["h"] = s["h"]
    if c["save8"]:
        B.moe_fp8_block_dequantize(codes, scales, "rows", s["y8"])
        out["y8"] = s["y8"]
    if c["step"]:
        ws = _workspace(s, B.moe_rmsnorm_workspace_size(n))
        B.moe_rmsnorm_bwd(n, s["dy"], s["h"] if c["residual"] else s["x"], s["rstd"], s["gamma"], s["dres"], s["dx"],
                          s["dgamma"], ws)
        out["dx"], out["dgamma"] = s["dx"], s["dgamma"]
    return out


def _own_balance(s):
    from moe_expert_ffn_03_gb300 import binding as B
    c = s["case"]
    b = B.balance(c["rows"], c["E"], c["k"], alpha=s["alpha"], beta=s["beta"])
    ws = _workspace(s, B.moe_balance_loss_workspace_size(b))
    B.moe_balance_loss_fwd(b, s["logits"], s["idx"], s["mask"], s["counts"], s["prob"], s["loss"], ws)
    B.moe_balance_loss_bwd(b, s["logits"], s["mask"], s["counts"], s["grad"], s["dlogits"])
    return {"counts": s["counts"], "prob": s["prob"], "loss": s["loss"], "dlogits": s["dlogits"]}


def _own_quant(s):
    from moe_expert_ffn_03_gb300 import binding as B
    kind = "tiles" if s["case"]["tiles"] else "tokens"
    B.moe_fp8_block_quantize(s["src"], s["codes"], s["scales"], s["split_sizes"], s["tcodes"], s["tscales"], kind)
    B.moe_fp8_block_dequantize(s["codes"], s["scales"], "rows", s["back"])
    B.moe_fp8_block_dequantize(s["tcodes"], s["tscales"], kind, s["tback"])
    return {"rows": s["back"], "tokens": s["tback"]}


def _own_weights(s):
    from moe_expert_ffn_03_gb300 import binding as B
    B.moe_fp8_block_quantize_weights(s["w"], s["codes"], s["scales"])
    B.moe_fp8_block_dequantize(s["codes"], s["scales"], "tiles", s["back"])
    return {"back": s["back"]}


def _own_linear(s):
    from moe_expert_ffn_03_gb300 import binding as B
    c = s["case"]
    d = B.grouped(c["rows"], c["K"], c["N"], c["E"])
    ws = _workspace(s, B.moe_grouped_linear_fp8_workspace_size(d))
    B.moe_grouped_linear_fp8_fwd(d, s["x"], s["x_scales"], s["split_sizes"], s["w"], s["w_scales"], s["y"], ws)
    out = {"y": s["y"]}
    if c["step"]:
        B.moe_grouped_linear_fp8_dgrad(d, s["dy"], s["dy_scales"], s["split_sizes"], s["w"], s["w_scales"], s["dx"], ws)
        B.moe_grouped_linear_fp8_wgrad(d, s["xt"], s["xt_scales"], s["dyt"], s["dyt_scales"], s["split_sizes"], s["dw"], ws)
        out["dx"], out["dw"] = s["dx"], s["dw"]
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rms": _own_rms, "balance": _own_balance, "quant": _own_quant, "weights": _own_weights,
                "linear8": _own_linear}[op](state)
    return {"rms": _plain_rms, "balance": _plain_balance, "quant": _plain_quant, "weights": _plain_weights,
            "linear8": _plain_linear}[op](state)


# ---- work ---------------------------------------------------------------------------------------
def _up(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    op = case["op"]
    if op == "rms":
        R, H, b = case["rows"], case["H"], 4 if case["f32"] else 2
        n = R * H
        total = n * b * (4 if case["residual"] else 2) + H * b + 4 * R
        flops = 5 * n
        if case["save8"]:                                               # codes and scales written, read, given back in bf16
            total += 2 * (n + 4 * R * _up(H)) + 2 * n
            flops += 3 * n
        if case["step"]:
            total += n * b * (4 if case["residual"] else 3) + 2 * H * b + 4 * R
            flops += 9 * n
        return {"bytes": total, "flops": flops}
    if op == "balance":
        T, E, k = case["rows"], case["E"], case["k"]
        return {"bytes": 4 * T * E * 3 + 4 * T * k + (2 * T if case["masked"] else 0) + 12 * E, "flops": 16 * T * E}
    if op == "quant":
        R, C, b = case["rows"], case["cols"], 4 if case["f32"] else 2
        n = R * C
        scales = 4 * R * _up(C) + 4 * _up(R) * (_up(C) if case["tiles"] else C)
        return {"bytes": n * b + 2 * (2 * n + scales) + 4 * n, "flops": 8 * n}
    if op == "weights":
        n = case["E"] * case["N"] * case["K"]
        scales = 4 * case["E"] * _up(case["N"]) * _up(case["K"])
        return {"bytes": n * (4 if case["f32"] else 2) + 2 * (n + scales) + 2 * n, "flops": 4 * n}
    R, K, N, E = case["rows"], case["K"], case["N"], case["E"]
    used = sum(n > 0 for n in _counts(case, torch.Generator().manual_seed(0)))   # experts that have rows
    weights = used * (N * K + 4 * _up(N) * _up(K))
    total, flops = R * K + 4 * R * _up(K) + weights + 2 * R * N, 2 * R * K * N
    if case["step"]:
        total += R * N + 4 * R * _up(N) + weights + 2 * R * K
        total += R * K + R * N + 4 * _up(R) * (N + _up(K)) + 2 * E * N * K
        flops *= 3
    return {"bytes": total, "flops": flops}


# ---- 64 bits ------------------------------------------------------------------------------------
def _e4m3_64(v):
    """v (float64, |v| <= 448) to the nearest E4M3 value, ties to even: three fraction bits, the exponent at least -6."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _kept_64(v, high, wide):
    """v (float64 [R][C]) through 8 bits, with blocks of `high` rows and `wide` columns from the first row on."""
    R, C = v.shape
    p = v.new_zeros(-(-R // high) * high, -(-C // wide) * wide)
    p[:R, :C] = v
    b = p.view(p.shape[0] // high, high, p.shape[1] // wide, wide)
    q = torch.clamp(torch.linalg.vector_norm(b, float("inf"), (1, 3), keepdim=True), min=TINY) / 448.0
    return (_e4m3_64(b / q) * q).view(p.shape)[:R, :C]


def _values_64(codes):
    """The values of E4M3 codes from their bits: sign, four exponent bits, three fraction bits."""
    c = codes.to(torch.int32)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, torch.ldexp(m, torch.full_like(e, -9)), torch.ldexp(8.0 + m, e - 10))
    return torch.where(c >= 128, -v, v)


def _stretched(scales, n, dim):
    """A scale for every one of n indices of a dimension cut into blocks of 128."""
    at = torch.arange(n, device=scales.device) // BLOCK
    return scales.double().index_select(dim, at)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = lambda k: s[k].double()  # noqa: E731
    if op == "rms":
        h = f("x") + f("residual") if case["residual"] else f("x")
        H = case["H"]
        r = (torch.einsum("rh,rh->r", h, h) / H + EPS).rsqrt()[:, None]
        n = h * r
        y = n * f("gamma")
        out = {"y": y}
        if case["residual"]:
            out["h"] = h
        if case["save8"]:
            out["y8"] = _kept_64(y, 1, BLOCK)
        if case["step"]:
            d = f("dy") * f("gamma")
            dx = r * (d - n * (torch.einsum("rh,rh->r", d, n) / H)[:, None])
            out["dx"] = dx + f("dres") if case["residual"] else dx
            out["dgamma"] = torch.einsum("rh,rh->h", f("dy"), n)
        return out
    if op == "balance":
        T, E, k = case["rows"], case["E"], case["k"]
        rows = torch.arange(T, device="cuda") if s["mask"] is None else s["mask"].nonzero().squeeze(1)
        n = max(1, rows.numel())
        x = f("logits")[rows].requires_grad_()
        counts = torch.bincount(s["idx"][rows].flatten().long(), minlength=E)
        P = torch.softmax(x, 1).sum(0) / n
        bal = E * (counts.double() * P).sum() / (k * n)
        z = torch.logsumexp(x, 1).square().sum() / n
        loss = s["alpha"] * bal + s["beta"] * z
        g, = torch.autograd.grad(loss, x)
        dl = torch.zeros(T, E, dtype=torch.float64, device=x.device).index_copy_(0, rows, g * f("grad"))
        return {"counts": torch.cat([counts, torch.tensor([rows.numel()], device=x.device)]), "prob": P.detach(),
                "loss": torch.stack([loss, bal, z]).detach(), "dlogits": dl}
    if op == "quant":
        v = f("src")
        out = torch.zeros(s["blocks"] * BLOCK, case["cols"], dtype=torch.float64, device=v.device)
        r0 = b0 = 0
        for n in s["counts"]:
            if n:
                out[b0: b0 + n] = _kept_64(v[r0: r0 + n], BLOCK, BLOCK if case["tiles"] else 1)
            r0, b0 = r0 + n, b0 + -(-n // BLOCK) * BLOCK
        return {"rows": _kept_64(v, 1, BLOCK), "tokens": out}
    if op == "weights":
        return {"back": torch.stack([_kept_64(w.double(), BLOCK, BLOCK) for w in s["w"]])}
    R, K, N, E = case["rows"], case["K"], case["N"], case["E"]
    ends = torch.cumsum(s["split_sizes"].long(), 0)
    owner = torch.searchsorted(ends, torch.arange(R, device=ends.device), right=True)        # the expert of each row
    x = _values_64(s["x"]) * _stretched(s["x_scales"], K, 0).t()
    out = {"y": torch.zeros(R, N, dtype=torch.float64, device=ends.device)}
    if case["step"]:
        dy = _values_64(s["dy"]) * _stretched(s["dy_scales"], N, 0).t()
        out["dx"] = torch.zeros(R, K, dtype=torch.float64, device=ends.device)
        out["dw"] = torch.zeros(E, N, K, dtype=torch.float64, device=ends.device)
        xt = _values_64(s["xt"]) * _stretched(_stretched(s["xt_scales"], K, 1), s["xt"].shape[0], 0)
        dyt = _values_64(s["dyt"]) * _stretched(s["dyt_scales"], s["dyt"].shape[0], 0)
        used = (torch.tensor(s["counts"]) + BLOCK - 1) // BLOCK
        first = torch.cumsum(used, 0) - used
    for e in owner.unique().tolist():
        at = (owner == e).nonzero().squeeze(1)
        w = _values_64(s["w"][e]) * _stretched(_stretched(s["w_scales"][e], N, 0), K, 1)
        out["y"].index_copy_(0, at, torch.einsum("rk,nk->rn", x.index_select(0, at), w))
        if case["step"]:
            out["dx"].index_copy_(0, at, torch.einsum("rn,nk->rk", dy.index_select(0, at), w))
            b = slice(int(first[e]) * BLOCK, int(first[e] + used[e]) * BLOCK)
            out["dw"][e] = torch.einsum("tn,tk->nk", dyt[b], xt[b])
    return out
