"""What is measured of the 8-bit layer around the dispatch: the norm in front of it, its rows in 8 bits, the
experts' product in 8-bit integers, and the router's balance loss.

Five operators, each in a plain form (elementary torch operations in 32 bits) and through the framework's calls:

* ``product``: the experts' product of INT8 rows with a scale each (as the quantised dispatch leaves them) and
  INT8 weights with a scale for each output channel, the groups' rows one after the other, plain or with the
  gated activation silu(gate) * up;
* ``rows8``: rows to 8 bits with one scale a row (INT8 or E4M3) and back to the values those stand for;
* ``norm8``: the residual's addition and the root-mean-square norm with its output in 8 bits, and the values
  those stand for;
* ``norm_step``: a training pass of the same norm with a bf16 output: forward, and the gradients of the rows
  and of the weight;
* ``balance``: a training pass of the router's balance loss: the loss, the experts' counts and the gradient of
  the router's logits.

Rows in 8 bits: scale = amax / top (127 for INT8, 448 for E4M3), codes are the values over the scale, rounded to
the nearest, ties to the even code. A row of zeros has scale 0.
"""

import math

import torch

own = False

DEV = "cuda"
E4M3, INT8 = 1, 2  # the framework's moe_quant values
TOP = {E4M3: 448.0, INT8: 127.0}
EPS = 1e-6
COEF = 0.01


def listed():
    return [
        # serving, one token: 8 rows over one rank's 32 experts, gate and up; the weights' bytes bound it
        {"name": "product, one token", "op": "product", "G": 32, "N": 8, "H": 7168, "O": 4096, "gated": True},
        # serving, a decode batch: 128 tokens of each of 8 ranks, the down projection
        {"name": "product, decode batch", "op": "product", "G": 32, "N": 1024, "H": 2048, "O": 7168, "gated": False},
        # odd sizes: rows, hidden size and outputs that fill no tile
        {"name": "product, ragged", "op": "product", "G": 16, "N": 3001, "H": 1040, "O": 1000, "gated": False},
        # prefill: 4096 tokens of each of 8 ranks, 8 experts each, on one rank's 32 experts; gate and up
        {"name": "product, prefill", "op": "product", "G": 32, "N": 32768, "H": 7168, "O": 4096, "gated": True},
        # a padded window of odd sizes whose last rows are unused, and a whole one between the two products
        {"name": "rows in 8 bits, ragged", "op": "rows8", "N": 1500, "used": 1367, "H": 2064, "quant": E4M3},
        {"name": "rows in 8 bits, window", "op": "rows8", "N": 32768, "used": 32768, "H": 7168, "quant": INT8},
        # a decode batch of 128 tokens, then one prefill step's 4096 tokens, on their way into a shared expert
        {"name": "norm to 8 bits, decode", "op": "norm8", "S": 128, "H": 7168, "quant": INT8, "residual": True, "weight": "bf16"},
        {"name": "norm to 8 bits, 4096 tokens", "op": "norm8", "S": 4096, "H": 7168, "quant": INT8, "residual": True, "weight": "fp32"},
        # a training step: a padded odd batch, then the bench workload's tokens
        {"name": "norm training, ragged", "op": "norm_step", "S": 1531, "H": 2064, "residual": True, "weight": "fp32"},
        {"name": "norm training, 4096 tokens", "op": "norm_step", "S": 4096, "H": 7168, "residual": True, "weight": "bf16"},
        # the router of a micro-batch, and of a large batch with popular experts and a padded end
        {"name": "balance, micro-batch", "op": "balance", "S": 128, "E": 16, "K": 2, "mask": 0.0, "zipf": 0.0, "score": "softmax", "logits": "bf16", "limited": False},
        {"name": "balance, skewed", "op": "balance", "S": 8192, "E": 256, "K": 8, "mask": 0.05, "zipf": 1.2, "score": "sigmoid", "logits": "fp32", "limited": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("product", "product", "rows8", "norm8", "norm_step", "balance"))
    if op == "product":
        groups, hidden, gated = rng.randint(1, 64), 16 * rng.randint(4, 448), rng.random() < 0.5
        outs = min(_log(rng, 64, 7168), 32 * 4096 * 7168 // (groups * hidden))
        outs += outs % 2 if gated else 0
        return {"op": op, "G": groups, "N": min(_log(rng, 1, 32768), 32768 * 4096 * 7168 // (outs * hidden)), "H": hidden, "O": outs, "gated": gated}
    if op == "rows8":
        rows = _log(rng, 1, 32768)
        return {"op": op, "N": rows, "used": rng.choice((rows, rng.randint(1, rows))), "H": 16 * rng.randint(4, 448), "quant": rng.choice((E4M3, INT8))}
    if op == "balance":
        top = rng.randint(1, 8)
        return {"op": op, "S": _log(rng, 1, 8192), "E": rng.randint(2 * top, 256), "K": top, "mask": rng.choice((0.0, 0.05, 0.4)), "zipf": rng.choice((0.0, 1.2)),
                "score": rng.choice(("softmax", "sigmoid")), "logits": rng.choice(("bf16", "fp32")), "limited": rng.random() < 0.5}
    case = {"op": op, "S": _log(rng, 1, 4096), "H": 16 * rng.randint(4, 448), "residual": rng.random() < 0.8, "weight": rng.choice(("bf16", "fp32"))}
    return {**case, "quant": rng.choice((E4M3, INT8))} if op == "norm8" else case


# ---------------------------------------------------------------- inputs


def _rows(g, n, H):
    """bf16 rows: normal values, each row with a scale of its own, as activations behind a product have."""
    spread = torch.exp2(torch.randn((n, 1), generator=g, device=DEV))
    return (torch.randn((n, H), generator=g, device=DEV) * spread).to(torch.bfloat16)


def _held(x, quant):
    """What fp32 rows hold in 8 bits: their codes as numbers, and the scales [rows, 1]."""
    scale = x.abs().amax(dim=-1, keepdim=True) / TOP[quant]
    q = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0)
    if quant == INT8:
        return torch.round(q).clamp(-127, 127), scale
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).float(), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s, op = {"case": dict(case)}, case["op"]
    if op == "product":
        G, N, H, O = case["G"], case["N"], case["H"], case["O"]
        # every group as popular as the others up to a factor, so small batches leave groups empty
        pop = torch.softmax(0.3 * torch.randn(G, generator=g, device=DEV), dim=0)
        count = torch.bincount(torch.multinomial(pop, N, replacement=True, generator=g), minlength=G)
        s["base"] = torch.cat((count.new_zeros(1), torch.cumsum(count, 0))).to(torch.int32)
        s["most"] = int(count.max())
        codes, scales = _held(_rows(g, N, H).float(), INT8)
        s["a"], s["a_scales"] = codes.to(torch.int8), scales.view(N)
        s["w"] = torch.empty((G, O, H), dtype=torch.int8, device=DEV)
        s["w_scales"] = torch.empty((G, O), device=DEV)
        for e in range(G):
            codes, scales = _held(torch.randn((O, H), generator=g, device=DEV).mul_(1 / math.sqrt(H)), INT8)
            s["w"][e], s["w_scales"][e] = codes.to(torch.int8), scales.view(O)
        return s
    if op == "rows8":
        s["x"] = _rows(g, case["N"], case["H"])
        s["count"] = torch.tensor([case["used"]], dtype=torch.int32, device=DEV)
        s["out"] = torch.zeros((case["N"], case["H"]), dtype=torch.bfloat16, device=DEV)  # rows behind the used ones stay zero
        return s
    if op == "balance":
        S, E, K = case["S"], case["E"], case["K"]
        kind = torch.bfloat16 if case["logits"] == "bf16" else torch.float32
        pop = -case["zipf"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
        logits = torch.randn((S, E), generator=g, device=DEV) + pop
        if case["limited"]:  # each token may go to one half of the experts only
            half = torch.rand((S, 1), generator=g, device=DEV) < 0.5
            logits = torch.where((torch.arange(E, device=DEV) % 2 == 0) == half, logits, -math.inf)
        s["logits"] = logits.to(kind)
        entry = torch.topk(s["logits"].float(), K, dim=1).indices.to(torch.int32)
        dropped = torch.rand((S, K), generator=g, device=DEV) < case["mask"]  # over an expert's capacity
        padded = torch.arange(S, device=DEV).unsqueeze(1) >= S - int(S * case["mask"])  # the batch's padding
        s["topk_idx"] = torch.where(dropped | padded, -1, entry).contiguous()
        s["d_loss"] = torch.ones(1, device=DEV)
        return s
    S, H = case["S"], case["H"]
    s["x"] = _rows(g, S, H)
    s["residual"] = _rows(g, S, H).mul_(2) if case["residual"] else None
    s["weight"] = (1 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16 if case["weight"] == "bf16" else torch.float32)
    if op == "norm_step":
        s["dy"] = _rows(g, S, H)
        s["d_sum"] = _rows(g, S, H) if case["residual"] else None
    return s


# ---------------------------------------------------------------- plain forms


def _product(s):
    case, base = s["case"], s["base"].long()
    G, N, H, O = case["G"], case["N"], case["H"], case["O"]
    row = torch.arange(N, device=DEV)
    group = torch.searchsorted(base, row, right=True) - 1
    a = torch.zeros((G, s["most"], H), device=DEV)
    a[group, row - base[group]] = s["a"].float()
    c = torch.bmm(s["w"].float(), a.transpose(1, 2).contiguous())  # [G, O, most]
    c = c.transpose(1, 2)[group, row - base[group]] * s["a_scales"].unsqueeze(1) * s["w_scales"][group]
    if case["gated"]:
        gate, up = c[:, : O // 2], c[:, O // 2 :]
        c = gate / (1 + torch.exp(-gate)) * up
    return c.to(torch.bfloat16)


def _normed(s):
    """The rows that are normed, in bf16, the normed rows in 32 bits without the weight, and 1 / rms [S, 1]."""
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    # mean and root in 64 bits: codes lie next to borders
    r = torch.rsqrt(h.double().square().mean(dim=-1, keepdim=True) + EPS).float()
    return h, h.float() * r, r


def _norm_step(s):
    h, n, r = _normed(s)
    dy, w = s["dy"].float(), s["weight"].float()
    back = w * dy
    dx = r * (back - n * (n * back).mean(dim=-1, keepdim=True))
    if s["d_sum"] is not None:
        dx = dx + s["d_sum"].float()
    d_weight = (dy * n).sum(dim=0)
    return (n * w).to(torch.bfloat16), h, dx.to(torch.bfloat16), d_weight


def _balance(s):
    case, entry = s["case"], s["topk_idx"].long()
    E = case["E"]
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV).scatter_add_(0, torch.where(entry >= 0, entry, E).flatten(), torch.ones_like(entry).flatten())[:E]
    lives = (entry >= 0).any(dim=1, keepdim=True)
    tokens = lives.sum()
    logits = torch.where(lives, s["logits"].float(), 0.0)
    if case["score"] == "sigmoid":
        e = 1 / (1 + torch.exp(-logits))
        turn = 1 - e
    else:
        e, turn = torch.exp(logits - logits.amax(dim=1, keepdim=True)), 1.0
    p = torch.where(lives, e / e.sum(dim=1, keepdim=True), 0.0)
    each = COEF * E / (counts.sum().double() * tokens.double()).clamp(min=1)  # an entry's weight
    loss = (each * (counts.double() * p.sum(dim=0).double()).sum()).float().view(1)
    # the gradient sees the counts' differences alone: taken from the mean, so that equal ones cancel exactly
    apart = (counts - torch.div(counts.sum(), E, rounding_mode="floor")).float()
    d_logits = s["d_loss"] * each.float() * p * (apart - (apart * p).sum(dim=1, keepdim=True)) * turn
    return loss, counts.to(torch.int32), tokens.to(torch.int32).view(1), d_logits.to(s["logits"].dtype)


def _plain(s):
    case = s["case"]
    if case["op"] == "product":
        return _product(s)
    if case["op"] == "norm_step":
        return _norm_step(s)
    if case["op"] == "balance":
        return _balance(s)
    if case["op"] == "norm8":
        h, n, _ = _normed(s)
        codes, scale = _held(n * s["weight"].float(), case["quant"])
        return h, (codes * scale).to(torch.bfloat16)
    used = case["used"]
    codes, scale = _held(s["x"][:used].float(), case["quant"])
    s["out"][:used] = (codes * scale).to(torch.bfloat16)
    return s["out"]


# ---------------------------------------------------------------- the framework's calls


def _framework(s):
    import combine_moe_layout_02_amd as moe

    case = s["case"]
    if case["op"] == "product":
        return moe.moe_scaled_product(moe.ScaledRows(s["a"], s["a_scales"]), moe.ScaledRows(s["w"], s["w_scales"]), s["base"],
                                      moe.MOE_MX_GATED if case["gated"] else moe.MOE_MX_PLAIN)
    if case["op"] == "rows8":
        rows8 = moe.moe_row_quantize(s["x"], case["quant"], num_rows=s["count"])
        return moe.moe_row_dequantize(rows8, case["quant"], num_rows=s["count"], out=s["out"])
    if case["op"] == "balance":
        score = moe.MOE_SCORE_SIGMOID if case["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX
        b = moe.moe_balance_loss(s["logits"], s["topk_idx"], COEF, score)
        d_logits = moe.moe_balance_loss_backward(s["d_loss"], s["logits"], s["topk_idx"], b.num_tokens_per_expert, b.num_tokens, COEF, score)
        return b.loss, b.num_tokens_per_expert, b.num_tokens, d_logits
    if case["op"] == "norm8":
        n = moe.moe_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], quant=case["quant"])
        return n.sum, moe.moe_row_dequantize(n.rows8, case["quant"])
    n = moe.moe_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
    dx, d_weight = moe.moe_rms_norm_backward(s["dy"], n.sum, s["weight"], EPS, d_sum=s["d_sum"])
    return n.out, n.sum, dx, d_weight


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "product":
        G, N, H, O = case["G"], case["N"], case["H"], case["O"]
        hit = G * (1 - (1 - 1 / G) ** N)  # groups with a row, whose weights have to be read
        return {"bytes": (hit * O + N) * (H + 4) + 2 * N * (O // 2 if case["gated"] else O) + 4 * (G + 1), "flops": 2 * N * O * H}
    if op == "rows8":
        # read the rows, write codes and scales; read those, write the values
        n = case["used"] * case["H"]
        return {"bytes": 6 * n + 8 * case["used"], "flops": 4 * n}
    if op == "balance":
        S, E, K = case["S"], case["E"], case["K"]
        size = 2 if case["logits"] == "bf16" else 4
        # the logits and the entries for the loss and again for the gradient, which is written
        return {"bytes": 3 * size * S * E + 8 * S * K + 8 * E + 16, "flops": 12 * S * E}
    n = case["S"] * case["H"]
    weight = case["H"] * (2 if case["weight"] == "bf16" else 4)
    added = 4 if case["residual"] else 0  # the residual read and the sum written
    if op == "norm8":
        # read the rows, write codes and scales; read those, write the values
        return {"bytes": n * (2 + added + 4) + 8 * case["S"] + weight, "flops": 8 * n}
    # forward: read the rows, write the normed ones; back: read dy, the sum (and its own gradient), write dx
    return {"bytes": n * (4 + added + 6 + (2 if case["residual"] else 0)) + 2 * weight + 4 * case["H"], "flops": 17 * n}


# ---------------------------------------------------------------- the definitions in 64 bits


def _held64(y, quant):
    """Rows in 64 bits after 8 bits with a scale a row: multiples of the scale (INT8), or of the scale's
    multiples that three bits behind the leading one reach, no finer than 2^-9 of it (E4M3)."""
    top = TOP[quant]
    scale = y.abs().max(dim=1, keepdim=True).values / top
    q = y / torch.where(scale > 0, scale, torch.ones_like(scale))
    if quant == INT8:
        return torch.round(q) * scale
    power = torch.floor(torch.log2(torch.where(q == 0, torch.ones_like(q), q.abs()))).clamp(min=-6)
    step = torch.exp2(power - 3)
    return (torch.round(q / step) * step).clamp(-top, top) * scale


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "product":
        base, O = s["base"].tolist(), case["O"]
        out = torch.zeros((case["N"], O), dtype=torch.float64, device=DEV)
        for e in range(case["G"]):
            rows = slice(base[e], base[e + 1])
            if base[e + 1] > base[e]:
                w = s["w"][e].double() * s["w_scales"][e].double()[:, None]
                out[rows] = (s["a"][rows].double() * s["a_scales"][rows].double()[:, None]) @ w.t().contiguous()
        gate, up = out[:, : O // 2], out[:, O // 2 :]
        return torch.sigmoid(gate) * gate * up if case["gated"] else out
    if op == "rows8":
        out = s["out"].double()
        out[: case["used"]] = _held64(s["x"][: case["used"]].double(), case["quant"])
        return out
    if op == "balance":
        E, entry = case["E"], s["topk_idx"]
        counts = torch.stack([(entry == e).sum() for e in range(E)]).double()
        lives = (entry >= 0).sum(dim=1) > 0
        tokens = float(lives.sum())
        d_logits = torch.zeros((case["S"], E), dtype=torch.float64, device=DEV)
        if not tokens:
            return torch.zeros(1, dtype=torch.float64, device=DEV), None, None, d_logits
        l = s["logits"][lives].double()
        p = torch.softmax(torch.nn.functional.logsigmoid(l) if case["score"] == "sigmoid" else l, dim=1)
        weight = COEF * E * counts / (float(counts.sum()) * tokens)
        inner = p * (weight - (p @ weight)[:, None])
        d_logits[lives] = inner * torch.sigmoid(-l) if case["score"] == "sigmoid" else inner
        return (p @ weight).sum().reshape(1), None, None, d_logits
    total = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
    h, w = total.to(torch.bfloat16).double(), s["weight"].double()  # the sum is held in bf16, and that is normed
    root = torch.sqrt((h * h).sum(dim=1, keepdim=True) / case["H"] + EPS)
    if op == "norm8":
        return total, _held64(h / root * w, case["quant"])
    dy = s["dy"].double()
    # y_i = w_i h_i / root and d root / d h_j = h_j / (H root)
    dx = w * dy / root - h * ((dy * w * h).sum(dim=1, keepdim=True) / (case["H"] * root**3))
    if s["d_sum"] is not None:
        dx = dx + s["d_sum"].double()
    return h / root * w, total, dx, (dy * h / root).sum(dim=0)
