"""The operators between the products of an expert layer, and the loss, measured.

  route     scores of a router's logits, the choice of each token's experts (bias,
            groups, top-k) and their weights; the gradient of the logits;
  dispatch  the rows of the experts' operands from the tokens': where each row
            goes, and the rows (bf16, or 8 bits with their scales), in the
            layouts of the grouped products;
  combine   the weighted sum of the experts' output rows back into the residual
            stream (without weights: the gradient of dispatch), and its gradient;
  loss      softmax cross entropy of x W^T over a large vocabulary, without the
            logits in memory; the gradients of x and W.

`own` False: the operators in elementary torch operations in 32 bits (the
choice of experts in 64, where values lie next to each other), rounded once at
the end.  `own` True: the package's calls.
"""
import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16
GROUP = 128
ALIGN = 128        # rows of an expert's segment in the contiguous layout
LEAST = 1e-20      # added to the sum that renormalised weights are divided by


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one decoding step of a handful of sequences: sigmoid scores with a bias for
        # balance, 4 of 8 groups of experts, 8 of 256 experts
        {"name": "route decode 7x256", "op": "route", "dir": "fwd", "T": 7, "G": 256, "k": 8,
         "sigmoid": True, "bias": True, "groups": 8, "top_groups": 4, "best": 2, "renorm": True,
         "scale": 2.5, "bf16": False},
        # a training step: softmax scores of a bf16 product's output, no groups
        {"name": "route train 16384x128", "op": "route", "dir": "fwd", "T": 16384, "G": 128, "k": 6,
         "sigmoid": False, "bias": False, "groups": 1, "top_groups": 1, "best": 1, "renorm": True,
         "scale": 1.0, "bf16": True},
        # gradient of the logits of a training step
        {"name": "route grad 8192x256", "op": "route", "dir": "bwd", "T": 8192, "G": 256, "k": 8,
         "sigmoid": True, "bias": True, "groups": 8, "top_groups": 4, "best": 2, "renorm": True,
         "scale": 2.5, "bf16": False},
        # decoding: the quantised rows into the masked layout of 8 experts
        {"name": "dispatch decode masked", "op": "dispatch", "T": 61, "K": 7168, "G": 8, "k": 2,
         "layout": "masked", "rows": 128, "form": "fp8"},
        # prefill: the quantised rows into the contiguous layout (segments of whole blocks)
        {"name": "dispatch prefill contiguous", "op": "dispatch", "T": 4096, "K": 7168, "G": 32,
         "k": 4, "layout": "contiguous", "rows": 20480, "form": "fp8"},
        # training in bf16: ragged rows, an odd number of tokens
        {"name": "dispatch train ragged", "op": "dispatch", "T": 8191, "K": 4096, "G": 64, "k": 4,
         "layout": "ragged", "rows": 32764, "form": "bf16"},
        # decoding: the experts' rows back into the residual stream
        {"name": "combine decode 61x7168", "op": "combine", "dir": "fwd", "T": 61, "K": 7168, "G": 8,
         "k": 2, "weights": True, "residual": True},
        # training: eight rows a token
        {"name": "combine train 4096x7168", "op": "combine", "dir": "fwd", "T": 4096, "K": 7168,
         "G": 32, "k": 8, "weights": True, "residual": True},
        # gradient of the same: of the rows and of their weights
        {"name": "combine grad 4096x7168", "op": "combine", "dir": "bwd", "T": 4096, "K": 7168,
         "G": 32, "k": 8, "weights": True, "residual": False},
        # the loss of a few tokens (scoring one sequence's continuation)
        {"name": "loss 61x32000", "op": "loss", "dir": "fwd", "T": 61, "V": 32000, "K": 2048,
         "ignored": 0.0},
        # the loss of a training step, a large vocabulary
        {"name": "loss 4096x131072", "op": "loss", "dir": "fwd", "T": 4096, "V": 131072, "K": 2048,
         "ignored": 0.1},
        # its gradients, a vocabulary of an odd size and some padding tokens
        {"name": "loss grad 4095x50003", "op": "loss", "dir": "bwd", "T": 4095, "V": 50003, "K": 4096,
         "ignored": 0.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, unit):
    return max(lo, min(hi, (_log(rng, lo, hi) + unit - 1) // unit * unit))


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "loss"])
    if op == "route":
        G = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512])
        groups = rng.choice([1, 1, 2, 4, 8])
        groups = groups if G % groups == 0 and G // groups >= 4 else 1
        top_groups = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(16, G // groups * top_groups))
        while True:
            T = _log(rng, 1, 32768)
            if T * G <= 16384 * 128:
                break
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "T": T, "G": G, "k": k,
                "sigmoid": rng.random() < 0.5, "bias": rng.random() < 0.5, "groups": groups,
                "top_groups": top_groups, "best": rng.choice([1, 2]),
                # (the weight of a single choice, renormalised, is the scale)
                "renorm": k > 1 and rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5, 16.0]), "bf16": rng.random() < 0.5}
    if op == "dispatch":
        layout = rng.choice(["ragged", "masked", "contiguous"])
        while True:
            G, K = _log(rng, 4, 256), _mult(rng, 512, 8192, GROUP)
            k = rng.randint(1, min(8, G))
            if layout == "masked":
                T = _log(rng, 1, 256)
                rows = (T + 127) // 128 * 128
                total = G * rows
            else:
                T = _log(rng, 1, 16384)
                rows = T * k if layout == "ragged" else (T * k // ALIGN + G) * ALIGN
                total = rows
            if total * K <= 32764 * 4096:
                break
        form = "bf16" if layout == "ragged" else rng.choice(["bf16", "fp8", "ue8m0"])
        return {"op": op, "T": T, "K": K, "G": G, "k": k, "layout": layout, "rows": rows, "form": form}
    if op == "combine":
        while True:
            G, K = _log(rng, 4, 256), _mult(rng, 256, 8192, 8)
            k = rng.randint(1, min(8, G))
            T = _log(rng, 1, 16384)
            if T * k * K <= 4096 * 8 * 7168:
                break
        if rng.random() < 0.4:
            return {"op": op, "dir": "bwd", "T": T, "K": K, "G": G, "k": k, "weights": True,
                    "residual": False}
        return {"op": op, "dir": "fwd", "T": T, "K": K, "G": G, "k": k,
                "weights": rng.random() < 0.7, "residual": rng.random() < 0.7}
    way = rng.choice(["fwd", "bwd"])
    while True:
        T, V, K = _log(rng, 1, 4096), _log(rng, 1000, 131072), _mult(rng, 256, 7168, 8)
        if T * V * K * (3 if way == "bwd" else 1) <= 4096 * 131072 * 2048:
            break
    return {"op": op, "dir": way, "T": T, "V": V, "K": K, "ignored": rng.choice([0.0, 0.1])}


# ----------------------------------------------------------------- inputs ----
def _choices(gen, T, G, k):
    """Experts of each token as a router chooses them: different ones, some experts
    more popular than others."""
    popular = torch.randn(G, device=DEV, generator=gen) * 0.5
    noise = -torch.log(-torch.log(torch.rand(T, G, device=DEV, generator=gen).clamp(1e-7, 1 - 1e-7)))
    return (popular + noise).topk(k, dim=1).indices.to(torch.int32)


def _places(experts, G):
    """(rows of each expert, index of each choice among its expert's), in order."""
    flat = experts.flatten().long()
    order = flat.argsort(stable=True)
    sizes = torch.zeros(G, dtype=torch.long, device=DEV).index_add_(0, flat, torch.ones_like(flat))
    first = sizes.cumsum(0) - sizes
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device=DEV) - first[flat[order]]
    return sizes, place.view(experts.shape)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFF)

    def normal(*shape, scale=1.0, dtype=BF16):
        x = torch.empty(shape, dtype=dtype, device=DEV)
        x.normal_(0.0, scale, generator=gen)
        return x

    def zeros(*shape, dtype=BF16):
        return torch.zeros(shape, dtype=dtype, device=DEV)

    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    s = {"case": case}
    T = case["T"]
    if case["op"] == "route":
        G, k = case["G"], case["k"]
        s["logits"] = normal(T, G, scale=1.5, dtype=f32).to(BF16 if case["bf16"] else f32)
        s["bias"] = normal(G, scale=0.05, dtype=f32) if case["bias"] else None
        if case["dir"] == "fwd":
            s["experts"], s["weights"] = zeros(T, k, dtype=i32), zeros(T, k, dtype=f32)
        else:
            s["experts"] = _choose(s["logits"].double(), s["bias"], case).to(i32)
            s["d_weights"] = normal(T, k, scale=0.1, dtype=f32)
            s["d_logits"] = torch.zeros_like(s["logits"])
        return s
    if case["op"] == "dispatch":
        K, G, k, rows = case["K"], case["G"], case["k"], case["rows"]
        s["experts"] = _choices(gen, T, G, k)
        s["row_of"], s["sizes"] = zeros(T, k, dtype=i32), zeros(G, dtype=i32)
        lead = (G, rows) if case["layout"] == "masked" else (rows,)
        s["m_indices"] = zeros(rows, dtype=i32) if case["layout"] == "contiguous" else None
        if case["form"] == "bf16":
            s["X"], s["A"] = normal(T, K), zeros(*lead, K)
            return s
        # rows as the quantiser leaves them: codes of any finite value, positive scales
        ld, ld_out = (T + 3) // 4 * 4, (rows + 3) // 4 * 4
        s["X"] = normal(T, K, scale=100.0, dtype=f32).clamp(-448, 448).to(torch.float8_e4m3fn).view(u8)
        s["A"] = zeros(*lead, K, dtype=u8)
        s["ld"], s["ld_out"] = ld, ld_out
        if case["form"] == "ue8m0":
            e = torch.randint(118, 124, ((K + 511) // 512, ld, 4), device=DEV, generator=gen, dtype=i32)
            s["sa"] = e.to(u8).view(i32).squeeze(-1).contiguous()
            s["sa_out"] = zeros(*lead[:-1], (K + 511) // 512, ld_out, dtype=i32)
        else:
            s["sa"] = (0.01 * (1.0 + normal(K // GROUP, ld, dtype=f32).abs())).contiguous()
            s["sa_out"] = zeros(*lead[:-1], K // GROUP, ld_out, dtype=f32)
        return s
    if case["op"] == "combine":
        K, G, k = case["K"], case["G"], case["k"]
        sizes, place = _places(e := _choices(gen, T, G, k), G)
        s["row_of"] = ((sizes.cumsum(0) - sizes)[e.long()] + place).to(i32)
        w = torch.rand(T, k, device=DEV, generator=gen) + 0.05
        s["weights"] = (w / w.sum(1, keepdim=True)).contiguous() if case["weights"] else None
        s["Y"] = normal(T * k, K)
        if case["dir"] == "fwd":
            s["R"] = normal(T, K, scale=2.0) if case["residual"] else None
            s["out"] = zeros(T, K)
        else:
            s["dO"] = normal(T, K, scale=0.02)
            s["dY"], s["dw"] = zeros(T * k, K), zeros(T, k, dtype=f32)
        return s
    V, K = case["V"], case["K"]
    s["X"] = normal(T, K)
    s["W"] = normal(V, K, scale=2.0 * K ** -0.5)
    # frequent words are far likelier than rare ones; a token without a target is padding
    t = (V * torch.rand(T, device=DEV, generator=gen) ** 3).long().clamp_max(V - 1)
    skip = torch.rand(T, device=DEV, generator=gen) < case["ignored"]
    s["targets"] = torch.where(skip, -1, t).to(i32)
    if case["dir"] == "fwd":
        s["loss"], s["lse"] = zeros(T, dtype=f32), zeros(T, dtype=f32)
    else:
        s["lse"] = torch.logsumexp((s["X"].float() @ s["W"].float().t()), dim=1)
        s["d_loss"] = torch.full((T,), 1.0 / T, device=DEV)
        s["dX"], s["dW"] = zeros(T, K), zeros(V, K)
    if own:
        import moe_grouped_gemm_bf16_gb300 as dg
        n = (dg.linear_cross_entropy_backward_workspace_bytes if case["dir"] == "bwd"
             else dg.linear_cross_entropy_workspace_bytes)(T, V, K)
        s["work"] = torch.empty(max(n, 16), dtype=u8, device=DEV)
    return s


# ------------------------------------------------------------ plain forms ----
def _choose(x, bias, case):
    """Chosen experts [T, k] from the logits in 64 bits."""
    c = 1.0 / (1.0 + torch.exp(-x)) if case["sigmoid"] else _softmax(x)
    if bias is not None:
        c = c + bias.double()
    if case["groups"] > 1:
        g = c.unflatten(1, (case["groups"], -1))
        best = g.sort(dim=2, descending=True).values[..., :case["best"]].sum(2)
        keep = best.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        on = torch.zeros_like(best, dtype=torch.bool).scatter_(1, keep, True)
        c = torch.where(on[..., None], g, -math.inf).flatten(1)
    return c.sort(dim=1, descending=True, stable=True).indices[:, :case["k"]]


def _softmax(x):
    e = torch.exp(x - x.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _route_plain(s):
    c = s["case"]
    x = s["logits"].float()
    p = 1.0 / (1.0 + torch.exp(-x)) if c["sigmoid"] else _softmax(x)
    if c["dir"] == "fwd":
        e = _choose(s["logits"].double(), s["bias"], c)
        w = p.gather(1, e)
        if c["renorm"]:
            w = w / (w.sum(1, keepdim=True) + LEAST)
        return {"experts": e.to(torch.int32), "weights": w * c["scale"]}
    e, dw = s["experts"].long(), s["d_weights"] * c["scale"]
    if c["renorm"]:
        w = p.gather(1, e)
        total = w.sum(1, keepdim=True) + LEAST
        dw = (dw - (dw * w / total).sum(1, keepdim=True)) / total
    dp = torch.zeros_like(p).scatter_(1, e, dw)
    if c["sigmoid"]:
        d = dp * p * (1.0 - p)
    else:
        d = p * (dp - (dp * p).sum(1, keepdim=True))
    return {"d_logits": d.to(s["logits"].dtype)}


def _dispatch_plain(s):
    c = s["case"]
    G, k, rows = c["G"], c["k"], c["rows"]
    e = s["experts"].long()
    sizes, place = _places(s["experts"], G)
    out = {"sizes": sizes.to(torch.int32)}
    if c["layout"] == "masked":
        row = e * rows + place
    else:
        room = (sizes + ALIGN - 1) // ALIGN * ALIGN if c["layout"] == "contiguous" else sizes
        end = room.cumsum(0)
        row = (end - room)[e] + place
        if c["layout"] == "contiguous":
            m = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
            m[row.flatten()] = s["experts"].flatten()
            out["m_indices"] = m
    out["row_of"] = row.to(torch.int32)
    flat = row.flatten()
    token = torch.arange(c["T"], device=DEV).repeat_interleave(k, output_size=c["T"] * k)
    a = torch.zeros_like(s["A"]).view(-1, c["K"])
    a[flat] = s["X"][token]
    a = a.view(s["A"].shape)
    out["A"] = a
    if c["form"] != "bf16":
        out["A"] = a.view(torch.float8_e4m3fn)
        sa = torch.zeros_like(s["sa_out"]).view(-1, s["sa"].shape[0], s["ld_out"])
        g = flat // rows if c["layout"] == "masked" else torch.zeros_like(flat)
        sa[g, :, flat - g * rows] = s["sa"][:, token].t()
        out["sa"] = _scales(sa.view(s["sa_out"].shape), c["form"])
    return out


def _scales(sa, form):
    """The scales as the values that they stand for."""
    return sa.view(torch.float8_e8m0fnu).unflatten(-1, (-1, 4)) if form == "ue8m0" else sa


def _combine_plain(s):
    c = s["case"]
    y = s["Y"][s["row_of"].long()].float()     # [T, k, K]
    if c["dir"] == "fwd":
        out = (y * s["weights"][..., None] if c["weights"] else y).sum(1)
        if c["residual"]:
            out = out + s["R"].float()
        return {"out": out.to(BF16)}
    d = s["dO"].float()[:, None]
    dy = torch.zeros_like(s["Y"])
    dy[s["row_of"].flatten().long()] = (d * s["weights"][..., None]).to(BF16).flatten(0, 1)
    return {"dY": dy, "dw": (y * d).sum(2)}


def _loss_plain(s):
    c = s["case"]
    x, w, t = s["X"].float(), s["W"].float(), s["targets"].long()
    there, at = t >= 0, t.clamp_min(0)[:, None]
    z = x @ w.t()
    if c["dir"] == "fwd":
        top = z.amax(dim=1)
        lse = torch.log(torch.exp(z - top[:, None]).sum(1)) + top
        return {"loss": torch.where(there, lse - z.gather(1, at)[:, 0], 0.0), "lse": lse}
    g = torch.exp(z - s["lse"][:, None])
    g.scatter_add_(1, at, torch.full_like(at, -1, dtype=g.dtype))
    g = g * torch.where(there, s["d_loss"], 0.0)[:, None]
    return {"dX": (g @ w).to(BF16), "dW": (g.t() @ x).to(BF16)}


# -------------------------------------------------------------------- run ----
def _own(s):
    import moe_grouped_gemm_bf16_gb300 as dg

    c = s["case"]
    T = c["T"]
    if c["op"] == "route":
        how = (T, c["G"], c["k"], c["sigmoid"])
        if c["dir"] == "fwd":
            (dg.route_top_k_bf16 if c["bf16"] else dg.route_top_k_fp32)(
                s["logits"], s["bias"], s["experts"], s["weights"], *how, c["groups"],
                c["top_groups"], c["best"], c["renorm"], c["scale"])
            return {"experts": s["experts"], "weights": s["weights"]}
        (dg.route_top_k_backward_bf16 if c["bf16"] else dg.route_top_k_backward_fp32)(
            s["logits"], s["experts"], s["d_weights"], s["d_logits"], *how, c["renorm"], c["scale"])
        return {"d_logits": s["d_logits"]}
    if c["op"] == "dispatch":
        K, G, k, rows = c["K"], c["G"], c["k"], c["rows"]
        out = {"sizes": s["sizes"], "row_of": s["row_of"]}
        total, groups = rows, 1
        if c["layout"] == "masked":
            dg.expert_rows_masked(s["experts"], s["sizes"], s["row_of"], T, k, G, rows)
            total, groups = G * rows, G
        elif c["layout"] == "contiguous":
            dg.expert_rows_contiguous(s["experts"], s["sizes"], s["row_of"], s["m_indices"], T, k, G,
                                      rows)
            out["m_indices"] = s["m_indices"]
        else:
            dg.expert_rows_ragged(s["experts"], s["sizes"], s["row_of"], T, k, G)
        if c["form"] == "bf16":
            dg.dispatch_rows_bf16(s["X"], s["row_of"], s["A"], T, K, k, total)
            out["A"] = s["A"]
        else:
            call = dg.dispatch_rows_fp8_1x128_ue8m0 if c["form"] == "ue8m0" else dg.dispatch_rows_fp8_1x128
            call(s["X"], s["sa"], s["ld"], s["row_of"], s["A"], s["sa_out"], s["ld_out"], T, K, k,
                 groups, rows)
            out["A"], out["sa"] = s["A"].view(torch.float8_e4m3fn), _scales(s["sa_out"], c["form"])
        return out
    if c["op"] == "combine":
        K, k = c["K"], c["k"]
        if c["dir"] == "fwd":
            dg.combine_rows(s["Y"], s["row_of"], s["weights"], s["R"], s["out"], T, K, k, T * k)
            return {"out": s["out"]}
        dg.combine_rows_backward(s["dO"], s["Y"], s["row_of"], s["weights"], s["dY"], s["dw"], T, K, k,
                                 T * k)
        return {"dY": s["dY"], "dw": s["dw"]}
    V, K = c["V"], c["K"]
    if c["dir"] == "fwd":
        dg.linear_cross_entropy(s["X"], s["W"], s["targets"], s["loss"], s["lse"], s["work"],
                                s["work"].numel(), T, V, K)
        return {"loss": s["loss"], "lse": s["lse"]}
    dg.linear_cross_entropy_backward(s["X"], s["W"], s["targets"], s["lse"], s["d_loss"], s["dX"],
                                     s["dW"], s["work"], s["work"].numel(), T, V, K)
    return {"dX": s["dX"], "dW": s["dW"]}


def run(state):
    if own:
        return _own(state)
    return {"route": _route_plain, "dispatch": _dispatch_plain, "combine": _combine_plain,
            "loss": _loss_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------- work ----
def work(case):
    T = case["T"]
    if case["op"] == "route":
        G, k, size = case["G"], case["k"], 2 if case["bf16"] else 4
        if case["dir"] == "fwd":
            return {"bytes": T * G * size + (4 * G if case["bias"] else 0) + 8 * T * k,
                    "flops": 6 * T * G}
        # sigmoid scores, and renormalised softmax ones, need the chosen logits only
        few = case["sigmoid"] or case["renorm"]
        return {"bytes": T * (k if few else G) * size + T * G * size + 8 * T * k, "flops": 6 * T * G}
    if case["op"] == "dispatch":
        K, k = case["K"], case["k"]
        row = 2 * K if case["form"] == "bf16" else K + (K // GROUP) * (4 if case["form"] == "fp8" else 1)
        b = T * row + T * k * row + 8 * T * k + 4 * case["G"]
        return {"bytes": b + (4 * case["rows"] if case["layout"] == "contiguous" else 0), "flops": T * k}
    if case["op"] == "combine":
        K, k = case["K"], case["k"]
        n, index = T * k * K, 4 * T * k * (2 if case["weights"] else 1)
        if case["dir"] == "fwd":
            return {"bytes": 2 * n + 2 * T * K * (2 if case["residual"] else 1) + index,
                    "flops": 2 * n}
        return {"bytes": 4 * n + 2 * T * K + index + 4 * T * k, "flops": 3 * n}
    V, K = case["V"], case["K"]
    if case["dir"] == "fwd":
        return {"bytes": 2 * K * (T + V) + 12 * T, "flops": 2 * T * V * K}
    # the logits again, and a product for each gradient
    return {"bytes": 4 * K * (T + V) + 12 * T, "flops": 6 * T * V * K}


# ------------------------------------------------------------------ exact ----
def _rank(c):
    """Rank of each entry of a row, larger ones first, equal ones by their index."""
    n = c.shape[1]
    i = torch.arange(n, device=c.device)
    rank = torch.zeros(c.shape, dtype=torch.int64, device=c.device)
    for j in range(n):
        v = c[:, j:j + 1]
        rank += ((v > c) | ((v == c) & (j < i))).long()
    return rank


def _exact_route(case, s):
    x = s["logits"].double()
    p = torch.sigmoid(x) if case["sigmoid"] else torch.softmax(x, dim=1)
    if case["dir"] == "fwd":
        c = p if s["bias"] is None else p + s["bias"].double()
        n = case["groups"]
        if n > 1:
            per = case["G"] // n
            value = torch.stack([c[:, i * per:(i + 1) * per].topk(case["best"], dim=1).values.sum(1)
                                 for i in range(n)], dim=1)
            kept = (_rank(value) < case["top_groups"]).repeat_interleave(per, dim=1)
            c = c.masked_fill(~kept, -math.inf)
        rank = _rank(c)
        e = torch.stack([(rank == j).double().argmax(1) for j in range(case["k"])], dim=1)
        w = torch.take_along_dim(p, e, 1)
        if case["renorm"]:
            w = w / (w.sum(1, keepdim=True) + LEAST)
        return {"experts": e.to(torch.int32), "weights": case["scale"] * w}
    # through the chain rule, by autograd in 64 bits
    x.requires_grad_()
    with torch.enable_grad():
        p = torch.sigmoid(x) if case["sigmoid"] else torch.softmax(x, dim=1)
        w = torch.take_along_dim(p, s["experts"].long(), 1)
        if case["renorm"]:
            w = w / (w.sum(1, keepdim=True) + LEAST)
        (case["scale"] * w * s["d_weights"].double()).sum().backward()
    return {"d_logits": x.grad}


def _exact_dispatch(case, s):
    """Row by row: the choices of one expert after the other."""
    G, k, rows = case["G"], case["k"], case["rows"]
    flat = s["experts"].flatten()
    row = torch.empty(flat.shape, dtype=torch.int32, device=DEV)
    sizes = torch.empty(G, dtype=torch.int32, device=DEV)
    owner = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    a = torch.zeros(s["A"].shape, dtype=torch.float64, device=DEV).view(-1, case["K"])
    x = s["X"].double() if case["form"] == "bf16" else s["X"].view(torch.float8_e4m3fn).double()
    out = {}
    if case["form"] != "bf16":
        to = _scales(s["sa_out"], case["form"]).double()
        of = _scales(s["sa"], case["form"]).double()
    first = 0
    for e in range(G):
        pair = (flat == e).nonzero()[:, 0]
        n = pair.numel()
        if case["layout"] == "masked":
            first = e * rows
        at = torch.arange(first, first + n, device=DEV)
        sizes[e], row[pair] = n, at.to(torch.int32)
        a[at] = x[pair // k]
        if case["form"] != "bf16":
            into = to[e] if case["layout"] == "masked" else to
            into[:, at % rows if case["layout"] == "masked" else at] = of[:, pair // k]
        if case["layout"] == "contiguous":
            owner[at] = e
            n = (n + ALIGN - 1) // ALIGN * ALIGN
        first += n
    out.update(sizes=sizes, row_of=row.view(-1, k), A=a.view(s["A"].shape))
    if case["layout"] == "contiguous":
        out["m_indices"] = owner
    if case["form"] != "bf16":
        out["sa"] = to
    return out


def _exact_combine(case, s):
    at = s["row_of"].long()
    if case["dir"] == "fwd":
        out = s["R"].double() if case["residual"] else torch.zeros(case["T"], case["K"], device=DEV).double()
        for j in range(case["k"]):
            y = s["Y"][at[:, j]].double()
            out = out + (y * s["weights"][:, j:j + 1].double() if case["weights"] else y)
        return {"out": out}
    d = s["dO"].double()
    dy = torch.zeros(s["Y"].shape, dtype=torch.float64, device=DEV)
    dw = torch.empty(s["weights"].shape, dtype=torch.float64, device=DEV)
    for j in range(case["k"]):
        dy[at[:, j]] = d * s["weights"][:, j:j + 1].double()
        dw[:, j] = torch.einsum("tk,tk->t", d, s["Y"][at[:, j]].double())
    return {"dY": dy, "dw": dw}


def _exact_loss(case, s):
    T, V, K = case["T"], case["V"], case["K"]
    if T * V * K * (6 if case["dir"] == "bwd" else 2) > 1.2e13:   # (beyond 20 seconds)
        return None
    x, t = s["X"].double(), s["targets"].long()
    step = max(1, (1 << 28) // V)      # tokens at a time: 2 GB of logits
    if case["dir"] == "fwd":
        w = s["W"].double().t().contiguous()
        lse, loss = [], []
        for i in range(0, T, step):
            z, y = x[i:i + step] @ w, t[i:i + step]
            lse.append(torch.logsumexp(z, dim=1))
            hit = z[torch.arange(z.shape[0], device=DEV), y.clamp_min(0)]
            loss.append((lse[-1] - hit) * (y >= 0))
        return {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    w = s["W"].double()
    dx, dw = torch.empty_like(x), torch.zeros_like(w)
    for i in range(0, T, step):
        xi, y = x[i:i + step], t[i:i + step]
        p = torch.exp(xi @ w.t() - s["lse"][i:i + step, None].double())
        there = (y >= 0).nonzero()[:, 0]
        p[there, y[there]] -= 1.0
        p *= (s["d_loss"][i:i + step].double() * (y >= 0))[:, None]
        dx[i:i + step] = p @ w
        dw += p.t() @ xi
    return {"dX": dx, "dW": dw}


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    return {"route": _exact_route, "dispatch": _exact_dispatch, "combine": _exact_combine,
            "loss": _exact_loss}[case["op"]](case, s)
