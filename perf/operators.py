"""The operators of an expert layer around the grouped FP8 products, measured.

Three operators, each with the direction that training needs:

  norm     root-mean-square norm of x + residual, with its output in 8 bits and
           one scale per row and 128 columns (the left operand of the FP8
           products), and its gradient;
  swiglu   silu(gate) * up between the two products of an expert, its output in
           8 bits with scales, the 8-bit checkpoint of gate and up, and the
           gradient computed from that checkpoint;
  product  bf16 products grouped by expert with ragged sizes: y = x W^T ("nt"),
           dx = dy W ("nn") and dW = dy^T x ("tn").

`own` False: the operators in elementary torch operations in 32 bits, rounded
once at the end.  `own` True: the package's calls.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
FLOOR = 1e-4      # smallest group maximum a scale is made from
EPS = 1e-6
GROUP = 128
DEV = "cuda"


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # the attention output of a handful of sequences joining the residual stream
        # in one decoding step; the quantised rows feed the experts' FP8 products
        {"name": "norm decode 7x7168", "op": "norm", "dir": "fwd", "M": 7, "K": 7168,
         "residual": True, "both": False, "ue8m0": False},
        # the same in a prefill or training step of 4096 tokens; the bf16 output is kept too,
        # for the router and the weight gradient
        {"name": "norm prefill 4096x7168", "op": "norm", "dir": "fwd", "M": 4096, "K": 7168,
         "residual": True, "both": True, "ue8m0": False},
        # gradient of a short, odd batch of a narrow layer, no gradient on the residual
        {"name": "norm grad 333x2048", "op": "norm", "dir": "bwd", "M": 333, "K": 2048,
         "residual": False},
        # gradient of a training step of 8192 tokens, joined with the residual's gradient
        {"name": "norm grad 8192x7168", "op": "norm", "dir": "bwd", "M": 8192, "K": 7168,
         "residual": True},
        # decoding under a CUDA graph: 8 experts with room for 128 rows each, a few filled
        # (the masked layout), power-of-two scales, no checkpoint
        {"name": "swiglu decode masked", "op": "swiglu", "dir": "fwd", "G": 8, "M": 128,
         "I": 2048, "filled": 211, "ckpt": False, "ue8m0": True},
        # training: the routed rows of 4 experts, with the checkpoint of gate and up
        {"name": "swiglu train 32647x2048", "op": "swiglu", "dir": "fwd", "G": 1, "M": 32647,
         "I": 2048, "filled": 32647, "ckpt": True, "ue8m0": False},
        # gradient of a small odd batch of a narrow expert
        {"name": "swiglu grad 515x1536", "op": "swiglu", "dir": "bwd", "G": 1, "M": 515,
         "I": 1536, "filled": 515},
        # gradient of the training rows above
        {"name": "swiglu grad 32647x2048", "op": "swiglu", "dir": "bwd", "G": 1, "M": 32647,
         "I": 2048, "filled": 32647},
        # one decoding step: 61 routed rows on 8 experts, two of them without a row; the
        # time is that of reading the weights
        {"name": "product nt decode", "op": "product", "form": "nt", "G": 8, "active": 6,
         "tokens": 61, "N": 4096, "K": 7168},
        # forward of the gate and up projections on the training rows
        {"name": "product nt train", "op": "product", "form": "nt", "G": 4, "active": 4,
         "tokens": 32647, "N": 4096, "K": 7168},
        # gradient with respect to the activations, many small experts, ragged, some empty
        {"name": "product nn ragged", "op": "product", "form": "nn", "G": 32, "active": 29,
         "tokens": 5003, "N": 2048, "K": 7168},
        # weight gradient of the down projection, one expert without rows
        {"name": "product tn train", "op": "product", "form": "tn", "G": 4, "active": 3,
         "tokens": 16391, "N": 2048, "K": 7168},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, unit):
    while True:
        v = max(lo, min(hi, (_log(rng, lo, hi) + unit - 1) // unit * unit))
        if v != 3072:
            return v


def draw(rng):
    op = rng.choice(["norm", "swiglu", "product"])
    if op == "norm":
        while True:
            M, K = _log(rng, 1, 8192), _mult(rng, 512, 16384, GROUP)
            if M * K <= 4096 * 7168:
                break
        if rng.random() < 0.5:
            return {"op": op, "dir": "bwd", "M": M, "K": K, "residual": rng.random() < 0.5}
        return {"op": op, "dir": "fwd", "M": M, "K": K, "residual": rng.random() < 0.7,
                "both": rng.random() < 0.5, "ue8m0": rng.random() < 0.25}
    if op == "swiglu":
        G = rng.choice([1, 1, 2, 4, 8])
        while True:
            M, I = _log(rng, 1, 32647), _mult(rng, 256, 4096, GROUP)
            if G * M * I <= 32647 * 2048:
                break
        filled = G * M if G == 1 else rng.randint(1, G * M)
        if rng.random() < 0.5:
            return {"op": op, "dir": "bwd", "G": G, "M": M, "I": I, "filled": filled}
        return {"op": op, "dir": "fwd", "G": G, "M": M, "I": I, "filled": filled,
                "ckpt": rng.random() < 0.5, "ue8m0": rng.random() < 0.25}
    form = rng.choice(["nt", "nn", "tn"])
    while True:
        G = _log(rng, 1, 64)
        tokens = _log(rng, 1, 32647)
        N, K = _mult(rng, 256, 8192, 8), _mult(rng, 256, 8192, 8)
        if G * N * K <= 32 * 2048 * 7168 and tokens * N * K <= 32647 * 2048 * 7168:
            break
    active = min(tokens, rng.randint(max(1, G // 2), G))
    return {"op": op, "form": form, "G": G, "active": active, "tokens": tokens, "N": N, "K": K}


# ----------------------------------------------------------------- inputs ----
def _filled(case, rng):
    """Valid rows of each of the G groups of the masked layout, `filled` in all."""
    G, M, left = case["G"], case["M"], case["filled"]
    got = []
    for g in range(G):
        room = (G - 1 - g) * M
        lo, hi = max(0, left - room), min(M, left)
        mean = left / (G - g)
        got.append(max(lo, min(hi, int(round(rng.uniform(0.3, 1.7) * mean)))))
        left -= got[-1]
    return got


def _sizes(case, rng):
    """Rows of each expert: `active` of the G experts share the tokens unevenly."""
    G, active, tokens = case["G"], case["active"], case["tokens"]
    w = [rng.uniform(0.4, 1.6) for _ in range(active)]
    rest, total = tokens - active, sum(w)
    got = [1 + int(rest * x / total) for x in w]
    got[-1] += tokens - sum(got)
    at = sorted(rng.sample(range(G), active))
    sizes = [0] * G
    for e, n in zip(at, got):
        sizes[e] = n
    return sizes


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFF)
    rng = random.Random(int(seed))
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8

    def normal(*shape, scale=1.0, dtype=bf):
        x = torch.empty(shape, dtype=dtype, device=DEV)
        x.normal_(0.0, scale, generator=gen)
        return x

    s = {"case": case}
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        # a few columns of the residual stream are far larger than the others
        loud = torch.ones(K, dtype=f32, device=DEV)
        loud[torch.randint(0, K, (max(1, K // 500),), device=DEV, generator=gen)] = 30.0
        s["W"] = (1.0 + 0.1 * normal(K, dtype=f32)).to(bf)
        if case["dir"] == "fwd":
            ld = (M + 3) // 4 * 4
            s["X"] = normal(M, K)
            s["R"] = (normal(M, K, dtype=f32) * loud).to(bf) if case["residual"] else None
            s["H"] = torch.zeros(M, K, dtype=bf, device=DEV) if case["residual"] else None
            s["Y"] = torch.zeros(M, K, dtype=bf, device=DEV) if case["both"] else None
            s["Q"] = torch.zeros(M, K, dtype=u8, device=DEV)
            s["rstd"] = torch.zeros(M, dtype=f32, device=DEV)
            s["ld"] = ld
            s["sa"] = (torch.zeros((K + 511) // 512, ld, dtype=torch.int32, device=DEV)
                       if case["ue8m0"] else torch.zeros(K // GROUP, ld, dtype=f32, device=DEV))
        else:
            s["H"] = (normal(M, K, dtype=f32) * loud).to(bf)
            s["rstd"] = torch.rsqrt(s["H"].float().square().mean(dim=1) + EPS)
            s["dY"] = normal(M, K, scale=0.02)
            s["dR"] = normal(M, K, scale=0.02) if case["residual"] else None
            s["dX"] = torch.zeros(M, K, dtype=bf, device=DEV)
            s["dW"] = torch.zeros(K, dtype=f32, device=DEV)
            # the partial sums of the weight's gradient: the whole of what any size needs
            s["work"] = torch.zeros(64 << 20, dtype=u8, device=DEV)
        return s
    if case["op"] == "swiglu":
        G, M, I = case["G"], case["M"], case["I"]
        ld = (M + 3) // 4 * 4
        rows = _filled(case, rng)
        s["ld"] = ld
        s["masked_m"] = torch.tensor(rows, dtype=torch.int32, device=DEV) if G > 1 else None
        s["rows"] = torch.arange(M, device=DEV)[None, :, None] < torch.tensor(
            rows, device=DEV)[:, None, None]
        if case["dir"] == "fwd":
            s["GU"] = normal(G, M, 2 * I, scale=1.5)
            s["Y"] = None
            s["Q"] = torch.zeros(G, M, I, dtype=u8, device=DEV)
            s["sa"] = (torch.zeros(G, (I + 511) // 512, ld, dtype=torch.int32, device=DEV)
                       if case["ue8m0"] else torch.zeros(G, I // GROUP, ld, dtype=f32, device=DEV))
            s["CQ"] = torch.zeros(G, M, 2 * I, dtype=u8, device=DEV) if case["ckpt"] else None
            s["csa"] = (torch.zeros(G, 2 * I // GROUP, ld, dtype=f32, device=DEV)
                        if case["ckpt"] else None)
        else:
            # a checkpoint as the forward pass leaves it
            gu = normal(G, M, 2 * I, scale=1.5)
            codes, scale = _codes(gu.float())
            s["CQ"] = codes.view(u8).contiguous()
            s["csa"] = _scale_rows(scale, ld)
            s["dY"] = normal(G, M, I, scale=0.02)
            s["dGU"] = torch.zeros(G, M, 2 * I, dtype=bf, device=DEV)
            s["Y"] = torch.zeros(G, M, I, dtype=bf, device=DEV)
        return s
    G, N, K, T = case["G"], case["N"], case["K"], case["tokens"]
    sizes = _sizes(case, rng)
    s["sizes"] = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    s["most"] = max(sizes)
    if case["form"] == "nt":       # y [T, N] = x [T, K] W[e] [N, K]^T
        s["A"], s["B"] = normal(T, K), normal(G, N, K, scale=K ** -0.5)
        s["D"] = torch.zeros(T, N, dtype=bf, device=DEV)
    elif case["form"] == "nn":     # dx [T, N] = dy [T, K] W[e] [K, N]
        s["A"], s["B"] = normal(T, K, scale=0.02), normal(G, K, N, scale=N ** -0.5)
        s["D"] = torch.zeros(T, N, dtype=bf, device=DEV)
    else:                          # dW[e] [N, K] = dy [T, N]^T x [T, K]
        s["A"], s["B"] = normal(T, N, scale=0.02), normal(T, K)
        s["D"] = torch.zeros(G, N, K, dtype=bf, device=DEV)
    return s


# ------------------------------------------------------------ plain forms ----
def _codes(x, pow2=False):
    """x [..., K] in 32 bits -> (e4m3 codes [..., K], scales [..., K/128]): one
    scale per 128 columns, amax / 448 or the power of two not below it."""
    g = x.unflatten(-1, (-1, GROUP))
    a = g.abs().amax(dim=-1).clamp_min(FLOOR)
    if pow2:
        m, e = torch.frexp(a / E4M3_MAX)
        scale = torch.ldexp(torch.ones_like(a), e - (m == 0.5).int())
        q = g / scale[..., None]
    else:
        scale = a / E4M3_MAX
        q = g * (E4M3_MAX / a)[..., None]
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).flatten(-2), scale


def _scale_rows(scale, ld):
    """[..., M, K/128] -> [..., K/128, ld], the columns past M zero."""
    t = scale.transpose(-1, -2)
    return torch.nn.functional.pad(t, (0, ld - t.shape[-1])).contiguous()


def _e8m0_rows(scale, ld, valid=None):
    """Power-of-two scales [..., M, K/128] -> the 8-bit exponents
    [..., ceil(K/512), ld, 4] as the values they stand for."""
    code = (torch.frexp(scale)[1] + 126).to(torch.uint8)
    if valid is not None:
        code = torch.where(valid, code, torch.zeros_like(code))
    t = code.transpose(-1, -2)
    kb = t.shape[-2]
    t = torch.nn.functional.pad(t, (0, ld - t.shape[-1], 0, -kb % 4))
    t = t.unflatten(-2, (-1, 4)).transpose(-1, -2).contiguous()
    return t.view(torch.float8_e8m0fnu)


def _norm_plain(s):
    c = s["case"]
    if c["dir"] == "fwd":
        h = s["X"].float()
        if c["residual"]:
            h = h + s["R"].float()
        rstd = torch.rsqrt(h.square().mean(dim=1) + EPS)
        y = h * rstd[:, None] * s["W"].float()
        q, scale = _codes(y, c["ue8m0"])
        return {"H": h.to(torch.bfloat16) if c["residual"] else None,
                "Y": y.to(torch.bfloat16) if c["both"] else None, "Q": q, "rstd": rstd,
                "sa": _e8m0_rows(scale, s["ld"]) if c["ue8m0"] else _scale_rows(scale, s["ld"])}
    xhat = s["H"].float() * s["rstd"][:, None]
    dy = s["dY"].float()
    g = dy * s["W"].float()
    dx = (g - xhat * (g * xhat).mean(dim=1, keepdim=True)) * s["rstd"][:, None]
    if c["residual"]:
        dx = dx + s["dR"].float()
    return {"dX": dx.to(torch.bfloat16), "dW": (dy * xhat).sum(dim=0)}


def _swiglu_plain(s):
    c, rows = s["case"], s["rows"]
    I = c["I"]
    if c["dir"] == "fwd":
        gu = s["GU"].float()
        g, u = gu[..., :I], gu[..., I:]
        y = torch.where(rows, g / (1.0 + torch.exp(-g)) * u, 0.0)
        q, scale = _codes(y, c["ue8m0"])
        out = {"Q": q, "sa": (_e8m0_rows(scale, s["ld"], rows) if c["ue8m0"]
                              else _scale_rows(torch.where(rows, scale, 0.0), s["ld"]))}
        if c["ckpt"]:
            cq, cs = _codes(torch.where(rows, gu, 0.0))
            out["CQ"], out["csa"] = cq, _scale_rows(torch.where(rows, cs, 0.0), s["ld"])
        return out
    cs = s["csa"][..., :c["M"]].transpose(-1, -2)
    gu = (s["CQ"].view(torch.float8_e4m3fn).float().unflatten(-1, (-1, GROUP))
          * cs[..., None]).flatten(-2)
    g, u, dy = gu[..., :I], gu[..., I:], s["dY"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    dg = dy * u * sig * (1.0 + g * (1.0 - sig))
    du = dy * g * sig
    dgu = torch.where(rows, torch.cat([dg, du], dim=-1), 0.0)
    return {"dGU": dgu.to(torch.bfloat16), "Y": torch.where(rows, g * sig * u, 0.0).to(torch.bfloat16)}


def _product_plain(s):
    c = s["case"]
    G, T = c["G"], c["tokens"]
    n = s["sizes"].long()
    e = torch.repeat_interleave(torch.arange(G, device=DEV), n, output_size=T)
    at = torch.arange(T, device=DEV) - (n.cumsum(0) - n)[e]

    def by_expert(x):  # rows side by side per expert, zeros behind the last
        p = torch.zeros(G, s["most"], x.shape[1], device=DEV)
        p[e, at] = x.float()
        return p

    if c["form"] == "tn":
        d = torch.matmul(by_expert(s["A"]).transpose(1, 2), by_expert(s["B"]))
        return {"D": d.to(torch.bfloat16)}
    b = s["B"].float()
    d = torch.matmul(by_expert(s["A"]), b.transpose(1, 2) if c["form"] == "nt" else b)
    return {"D": d[e, at].to(torch.bfloat16)}


# -------------------------------------------------------------------- run ----
def _own(s):
    import moe_grouped_gemm_bf16_gb300 as dg

    c = s["case"]
    e4m3, e8m0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        if c["dir"] == "fwd":
            call = (dg.rms_norm_quantize_fp8_1x128_ue8m0 if c["ue8m0"]
                    else dg.rms_norm_quantize_fp8_1x128)
            call(s["X"], s["R"], s["W"], s["H"], s["Y"], s["Q"], s["sa"], s["rstd"], M, K, s["ld"],
                 EPS)
            return {"H": s["H"], "Y": s["Y"], "Q": s["Q"].view(e4m3), "rstd": s["rstd"],
                    "sa": s["sa"].view(e8m0).unflatten(-1, (-1, 4)) if c["ue8m0"] else s["sa"]}
        dg.rms_norm_backward(s["dY"], s["H"], s["rstd"], s["W"], s["dR"], s["dX"], s["dW"],
                             s["work"], s["work"].numel(), M, K)
        return {"dX": s["dX"], "dW": s["dW"]}
    if c["op"] == "swiglu":
        G, M, I = c["G"], c["M"], c["I"]
        if c["dir"] == "fwd":
            call = (dg.swiglu_quantize_fp8_1x128_ue8m0 if c["ue8m0"]
                    else dg.swiglu_quantize_fp8_1x128)
            call(s["GU"], s["Y"], s["Q"], s["sa"], s["CQ"], s["csa"], G, M, I, s["ld"],
                 masked_m=s["masked_m"])
            out = {"Q": s["Q"].view(e4m3),
                   "sa": s["sa"].view(e8m0).unflatten(-1, (-1, 4)) if c["ue8m0"] else s["sa"]}
            if c["ckpt"]:
                out["CQ"], out["csa"] = s["CQ"].view(e4m3), s["csa"]
            return out
        dg.swiglu_backward_fp8_1x128(s["CQ"], s["csa"], s["dY"], s["dGU"], s["Y"], G, M, I, s["ld"],
                                     masked_m=s["masked_m"])
        return {"dGU": s["dGU"], "Y": s["Y"]}
    G, N, K, T = c["G"], c["N"], c["K"], c["tokens"]
    if c["form"] == "tn":
        dg.k_grouped_gemm_bf16_tn_ragged(s["A"], s["B"], s["D"], s["sizes"], G, N, K, T)
    elif c["form"] == "nt":
        dg.m_grouped_gemm_bf16_nt_ragged(s["A"], s["B"], s["D"], s["sizes"], T, N, K, G)
    else:
        dg.m_grouped_gemm_bf16_nn_ragged(s["A"], s["B"], s["D"], s["sizes"], T, N, K, G)
    return {"D": s["D"]}


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm_plain, "swiglu": _swiglu_plain,
            "product": _product_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------- work ----
def work(case):
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        n = M * K
        if case["dir"] == "fwd":
            b = 2 * n + n + M * 4 + 2 * K                      # x, codes, rstd, weight
            b += 4 * n if case["residual"] else 0              # residual in, sum out
            b += 2 * n if case["both"] else 0                  # bf16 output
            b += M * (K // GROUP) * (1 if case["ue8m0"] else 4)
            return {"bytes": b, "flops": 8 * n}
        b = 6 * n + M * 4 + 6 * K + (2 * n if case["residual"] else 0)
        return {"bytes": b, "flops": 12 * n}
    if case["op"] == "swiglu":
        n, kb = case["filled"] * case["I"], case["filled"] * (case["I"] // GROUP)
        # at least the row counts are read
        least = 4 * case["G"]
        if case["dir"] == "fwd":
            b = 5 * n + kb * (1 if case["ue8m0"] else 4) + least
            b += 2 * n + 8 * kb if case["ckpt"] else 0
            return {"bytes": b, "flops": 10 * n}
        return {"bytes": 2 * n + 8 * kb + 2 * n + 4 * n + 2 * n + least, "flops": 16 * n}
    G, N, K, T = case["G"], case["N"], case["K"], case["tokens"]
    # nt: x and y over K and N columns; nn the same; tn: both operands by rows, every dW written
    weights = (G if case["form"] == "tn" else case["active"]) * N * K
    return {"bytes": 2 * (T * (N + K) + weights) + 4 * G, "flops": 2 * T * N * K}


# ------------------------------------------------------------------ exact ----
def _exact_groups(y):
    a = y.reshape(*y.shape[:-1], -1, GROUP).abs().max(dim=-1).values
    return torch.maximum(a, torch.full_like(a, FLOOR))


def _exact_quant(y, ld, ue8m0):
    """Definition of the 8-bit output in 64 bits: (codes' values, scales in their layout)."""
    a = _exact_groups(y)
    s = torch.exp2(torch.ceil(torch.log2(a / E4M3_MAX))) if ue8m0 else a / E4M3_MAX
    q = (y.reshape(*y.shape[:-1], -1, GROUP) / s.unsqueeze(-1)).reshape(y.shape)
    kb, M = s.shape[-1], s.shape[-2]
    rows = (kb + 3) // 4 * 4 if ue8m0 else kb
    # an exponent of zero stands for 2^-127 where no scale is written
    out = torch.full((*s.shape[:-2], rows, ld), 2.0 ** -127 if ue8m0 else 0.0,
                     dtype=torch.float64, device=y.device)
    out[..., :kb, :M] = s.transpose(-1, -2)
    if ue8m0:
        out = out.reshape(*s.shape[:-2], rows // 4, 4, ld).transpose(-1, -2).contiguous()
    return q, out


def _exact_blank(q, s, valid, ue8m0):
    """Rows without a token hold zero codes and no scale."""
    blank = 2.0 ** -127 if ue8m0 else 0.0
    M = valid.shape[1]
    if ue8m0:
        s[:, :, :M, :] = torch.where(valid[:, None, :, None], s[:, :, :M, :], blank)
    else:
        s[:, :, :M] = torch.where(valid[:, None, :], s[:, :, :M], blank)
    return q * valid[..., None], s


def exact(case, seed):
    """The definitions in 64 bits.  The values behind 8-bit codes are those before the
    rounding to 8 bits, in units of the scale."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        W = s["W"].double()
        if case["dir"] == "fwd":
            h = s["X"].double() + (s["R"].double() if case["residual"] else 0.0)
            r = 1.0 / torch.sqrt((h * h).sum(1) / case["K"] + EPS)
            y = h * r[:, None] * W[None, :]
            q, sa = _exact_quant(y, s["ld"], case["ue8m0"])
            return {"H": h if case["residual"] else None, "Y": y if case["both"] else None,
                    "Q": q, "rstd": r, "sa": sa}
        h, dy, r = s["H"].double(), s["dY"].double(), s["rstd"].double()
        K = case["K"]
        # d/dh_j of sum_k dy_k w_k h_k r(h): r w_j dy_j - h_j r^3 / K sum_k dy_k w_k h_k
        dot = (dy * W * h).sum(1)
        dx = W * dy * r[:, None] - h * (r ** 3 * dot / K)[:, None]
        if case["residual"]:
            dx = dx + s["dR"].double()
        return {"dX": dx, "dW": torch.einsum("mk,mk,m->k", dy, h, r)}
    if case["op"] == "swiglu":
        I, M, ld = case["I"], case["M"], s["ld"]
        if s["masked_m"] is None:
            n = torch.tensor([M], device=DEV)
        else:
            n = s["masked_m"].long()
        valid = torch.arange(M, device=DEV).unsqueeze(0) < n.unsqueeze(1)
        if case["dir"] == "fwd":
            g, u = s["GU"][..., :I].double(), s["GU"][..., I:].double()
            y = g * u * torch.sigmoid(g)
            q, sa = _exact_blank(*_exact_quant(y, ld, case["ue8m0"]), valid, case["ue8m0"])
            out = {"Q": q, "sa": sa}
            if case["ckpt"]:
                out["CQ"], out["csa"] = _exact_blank(
                    *_exact_quant(s["GU"].double(), ld, False), valid, False)
            return out
        sc = s["csa"].double()[:, :, :M].permute(0, 2, 1).repeat_interleave(GROUP, dim=2)
        x = s["CQ"].view(torch.float8_e4m3fn).double() * sc
        g, u, dy = x[..., :I], x[..., I:], s["dY"].double()
        t = torch.sigmoid(g)
        d = torch.cat([dy * u * (t + g * t * (1.0 - t)), dy * g * t], dim=-1)
        return {"dGU": d * valid[..., None], "Y": g * t * u * valid[..., None]}
    # one expert after the other
    A, B, form = s["A"], s["B"], case["form"]
    D = torch.zeros(s["D"].shape, dtype=torch.float64, device=DEV)
    first = 0
    for e, n in enumerate(s["sizes"].tolist()):
        rows = slice(first, first + n)
        first += n
        if n == 0:
            continue
        if form == "nt":
            D[rows] = A[rows].double() @ B[e].double().t()
        elif form == "nn":
            D[rows] = A[rows].double() @ B[e].double()
        else:
            D[e] = A[rows].double().t() @ B[rows].double()
    return {"D": D}
