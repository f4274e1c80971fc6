"""One mixture-of-experts layer on the library's operators: a training step and a
decoding step.

    python examples/moe_layer.py [--tokens 4096] [--hidden 7168] [--inter 2048]
                                 [--experts 8] [--top-k 2]

Training, in bf16 with an 8-bit activation checkpoint:

    norm(x + residual) -> router -> rows grouped by expert (ragged, no padding)
    -> product nt (gate | up) -> gated activation, checkpoint of its input
    -> product nt (down) -> weighted sum back into the residual stream

and backward through product nn, the gated activation's gradient from the
checkpoint (which also gives the activation again for the weight gradient),
product tn, and the norm's gradient.  Decoding, in FP8: the norm writes the
quantised rows, which go through the masked grouped GEMM, the gated activation
with 8-bit output, and the masked grouped GEMM again.

The router, the permutation of rows and the weighted sum are plain torch.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import moe_grouped_gemm_bf16_gb300 as dg  # noqa: E402

EPS = 1e-6
BF16 = torch.bfloat16


def _empty(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="cuda")


class Weights:
    """Norm weight [H], router [H, G], W1 [G, 2I, H] (gate rows, then up rows),
    W2 [G, H, I], all bf16."""

    def __init__(self, hidden, inter, experts, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, scale: (torch.randn(*s, generator=g, device="cuda") * scale).to(BF16)
        self.hidden, self.inter, self.experts = hidden, inter, experts
        self.norm = (1.0 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).to(BF16)
        self.router = rand(hidden, experts, scale=hidden ** -0.5)
        self.w1 = rand(experts, 2 * inter, hidden, scale=hidden ** -0.5)
        self.w2 = rand(experts, hidden, inter, scale=inter ** -0.5)


def route(y, w, top_k):
    """(weights [T, k] fp32, experts [T, k]) of each token."""
    p = torch.softmax((y @ w.router).float(), dim=-1)
    return p.topk(top_k, dim=-1)


def train_step(w, x, residual, d_out, top_k):
    """Forward and backward of the layer.  Returns (out, gradients): out is the
    residual stream after the layer, gradients a dict of dx (of x and of the
    residual alike), d_norm, dw1, dw2.  The routing is taken as given (its own
    gradient is not part of this example)."""
    T, H, I, G = x.shape[0], w.hidden, w.inter, w.experts
    h, y, rstd = _empty(T, H), _empty(T, H), _empty(T, dtype=torch.float32)
    dg.rms_norm_quantize_fp8_1x128(x, residual, w.norm, h, y, None, None, rstd, T, H, 0, EPS)
    gate, expert = route(y, w, top_k)

    # rows of the experts one after the other; their counts stay on the device
    R = T * top_k
    order = expert.flatten().argsort(stable=True)
    token = order // top_k
    sizes = torch.bincount(expert.flatten(), minlength=G).to(torch.int32)
    rows = y[token]
    gu, out_rows = _empty(R, 2 * I), _empty(R, H)
    dg.m_grouped_gemm_bf16_nt_ragged(rows, w.w1, gu, sizes, R, 2 * I, H, G)
    act = _empty(R, I)
    ld = dg.get_tma_aligned_size(R, 4)
    ckpt, ckpt_scale = _empty(R, 2 * I, dtype=torch.uint8), _empty(2 * I // 128, ld, dtype=torch.float32)
    dg.swiglu_quantize_fp8_1x128(gu, act, None, None, ckpt, ckpt_scale, 1, R, I, ld)
    dg.m_grouped_gemm_bf16_nt_ragged(act, w.w2, out_rows, sizes, R, H, I, G)
    share = gate.flatten()[order].unsqueeze(1)
    out = h.float().index_add_(0, token, out_rows.float() * share).to(BF16)
    del gu, act   # the backward pass needs neither: it has the checkpoint

    d_rows = (d_out[token].float() * share).to(BF16)
    d_act = _empty(R, I)
    dg.m_grouped_gemm_bf16_nn_ragged(d_rows, w.w2, d_act, sizes, R, I, H, G)
    d_gu, act = _empty(R, 2 * I), _empty(R, I)
    dg.swiglu_backward_fp8_1x128(ckpt, ckpt_scale, d_act, d_gu, act, 1, R, I, ld)
    dw2, dw1 = _empty(G, H, I), _empty(G, 2 * I, H)
    dg.k_grouped_gemm_bf16_tn_ragged(d_rows, act, dw2, sizes, G, H, I, R)
    dg.k_grouped_gemm_bf16_tn_ragged(d_gu, rows, dw1, sizes, G, 2 * I, H, R)
    d_in = _empty(R, H)
    dg.m_grouped_gemm_bf16_nn_ragged(d_gu, w.w1, d_in, sizes, R, H, 2 * I, G)
    dy = torch.zeros(T, H, device="cuda").index_add_(0, token, d_in.float()).to(BF16)
    dx, d_norm = _empty(T, H), _empty(H, dtype=torch.float32)
    n = dg.rms_norm_backward_workspace_bytes(T, H)
    work = _empty(max(n, 16), dtype=torch.uint8)
    dg.rms_norm_backward(dy, h, rstd, w.norm, d_out, dx, d_norm, work, n, T, H)
    return out, dict(dx=dx, d_norm=d_norm, dw1=dw1, dw2=dw2)


def quantize_weight(x):
    """[G, N, K] bf16 -> e4m3 codes and fp32 scales [G, N/128, K/128] (128 x 128
    blocks), once, when a model is loaded."""
    G, N, K = x.shape
    b = x.float().unflatten(2, (-1, 128)).unflatten(1, (-1, 128))   # [G, N/128, 128, K/128, 128]
    s = b.abs().amax(dim=(2, 4)).clamp_min(1e-4) / 448.0
    q = (b / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(G, N, K), s.contiguous()


def decode_step(w, w1q, w2q, x, residual, top_k, max_m):
    """One decoding step in FP8 (w1q, w2q: quantize_weight of the experts), with
    room for max_m rows per expert: as many as tokens, which may all choose one."""
    T, H, I, G = x.shape[0], w.hidden, w.inter, w.experts
    if T > max_m:
        raise ValueError(f"{T} tokens, room for {max_m} rows per expert")
    ld = dg.get_tma_aligned_size(T, 4)
    h, y = _empty(T, H), _empty(T, H)
    q, sa = _empty(T, H, dtype=torch.uint8), _empty(H // 128, ld, dtype=torch.float32)
    dg.rms_norm_quantize_fp8_1x128(x, residual, w.norm, h, y, q, sa, None, T, H, ld, EPS)
    gate, expert = route(y, w, top_k)

    # row j of expert e's block: the j-th of the (token, choice) pairs routed to it
    flat = expert.flatten()
    hot = torch.nn.functional.one_hot(flat, G)
    place = (hot.cumsum(0) - hot).gather(1, flat[:, None]).squeeze(1)
    masked_m = hot.sum(0).to(torch.int32)
    token = torch.arange(T, device="cuda").repeat_interleave(top_k, output_size=T * top_k)
    lm = dg.get_tma_aligned_size(max_m, 4)
    a = torch.zeros(G, max_m, H, dtype=torch.uint8, device="cuda")
    sa_e = torch.zeros(G, H // 128, lm, device="cuda")
    a[flat, place] = q[token]
    sa_e[flat, :, place] = sa[:, token].t()
    gu, out_rows = _empty(G, max_m, 2 * I), _empty(G, max_m, H)
    expected = max(1, T * top_k // G)
    dg.m_grouped_gemm_fp8_fp8_bf16_nt_masked(a, sa_e, lm, w1q[0], w1q[1], gu, masked_m, G, max_m, 2 * I,
                                             H, expected)
    aq, sq = _empty(G, max_m, I, dtype=torch.uint8), _empty(G, I // 128, lm, dtype=torch.float32)
    dg.swiglu_quantize_fp8_1x128(gu, None, aq, sq, None, None, G, max_m, I, lm, masked_m=masked_m)
    dg.m_grouped_gemm_fp8_fp8_bf16_nt_masked(aq, sq, lm, w2q[0], w2q[1], out_rows, masked_m, G, max_m, H,
                                             I, expected)
    return h.float().index_add_(0, token, out_rows[flat, place].float() * gate.flatten()[:, None]).to(BF16)


def reference_step(w, x, residual, d_out, top_k):
    """The training step by torch autograd in fp32, for comparison."""
    leaves = [t.float().requires_grad_() for t in (x.float() + residual.float(), w.norm, w.w1, w.w2)]
    h, wn, w1, w2 = leaves
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * wn
    with torch.no_grad():
        gate, expert = route(y.to(BF16), w, top_k)
    out = h
    for e in range(w.experts):
        t, k = (expert == e).nonzero(as_tuple=True)
        g, u = (y[t] @ w1[e].t()).chunk(2, dim=-1)
        out = out.index_add(0, t, (g * torch.sigmoid(g) * u) @ w2[e].t() * gate[t, k][:, None])
    (out * d_out.float()).sum().backward()
    return out.detach(), dict(zip(("dx", "d_norm", "dw1", "dw2"), (t.grad for t in leaves)))


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def run(tokens, hidden, inter, experts, top_k, seed=0):
    """Both steps against the reference: a dict of relative errors (of the
    decoding step, that of what the layer adds to the residual stream)."""
    w = Weights(hidden, inter, experts, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    rand = lambda scale: (torch.randn(tokens, hidden, generator=g, device="cuda") * scale).to(BF16)
    x, residual, d_out = rand(1.0), rand(2.0), rand(0.02)
    out, grads = train_step(w, x, residual, d_out, top_k)
    want, want_grads = reference_step(w, x, residual, d_out, top_k)
    base = x.float() + residual.float()
    err = {"out": relative(out, want)}
    err.update({k: relative(grads[k], want_grads[k]) for k in grads})
    n = min(tokens, 32)
    dec = decode_step(w, quantize_weight(w.w1), quantize_weight(w.w2), x[:n].contiguous(),
                      residual[:n].contiguous(), top_k, max_m=128)
    err["decode"] = relative(dec.float() - base[:n], want[:n] - base[:n])
    status = dg.get_device_status()
    assert status == 0, dg.STATUS_NAMES.get(status, status)
    return err


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 4096), ("hidden", 7168), ("inter", 2048), ("experts", 8), ("top-k", 2)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    for k, v in run(a.tokens, a.hidden, a.inter, a.experts, a.top_k).items():
        print(f"{k:8s} relative error {v:.2e}")
    w = Weights(a.hidden, a.inter, a.experts)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(BF16)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(3):
        train_step(w, x, x, x, a.top_k)
    start.record()
    for _ in range(10):
        train_step(w, x, x, x, a.top_k)
    end.record()
    torch.cuda.synchronize()
    print(f"training step {start.elapsed_time(end) / 10:.2f} ms")


if __name__ == "__main__":
    main()
