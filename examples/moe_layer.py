"""One mixture-of-experts layer on the library's operators: a training step and a
decoding step.

    python examples/moe_layer.py [--tokens 4096] [--hidden 7168] [--inter 2048]
                                 [--experts 8] [--top-k 2] [--vocabulary 32000]

Training, in bf16 with an 8-bit activation checkpoint:

    norm(x + residual) -> router -> routing -> rows grouped by expert (ragged, no
    padding) -> product nt (gate | up) -> gated activation, checkpoint of its input
    -> product nt (down) -> weighted sum back into the residual stream
    -> cross entropy of its product with an output matrix

and backward through the cross entropy's gradient, the weighted sum's, product nn,
the gated activation's gradient from the checkpoint (which also gives the activation
again for the weight gradient), product tn, the routing's and the norm's gradient.
Decoding, in FP8: the norm writes the quantised rows, which are dispatched into the
masked layout and go through the masked grouped GEMM, the gated activation with 8-bit
output, and the masked grouped GEMM again.

The router's own product (a few columns) is plain torch.
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
    W2 [G, H, I], output matrix [V, H], all bf16."""

    def __init__(self, hidden, inter, experts, seed=0, vocabulary=1000):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, scale: (torch.randn(*s, generator=g, device="cuda") * scale).to(BF16)
        self.hidden, self.inter, self.experts, self.vocabulary = hidden, inter, experts, vocabulary
        self.norm = (1.0 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).to(BF16)
        self.router = rand(hidden, experts, scale=hidden ** -0.5)
        self.w1 = rand(experts, 2 * inter, hidden, scale=hidden ** -0.5)
        self.w2 = rand(experts, hidden, inter, scale=inter ** -0.5)
        self.head = rand(vocabulary, hidden, scale=0.5 * hidden ** -0.5)


def route(y, w, top_k):
    """(logits [T, G] bf16, weights [T, k] fp32, experts [T, k] int32) of each token."""
    T, G = y.shape[0], w.experts
    logits = y @ w.router
    weights, experts = _empty(T, top_k, dtype=torch.float32), _empty(T, top_k, dtype=torch.int32)
    dg.route_top_k_bf16(logits, None, experts, weights, T, G, top_k, renormalize=False)
    return logits, weights, experts


def forward(w, x, residual, top_k):
    """(out [T, H]: the residual stream after the layer, what backward needs)."""
    T, H, I, G = x.shape[0], w.hidden, w.inter, w.experts
    h, y, rstd = _empty(T, H), _empty(T, H), _empty(T, dtype=torch.float32)
    dg.rms_norm_quantize_fp8_1x128(x, residual, w.norm, h, y, None, None, rstd, T, H, 0, EPS)
    logits, gate, expert = route(y, w, top_k)

    # rows of the experts one after the other; their counts stay on the device
    R = T * top_k
    sizes, at = _empty(G, dtype=torch.int32), _empty(T, top_k, dtype=torch.int32)
    dg.expert_rows_ragged(expert, sizes, at, T, top_k, G)
    rows = _empty(R, H)
    dg.dispatch_rows_bf16(y, at, rows, T, H, top_k, R)
    gu, out_rows = _empty(R, 2 * I), _empty(R, H)
    dg.m_grouped_gemm_bf16_nt_ragged(rows, w.w1, gu, sizes, R, 2 * I, H, G)
    act = _empty(R, I)
    ld = dg.get_tma_aligned_size(R, 4)
    ckpt, ckpt_scale = _empty(R, 2 * I, dtype=torch.uint8), _empty(2 * I // 128, ld, dtype=torch.float32)
    dg.swiglu_quantize_fp8_1x128(gu, act, None, None, ckpt, ckpt_scale, 1, R, I, ld)
    dg.m_grouped_gemm_bf16_nt_ragged(act, w.w2, out_rows, sizes, R, H, I, G)
    out = _empty(T, H)
    dg.combine_rows(out_rows, at, gate, h, out, T, H, top_k, R)
    # (the activation itself is not kept: there is the checkpoint)
    return out, (h, y, rstd, logits, gate, expert, sizes, at, rows, ckpt, ckpt_scale, ld, out_rows)


def loss_and_gradient(w, out, targets):
    """(loss [T], d_out, d_head): the mean cross entropy's gradients."""
    T, H, V = out.shape[0], w.hidden, w.vocabulary
    loss, lse = _empty(T, dtype=torch.float32), _empty(T, dtype=torch.float32)
    n = max(dg.linear_cross_entropy_workspace_bytes(T, V, H),
            dg.linear_cross_entropy_backward_workspace_bytes(T, V, H))
    work = _empty(n, dtype=torch.uint8)
    dg.linear_cross_entropy(out, w.head, targets, loss, lse, work, n, T, V, H)
    d_loss = torch.full((T,), 1.0 / T, device="cuda")
    d_out, d_head = _empty(T, H), _empty(V, H)
    dg.linear_cross_entropy_backward(out, w.head, targets, lse, d_loss, d_out, d_head, work, n, T, V, H)
    return loss, d_out, d_head


def backward(w, saved, d_out, top_k):
    """Gradients of the layer: dx (of x and of the residual alike), d_norm, d_router, dw1,
    dw2."""
    h, y, rstd, logits, gate, expert, sizes, at, rows, ckpt, ckpt_scale, ld, out_rows = saved
    T, H, I, G, R = h.shape[0], w.hidden, w.inter, w.experts, rows.shape[0]
    d_rows, d_gate = _empty(R, H), _empty(T, top_k, dtype=torch.float32)
    dg.combine_rows_backward(d_out, out_rows, at, gate, d_rows, d_gate, T, H, top_k, R)
    d_act = _empty(R, I)
    dg.m_grouped_gemm_bf16_nn_ragged(d_rows, w.w2, d_act, sizes, R, I, H, G)
    d_gu, act = _empty(R, 2 * I), _empty(R, I)
    dg.swiglu_backward_fp8_1x128(ckpt, ckpt_scale, d_act, d_gu, act, 1, R, I, ld)
    dw2, dw1 = _empty(G, H, I), _empty(G, 2 * I, H)
    dg.k_grouped_gemm_bf16_tn_ragged(d_rows, act, dw2, sizes, G, H, I, R)
    dg.k_grouped_gemm_bf16_tn_ragged(d_gu, rows, dw1, sizes, G, 2 * I, H, R)
    d_in = _empty(R, H)
    dg.m_grouped_gemm_bf16_nn_ragged(d_gu, w.w1, d_in, sizes, R, H, 2 * I, G)
    d_logits = _empty(T, G)
    dg.route_top_k_backward_bf16(logits, expert, d_gate, d_logits, T, G, top_k, renormalize=False)
    dy = d_logits @ w.router.t()
    dg.combine_rows(d_in, at, None, dy, dy, T, H, top_k, R)   # (the dispatch's gradient, on the router's)
    dx, d_norm = _empty(T, H), _empty(H, dtype=torch.float32)
    n = dg.rms_norm_backward_workspace_bytes(T, H)
    work = _empty(max(n, 16), dtype=torch.uint8)
    dg.rms_norm_backward(dy, h, rstd, w.norm, d_out, dx, d_norm, work, n, T, H)
    return dict(dx=dx, d_norm=d_norm, d_router=y.t() @ d_logits, dw1=dw1, dw2=dw2)


def train_step(w, x, residual, targets, top_k):
    """(loss [T], out, gradients) of the layer and the output matrix."""
    out, saved = forward(w, x, residual, top_k)
    loss, d_out, d_head = loss_and_gradient(w, out, targets)
    return loss, out, dict(backward(w, saved, d_out, top_k), d_head=d_head)


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
    _, gate, expert = route(y, w, top_k)

    masked_m, at = _empty(G, dtype=torch.int32), _empty(T, top_k, dtype=torch.int32)
    dg.expert_rows_masked(expert, masked_m, at, T, top_k, G, max_m)
    lm = dg.get_tma_aligned_size(max_m, 4)
    a, sa_e = _empty(G, max_m, H, dtype=torch.uint8), _empty(G, H // 128, lm, dtype=torch.float32)
    dg.dispatch_rows_fp8_1x128(q, sa, ld, at, a, sa_e, lm, T, H, top_k, G, max_m)
    gu, out_rows = _empty(G, max_m, 2 * I), _empty(G, max_m, H)
    expected = max(1, T * top_k // G)
    dg.m_grouped_gemm_fp8_fp8_bf16_nt_masked(a, sa_e, lm, w1q[0], w1q[1], gu, masked_m, G, max_m, 2 * I,
                                             H, expected)
    aq, sq = _empty(G, max_m, I, dtype=torch.uint8), _empty(G, I // 128, lm, dtype=torch.float32)
    dg.swiglu_quantize_fp8_1x128(gu, None, aq, sq, None, None, G, max_m, I, lm, masked_m=masked_m)
    dg.m_grouped_gemm_fp8_fp8_bf16_nt_masked(aq, sq, lm, w2q[0], w2q[1], out_rows, masked_m, G, max_m, H,
                                             I, expected)
    out = _empty(T, H)
    dg.combine_rows(out_rows, at, gate, h, out, T, H, top_k, G * max_m)
    return out


def reference_step(w, x, residual, targets, top_k, expert):
    """The training step by torch autograd in fp32, for comparison (experts as chosen)."""
    leaves = [t.float().requires_grad_()
              for t in (x.float() + residual.float(), w.norm, w.router, w.w1, w.w2, w.head)]
    h, wn, router, w1, w2, head = leaves
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * wn
    gate = torch.softmax(y @ router, dim=-1).gather(1, expert.long())
    out = h
    for e in range(w.experts):
        t, k = (expert == e).nonzero(as_tuple=True)
        g, u = (y[t] @ w1[e].t()).chunk(2, dim=-1)
        out = out.index_add(0, t, (g * torch.sigmoid(g) * u) @ w2[e].t() * gate[t, k][:, None])
    loss = torch.nn.functional.cross_entropy(out @ head.t(), targets.long(), reduction="none")
    loss.mean().backward()
    names = ("dx", "d_norm", "d_router", "dw1", "dw2", "d_head")
    return loss.detach(), out.detach(), dict(zip(names, (t.grad for t in leaves)))


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def run(tokens, hidden, inter, experts, top_k, seed=0, vocabulary=1000):
    """Both steps against the reference: a dict of relative errors (of the
    decoding step, that of what the layer adds to the residual stream)."""
    w = Weights(hidden, inter, experts, seed, vocabulary)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    rand = lambda scale: (torch.randn(tokens, hidden, generator=g, device="cuda") * scale).to(BF16)
    x, residual = rand(1.0), rand(2.0)
    targets = torch.randint(0, vocabulary, (tokens,), generator=g, device="cuda").to(torch.int32)
    loss, out, grads = train_step(w, x, residual, targets, top_k)
    expert = forward(w, x, residual, top_k)[1][5]
    want_loss, want, want_grads = reference_step(w, x, residual, targets, top_k, expert)
    base = x.float() + residual.float()
    err = {"loss": relative(loss, want_loss), "out": relative(out, want)}
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
    for name, default in (("tokens", 4096), ("hidden", 7168), ("inter", 2048), ("experts", 8), ("top-k", 2),
                          ("vocabulary", 32000)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    for k, v in run(a.tokens, a.hidden, a.inter, a.experts, a.top_k, vocabulary=a.vocabulary).items():
        print(f"{k:8s} relative error {v:.2e}")
    w = Weights(a.hidden, a.inter, a.experts, vocabulary=a.vocabulary)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(BF16)
    y = torch.randint(0, a.vocabulary, (a.tokens,), device="cuda").to(torch.int32)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(3):
        train_step(w, x, x, y, a.top_k)
    start.record()
    for _ in range(10):
        train_step(w, x, x, y, a.top_k)
    end.record()
    torch.cuda.synchronize()
    print(f"training step {start.elapsed_time(end) / 10:.2f} ms")


if __name__ == "__main__":
    main()
