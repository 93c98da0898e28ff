"""Definitions in 64 bits of the experts' products, the gated activation and
the balance loss, and the inputs their GPU tests share."""
from __future__ import annotations

import torch

import combine_ep_get_dispatch_amd as M

E4M3 = torch.float8_e4m3fn


def scales64(sc):
    if sc.dtype == torch.float32:
        return sc.double()
    return torch.exp2(sc.double() - 127)


def rows64(x, sc):
    """Dequantised rows [R][K]."""
    return x.double() * scales64(sc).repeat_interleave(128, -1)


def weights64(w, sc):
    n = w.shape[-2]
    return w.double() * scales64(sc).repeat_interleave(128, -1).repeat_interleave(128, -2)[..., :n, :]


def spans(counts, stride=0, cap=0, base=0):
    """(first row, rows) per expert."""
    if stride:
        return [(e * stride + base, min(c, cap)) for e, c in enumerate(counts)]
    out, at = [], 0
    for c in counts:
        out.append((at, c))
        at += c
    return out


class Problem:
    """Rows, weights and bounds of one product on the GPU.  Every byte of the
    row buffers that no expert owns holds NaN, so that reading it shows."""

    def __init__(self, counts, N, K, fmt, seed=0, spare=5, padded=None, expected=0):
        g = torch.Generator().manual_seed(seed)
        self.counts, self.N, self.K, self.fmt = list(counts), N, K, fmt
        E = self.E = len(counts)
        if padded:
            stride, cap, base = padded
            self.rows = M.moedisp_rows.padded(E, cap, stride, base, expected)
            self.bounds = torch.tensor(counts, dtype=torch.int32).cuda()
            self.spans = spans(counts, stride, cap, base)
        else:
            R = sum(counts) + spare
            self.rows = M.moedisp_rows.contiguous(E, R, expected)
            off = [0]
            for c in counts:
                off.append(off[-1] + c)
            self.bounds = torch.tensor(off, dtype=torch.int32).cuda()
            self.spans = spans(counts)
        R = self.R = self.rows.max_rows
        kb, nb = K // 128, -(-N // 128)
        x = torch.full((R, K), 0x7F, dtype=torch.uint8).view(E4M3)
        xs = torch.full((R, kb), float("nan")) if fmt == M.SCALE_FP32 else torch.full((R, kb), 255, dtype=torch.uint8)
        live = torch.zeros(R, dtype=torch.bool)
        for lo, c in self.spans:
            live[lo:lo + c] = True
            x[lo:lo + c] = (torch.randn(c, K, generator=g) * 150).clamp(-448, 448).to(E4M3)
            xs[lo:lo + c] = self._scales(g, c, kb)
        self.live = live.cuda()
        self.x, self.xs = x.cuda(), xs.cuda()
        self.w = (torch.randn(E, N, K, generator=g) * 150).clamp(-448, 448).to(E4M3).cuda()
        self.ws_ = self._scales(g, E, nb, kb).cuda()
        self.dy = torch.full((R, N), float("nan"), dtype=torch.bfloat16)
        for lo, c in self.spans:
            self.dy[lo:lo + c] = torch.randn(c, N, generator=g).to(torch.bfloat16)
        self.dy = self.dy.cuda()
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def _scales(self, g, *shape):
        if self.fmt == M.SCALE_FP32:
            return torch.exp(torch.randn(*shape, generator=g)) / 150
        return torch.randint(115, 124, shape, generator=g, dtype=torch.uint8)

    def gemm(self, out_dtype, fill=7.0, stream=None):
        dt = torch.float32 if out_dtype == M.FP32 else torch.bfloat16
        y = torch.full((self.R, self.N), fill, dtype=dt, device="cuda")
        M.ep_expert_gemm(self.rows, self.N, self.K, self.fmt, self.x, self.xs, self.w, self.ws_, self.bounds, y,
                         out_dtype, self.ws, stream)
        return y

    def gemm64(self):
        """(y, sum of the products' magnitudes) per row, zeros elsewhere."""
        y = torch.zeros(self.R, self.N, dtype=torch.float64, device="cuda")
        s = torch.zeros_like(y)
        for e, (lo, c) in enumerate(self.spans):
            x, w = rows64(self.x[lo:lo + c], self.xs[lo:lo + c]), weights64(self.w[e], self.ws_[e])
            y[lo:lo + c] = x @ w.t()
            s[lo:lo + c] = x.abs() @ w.abs().t()
        return y, s

    def wgrad(self, out_dtype, accumulate=False, dw=None):
        dt = torch.float32 if out_dtype == M.FP32 else torch.bfloat16
        if dw is None:
            dw = torch.full((self.E, self.N, self.K), 7.0, dtype=dt, device="cuda")
        M.ep_expert_wgrad(self.rows, self.N, self.K, self.fmt, self.x, self.xs, self.dy, self.bounds, dw, out_dtype,
                          accumulate, self.ws)
        return dw

    def wgrad64(self):
        d = torch.zeros(self.E, self.N, self.K, dtype=torch.float64, device="cuda")
        s = torch.zeros_like(d)
        for e, (lo, c) in enumerate(self.spans):
            x, dy = rows64(self.x[lo:lo + c], self.xs[lo:lo + c]), self.dy[lo:lo + c].double()
            d[e] = dy.t() @ x
            s[e] = dy.abs().t() @ x.abs()
        return d, s

    def status(self):
        return M.ep_check_status(self.ws)


def swiglu64(gu):
    g, u = gu.double().chunk(2, -1)
    return g * torch.sigmoid(g) * u


def swiglu_backward64(gu, dh):
    g, u = gu.double().chunk(2, -1)
    s, d = torch.sigmoid(g), dh.double()
    return torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], -1)


def balance64(z, idx, S, k, coef, score, d_loss=1.0):
    """(loss, counts, tokens, d_logits) of logits [S*L][E] in 64 bits."""
    T, E = z.shape
    L = T // S if S else 0
    z = z.double().view(S, L, E)
    idx = idx.view(S, L, k).long()
    if score == M.SCORE_SOFTMAX:
        p, slope = torch.softmax(z, -1), 1.0
    else:
        sg = torch.sigmoid(z)
        p, slope = sg / sg.sum(-1, keepdim=True), 1 - sg
    p = torch.nan_to_num(p, nan=0.0)
    live = (idx >= 0).any(-1)
    p = p * live[..., None]
    counts = torch.stack([torch.bincount(i[i >= 0], minlength=E) for i in idx]) if S else torch.zeros(0, E)
    n = live.sum(1).double()
    some = (n > 0).sum().clamp(min=1)
    w = coef * E * counts.double() / (some * k * n.clamp(min=1)[:, None] ** 2)
    loss = (w * p.sum(1)).sum()
    w = (w * d_loss)[:, None, :]
    dz = p * slope * (w - (p * w).sum(-1, keepdim=True))
    return loss, counts, n.long(), dz.view(T, E)
