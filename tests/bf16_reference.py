"""Definitions in 64 bits of the experts' bf16 products, their products with
4-bit weights and the router's choice, and the inputs their GPU tests share."""
from __future__ import annotations

import torch

import combine_ep_get_dispatch_amd as M
from experts_reference import spans

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E2M1 = E2M1 + [-v for v in E2M1]


def group_of(fmt):
    return 128 if fmt == M.W4_INT4 else 32


def unpack4(w, fmt):
    """Values float64 [..., k] of packed codes [..., k/2]."""
    lut = torch.arange(-8, 8, dtype=torch.float64) if fmt == M.W4_INT4 else torch.tensor(E2M1, dtype=torch.float64)
    lut = lut.to(w.device)
    return torch.stack([lut[(w & 15).long()], lut[(w >> 4).long()]], -1).flatten(-2)


def scales4(sc, fmt):
    """Scales [..., k/g, n] as float64 [..., n, k]."""
    real = sc.double() if fmt == M.W4_INT4 else torch.exp2(sc.double() - 127)
    return real.repeat_interleave(group_of(fmt), -2).transpose(-1, -2)


def weights4(w, sc, fmt):
    return unpack4(w, fmt) * scales4(sc, fmt)


def hint_for(E, N, K, field, tile):
    """expected_rows for which the plan takes this tile."""
    for rows in [*range(1, 64), *range(64, 2000, 5)]:
        if M.ep_bf16_plan_query(M.moedisp_rows.contiguous(E, 4096, rows), N, K)[field] == tile:
            return rows
    raise AssertionError(f"no hint takes {field} {tile}")


class Bf16Problem:
    """Rows, weights and bounds of one product on the GPU.  Every byte of the
    row buffers that no expert owns holds NaN, so that reading it shows."""

    def __init__(self, counts, N, K, seed=0, spare=5, padded=None, expected=0):
        g = self.g = torch.Generator().manual_seed(seed)
        self.counts, self.N, self.K = list(counts), N, K
        E = self.E = len(counts)
        if padded:
            stride, cap, base = padded
            self.rows = M.moedisp_rows.padded(E, cap, stride, base, expected)
            self.bounds = torch.tensor(counts, dtype=torch.int32).cuda()
            self.spans = spans(counts, stride, cap, base)
        else:
            self.rows = M.moedisp_rows.contiguous(E, sum(counts) + spare, expected)
            off = [0]
            for c in counts:
                off.append(off[-1] + c)
            self.bounds = torch.tensor(off, dtype=torch.int32).cuda()
            self.spans = spans(counts)
        R = self.R = self.rows.max_rows
        live = torch.zeros(R, dtype=torch.bool)
        for lo, c in self.spans:
            live[lo:lo + c] = True
        self.live = live.cuda()
        self.x, self.dy = self.rows_of(K), self.rows_of(N)
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def rows_of(self, width):
        x = torch.full((self.R, width), float("nan"))
        for lo, c in self.spans:
            x[lo:lo + c] = torch.randn(c, width, generator=self.g)
        return x.to(torch.bfloat16).cuda()

    def weights(self, layout):
        shape = (self.E, self.N, self.K) if layout == M.WEIGHTS_NK else (self.E, self.K, self.N)
        return torch.randn(*shape, generator=self.g).to(torch.bfloat16).cuda()

    def quantised(self, fmt):
        w = torch.randint(0, 256, (self.E, self.N, self.K // 2), generator=self.g, dtype=torch.uint8).cuda()
        if fmt == M.W4_INT4:
            sc = torch.exp(torch.randn(self.E, self.K // 128, self.N, generator=self.g)).to(torch.bfloat16)
        else:
            sc = torch.randint(120, 131, (self.E, self.K // 32, self.N), generator=self.g, dtype=torch.uint8)
        return w, sc.cuda()

    def _y(self, out_dtype, fill):
        dt = torch.float32 if out_dtype == M.FP32 else torch.bfloat16
        return torch.full((self.R, self.N), fill, dtype=dt, device="cuda")

    def gemm(self, w, layout, out_dtype, fill=7.0, stream=None):
        y = self._y(out_dtype, fill)
        M.ep_expert_gemm_bf16(self.rows, self.N, self.K, layout, self.x, w, self.bounds, y, out_dtype, self.ws, stream)
        return y

    def gemm4(self, w, sc, fmt, out_dtype, fill=7.0, stream=None):
        y = self._y(out_dtype, fill)
        M.ep_expert_gemm_w4(self.rows, self.N, self.K, fmt, self.x, w, sc, self.bounds, y, out_dtype, self.ws, stream)
        return y

    def product64(self, weights):
        """(y, sum of the products' magnitudes, sum of x's magnitudes) per row,
        zeros elsewhere; weights(e) is float64 [N][K]."""
        y = torch.zeros(self.R, self.N, dtype=torch.float64, device="cuda")
        s = torch.zeros_like(y)
        for e, (lo, c) in enumerate(self.spans):
            if c:
                x, w = self.x[lo:lo + c].double(), weights(e)
                y[lo:lo + c] = x @ w.t()
                s[lo:lo + c] = x.abs() @ w.abs().t()
        return y, s

    def wgrad(self, out_dtype, accumulate=False, dw=None):
        dt = torch.float32 if out_dtype == M.FP32 else torch.bfloat16
        if dw is None:
            dw = torch.full((self.E, self.N, self.K), 7.0, dtype=dt, device="cuda")
        M.ep_expert_wgrad_bf16(self.rows, self.N, self.K, self.x, self.dy, self.bounds, dw, out_dtype, accumulate,
                               self.ws)
        return dw

    def wgrad64(self):
        d = torch.zeros(self.E, self.N, self.K, dtype=torch.float64, device="cuda")
        s = torch.zeros_like(d)
        for e, (lo, c) in enumerate(self.spans):
            x, dy = self.x[lo:lo + c].double(), self.dy[lo:lo + c].double()
            d[e] = dy.t() @ x
            s[e] = dy.abs().t() @ x.abs()
        return d, s

    def status(self):
        return M.ep_check_status(self.ws)


def to41(v):
    """binary64 values to the nearest of 41 bits, as the choice compares them."""
    return ((v + 0.0).view(torch.int64) + 2048 & ~4095).view(torch.float64)


def router64(z, k, score, bias=None, live=None, groups=1, topk_groups=1, group_best=2, normalise=True, scale=1.0):
    """(idx, weights) of logits [T][E] in 64 bits; weights carry the gradient of z."""
    T, E = z.shape
    zd = z if z.dtype == torch.float64 else z.double()
    dead = ~(zd.detach() > -torch.inf)
    zz = torch.where(dead, -torch.inf, zd)
    if score == M.SCORE_SOFTMAX:
        p = torch.nan_to_num(torch.softmax(zz, 1), nan=0.0)
    else:
        p = torch.sigmoid(zz)
    with torch.no_grad():
        by_score = bias is not None or groups > 1
        key = p.detach().clone() if by_score else zz.detach().clone()
        if bias is not None:
            key = key + bias.double()
        if by_score:
            key = torch.where(torch.isfinite(key), to41(key), key)
        key = torch.where(dead | torch.isnan(key), -torch.inf, key)
        if groups > 1:
            v = key.view(T, groups, E // groups).sort(2, descending=True).values[..., :group_best]
            some = v[..., 0] > -torch.inf
            v = torch.where(v > -torch.inf, v, 0.0).sum(2)
            v = torch.where(some, torch.where(torch.isfinite(v), to41(v), v), -torch.inf)
            order = v.argsort(dim=1, descending=True, stable=True)[:, :topk_groups]
            kept = torch.zeros(T, groups, dtype=torch.bool, device=z.device).scatter_(1, order, True)
            key = torch.where(kept.repeat_interleave(E // groups, 1), key, -torch.inf)
        order = key.argsort(dim=1, descending=True, stable=True)[:, :k]
        taken = key.gather(1, order) > -torch.inf
        if live is not None:
            taken &= live.bool()[:, None]
    s = torch.where(taken, p.gather(1, order), 0.0)
    if normalise:
        # shares of scores that may vanish: of their logarithms
        lz = zz.gather(1, order)
        ls = lz if score == M.SCORE_SOFTMAX else torch.nn.functional.logsigmoid(lz)
        ls = torch.where(taken, ls, -torch.inf)
        w = torch.nan_to_num(torch.softmax(ls, 1), nan=0.0)
        w = torch.where(taken, w, 0.0)
    else:
        w = s
    return torch.where(taken, order, -1), scale * w
