"""Measured cases of the bf16 and 4-bit paths around dispatch and combine: the
experts' bf16 products with both gradients, their products with 4-bit weights,
the gated activation in bf16, and the router's choice with its gradient."""
import math

import torch

own = False

GROUP_E2M1 = 32     # channels per scale
GROUP_INT4 = 128


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(name, op, **kw):
    return dict(name=name, op=op, **kw)


def listed():
    return [
        # prefill, 4096 tokens top-8 over 256 experts: the gate-and-up product of
        # about 128 rows an expert, bound by the weights' bytes and the products alike
        _case("product_prefill", "product", T=4096, E=256, topk=8, K=7168, N=4096, wt="nk", out="bf16", zipf=0.0,
              mask=0.0),
        # a large batch over few experts, 4096 rows an expert: bound by arithmetic
        _case("product_large", "product", T=16384, E=8, topk=2, K=4096, N=8192, wt="nk", out="bf16", zipf=0.0,
              mask=0.0),
        # the gradient of the down product's rows under skewed routing with masked
        # slots, from the weights as they lie: experts from none to thousands of rows
        _case("product_gradient", "product", T=4096, E=256, topk=8, K=7168, N=2048, wt="kn", out="bf16", zipf=1.2,
              mask=0.05),
        # weight gradients of a large batch over few experts
        _case("wgrad_large", "wgrad", T=16384, E=8, topk=2, K=4096, N=4096, out="bf16", zipf=0.0, mask=0.0),
        # weight gradients of many experts with few rows, sizes that fill no tile,
        # in fp32: bound by the writes
        _case("wgrad_many", "wgrad", T=2048, E=64, topk=4, K=1992, N=7176, out="fp32", zipf=1.2, mask=0.05),
        # one token top-8 over 256 experts: eight matrix-vector products
        _case("w4_token", "w4", T=1, E=256, topk=8, K=7168, N=4096, fmt="e2m1", out="bf16", layout="contiguous",
              capacity=0, zipf=0.0, mask=0.0),
        # a decode step of 128 tokens in the padded layout, about 4 rows an expert
        _case("w4_decode", "w4", T=128, E=256, topk=8, K=7168, N=4096, fmt="e2m1", out="bf16", layout="padded",
              capacity=64, zipf=0.0, mask=0.0),
        # a batch of 500 tokens over 8 experts, 4-bit integers, a last column tile that is cut
        _case("w4_batch", "w4", T=500, E=8, topk=2, K=4096, N=8208, fmt="int4", out="bf16", layout="contiguous",
              capacity=0, zipf=0.0, mask=0.05),
        # the activation between the two products of a prefill step
        _case("swiglu_prefill", "swiglu", T=4096, E=256, topk=8, I=2048, mask=0.0),
        # and of the tiny configuration: latency
        _case("swiglu_tiny", "swiglu", T=128, E=8, topk=2, I=256, mask=0.1),
        # the choice of a decode step: sigmoid scores, a bias that balances, 4 of 8 groups
        _case("router_decode", "router", T=128, E=256, topk=8, score="sigmoid", dtype="fp32", bias=True, groups=8,
              topk_groups=4, group_best=2, normalise=True, backward=False, pad=0.0),
        # the choice and its gradient in a large training batch of padded sequences, bf16 logits
        _case("router_training", "router", T=131072, E=256, topk=8, score="softmax", dtype="bf16", bias=False,
              groups=1, topk_groups=1, group_best=1, normalise=False, backward=True, pad=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "wgrad", "w4", "w4", "swiglu", "router", "router"])
    if op == "router":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.randint(4, 32) if groups > 1 else rng.choice([8, 16, 60, 64, 100, 128, 160, 256])
        topk_groups = rng.randint(1, groups)
        return dict(op=op, T=_log_int(rng, 1, 32768), E=E, topk=rng.randint(1, min(8, E // groups * topk_groups)),
                    score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["fp32", "bf16"]),
                    bias=rng.random() < 0.5, groups=groups, topk_groups=topk_groups, group_best=rng.choice([1, 2]),
                    normalise=rng.random() < 0.5, backward=rng.random() < 0.7, pad=rng.choice([0.0, 0.1, 0.5]))
    E = rng.randint(2, 64)
    topk = rng.randint(1, min(8, E))
    mask = rng.choice([0.0, 0.05, 0.3])
    if op == "swiglu":
        return dict(op=op, T=_log_int(rng, 1, 4096), E=E, topk=topk, I=128 * rng.randint(1, 16), mask=mask)
    zipf = rng.choice([0.0, 0.0, 1.2])
    out = rng.choice(["bf16", "fp32"])
    if op == "w4":
        T = _log_int(rng, 1, 512)
        padded = rng.random() < 0.5
        return dict(op=op, T=T, E=E, topk=topk, K=128 * rng.randint(1, 32), N=16 * _log_int(rng, 1, 256),
                    fmt=rng.choice(["e2m1", "int4"]), out=out, layout="padded" if padded else "contiguous",
                    capacity=T + rng.randint(0, 7) if padded else 0, zipf=zipf, mask=mask)
    K, N = 8 * _log_int(rng, 1, 512), 8 * _log_int(rng, 1, 512)
    T = _log_int(rng, 1, 4096)
    if op == "wgrad":
        return dict(op=op, T=T, E=E, topk=topk, K=K, N=N, out=out, zipf=zipf, mask=mask)
    return dict(op=op, T=T, E=E, topk=topk, K=K, N=N, wt=rng.choice(["nk", "kn"]), out=out, zipf=zipf, mask=mask)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6841 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _routing(g, T, E, topk, zipf, mask):
    """int32 [T][topk]: distinct experts per token, -1 in the masked share of the slots."""
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    keys = -torch.log(-torch.log(u))
    if zipf > 0:
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1
        keys = keys - zipf * torch.log(rank)
    idx = keys.topk(topk, dim=1).indices.to(torch.int32).contiguous()
    masked = round(mask * T * topk)
    idx.view(-1)[torch.randperm(T * topk, generator=g, device="cuda")[:masked]] = -1
    return idx


def _weights(g, *shape):
    """bf16 weights of variance 1/channels, expert by expert."""
    w = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    for e in range(shape[0]):
        w[e] = _randn(g, *shape[1:])
    return w


def _quantised(g, fmt, N, K):
    """N(0, 1) weights as 4-bit codes uint8 [N][K/2] (low half first): nearest
    multiples of 1/2 sigma (e2m1) or of 0.4 sigma (int4)."""
    v = _randn(g, N, K)
    if fmt == "int4":
        c = (v * 2.5).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
    else:
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
        c = torch.bucketize(v.abs() * 2, edges, out_int32=True).to(torch.uint8)
        c |= (v < 0).to(torch.uint8) << 3
    return c[:, 0::2] | (c[:, 1::2] << 4)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=dict(case))
    op = case["op"]
    T, E, k = case["T"], case["E"], case["topk"]
    if op == "router":
        dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        s["logits"] = _randn(g, T, E).to(dt)
        s["bias"] = 0.1 * _randn(g, E) if case["bias"] else None
        # padding tokens have no choice
        s["live"] = (torch.rand(T, generator=g, device="cuda") >= case["pad"]).to(torch.uint8) if case["pad"] else None
        s["d_weights"] = _randn(g, T, k)
        s["idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(T, k, device="cuda")
        s["d_logits"] = torch.empty_like(s["logits"])
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return s
    idx = _routing(g, T, E, k, case.get("zipf", 0.0), case["mask"]).reshape(-1).long()
    counts = torch.bincount(idx[idx >= 0], minlength=E).to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    s["counts"], s["offsets"] = counts, offsets
    s["host_counts"] = counts.tolist()
    s["R"] = int(offsets[-1])
    s["most"] = max(s["host_counts"])
    s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    if op == "swiglu":
        s["gu"] = _randn(g, T * k, 2 * case["I"]).to(torch.bfloat16)
        s["h"] = torch.empty(T * k, case["I"], dtype=torch.bfloat16, device="cuda")
        return s
    K, N = case["K"], case["N"]
    odt = torch.float32 if case["out"] == "fp32" else torch.bfloat16
    rows = E * case["capacity"] if case.get("layout") == "padded" else T * k
    s["x"] = _randn(g, rows, K).to(torch.bfloat16)
    if op == "wgrad":
        s["dy"] = _randn(g, rows, N).to(torch.bfloat16)
        s["dw"] = torch.zeros(E, N, K, dtype=odt, device="cuda")
        return s
    s["y"] = torch.zeros(rows, N, dtype=odt, device="cuda")
    if op == "product":
        s["w"] = _weights(g, E, N, K) if case["wt"] == "nk" else _weights(g, E, K, N)
        return s
    s["w"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    for e in range(E):
        s["w"][e] = _quantised(g, case["fmt"], N, K)
    if case["fmt"] == "int4":
        s["scales"] = (0.4 / math.sqrt(K) * torch.exp(0.2 * _randn(g, E, K // GROUP_INT4, N))).to(torch.bfloat16)
    else:
        e0 = 127 + round(math.log2(0.5 / math.sqrt(K)))
        s["scales"] = (e0 + torch.randint(-1, 2, (E, K // GROUP_E2M1, N), generator=g, device="cuda")).to(torch.uint8)
    return s


# ---------------------------------------------------------------------------
# the operators: the framework's calls, or elementary torch operations
# ---------------------------------------------------------------------------

def run(s):
    return {"product": _product, "wgrad": _wgrad, "w4": _w4, "swiglu": _swiglu, "router": _router}[s["case"]["op"]](s)


def _rows(M, c):
    if c.get("layout") == "padded":
        return M.moedisp_rows.padded(c["E"], c["capacity"], expected_rows=-(-c["T"] * c["topk"] // c["E"]))
    return M.moedisp_rows.contiguous(c["E"], c["T"] * c["topk"])


def _out(M, c):
    return M.FP32 if c["out"] == "fp32" else M.BF16


def _by_expert(rows, s):
    """Contiguous rows [R][*] as float [E][most][*], zeros past an expert's count."""
    i = torch.arange(s["most"], device=rows.device)
    valid = i[None, :] < s["counts"][:, None]
    at = torch.where(valid, s["offsets"][:-1, None] + i[None, :], 0).long()
    return torch.where(valid[..., None], rows[at].float(), 0.0), valid


def _product(s):
    c = s["case"]
    if own:
        import combine_ep_get_dispatch_amd as M
        M.ep_expert_gemm_bf16(_rows(M, c), c["N"], c["K"], M.WEIGHTS_NK if c["wt"] == "nk" else M.WEIGHTS_KN, s["x"],
                              s["w"], s["offsets"], s["y"], _out(M, c), s["ws"])
        return s["y"][:s["R"]]
    x, valid = _by_expert(s["x"], s)
    w = s["w"].float()
    return torch.bmm(x, w.transpose(1, 2) if c["wt"] == "nk" else w)[valid].to(s["y"].dtype)


def _wgrad(s):
    c = s["case"]
    if own:
        import combine_ep_get_dispatch_amd as M
        M.ep_expert_wgrad_bf16(_rows(M, c), c["N"], c["K"], s["x"], s["dy"], s["offsets"], s["dw"], _out(M, c), False,
                               s["ws"])
        return s["dw"]
    x, _ = _by_expert(s["x"], s)
    dy, _ = _by_expert(s["dy"], s)
    return torch.bmm(dy.transpose(1, 2), x).to(s["dw"].dtype)


def _codes(w, fmt):
    """float32 [N][K] of packed codes [N][K/2]."""
    c = torch.stack([w & 15, w >> 4], -1).view(w.shape[0], -1)
    if fmt == "int4":
        return c.float() - 8
    m = (c & 7).float()     # 0, 0.5, 1, 1.5, 2, 3, 4, 6
    m = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    return torch.where(c >= 8, -m, m)


def _scales(sc, fmt, K):
    """float32 [N][K] of the scales [K/group][N]."""
    if fmt == "int4":
        return sc.float().repeat_interleave(GROUP_INT4, 0).t()
    return torch.ldexp(torch.ones((), device=sc.device), sc.int() - 127).repeat_interleave(GROUP_E2M1, 0).t()


def _spans(s):
    """(expert, first row, rows) of the experts with rows."""
    c, at = s["case"], 0
    for e, n in enumerate(s["host_counts"]):
        if n:
            yield e, e * c["capacity"] if c["layout"] == "padded" else at, n
        at += n


def _w4(s):
    c = s["case"]
    padded = c["layout"] == "padded"
    if own:
        import combine_ep_get_dispatch_amd as M
        M.ep_expert_gemm_w4(_rows(M, c), c["N"], c["K"], M.W4_INT4 if c["fmt"] == "int4" else M.W4_E2M1, s["x"],
                            s["w"], s["scales"], s["counts"] if padded else s["offsets"], s["y"], _out(M, c), s["ws"])
        return s["y"] if padded else s["y"][:s["R"]]
    y = torch.zeros_like(s["y"])
    for e, lo, n in _spans(s):
        w = _codes(s["w"][e], c["fmt"]) * _scales(s["scales"][e], c["fmt"], c["K"])
        y[lo:lo + n] = (s["x"][lo:lo + n].float() @ w.t()).to(y.dtype)
    return y if padded else y[:s["R"]]


def _swiglu(s):
    c = s["case"]
    R, I = s["R"], c["I"]
    if own:
        import combine_ep_get_dispatch_amd as M
        M.ep_swiglu(_rows(M, c), I, s["gu"], s["offsets"], s["h"], s["ws"])
        return s["h"][:R]
    g, u = s["gu"][:R, :I].float(), s["gu"][:R, I:].float()
    return (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)


SCALE = 2.5


def _best(v, n):
    """Indices of the n largest of each row, the lowest index first among equals."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[..., :n]


def _router(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["topk"]
    if own:
        import combine_ep_get_dispatch_amd as M
        r = M.moedisp_router.make(T, E, k, M.SCORE_SOFTMAX if c["score"] == "softmax" else M.SCORE_SIGMOID,
                                  M.FP32 if c["dtype"] == "fp32" else M.BF16, groups=c["groups"],
                                  topk_groups=c["topk_groups"], group_best=c["group_best"], normalise=c["normalise"],
                                  scale=SCALE)
        M.ep_router_topk(r, s["logits"], s["bias"], s["live"], s["idx"], s["weights"])
        if not c["backward"]:
            return s["idx"], s["weights"]
        M.ep_router_topk_backward(r, s["logits"], s["idx"], s["d_weights"], s["d_logits"], s["ws"])
        return s["idx"], s["weights"], s["d_logits"]
    z = s["logits"].float()
    soft = c["score"] == "softmax"
    # the choice, in 64 bits: values next to a border
    choice = z.double()
    if s["bias"] is not None or c["groups"] > 1:
        if soft:
            ex = torch.exp(choice - choice.amax(1, keepdim=True))
            choice = ex / ex.sum(1, keepdim=True)
        else:
            choice = 1 / (1 + torch.exp(-choice))
        if s["bias"] is not None:
            choice = choice + s["bias"].double()
    if c["groups"] > 1:
        per = E // c["groups"]
        by_group = choice.view(T, c["groups"], per)
        value = by_group.gather(2, _best(by_group, min(c["group_best"], per))).sum(-1)
        kept = torch.zeros(T, c["groups"], dtype=torch.bool, device=z.device)
        kept.scatter_(1, _best(value, c["topk_groups"]), True)
        choice = torch.where(kept.repeat_interleave(per, 1), choice, -math.inf)
    idx = _best(choice, k)
    # the chosen experts' weights
    if soft:
        ex = torch.exp(z - z.amax(1, keepdim=True))
        score = ex / ex.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-z))
    p = score.gather(1, idx)
    share = p / p.sum(1, keepdim=True) if c["normalise"] else p
    live = torch.ones(T, 1, dtype=torch.bool, device=z.device) if s["live"] is None else s["live"].bool()[:, None]
    out = (torch.where(live, idx, -1).to(torch.int32), torch.where(live, SCALE * share, 0.0))
    if not c["backward"]:
        return out
    gr = SCALE * s["d_weights"]
    mean = (gr * share).sum(1, keepdim=True)
    if c["normalise"]:
        d = share * (gr - mean) * (1.0 if soft else 1 - p)
    else:
        d = gr * p * (1.0 if soft else 1 - p)
    dz = torch.zeros_like(z).scatter_(1, idx, d)
    if soft and not c["normalise"]:
        dz = dz - score * mean
    return (*out, torch.where(live, dz, 0.0).to(s["logits"].dtype))


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _hit(case):
    """Experts with at least one row, for routing by the case's law."""
    p = [1.0 / (r + 1) ** case["zipf"] for r in range(case["E"])]
    tot = sum(p)
    return sum(1 - (1 - min(1.0, case["topk"] * (1 - case["mask"]) * q / tot)) ** case["T"] for q in p)


def work(case):
    op = case["op"]
    T, E, k = case["T"], case["E"], case["topk"]
    if op == "router":
        eb = 4 if case["dtype"] == "fp32" else 2
        # the choice reads the logits; the gradient reads a softmax row again where the weights are not normalised,
        # else the chosen logits, and writes a row
        b = T * (E * eb + 8 * k)
        if case["backward"]:
            again = E if case["score"] == "softmax" and not case["normalise"] else k
            b += T * (again * eb + 8 * k + E * eb)
        return {"bytes": b, "flops": T * E * (20.0 if case["backward"] else 10.0)}
    R = T * k - round(case["mask"] * T * k)
    if op == "swiglu":
        return {"bytes": R * case["I"] * 6, "flops": 8.0 * R * case["I"]}
    K, N = case["K"], case["N"]
    ob = 4 if case["out"] == "fp32" else 2
    flops = 2.0 * R * N * K
    if op == "wgrad":
        return {"bytes": R * (N + K) * 2 + E * N * K * ob, "flops": flops}
    if op == "product":
        return {"bytes": R * K * 2 + _hit(case) * N * K * 2 + R * N * ob, "flops": flops}
    sb = 2 * K // GROUP_INT4 if case["fmt"] == "int4" else K // GROUP_E2M1
    return {"bytes": R * K * 2 + _hit(case) * N * (K // 2 + sb) + R * N * ob, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _lut(fmt):
    if fmt == "int4":
        return torch.arange(-8, 8, dtype=torch.float64, device="cuda")
    half = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(half + [-v for v in half], dtype=torch.float64, device="cuda")


def _w64(w, sc, fmt):
    lut = _lut(fmt)
    N = w.shape[0]
    v = torch.empty(N, 2 * w.shape[1], dtype=torch.float64, device="cuda")
    v[:, 0::2] = lut[(w & 15).int()]
    v[:, 1::2] = lut[(w >> 4).int()]
    real = sc.double() if fmt == "int4" else torch.exp2(sc.double() - 127)
    v.view(N, sc.shape[0], -1).mul_(real.t()[..., None])
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "router":
        return _router64(case, s)
    if op == "swiglu":
        g, u = s["gu"][:s["R"]].double().chunk(2, dim=1)
        return g * torch.sigmoid(g) * u
    N, K = case["N"], case["K"]
    out = torch.zeros_like(s["dw"] if op == "wgrad" else s["y"], dtype=torch.float64)
    at = 0
    for e, n in enumerate(s["host_counts"]):
        lo = e * case["capacity"] if case.get("layout") == "padded" else at
        at += n
        if not n:
            continue
        x = s["x"][lo:lo + n].double()
        if op == "wgrad":
            out[e] = s["dy"][lo:lo + n].double().t() @ x
        elif op == "w4":
            out[lo:lo + n] = x @ _w64(s["w"][e], s["scales"][e], case["fmt"]).t()
        else:
            w = s["w"][e].double()
            out[lo:lo + n] = x @ (w.t() if case["wt"] == "nk" else w)
    return out if op == "wgrad" or case.get("layout") == "padded" else out[:s["R"]]


def _router64(case, s):
    T, E, k, G = case["T"], case["E"], case["topk"], case["groups"]
    z = s["logits"].double().requires_grad_()
    score = torch.softmax(z, 1) if case["score"] == "softmax" else torch.sigmoid(z)
    with torch.no_grad():
        key = z.detach().clone() if s["bias"] is None and G == 1 else score.detach().clone()
        if s["bias"] is not None:
            key += s["bias"].double()
        if G > 1:
            grp = torch.arange(E, device="cuda") // (E // G)
            ranked = torch.sort(key.view(T, G, -1), dim=2, descending=True).values
            of_group = ranked[..., :case["group_best"]].sum(2)
            order = torch.argsort(of_group, dim=1, descending=True, stable=True)
            rank = torch.empty_like(order).scatter_(1, order, torch.arange(G, device="cuda").expand(T, G))
            key[(rank >= case["topk_groups"])[:, grp]] = -math.inf
        idx = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
    live = s["live"].bool() if s["live"] is not None else torch.ones(T, dtype=torch.bool, device="cuda")
    picked = score.gather(1, idx)
    wt = SCALE * (picked / picked.sum(1, keepdim=True) if case["normalise"] else picked) * live[:, None]
    idx = torch.where(live[:, None], idx, -1)
    if not case["backward"]:
        return idx, wt.detach()
    (wt * s["d_weights"].double()).sum().backward()
    return idx, wt.detach(), z.grad
