"""Experts in 16 bits, their gradients and low-rank adapters, measured.

Five operators beside the compressed path:

  product       grouped product of rows with 16-bit expert weights, with a
                SwiGLU (optionally keeping what enters it) or a plain epilogue
  grad_rows     its gradient by the rows: dY W_e, plain or continued through
                the SwiGLU that made the product's input
  grad_weights  its gradient by the weights: dW_e = sum over the expert's rows
                of dY^T A, zeros for an expert without rows
  combine_grad  the gradient of the gate-weighted combine by the experts'
                outputs, the gates and the router's logits
  adapters      low-rank adapters of many requests added to a shared
                projection's output: out_t = y_t + s_a B_a (A_a x_t), a the
                adapter of token t's request, out_t = y_t where it has none

`own` false: plain forms, elementary torch operations in 32 bits, one rounding
at the end.  `own` true: the library's calls.
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one token through gate/up of a 64-expert layer: the shortest call, 8 experts' weights are read
        dict(name="product_token", op="product", T=1, k=8, E=64, N=2048, K=2048, dtype="bf16", epi="swiglu", pre=False,
             zipf=False),
        # a decode batch's down product: few rows an expert, popular ones fuller
        dict(name="product_decode", op="product", T=32, k=8, E=64, N=2048, K=1024, dtype="bf16", epi="fp16", pre=False,
             zipf=True),
        # gate/up of a training batch, what enters the SwiGLU is kept for the gradient
        dict(name="product_batch", op="product", T=8192, k=8, E=64, N=2048, K=2048, dtype="bf16", epi="swiglu", pre=True,
             zipf=False),
        # down of the wide experts, about 128 rows each
        dict(name="product_wide", op="product", T=512, k=2, E=8, N=4096, K=14336, dtype="fp16", epi="fp16", pre=False,
             zipf=False),
        # from the experts' outputs back through down and the SwiGLU, the training batch
        dict(name="grad_rows_batch", op="grad_rows", T=8192, k=8, E=64, N=2048, K=1024, dtype="bf16", epi="swiglu_grad",
             zipf=False),
        # back through gate/up of the wide experts, uneven segments, an odd number of tokens
        dict(name="grad_rows_wide", op="grad_rows", T=509, k=2, E=8, N=28672, K=4096, dtype="fp16", epi="fp16", zipf=True),
        # gate/up weights' gradient of the training batch
        dict(name="grad_weights_batch", op="grad_weights", T=8192, k=8, E=64, N=2048, K=2048, dtype="bf16", out="bf16",
             zipf=False),
        # few rows for many weights: the wide experts' down weights, kept in 32 bits
        dict(name="grad_weights_wide", op="grad_weights", T=509, k=2, E=8, N=4096, K=14336, dtype="bf16", out="fp32",
             zipf=True),
        # a small odd batch: the launch
        dict(name="combine_grad_few", op="combine_grad", T=33, k=8, E=64, H=2048, dtype="bf16", none=0.0),
        # the training batch
        dict(name="combine_grad_batch", op="combine_grad", T=8192, k=8, E=64, H=2048, dtype="bf16", none=0.0),
        # a decode step of 32 requests over 16 adapters, some requests without one
        dict(name="adapters_decode", op="adapters", T=32, n=16, K=4096, N=4096, r=16, dtype="bf16", run=1, none=0.2),
        # 256 requests of 16 tokens before the wide projection, 16 adapters by popularity
        dict(name="adapters_prompt", op="adapters", T=4096, n=16, K=4096, N=14336, r=32, dtype="bf16", run=16, none=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["product", "product", "grad_rows", "grad_weights", "combine_grad", "adapters"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "combine_grad":
        H, k = 8 * _log(rng, 16, 512), rng.randint(1, 8)
        E = max(k, _log(rng, 4, 256))
        return dict(op=op, T=_log(rng, 1, min(8192, 134_000_000 // (H * k))), k=k, E=E, H=H, dtype=dtype,
                    none=rng.choice([0.0, 0.0, 0.1]))
    if op == "adapters":
        K, N = 8 * _log(rng, 32, 1792), 8 * _log(rng, 32, 1792)
        return dict(op=op, T=_log(rng, 1, min(8192, 75_000_000 // (K + N))), n=_log(rng, 1, 64), K=K, N=N,
                    r=8 * _log(rng, 1, 16), dtype=dtype, run=rng.choice([1, 1, 7, 64]), none=rng.choice([0.0, 0.2]))
    # no more weights than the wide layer's, no more products or rows than the training batch's
    E, k, zipf = _log(rng, 1, 64), rng.randint(1, 8), rng.random() < 0.4
    N, K = 16 * _log(rng, 4, 256), 8 * _log(rng, 8, 1024)
    E = max(1, min(E, 450_000_000 // (N * K)))
    k = min(k, E)
    T = _log(rng, 1, min(8192, 270_000_000_000 // (k * N * K), 450_000_000 // (k * (N + 4 * K))))
    c = dict(op=op, T=T, k=k, E=E, N=N, K=K, dtype=dtype, zipf=zipf)
    if op == "product":
        epi = rng.choice(["swiglu", "swiglu", "bf16", "fp16"])
        return dict(c, epi=epi, pre=epi == "swiglu" and rng.random() < 0.5)
    if op == "grad_rows":
        return dict(c, epi=rng.choice(["swiglu_grad", "swiglu_grad", "bf16", "fp16"]))
    return dict(c, out=rng.choice(["bf16", "fp16", "fp32"]))


# -------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _acts(g, rows, width):
    """Normal activations with a few strong channels, as a residual stream has."""
    x = torch.randn(rows, width, generator=g, device=DEV)
    strong = torch.rand(width, generator=g, device=DEV) < 0.01
    return x * torch.where(strong, 8.0, 1.0)


def _logits(g, T, E, zipf):
    x = torch.randn(T, E, generator=g, device=DEV)
    if zipf:
        rank = torch.randperm(E, generator=g, device=DEV).float() + 1
        x = x - 1.1 * torch.log(rank)
    return x


def _weights(g, n, N, K, dt):
    w = torch.empty(n, N, K, dtype=dt, device=DEV)
    for e in range(n):
        w[e] = torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K)
    return w


def _grouping(s, flat, E):
    """(token, slot) pairs by expert (an id outside 0..E-1 after the others), as the library's grouping gives them."""
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    s["pairs"] = torch.sort(key, stable=True).indices.int()
    s["pos"] = torch.sort(s["pairs"].long()).indices.int()
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    s["most"] = max(1, int(counts.max()))  # rows of the fullest segment, for the plain form's padding
    s["valid"] = int(counts.sum())


def prepare(case, seed):
    g, c = _gen(seed), case
    s, dt, op = dict(case=c), DTYPES[c["dtype"]], c["op"]
    if op == "adapters":
        runs = -(-c["T"] // c["run"])
        ids = torch.sort(_logits(g, runs, c["n"], True), dim=-1, descending=True).indices[:, 0]
        ids = torch.where(torch.rand(runs, generator=g, device=DEV) < c["none"], -1, ids)
        _grouping(s, ids.repeat_interleave(c["run"])[: c["T"]], c["n"])
        s["x"] = _acts(g, c["T"], c["K"]).to(dt)
        s["y"] = torch.randn(c["T"], c["N"], generator=g, device=DEV).to(dt)
        s["A"] = _weights(g, c["n"], c["r"], c["K"], dt)
        s["B"] = _weights(g, c["n"], c["N"], c["r"], dt)
        s["scale"] = 0.5 + torch.rand(c["n"], generator=g, device=DEV)
        return s
    logits = _logits(g, c["T"], c["E"], c.get("zipf", False))
    top = torch.sort(logits, dim=-1, descending=True)
    ids = top.indices[:, : c["k"]].int()
    P = c["T"] * c["k"]
    if op == "combine_grad":
        ids = torch.where(torch.rand(ids.shape, generator=g, device=DEV) < c["none"], -1, ids)
        s["w"] = torch.softmax(top.values[:, : c["k"]], -1)
        s["ids"] = ids.contiguous()
        s["dout"] = torch.randn(c["T"], c["H"], generator=g, device=DEV).to(torch.bfloat16)
        s["y"] = torch.randn(P, c["H"], generator=g, device=DEV).to(torch.float16)
        _grouping(s, ids.flatten().long(), c["E"])
        return s
    _grouping(s, ids.flatten().long(), c["E"])
    if op != "grad_weights":
        s["w"] = _weights(g, c["E"], c["N"], c["K"], dt)
    if op != "grad_rows":
        s["a"] = _acts(g, c["T"], c["K"]).to(dt)
    if op != "product":
        s["dy"] = torch.randn(P, c["N"], generator=g, device=DEV).to(dt)
    if c.get("epi") == "swiglu_grad":
        s["pre"] = torch.randn(P, 2 * c["K"], generator=g, device=DEV).to(dt)
    return s


# --------------------------------------------------------------- plain forms
def _slots(offsets, rows, most):
    """Where the grouped rows lie when every segment is padded to `most` rows."""
    i = torch.arange(rows, device=DEV)
    e = torch.searchsorted(offsets[1:].contiguous(), i.int(), right=True)
    return e * most + i - offsets[e]


def _padded(a, slot, E, most):
    out = a.new_zeros(E * most, a.shape[1])
    out[slot] = a
    return out.view(E, most, -1)


def _swiglu_grad(dh, pre):
    g, u = pre.float().chunk(2, -1)
    sig = 1 / (1 + torch.exp(-g))
    return torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], -1)


def _run_plain(s, c):
    op = c["op"]
    if op == "combine_grad":
        T, k, nv = c["T"], c["k"], s["valid"]
        live = (s["pos"] < nv).view(T, k)
        dout = s["dout"].float()
        y = s["y"].float()[s["pos"].long()].view(T, k, -1)
        dw = torch.where(live, (y * dout[:, None]).sum(-1), 0.0)
        at = s["pairs"][:nv].long()
        dy = dout[at // k] * s["w"].flatten()[at][:, None]
        dl = s["w"] * (dw - (s["w"] * dw).sum(-1, keepdim=True))
        dlogits = torch.zeros(T, c["E"] + 1, device=DEV).scatter_(1, torch.where(live, s["ids"], c["E"]).long(), dl)
        return dict(dy=dy.to(DTYPES[c["dtype"]]), dw=dw, dlogits=dlogits[:, : c["E"]].contiguous())
    most = s["most"]
    if op == "adapters":
        at = s["pairs"][: s["valid"]].long()
        slot = _slots(s["offsets"], s["valid"], most)
        xs = _padded(s["x"].float()[at], slot, c["n"], most)
        v = torch.bmm(xs, s["A"].float().transpose(1, 2).contiguous()) * s["scale"][:, None, None]
        d = torch.bmm(v, s["B"].float().transpose(1, 2).contiguous()).view(c["n"] * most, -1)[slot]
        out = s["y"].clone()
        out[at] = (s["y"].float()[at] + d).to(out.dtype)
        return out
    P = c["T"] * c["k"]
    slot = _slots(s["offsets"], P, most)
    if op == "product":
        a = _padded(s["a"].float()[(s["pairs"] // c["k"]).long()], slot, c["E"], most)
        y = torch.bmm(a, s["w"].float().transpose(1, 2).contiguous()).view(c["E"] * most, -1)[slot]
        if c["epi"] != "swiglu":
            return y.to(DTYPES[c["epi"]])
        g, u = y.chunk(2, -1)
        h = (g / (1 + torch.exp(-g)) * u).to(s["w"].dtype)
        return dict(h=h, pre=y.to(s["w"].dtype)) if c["pre"] else h
    dy = _padded(s["dy"].float(), slot, c["E"], most)
    if op == "grad_rows":
        da = torch.bmm(dy, s["w"].float()).view(c["E"] * most, -1)[slot]
        return _swiglu_grad(da, s["pre"]).to(s["w"].dtype) if c["epi"] == "swiglu_grad" else da.to(DTYPES[c["epi"]])
    a = _padded(s["a"].float()[(s["pairs"] // c["k"]).long()], slot, c["E"], most)
    return torch.bmm(dy.transpose(1, 2).contiguous(), a).to(DTYPES[c["out"]])


# ------------------------------------------------------- the library's calls
def _run_own(s, c):
    import quantized_moe_expert_top_amd as q
    op, plain = c["op"], {"bf16": q.MOE_EPI_NONE, "fp16": q.MOE_EPI_NONE_F16, "fp32": q.MOE_EPI_NONE_F32}
    if op == "combine_grad":
        g = q.moe_unpermute_combine_grad(s["dout"], s["y"], s["pos"], s["w"], c["T"], c["k"], dtype=DTYPES[c["dtype"]],
                                         n_valid=s["offsets"][-1:], ids=s["ids"], E=c["E"])
        return dict(dy=g.dy[: s["valid"]], dw=g.dw, dlogits=g.dlogits)
    if op == "adapters":
        return q.moe_adapter_add(s["y"], s["x"], s["A"], s["B"], s["offsets"], s["pairs"], scale=s["scale"])
    P = c["T"] * c["k"]
    if op == "product":
        if c["epi"] != "swiglu":
            return q.moe_grouped_gemm(s["w"], s["a"], s["offsets"], P, plain[c["epi"]], gather_pair=s["pairs"], k=c["k"])
        pre = torch.empty(P, c["N"], dtype=s["w"].dtype, device=DEV) if c["pre"] else None
        h = q.moe_grouped_gemm(s["w"], s["a"], s["offsets"], P, q.MOE_EPI_SWIGLU, gather_pair=s["pairs"], k=c["k"], pre=pre)
        return dict(h=h, pre=pre) if c["pre"] else h
    if op == "grad_rows":
        if c["epi"] == "swiglu_grad":
            return q.moe_grouped_gemm_grad_rows(s["w"], s["dy"], s["offsets"], P, q.MOE_EPI_SWIGLU_GRAD, pre=s["pre"])
        return q.moe_grouped_gemm_grad_rows(s["w"], s["dy"], s["offsets"], P, plain[c["epi"]])
    return q.moe_grouped_gemm_grad_weights(s["dy"], s["a"], s["offsets"], c["E"], P, plain[c["out"]],
                                           gather_pair=s["pairs"], k=c["k"])


def run(s):
    return (_run_own if own else _run_plain)(s, s["case"])


# ---------------------------------------------------------- what a pass needs
def _touched(T, k, E):
    return E * (1 - (1 - k / E) ** T)


def work(case):
    c, op = case, case["op"]
    if op == "combine_grad":
        P, b = c["T"] * c["k"], DTYPES[c["dtype"]].itemsize
        return dict(bytes=2.0 * c["T"] * c["H"] + (2.0 + b) * P * c["H"] + 16.0 * P + 4.0 * c["T"] * c["E"], flops=3.0 * P * c["H"])
    if op == "adapters":
        live = c["T"] * (1 - c["none"])
        used = _touched(max(1, live / c["run"]), 1, c["n"])
        return dict(bytes=2.0 * used * c["r"] * (c["K"] + c["N"]) + 2.0 * live * c["K"] + 4.0 * c["T"] * c["N"],
                    flops=2.0 * live * c["r"] * (c["K"] + c["N"]))
    M, N, K = c["T"] * c["k"], c["N"], c["K"]
    flops, w = 2.0 * M * N * K, 2.0 * _touched(c["T"], c["k"], c["E"]) * N * K
    if op == "product":
        n_out = (N // 2 + (N if c["pre"] else 0)) if c["epi"] == "swiglu" else N
        return dict(bytes=w + 2.0 * c["T"] * K + 4.0 * M + 2.0 * M * n_out, flops=flops)
    if op == "grad_rows":
        return dict(bytes=w + 2.0 * M * N + 2.0 * M * K * (4 if c["epi"] == "swiglu_grad" else 1), flops=flops)
    return dict(bytes=DTYPES[c["out"]].itemsize * c["E"] * N * K + 2.0 * M * N + 2.0 * c["T"] * K + 4.0 * M, flops=flops)


# ------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    op, o = c["op"], s["offsets"].tolist()
    if op == "combine_grad":
        T, k = c["T"], c["k"]
        pos, w, dout = s["pos"].long().view(T, k), s["w"].double(), s["dout"].double()
        dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
        dy = torch.zeros(T * k, c["H"], dtype=torch.float64, device=DEV)
        for j in range(k):
            live = pos[:, j] < s["valid"]
            p = pos[live, j]
            dw[live, j] = torch.linalg.vecdot(s["y"][p].double(), dout[live])
            dy[p] = w[live, j, None] * dout[live]
        # softmax's Jacobian, slot by slot; a slot without an expert has no logit
        dl = torch.zeros(T, c["E"], dtype=torch.float64, device=DEV)
        for j in range(k):
            jac = -w[:, j, None] * w
            jac[:, j] += w[:, j]
            live = pos[:, j] < s["valid"]
            dl[live, s["ids"][live, j].long()] = torch.linalg.vecdot(jac, dw)[live]
        return dict(dy=dy[: s["valid"]], dw=dw, dlogits=dl)
    if op == "adapters":
        out = s["y"].double()
        for a in range(c["n"]):
            t = s["pairs"][o[a] : o[a + 1]].long()
            if len(t):
                low = torch.mm(s["x"][t].double(), s["A"][a].double().t().contiguous())
                out[t] = out[t] + s["scale"][a].double() * torch.mm(low, s["B"][a].double().t().contiguous())
        return out
    P, N, K = c["T"] * c["k"], c["N"], c["K"]
    tokens = torch.div(s["pairs"], c["k"], rounding_mode="floor").long()
    if op == "grad_weights":
        if c["E"] * N * K > 500_000_000:
            return None
        out = torch.zeros(c["E"], N, K, dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            if o[e + 1] > o[e]:
                out[e] = s["dy"][o[e] : o[e + 1]].double().t().contiguous() @ s["a"][tokens[o[e] : o[e + 1]]].double()
        return out
    y = torch.zeros(P, N if op == "product" else K, dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        rows = slice(o[e], o[e + 1])
        if o[e + 1] > o[e]:
            w = s["w"][e].double()
            y[rows] = s["a"][tokens[rows]].double() @ w.t().contiguous() if op == "product" else s["dy"][rows].double() @ w
    if c["epi"] == "swiglu":
        gate, up = y[:, : N // 2], y[:, N // 2 :]
        h = torch.nn.functional.silu(gate) * up
        return dict(h=h, pre=y) if c["pre"] else h
    if c["epi"] != "swiglu_grad":
        return y
    gate, up = s["pre"][:, :K].double(), s["pre"][:, K:].double()
    sig = torch.sigmoid(gate)
    return torch.cat([y * up * (sig + gate * sig * torch.sigmoid(-gate)), y * gate * sig], 1)
