"""What is measured of the ragged grouped products, the int8 products and the block norms.

Each case names one call (or the short chain a user runs as one step) at the sizes of this
repository's layers and at odd ones. ``run`` computes it in plain torch operations, or, where
``own`` is true, through the public entry points of ``routing_expert_grouped_amd``.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
_EPS = 1e-6


# --------------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------------
# op of a case:
#   grouped_fwd   out[r] = rows[src r] W[e r], W [E][K][N]; gather: rows are the T tokens, read
#                 through the schedule's perm, else the R routed rows
#   grouped_dgrad dX[r] = dY[r] W[e r]^T
#   grouped_wgrad dW[e] = X_e^T dY_e in float32
#   grouped_step  the three of a training step of one expert matrix
#   int8_linear   quantise the tokens, dense int8 product (norm: the pre-norm writes the int8 rows)
#   int8_grouped  quantise the tokens once, grouped int8 product gathered through perm
#   post_norm     the norm after a block with gate and residual, and the next block's norm
#   post_norm_bwd its gradients
def listed():
    return [
        # the tiny layer's first expert product: launch latency counts
        dict(name="grouped_fwd_tiny", op="grouped_fwd", T=64, k=2, E=8, K=256, N=256, dt="bf16",
             gather=True, skew="router"),
        # serving a few tokens through the Qwen-shaped layer's 512 experts: every weight of the
        # experts that are hit is read once for one or two rows
        dict(name="grouped_fwd_decode", op="grouped_fwd", T=16, k=10, E=512, K=4096, N=2048,
             dt="bf16", gather=True, skew="router"),
        # the Qwen-shaped layer's 4096 tokens: about 80 rows per expert, ragged
        dict(name="grouped_fwd_layer", op="grouped_fwd", T=4096, k=10, E=512, K=4096, N=2048,
             dt="bf16", gather=True, skew="router"),
        # the Kimi-shaped expert share in training: few large skewed experts, each gradient
        dict(name="grouped_dgrad_share", op="grouped_dgrad", T=2048, k=8, E=6, K=7168, N=4096,
             dt="bf16", gather=False, skew="zipf"),
        dict(name="grouped_wgrad_share", op="grouped_wgrad", T=2048, k=8, E=6, K=7168, N=4096,
             dt="bf16", gather=False, skew="zipf"),
        # a training step of an odd-sized expert matrix in half precision
        dict(name="grouped_step_odd", op="grouped_step", T=499, k=3, E=7, K=1001, N=777,
             dt="fp16", gather=False, skew="router"),
        # one token through an int8 projection of the Kimi-shaped shared expert (gate | up), with
        # the norm before it
        dict(name="int8_norm_linear_token", op="int8_linear", T=1, K=7168, N=4096, dt="bf16",
             norm=True, bias=False),
        # a prompt through an int8 projection of the GLM-5.2-shaped layer's width
        dict(name="int8_linear_prompt", op="int8_linear", T=8192, K=6144, N=4096, dt="bf16",
             norm=False, bias=True),
        # the GLM-5.2-shaped layer's routed experts in int8, 8192 tokens
        dict(name="int8_grouped_layer", op="int8_grouped", T=8192, k=8, E=256, K=6144, N=4096,
             dt="bf16", skew="router"),
        # one token after a block
        dict(name="post_norm_token", op="post_norm", T=1, h=7168, dt="bf16", tau=True),
        # the GLM-5.2-shaped layer's tokens after a block
        dict(name="post_norm_layer", op="post_norm", T=8192, h=6144, dt="bf16", tau=True),
        # the Qwen-shaped layer's tokens in training
        dict(name="post_norm_bwd_layer", op="post_norm_bwd", T=4096, h=4096, dt="bf16", tau=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: a multiple of 128, of 8, or any number."""
    n = _log_int(rng, lo, hi)
    m = rng.choice((128, 128, 8, 1))
    return max(m, n // m * m)


def draw(rng):
    op = rng.choice(("grouped_fwd", "grouped_fwd", "grouped_dgrad", "grouped_wgrad",
                     "grouped_step", "int8_linear", "int8_linear", "int8_grouped", "int8_grouped",
                     "post_norm", "post_norm_bwd"))
    while True:
        T = _log_int(rng, 1, 8192)
        dt = rng.choice(("bf16", "bf16", "fp16"))
        if op in ("post_norm", "post_norm_bwd"):
            return dict(op=op, T=T, h=_width(rng, 64, 8192), dt=dt, tau=rng.random() < 0.5)
        K, N = _width(rng, 64, 8192), _width(rng, 64, 8192)
        if op == "int8_linear":
            c = dict(op=op, T=T, K=K, N=N, dt="bf16", norm=rng.random() < 0.5,
                     bias=rng.random() < 0.5)
        else:
            E = _log_int(rng, 1, 512)
            k = min(E, rng.randint(1, 10))
            c = dict(op=op, T=T, k=k, E=E, K=K, N=N, dt=dt,
                     skew=rng.choice(("router", "zipf", "one")))
            if op == "int8_grouped":
                c["dt"] = "bf16"
            else:
                c["gather"] = op == "grouped_fwd" and rng.random() < 0.5
        w = work(c)
        if w["flops"] <= 1.5e12 and w["bytes"] <= 4e9 and c.get("E", 1) * K * N <= 3e9:
            return c


# --------------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------------
def _dev():
    return torch.device("cuda")


def _gen(seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=_dev()) * scale).to(dtype)


def _tokens(g, T, h, dtype):
    """Hidden states: unit normals with a few channels that carry much larger values."""
    x = torch.randn(T, h, generator=g, device=_dev())
    ch = torch.randint(0, h, (max(1, h // 512),), generator=g, device=_dev())
    x[:, ch] *= 8.0
    return x.to(dtype)


def _schedule(g, c):
    """offsets (device int32 and host list) and perm of a routed batch: R = T k assignments sorted
    by expert, ascending inside an expert."""
    T, k, E = c["T"], c["k"], c["E"]
    if c["skew"] == "router":  # each token's k best of E noisy logits, some experts preferred
        logits = torch.randn(T, E, generator=g, device=_dev())
        logits += 0.7 * torch.randn(E, generator=g, device=_dev())
        assign = logits.topk(k, dim=1).indices.reshape(-1)
    elif c["skew"] == "zipf":  # an expert-parallel share: a heavy first expert
        p = torch.arange(1, E + 1, device=_dev(), dtype=torch.float32) ** -1.2
        assign = torch.multinomial(p, T * k, replacement=True, generator=g)
    else:  # every row to one expert, the others empty
        assign = torch.full((T * k,), E // 2, device=_dev(), dtype=torch.int64)
    perm = torch.argsort(assign, stable=True)
    counts = torch.bincount(assign, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=_dev())
    offsets[1:] = counts.cumsum(0)
    return offsets.to(torch.int32), offsets.tolist(), perm.to(torch.int32)


def _weights(g, E, K, N, dtype):
    w = torch.empty(E, K, N, dtype=dtype, device=_dev())
    for e in range(E):
        w[e] = _randn(g, K, N, scale=K ** -0.5)
    return w


def _int8_weights(g, E, N, K):
    """Quantised weights as a checkpoint holds them: codes [E][N][K], a scale per channel [E][N]."""
    q = torch.empty(E, N, K, dtype=torch.int8, device=_dev())
    for e in range(E):
        q[e] = (torch.randn(N, K, generator=g, device=_dev()) * 30.0).round_().clamp_(-127, 127)
    s = (0.5 + torch.rand(E, N, generator=g, device=_dev())) / (30.0 * K ** 0.5)
    return q, s


def _inputs(case, seed):
    """The inputs alone, in plain tensors."""
    c, g = case, _gen(seed)
    op = c["op"]
    s = {"case": c}
    dt = _DT[c["dt"]]
    if op.startswith("grouped"):
        s["offsets"], s["host_offsets"], s["perm"] = _schedule(g, c)
        R = c["T"] * c["k"]
        if op != "grouped_dgrad":
            s["x"] = _randn(g, c["T"] if c["gather"] else R, c["K"], dtype=dt)
        if op != "grouped_wgrad":
            s["w"] = _weights(g, c["E"], c["K"], c["N"], dt)
        if op != "grouped_fwd":
            s["dy"] = _randn(g, R, c["N"], dtype=dt)
    elif op == "int8_linear":
        s["x"] = _tokens(g, c["T"], c["K"], dt)
        s["q"], s["qs"] = _int8_weights(g, 1, c["N"], c["K"])
        s["wn"] = (1.0 + 0.1 * _randn(g, c["K"])).to(dt) if c["norm"] else None
        s["bias"] = _randn(g, 1, c["N"]) if c["bias"] else None
    elif op == "int8_grouped":
        s["offsets"], s["host_offsets"], s["perm"] = _schedule(g, c)
        s["x"] = _tokens(g, c["T"], c["K"], dt)
        s["q"], s["qs"] = _int8_weights(g, c["E"], c["N"], c["K"])
    else:
        T, h = c["T"], c["h"]
        s["res"] = _tokens(g, T, h, dt)
        s["y"] = _randn(g, T, h, scale=0.5, dtype=dt)
        s["w"] = (1.0 + 0.1 * _randn(g, h)).to(dt)
        s["gate"] = (0.3 * _randn(g, h)).to(dt)
        s["w_next"] = (1.0 + 0.1 * _randn(g, h)).to(dt)
        s["tau"] = torch.rand(T, generator=g, device=_dev()) if c["tau"] else None
        s["scale"] = 0.75
        if op == "post_norm_bwd":  # what the forward keeps: u and the two reciprocal norms
            s["du"] = _randn(g, T, h, dtype=dt)
            s["dz"] = _randn(g, T, h, dtype=dt)
            y = s["y"].double()
            ry = (y.square().mean(1, keepdim=True) + _EPS).rsqrt()
            v = y * ry * s["w"].double() * s["gate"].double()
            if s["tau"] is not None:
                v = v * s["tau"].double()[:, None]
            s["u"] = (s["scale"] * s["res"].double() + v).to(dt)
            ru = (s["u"].double().square().mean(1) + _EPS).rsqrt()
            s["rstd"], s["rstd_next"] = ry[:, 0].float(), ru.float()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and "q" in s:  # int8 weights are laid out once, when a model is loaded
        import routing_expert_grouped_amd as G
        E, N, K = s["q"].shape
        s["shape"] = G.make_gemm_shape(case["T"] * case.get("k", 1), K, N, E)
        s["packed"] = G.moe_int8_pack_weights(s["shape"], s["q"])
        del s["q"]
    elif own and "offsets" in s:
        import routing_expert_grouped_amd as G
        s["shape"] = G.make_gemm_shape(case["T"] * case["k"], case["K"], case["N"], case["E"])
    return s


# --------------------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------------------
def _segments(s):
    o = s["host_offsets"]
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def _rows_of(s):
    if s["case"]["gather"]:
        return s["x"].index_select(0, torch.div(s["perm"], s["case"]["k"], rounding_mode="floor"))
    return s["x"]


def _plain_fwd(s):
    x, w = _rows_of(s), s["w"]
    out = torch.zeros(x.shape[0], w.shape[2], dtype=x.dtype, device=x.device)
    for e, a, b in _segments(s):
        out[a:b] = (x[a:b].float() @ w[e].float()).to(x.dtype)
    return out


def _plain_dgrad(s):
    dy, w = s["dy"], s["w"]
    dx = torch.zeros(dy.shape[0], w.shape[1], dtype=dy.dtype, device=dy.device)
    for e, a, b in _segments(s):
        dx[a:b] = (dy[a:b].float() @ w[e].float().t()).to(dy.dtype)
    return dx


def _plain_wgrad(s):
    x, dy, c = _rows_of(s), s["dy"], s["case"]
    dw = torch.zeros(c["E"], c["K"], c["N"], dtype=torch.float32, device=dy.device)
    for e, a, b in _segments(s):
        dw[e] = x[a:b].float().t() @ dy[a:b].float()
    return dw


def _plain_quantise(p):
    """Codes rint(127 p / amax) of each row; 127 p of a product of two bf16 values is exact in
    float32, so the quotient is on the right side of every rounding border."""
    amax = p.abs().amax(1, keepdim=True)
    codes = torch.where(amax > 0, torch.round(p * 127.0 / amax), torch.zeros_like(p))
    return codes, amax


def _plain_int_product(a, q):
    """Exact integer product of integer-valued float32 rows a and int8 q [N][K]: float32 partial
    products over 1024 columns stay below 2^24, their sum is kept in int32."""
    acc = torch.zeros(a.shape[0], q.shape[0], dtype=torch.int32, device=a.device)
    for i in range(0, a.shape[1], 1024):
        acc += (a[:, i:i + 1024] @ q[:, i:i + 1024].float().t()).to(torch.int32)
    return acc


def _plain_int8_linear(s):
    x = s["x"].float()
    if s["wn"] is not None:
        r = torch.rsqrt(x.square().mean(1, keepdim=True) + _EPS)
        codes, amax = _plain_quantise(x * s["wn"].float())
        sa = amax * r / 127.0
    else:
        codes, amax = _plain_quantise(x)
        sa = amax / 127.0
    y = _plain_int_product(codes, s["q"][0]).float() * sa * s["qs"][0]
    if s["bias"] is not None:
        y = y + s["bias"][0]
    return y.to(s["x"].dtype)


def _plain_int8_grouped(s):
    c = s["case"]
    codes, amax = _plain_quantise(s["x"].float())
    src = torch.div(s["perm"], c["k"], rounding_mode="floor")
    rows, sa = codes.index_select(0, src), (amax / 127.0).index_select(0, src)
    out = torch.zeros(rows.shape[0], c["N"], dtype=s["x"].dtype, device=rows.device)
    for e, a, b in _segments(s):
        out[a:b] = (_plain_int_product(rows[a:b], s["q"][e]).float() * sa[a:b]
                    * s["qs"][e]).to(out.dtype)
    return out


def _plain_post_norm(s):
    dt = s["res"].dtype
    y = s["y"].float()
    v = y * torch.rsqrt(y.square().mean(1, keepdim=True) + _EPS) * s["w"].float()
    v = v * s["gate"].float()
    if s["tau"] is not None:
        v = v * s["tau"][:, None]
    u = (s["scale"] * s["res"].float() + v).to(dt)
    uf = u.float()
    z = uf * torch.rsqrt(uf.square().mean(1, keepdim=True) + _EPS) * s["w_next"].float()
    return u, z.to(dt)


def _plain_post_norm_bwd(s):
    dt = s["res"].dtype
    u, y = s["u"].float(), s["y"].float()
    nu, ny = u * s["rstd_next"][:, None], y * s["rstd"][:, None]
    dz, w, gate = s["dz"].float(), s["w"].float(), s["gate"].float()
    tau = s["tau"][:, None] if s["tau"] is not None else torch.ones_like(s["rstd"])[:, None]
    q = dz * s["w_next"].float()
    g = s["du"].float() + s["rstd_next"][:, None] * (q - nu * (q * nu).mean(1, keepdim=True))
    dn = g * w * gate * tau
    dy = s["rstd"][:, None] * (dn - ny * (dn * ny).mean(1, keepdim=True))
    col = (g * ny * tau).double().sum(0)  # long sums
    out = {"dres": (s["scale"] * g).to(dt), "dy": dy.to(dt),
           "dw": (col * gate.double()).float(), "dgate": (col * w.double()).float(),
           "dw_next": (dz * nu).double().sum(0).float()}
    if s["tau"] is not None:
        out["dtau"] = (g * ny * w * gate).double().sum(1).float()
    return out


_PLAIN = {
    "grouped_fwd": _plain_fwd,
    "grouped_dgrad": _plain_dgrad,
    "grouped_wgrad": _plain_wgrad,
    "grouped_step": lambda s: (_plain_fwd(s), _plain_dgrad(s), _plain_wgrad(s)),
    "int8_linear": _plain_int8_linear,
    "int8_grouped": _plain_int8_grouped,
    "post_norm": _plain_post_norm,
    "post_norm_bwd": _plain_post_norm_bwd,
}


def _own_run(s):
    import routing_expert_grouped_amd as G
    c = s["case"]
    op = c["op"]
    if op.startswith("grouped"):
        sh, off = s["shape"], s["offsets"]
        gather = dict(perm=s["perm"], k=c["k"]) if c["gather"] else {}
        if op == "grouped_fwd":
            return G.moe_grouped_gemm(sh, s["x"], s["w"], off, **gather)
        if op == "grouped_dgrad":
            return G.moe_grouped_gemm_dgrad(sh, s["dy"], s["w"], off)
        if op == "grouped_wgrad":
            return G.moe_grouped_gemm_wgrad(sh, s["x"], s["dy"], off, **gather)
        return (G.moe_grouped_gemm(sh, s["x"], s["w"], off),
                G.moe_grouped_gemm_dgrad(sh, s["dy"], s["w"], off),
                G.moe_grouped_gemm_wgrad(sh, s["x"], s["dy"], off))
    if op == "int8_linear":
        if c["norm"]:
            codes, scales, _ = G.moe_pre_norm_int8(s["x"], s["wn"], eps=_EPS)
        else:
            codes, scales = G.moe_quantize_int8(s["x"])
        return G.moe_gemm_int8(s["shape"], codes, scales, s["packed"], s["qs"], bias=s["bias"])
    if op == "int8_grouped":
        codes, scales = G.moe_quantize_int8(s["x"])
        return G.moe_grouped_gemm_int8(s["shape"], codes, scales, s["packed"], s["qs"],
                                       s["offsets"], perm=s["perm"], k=c["k"])
    if op == "post_norm":
        u, z, _, _ = G.moe_post_norm(s["res"], s["y"], s["w"], gate=s["gate"],
                                     token_gate=s["tau"], res_scale=s["scale"],
                                     w_next=s["w_next"], eps=_EPS)
        return u, z
    gr = G.moe_post_norm_backward(s["du"], s["y"], s["rstd"], s["w"], gate=s["gate"],
                                  token_gate=s["tau"], res_scale=s["scale"], dz=s["dz"],
                                  u=s["u"], rstd_next=s["rstd_next"], w_next=s["w_next"])
    out = {"dres": gr["dres"], "dy": gr["dy"], "dw": gr["dw"], "dgate": gr["dgate"],
           "dw_next": gr["dw_next"]}
    if s["tau"] is not None:
        out["dtau"] = gr["dtoken_gate"]
    return out


def run(state):
    return _own_run(state) if own else _PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------------------------------
def _experts_hit(c):
    """Experts with at least one row, in expectation over evenly drawn assignments (one expert for
    the case that sends every row to one)."""
    R, E = c["T"] * c["k"], c["E"]
    if c["skew"] == "one":
        return 1
    if c["skew"] == "zipf":
        p = [(e + 1) ** -1.2 for e in range(E)]
        t = sum(p)
        return sum(1.0 - (1.0 - q / t) ** R for q in p)
    return E * (1.0 - (1.0 - c["k"] / E) ** c["T"])


def work(case):
    c = case
    op = c["op"]
    el = 2
    if op.startswith("grouped"):
        R, K, N, E = c["T"] * c["k"], c["K"], c["N"], c["E"]
        hit = _experts_hit(c)
        xrows = c["T"] if c["gather"] else R
        one = {"grouped_fwd": (xrows * K + hit * K * N + R * N) * el,
               "grouped_dgrad": (R * N + hit * K * N + R * K) * el,
               "grouped_wgrad": (xrows * K + R * N) * el + E * K * N * 4}
        flops = 2 * R * K * N
        if op == "grouped_step":  # x, dy and W once, and the three outputs
            return {"bytes": int((R * K + R * N + hit * K * N + R * N + R * K) * el + E * K * N * 4),
                    "flops": 3 * flops}
        return {"bytes": int(one[op]), "flops": flops}
    if op == "int8_linear":
        T, K, N = c["T"], c["K"], c["N"]
        return {"bytes": T * K * el + N * K + 4 * N + T * N * el, "flops": 2 * T * K * N}
    if op == "int8_grouped":
        R, K, N = c["T"] * c["k"], c["K"], c["N"]
        hit = _experts_hit(c)
        return {"bytes": int(c["T"] * K * el + hit * (N * K + 4 * N) + R * N * el),
                "flops": 2 * R * K * N}
    T, h = c["T"], c["h"]
    if op == "post_norm":  # res, y -> u, z
        return {"bytes": 4 * T * h * el + 3 * h * el, "flops": 12 * T * h}
    # du, dz, u, y -> dres, dy and the small gradients
    return {"bytes": 6 * T * h * el + 3 * h * el + 3 * h * 4, "flops": 24 * T * h}


# --------------------------------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    c = case
    op = c["op"]
    f8 = torch.float64
    if op.startswith("grouped"):
        R, E, K, N = c["T"] * c["k"], c["E"], c["K"], c["N"]
        o = s["host_offsets"]
        src = (s["perm"].long() // c["k"]) if c["gather"] else torch.arange(R, device=_dev())
        fwd = torch.zeros(R, N, dtype=f8, device=_dev()) if op in ("grouped_fwd",
                                                                  "grouped_step") else None
        dx = torch.zeros(R, K, dtype=f8, device=_dev()) if op in ("grouped_dgrad",
                                                                 "grouped_step") else None
        dw = torch.zeros(E, K, N, dtype=f8, device=_dev()) if op in ("grouped_wgrad",
                                                                    "grouped_step") else None
        for e in range(E):
            r = slice(o[e], o[e + 1])
            if o[e] == o[e + 1]:
                continue
            we = s["w"][e].to(f8) if "w" in s else None
            xe = s["x"][src[r]].to(f8) if "x" in s else None
            if fwd is not None:
                fwd[r] = torch.mm(xe, we)
            if dx is not None:
                dx[r] = torch.mm(s["dy"][r].to(f8), we.T.contiguous())
            if dw is not None:
                dw[e] = torch.mm(xe.T.contiguous(), s["dy"][r].to(f8))
        return (fwd, dx, dw) if op == "grouped_step" else (fwd if fwd is not None else
                                                           dx if dx is not None else dw)
    if op.startswith("int8"):
        p = s["x"].to(f8)
        norm = torch.ones(p.shape[0], dtype=f8, device=_dev())
        if s.get("wn") is not None:
            norm = 1.0 / torch.sqrt(torch.mean(p * p, dim=1) + _EPS)
            p = p * s["wn"].to(f8)
        top = p.abs().max(dim=1).values
        safe = torch.where(top == 0, torch.ones_like(top), top)
        codes = torch.round(127.0 * p / safe[:, None])
        scale = top * norm / 127.0
        if op == "int8_linear":
            y = torch.mm(codes, s["q"][0].to(f8).T.contiguous()) * scale[:, None]
            y = y * s["qs"][0].to(f8)[None, :]
            return y + s["bias"][0].to(f8)[None, :] if s["bias"] is not None else y
        o = s["host_offsets"]
        tok = s["perm"].long() // c["k"]
        y = torch.empty(c["T"] * c["k"], c["N"], dtype=f8, device=_dev())
        for e in range(c["E"]):
            t = tok[o[e]:o[e + 1]]
            if len(t):
                y[o[e]:o[e + 1]] = (torch.mm(codes[t], s["q"][e].to(f8).T.contiguous())
                                    * scale[t][:, None] * s["qs"][e].to(f8)[None, :])
        return y
    d = {n: s[n].to(f8) for n in ("res", "y", "w", "gate", "w_next")}
    tau = s["tau"].to(f8) if s["tau"] is not None else torch.ones(c["T"], dtype=f8, device=_dev())
    if op == "post_norm":
        inv = 1.0 / torch.sqrt(torch.mean(d["y"] ** 2, dim=1) + _EPS)
        u = s["scale"] * d["res"] + (inv * tau)[:, None] * d["y"] * (d["w"] * d["gate"])[None, :]
        # the next norm reads u as it is stored, in the inputs' type
        us = u.to(s["res"].dtype).to(f8)
        inv2 = 1.0 / torch.sqrt(torch.mean(us ** 2, dim=1) + _EPS)
        return u, inv2[:, None] * us * d["w_next"][None, :]
    h = c["h"]
    ru, ry = s["rstd_next"].to(f8), s["rstd"].to(f8)
    u, dz = s["u"].to(f8), s["dz"].to(f8)
    q = dz * d["w_next"][None, :]
    g = s["du"].to(f8) + ru[:, None] * q - u * (ru ** 3 * (q * u).sum(1) / h)[:, None]
    wg = d["w"] * d["gate"]
    dn = g * wg[None, :] * tau[:, None]
    dy = ry[:, None] * dn - d["y"] * (ry ** 3 * (dn * d["y"]).sum(1) / h)[:, None]
    a = torch.mv((g * d["y"]).T.contiguous(), ry * tau)
    out = {"dres": s["scale"] * g, "dy": dy, "dw": a * d["gate"], "dgate": a * d["w"],
           "dw_next": torch.mv((dz * u).T.contiguous(), ru)}
    if s["tau"] is not None:
        out["dtau"] = torch.mv(g * d["y"], wg) * ry
    return out
