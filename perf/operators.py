"""Cases of the operators that stand around the expert products of an MoE layer.

Three groups: the residual addition + RMS norm with an 8-bit output (forward
and backward), the router (scores, top-k choice, per-expert counts, balance
loss; its gradient; the gradient of the combine's weights), and the gated
activation between the two expert products with MXFP8 output (forward and
backward).  With ``own`` false ``run`` computes them with elementary torch
operations in 32 bits; with ``own`` true it calls this package.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
E4M3_MAX = 448.0
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoded token of the DeepSeek-V3 layer: the norm before its experts, latency only
        dict(name="norm_fwd_token", op="norm_fwd", T=1, H=7168, residual=True, y=True, rstd=False, recipe="mx",
             tiled=False, w32=False),
        # the Llama4-Scout layer's training batch: residual, bf16 rows for the router, MXFP8 rows for a dense product
        dict(name="norm_fwd_scout", op="norm_fwd", T=16384, H=5120, residual=True, y=True, rstd=True, recipe="mx",
             tiled=True, w32=False),
        # Llama3-8B rows, a batch cut short by one token, rowwise FP8 only
        dict(name="norm_fwd_rowwise", op="norm_fwd", T=8191, H=4096, residual=True, y=False, rstd=True,
             recipe="rowwise", tiled=False, w32=True),
        # the Scout batch's backward, with the gradient that comes along the residual stream
        dict(name="norm_bwd_scout", op="norm_bwd", T=16384, H=5120, stream=True, w32=False),
        # a decode step of a few tokens through DeepSeek-V3's router (sigmoid scores, selection bias)
        dict(name="router_fwd_token", op="router_fwd", T=3, E=256, k=8, score="sigmoid", renorm=True, bias=True,
             dead=0, masked=0.0, bf16=False),
        # DeepSeek-V3's training batch, eight experts masked out, a few padding tokens
        dict(name="router_fwd_dsv3", op="router_fwd", T=4096, E=256, k=8, score="sigmoid", renorm=True, bias=True,
             dead=8, masked=0.03, bf16=False),
        # MoE-16B's batch: softmax over 64 experts, bf16 logits with many ties
        dict(name="router_fwd_moe16b", op="router_fwd", T=8192, E=64, k=6, score="softmax", renorm=False, bias=False,
             dead=0, masked=0.0, bf16=True),
        # the gradient of DeepSeek-V3's router
        dict(name="router_bwd_dsv3", op="router_bwd", T=4096, E=256, k=8, score="sigmoid", renorm=True, bias=True,
             dead=8, masked=0.03, bf16=False),
        # the gradient of the combine's weights, DeepSeek-V3's batch: every routed row against its token's gradient
        dict(name="weight_grad_dsv3", op="weight_grad", T=4096, N=7168, k=8),
        # a few decoded tokens between the two expert products, rows in 128x4 scale tiles
        dict(name="swiglu_fwd_token", op="swiglu_fwd", M=32, F=2048, E=1, y=False, dim1=False),
        # DeepSeek-V3's routed batch: 256 ragged groups, both directions for forward and weight gradient
        dict(name="swiglu_fwd_dsv3", op="swiglu_fwd", M=36448, F=2048, E=256, y=False, dim1=True),
        # MoE-16B's routed batch backward, both directions of the gradient of gate and up
        dict(name="swiglu_bwd_moe16b", op="swiglu_bwd", M=51136, F=1408, E=64, y=False, dim1=True),
    ]


def _logsize(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "router_fwd", "router_bwd", "weight_grad", "swiglu_fwd", "swiglu_bwd"])
    flag = lambda p=0.5: rng.random() < p  # noqa: E731
    if op in ("norm_fwd", "norm_bwd"):
        H = 32 * _logsize(rng, 8, 256)
        H += 32 * (H == 3072)
        T = _logsize(rng, 1, min(40000, 80_000_000 // H))
        if op == "norm_bwd":
            return dict(op=op, T=T, H=H, stream=flag(), w32=flag())
        recipe = rng.choice(["mx", "rowwise", "mx", "none"])
        return dict(op=op, T=T, H=H, residual=flag(0.7), y=recipe == "none" or flag(), rstd=flag(), recipe=recipe,
                    tiled=recipe == "mx" and flag(), w32=flag())
    if op in ("router_fwd", "router_bwd"):
        E = rng.choice([8, 16, 60, 64, 100, 128, 160, 256, 384, 512])
        k = rng.randint(1, min(E, 10))
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=_logsize(rng, 1, 4_000_000 // E), E=E, k=k, score=score, renorm=flag(),
                    bias=score == "sigmoid" and flag(), dead=rng.choice([0, 0, 1, 3]) if E > 8 + k else 0,
                    masked=rng.choice([0.0, 0.1]), bf16=flag())
    if op == "weight_grad":
        N, k = 8 * _logsize(rng, 16, 1024), rng.randint(1, 8)
        N += 8 * (N == 3072)
        return dict(op=op, T=_logsize(rng, 1, 250_000_000 // (N * (k + 1))), N=N, k=k)
    F = 32 * _logsize(rng, 4, 200)
    F += 32 * (F == 3072)
    rows = 32 * _logsize(rng, 1, 50_000_000 // F // 32)
    return dict(op=op, M=rows, F=F, E=min(_logsize(rng, 1, 256), rows // 32), y=flag(0.3), dim1=flag(0.7))


# ---------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------

def _up(a, b):
    return (a + b - 1) // b * b


def _tiled_bytes(rows, cols):
    """Bytes of the 128x4 layout of a [rows, cols] scale matrix."""
    return _up(rows, 128) * _up(cols, 4)


def work(case):
    op = case["op"]
    if op == "norm_fwd":
        T, H = case["T"], case["H"]
        per = 2 + (4 if case["residual"] else 0) + (2 if case["y"] else 0)
        out = {"mx": H + H / 32, "rowwise": H + 4, "none": 0}[case["recipe"]]
        return {"bytes": T * (H * per + out + (4 if case["rstd"] else 0)) + H * (4 if case["w32"] else 2),
                "flops": 8 * T * H}
    if op == "norm_bwd":
        T, H = case["T"], case["H"]
        return {"bytes": T * (H * (8 if case["stream"] else 6) + 4) + H * ((4 if case["w32"] else 2) + 4),
                "flops": 12 * T * H}
    if op in ("router_fwd", "router_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        b = 2 if case["bf16"] else 4
        if op == "router_fwd":
            return {"bytes": T * (E * b + 8 * k + 1) + 12 * E, "flops": T * E * (8 + k)}
        return {"bytes": T * (2 * E * b + 8 * k + 1) + 4 * E, "flops": 16 * T * E}
    if op == "weight_grad":
        T, N, k = case["T"], case["N"], case["k"]
        return {"bytes": T * (2 * N * (k + 1) + 8 * k), "flops": 2 * T * N * k}
    M, F = case["M"], case["F"]
    width = F if op == "swiglu_fwd" else 2 * F
    read = 4 * F if op == "swiglu_fwd" else 6 * F
    dirs = 2 if case["dim1"] else 1
    return {"bytes": M * (read + width * dirs * (1 + 1 / 32) + (2 * width if case["y"] else 0)),
            "flops": M * F * (8 if op == "swiglu_fwd" else 20)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, device=DEV, generator=gen) * scale).to(dtype)


def _rows(gen, T, H):
    """Activations as a residual stream has them: unit rows, a few large channels."""
    x = torch.randn(T, H, device=DEV, generator=gen)
    x *= 1.0 + 20.0 * (torch.rand(H, device=DEV, generator=gen) < 0.005)
    return x.to(BF16)


def _logits(gen, case):
    T, E = case["T"], case["E"]
    # popularity falls off over the experts, as a trained router's does
    pop = -0.5 * torch.log(1.0 + torch.arange(E, device=DEV, dtype=F32))
    pop = pop[torch.randperm(E, device=DEV, generator=gen)]
    x = torch.randn(T, E, device=DEV, generator=gen) * 1.5 + pop
    if case["dead"]:
        x[:, torch.randperm(E, device=DEV, generator=gen)[:case["dead"]]] = -math.inf
    return x.to(BF16 if case["bf16"] else F32)


def _offsets(gen, M, E):
    """Cumulative ends of E ragged groups of whole 32-row blocks, some empty."""
    share = torch.rand(E, device=DEV, generator=gen).pow(3)
    cum = share.cumsum(0) / share.sum()
    ends = (cum * (M // 32)).round().to(torch.int32) * 32
    ends[-1] = M
    return ends


def _choose(x, bias, score, k):
    """Expert ids by (key, id): the k largest keys, ties to the lowest id."""
    key = x
    if bias is not None:
        s = 1.0 / (1.0 + torch.exp(-x)) if score == "sigmoid" else _softmax(x)
        key = torch.where(x > -math.inf, s + bias, torch.full_like(x, -math.inf))
    return torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, s = case["op"], dict(case)
    s["plan"] = {}
    if op in ("norm_fwd", "norm_bwd"):
        T, H = case["T"], case["H"]
        s["w"] = _randn(gen, H, dtype=F32, scale=0.2).add_(1.0).to(F32 if case["w32"] else BF16)
    if op == "norm_fwd":
        s["x"] = _rows(gen, T, H)
        s["r"] = _rows(gen, T, H) if case["residual"] else None
        # the output buffers that a program keeps from step to step
        p = s["plan"]
        p["h"] = torch.empty(T, H, dtype=BF16, device=DEV) if case["residual"] else None
        p["y"] = torch.empty(T, H, dtype=BF16, device=DEV) if case["y"] else None
        p["rstd"] = torch.empty(T, dtype=F32, device=DEV) if case["rstd"] else None
        if case["recipe"] != "none":
            p["q"] = torch.empty(T, H, dtype=torch.uint8, device=DEV)
        if case["recipe"] == "mx":
            shape = (_tiled_bytes(T, H // 32),) if case["tiled"] else (T, H // 32)
            p["scale"] = torch.zeros(shape, dtype=torch.uint8, device=DEV)
        elif case["recipe"] == "rowwise":
            p["scale"] = torch.empty(T, dtype=F32, device=DEV)
    elif op == "norm_bwd":
        s["h"] = _rows(gen, T, H)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        s["dy"] = _randn(gen, T, H)
        s["dh"] = _randn(gen, T, H) if case["stream"] else None
    elif op in ("router_fwd", "router_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _logits(gen, case)
        s["bias"] = _randn(gen, E, dtype=F32, scale=0.05) if case["bias"] else None
        s["mask"] = None
        if case["masked"]:
            s["mask"] = (torch.rand(T, device=DEV, generator=gen) >= case["masked"]).to(torch.uint8)
        if op == "router_bwd":
            x = s["logits"].float()
            if s["mask"] is not None:
                x = torch.where(s["mask"][:, None] != 0, x, torch.full_like(x, -math.inf))
            idx = _choose(x, s["bias"], case["score"], k)
            live = torch.gather(x, 1, idx) > -math.inf
            counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
            counts.scatter_add_(0, idx.reshape(-1), live.reshape(-1).to(torch.int64))
            counts[E] = T if s["mask"] is None else s["mask"].sum()
            s["idx"], s["counts"] = idx.to(torch.int32), counts.to(torch.int32)
            s["dw"] = _randn(gen, T, k, dtype=F32)
            s["dloss"] = torch.rand(1, device=DEV, generator=gen) + 0.5
    elif op == "weight_grad":
        T, N, k = case["T"], case["N"], case["k"]
        rows = _up(T * k + 32, 32)
        s["y"] = _randn(gen, rows, N)
        s["dout"] = _randn(gen, T, N)
        s["row_of"] = torch.randperm(rows, device=DEV, generator=gen)[:T * k].reshape(T, k).to(torch.int32)
    else:
        M, F, E = case["M"], case["F"], case["E"]
        s["h"] = _randn(gen, M, 2 * F, scale=1.5)
        s["offs"] = _offsets(gen, M, E)
        width = F if op == "swiglu_fwd" else 2 * F
        if op == "swiglu_bwd":
            s["dout"] = _randn(gen, M, F)
        p = s["plan"]
        p["out"] = torch.empty(M, width, dtype=BF16, device=DEV) if case["y"] else None
        p["q0"] = torch.empty(M, width, dtype=torch.uint8, device=DEV)
        p["s0"] = torch.zeros((_up(M, 128) // 128 + E) * 128 * _up(width // 32, 4), dtype=torch.uint8, device=DEV)
        if case["dim1"]:
            p["q1"] = torch.empty(width, M, dtype=torch.uint8, device=DEV)
            p["s1"] = torch.zeros(_up(width, 128) * (_up(M // 32, 4) + 4 * E), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


# --- plain forms ------------------------------------------------------------

def _softmax(x):
    """Softmax over the last axis; a row of nothing but -inf is all zero."""
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    z = e.sum(-1, keepdim=True)
    return e / torch.where(z > 0, z, torch.ones_like(z))


def _mx(v):
    """[.., C] fp32 -> (e4m3 codes, e8m0 bytes [.., C / 32])."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    field = (b.abs().amax(-1).view(torch.int32) >> 23) & 0xFF
    byte = field.clamp(min=8) - 8
    inv = ((254 - byte) << 23).view(F32)                      # 2^-(byte - 127)
    q = (b * inv[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    return q.reshape(v.shape), byte.to(torch.uint8)


def _tile_index(rows, cols, width):
    """Byte of scale (row, col) in the 128x4 tile layout, `width` columns."""
    r, c = rows[:, None], cols[None, :]
    return (r // 128 * (width // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4


def _scatter_tiles(scales, rows, cols, width, total):
    out = torch.zeros(total, dtype=torch.uint8, device=DEV)
    out[_tile_index(rows, cols, width).reshape(-1)] = scales.reshape(-1)
    return out


def _padded_rows(offs, M):
    """Row of each token in the layout whose groups start at multiples of 128."""
    ends = offs.to(torch.int64)
    start = torch.cat([torch.zeros_like(ends[:1]), ends[:-1]])
    pad = (ends - start + 127) // 128 * 128
    first = pad.cumsum(0) - pad
    r = torch.arange(M, device=DEV)
    g = torch.searchsorted(ends, r, right=True)
    return first[g] + r - start[g]


def _plain_norm_fwd(s):
    a = s["x"].float()
    out = []
    if s["r"] is not None:
        a = a + s["r"].float()
        out.append(a.to(BF16))
    rstd = torch.rsqrt(a.square().mean(1) + EPS)
    y = a * rstd[:, None] * s["w"].float()
    if s["y"]:
        out.append(y.to(BF16))
    if s["rstd"]:
        out.append(rstd)
    if s["recipe"] == "mx":
        q, b = _mx(y)
        if s["tiled"]:
            T, C = b.shape
            b = _scatter_tiles(b, torch.arange(T, device=DEV), torch.arange(C, device=DEV), _up(C, 4),
                               _tiled_bytes(T, C))
        out += [q, b.view(E8M0)]
    elif s["recipe"] == "rowwise":
        scale = E4M3_MAX / y.abs().amax(1).clamp(min=1e-12)
        out += [(y * scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), 1.0 / scale]
    return out


def _plain_norm_bwd(s):
    dy, xh = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return [dx.to(BF16), (dy * xh).sum(0)]


def _scores(s):
    """(logits with masked tokens at -inf, scores, probabilities of the balance loss)."""
    x = s["logits"].float()
    if s["mask"] is not None:
        x = torch.where(s["mask"][:, None] != 0, x, torch.full_like(x, -math.inf))
    if s["score"] == "softmax":
        p = _softmax(x)
        return x, p, p
    sc = 1.0 / (1.0 + torch.exp(-x))
    z = sc.sum(1, keepdim=True)
    return x, sc, sc / torch.where(z > 0, z, torch.ones_like(z))


def _plain_router_fwd(s):
    T, E, k = s["T"], s["E"], s["k"]
    x, sc, p = _scores(s)
    idx = _choose(x, s["bias"], s["score"], k)
    w = torch.gather(sc, 1, idx)
    if s["renorm"]:
        z = w.sum(1, keepdim=True)
        w = w / torch.where(z > 0, z, torch.ones_like(z))
    w = w * 2.5
    live = torch.gather(x, 1, idx) > -math.inf
    counts = torch.zeros(E, dtype=torch.int64, device=DEV)
    counts.scatter_add_(0, idx.reshape(-1), live.reshape(-1).to(torch.int64))
    n = torch.full((1,), T, dtype=torch.int64, device=DEV) if s["mask"] is None else s["mask"].sum().reshape(1)
    psum = p.sum(0)
    nf = n.float().clamp(min=1.0)
    loss = (counts.float() * psum).sum().reshape(1) * (E / k) / (nf * nf)
    return [idx.to(torch.int32), w, torch.cat([counts, n]).to(torch.int32), psum, loss]


def _plain_router_bwd(s):
    E, k = s["E"], s["k"]
    x, sc, p = _scores(s)
    idx = s["idx"].to(torch.int64)
    n = s["counts"][E].float().clamp(min=1.0)
    c = s["dloss"] * (E / k) / (n * n) * s["counts"][:E].float()
    r = p * (c - (p * c).sum(1, keepdim=True))
    w, dw = torch.gather(sc, 1, idx), s["dw"]
    if s["renorm"]:
        z = w.sum(1, keepdim=True)
        w = w / torch.where(z > 0, z, torch.ones_like(z))
        u = w * (dw - (dw * w).sum(1, keepdim=True))
    else:
        u = w * dw
    u = u * 2.5
    if s["score"] == "softmax":
        d = (r - p * u.sum(1, keepdim=True)).scatter_add(1, idx, u)
    else:
        d = r.scatter_add(1, idx, u) * (1.0 - sc)
    return [d.to(s["logits"].dtype)]


def _plain_weight_grad(s):
    return [(s["y"].float()[s["row_of"].to(torch.int64)] * s["dout"].float()[:, None, :]).sum(-1)]


def _plain_quant(s, v):
    M, width = v.shape
    out = [v.to(BF16)] if s["y"] else []
    rows = _padded_rows(s["offs"], M)
    q, b = _mx(v)
    out += [q, _scatter_tiles(b, rows, torch.arange(width // 32, device=DEV), _up(width // 32, 4),
                              s["plan"]["s0"].numel()).view(E8M0)]
    if s["dim1"]:
        q, b = _mx(v.t().contiguous())
        out += [q, _scatter_tiles(b, torch.arange(width, device=DEV), rows[::32] // 32,
                                  _up(M // 32, 4) + 4 * s["E"], s["plan"]["s1"].numel()).view(E8M0)]
    return out


def _plain_swiglu_fwd(s):
    g, u = s["h"].float().chunk(2, dim=1)
    return _plain_quant(s, g / (1.0 + torch.exp(-g)) * u)


def _plain_swiglu_bwd(s):
    g, u = s["h"].float().chunk(2, dim=1)
    d = s["dout"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    return _plain_quant(s, torch.cat([d * u * sig * (1.0 + g * (1.0 - sig)), d * g * sig], dim=1))


_plain = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "router_fwd": _plain_router_fwd,
          "router_bwd": _plain_router_bwd, "weight_grad": _plain_weight_grad, "swiglu_fwd": _plain_swiglu_fwd,
          "swiglu_bwd": _plain_swiglu_bwd}


# --- the framework's operators ------------------------------------------------

def _own_norm_fwd(s):
    import mxfp8_moe_quantization_gb300 as F
    recipe = {"mx": F.MXFP8, "rowwise": F.ROWWISE, "none": None}[s["recipe"]]
    h, y, rstd, q, scale = F.fp8moe_add_rmsnorm_fwd(
        s["x"], s["w"], s["r"], eps=EPS, recipe=recipe, scale_layout=F.NO_GROUPS if s["tiled"] else F.SCALES_ROWMAJOR,
        need_y=s["y"], need_rstd=s["rstd"], **s["plan"])
    out = [t for t in (h, y, rstd) if t is not None]
    if q is not None:
        out += [q.view(E4M3), scale.view(E8M0) if s["recipe"] == "mx" else scale]
    return out


def _own_norm_bwd(s):
    import mxfp8_moe_quantization_gb300 as F
    return list(F.fp8moe_add_rmsnorm_bwd(s["dy"], s["h"], s["rstd"], s["w"], s["dh"]))


def _own_router_fwd(s):
    import mxfp8_moe_quantization_gb300 as F
    score = F.SCORE_SOFTMAX if s["score"] == "softmax" else F.SCORE_SIGMOID
    return list(F.fp8moe_router_fwd(s["logits"], s["k"], score=score, renormalize=s["renorm"], route_scale=2.5,
                                    bias=s["bias"], token_mask=s["mask"]))


def _own_router_bwd(s):
    import mxfp8_moe_quantization_gb300 as F
    score = F.SCORE_SOFTMAX if s["score"] == "softmax" else F.SCORE_SIGMOID
    return [F.fp8moe_router_bwd(s["logits"], s["idx"], s["counts"], s["dw"], s["dloss"], score=score,
                                renormalize=s["renorm"], route_scale=2.5, token_mask=s["mask"])]


def _own_weight_grad(s):
    import mxfp8_moe_quantization_gb300 as F
    return [F.fp8moe_route_weight_grad(s["dout"], s["y"], s["row_of"])]


def _own_swiglu(s, result):
    out, q0, s0, q1, s1 = result
    return ([out] if out is not None else []) + [q0.view(E4M3), s0.view(E8M0)] + (
        [q1.view(E4M3), s1.view(E8M0)] if q1 is not None else [])


def _own_swiglu_fwd(s):
    import mxfp8_moe_quantization_gb300 as F
    return _own_swiglu(s, F.fp8moe_swiglu_fwd(
        s["h"], s["offs"], F.GROUP_ROWS, F.GROUP_COLS, need_out=s["y"], dim0=True, dim1=s["dim1"], **s["plan"]))


def _own_swiglu_bwd(s):
    import mxfp8_moe_quantization_gb300 as F
    return _own_swiglu(s, F.fp8moe_swiglu_bwd(
        s["dout"], s["h"], s["offs"], F.GROUP_ROWS, F.GROUP_COLS, need_dh=s["y"], dim0=True, dim1=s["dim1"],
        **s["plan"]))


_own = {"norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "router_fwd": _own_router_fwd,
        "router_bwd": _own_router_bwd, "weight_grad": _own_weight_grad, "swiglu_fwd": _own_swiglu_fwd,
        "swiglu_bwd": _own_swiglu_bwd}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_64(v):
    """The nearest e4m3fn value (ties to even, saturating), in float64."""
    a = v.abs().clamp(max=E4M3_MAX)
    step = torch.exp2((torch.frexp(a)[1] - 1).clamp(min=-6).to(F64) - 3.0)
    return torch.copysign((torch.round(a / step) * step).clamp(max=E4M3_MAX), v)


def _mx_64(v):
    """[R, C] float64 -> (e4m3 values, scale values 2^e [R, C / 32])."""
    b = v.unflatten(1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 1 - 8).clamp(-127, 127), torch.full_like(amax, -127).int())
    scale = torch.exp2(e.to(F64))
    return _e4m3_64(b / scale[..., None]).flatten(1), scale


def _tile_order(full):
    """A padded [128 i, 4 j] matrix in the byte order of the 128x4 tiles."""
    R, C = full.shape
    return full.reshape(R // 128, 4, 32, C // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _place(scale, at_rows, at_cols, shape):
    full = torch.full(shape, 2.0 ** -127, dtype=F64, device=DEV)
    full[at_rows[:, None], at_cols[None, :]] = scale
    return _tile_order(full)


def _group_rows_64(offs):
    at, base, begin = [], 0, 0
    for end in offs.tolist():
        at.append(torch.arange(end - begin) + base)
        base += _up(end - begin, 128)
        begin = end
    return torch.cat(at).to(DEV)


def _exact_quant(s, v):
    M, width = v.shape
    out = [v] if s["y"] else []
    rows = _group_rows_64(s["offs"])
    q, sc = _mx_64(v)
    out += [q, _place(sc, rows, torch.arange(width // 32, device=DEV),
                      ((_up(M, 128) // 128 + s["E"]) * 128, _up(width // 32, 4)))]
    if s["dim1"]:
        q, sc = _mx_64(v.t().contiguous())
        out += [q, _place(sc, torch.arange(width, device=DEV), rows.reshape(-1, 32)[:, 0] // 32,
                          (_up(width, 128), _up(M // 32, 4) + 4 * s["E"]))]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        a = s["x"].to(F64) + (s["r"].to(F64) if case["residual"] else 0.0)
        rstd = ((a * a).sum(1) / case["H"] + EPS) ** -0.5
        y = a * s["w"].to(F64) * rstd[:, None]
        out = ([a] if case["residual"] else []) + ([y] if case["y"] else []) + ([rstd] if case["rstd"] else [])
        if case["recipe"] == "mx":
            q, sc = _mx_64(y)
            T, C = sc.shape
            if case["tiled"]:
                sc = _place(sc, torch.arange(T, device=DEV), torch.arange(C, device=DEV), (_up(T, 128), _up(C, 4)))
            out += [q, sc]
        elif case["recipe"] == "rowwise":
            inv = y.abs().amax(1).clamp(min=1e-12) / E4M3_MAX
            out += [_e4m3_64(y / inv[:, None]), inv]
        return out
    if op == "norm_bwd":
        h, dy, w, rstd = (s[n].to(F64) for n in ("h", "dy", "w", "rstd"))
        c = (dy * w * h).sum(1) * rstd.pow(3) / case["H"]
        dx = dy * w * rstd[:, None] - h * c[:, None]
        return [dx + s["dh"].to(F64) if case["stream"] else dx, torch.einsum("th,th,t->h", dy, h, rstd)]
    if op in ("router_fwd", "router_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        x = s["logits"].to(F64)
        if s["mask"] is not None:
            x = x.masked_fill(s["mask"][:, None] == 0, -math.inf)
        if case["score"] == "softmax":
            sc = p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True)).nan_to_num(0.0)
        else:
            sc = torch.sigmoid(x)
            p = (sc / sc.sum(1, keepdim=True)).nan_to_num(0.0)
        n = float(T if s["mask"] is None else int(s["mask"].sum()))
        if op == "router_fwd":
            key = x.float() if s["bias"] is None else (sc.float() + s["bias"]).masked_fill(x == -math.inf, -math.inf)
            idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
            w = sc.gather(1, idx)
            if case["renorm"]:
                w = (w / w.sum(1, keepdim=True)).nan_to_num(0.0)
            live = (x.gather(1, idx) > -math.inf).to(F64)
            counts = torch.zeros(E, dtype=F64, device=DEV).scatter_add_(0, idx.flatten(), live.flatten())
            loss = (counts @ p.sum(0)) * E / (k * max(n, 1.0) ** 2)
            return [None, w * 2.5, None, p.sum(0), loss.reshape(1)]
        # the gradient written with the whole Jacobians of scores and weights
        idx = s["idx"].long()
        gp = s["dloss"].to(F64) * E / (k * max(n, 1.0) ** 2) * s["counts"][:E].to(F64)
        sel, dw = sc.gather(1, idx), 2.5 * s["dw"].to(F64)
        if case["renorm"]:
            z = sel.sum(1, keepdim=True)
            gs = ((dw - (dw * sel).sum(1, keepdim=True) / z) / z).nan_to_num(0.0, 0.0, 0.0)
        else:
            gs = dw
        gsel = torch.zeros_like(sc).scatter_(1, idx, gs)
        if case["score"] == "softmax":
            g = gp + gsel
            return [p * (g - (p * g).sum(1, keepdim=True))]
        z = sc.sum(1, keepdim=True)
        g = ((gp - (p * gp).sum(1, keepdim=True)) / z).nan_to_num(0.0, 0.0, 0.0) + gsel
        return [g * sc * (1.0 - sc)]
    if op == "weight_grad":
        d, y, at = s["dout"].to(F64), s["y"], s["row_of"].long()
        return [torch.stack([(y[at[:, j]].to(F64) * d).sum(1) for j in range(case["k"])], 1)]
    g, u = s["h"][:, :case["F"]].to(F64), s["h"][:, case["F"]:].to(F64)
    sig = torch.sigmoid(g)
    if op == "swiglu_fwd":
        return _exact_quant(s, g * sig * u)
    d = s["dout"].to(F64)
    return _exact_quant(s, torch.cat([d * u * (sig + g * sig * (1.0 - sig)), d * g * sig], 1))
