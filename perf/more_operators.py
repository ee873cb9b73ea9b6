"""Cases of the expert layer for a few tokens, and of its training with
activations kept in 8 bits.

Five operators: the whole expert layer of a few tokens on MXFP8 weights (both
products, the activation and the weighted sum over the experts); the gated
activation that also writes its input as an MXFP8 checkpoint; its backward from
that checkpoint, which also gives the activation's operand for the weight
gradient; the norm's backward from an MXFP8 checkpoint; and the gradient of the
combine's weights from expert outputs kept in MXFP8.  With ``own`` false
``run`` computes them with elementary torch operations in 32 bits; with ``own``
true it calls this package.
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
        # one answered token through MoE-16B's expert layer: six experts, latency as much as bandwidth
        dict(name="decode_moe16b_token", op="decode", T=1, H=2048, F=1408, E=64, k=6, masked=0, away=0.0),
        # one answered token through DeepSeek-V3's
        dict(name="decode_dsv3_token", op="decode", T=1, H=7168, F=2048, E=256, k=8, masked=0, away=0.0),
        # a batch of 23 sequences, three of them ended (weights 0), a tenth of the choices on another device
        dict(name="decode_dsv3_batch", op="decode", T=23, H=7168, F=2048, E=256, k=8, masked=3, away=0.1),
        # Llama4-Scout's layer, one expert a token, a full batch of sequences
        dict(name="decode_scout_batch", op="decode", T=64, H=5120, F=8192, E=16, k=1, masked=0, away=0.0),
        # DeepSeek-V3's routed batch: 256 ragged groups, both directions for forward and weight gradient
        dict(name="swiglu_fwd_dsv3", op="swiglu_fwd", M=36448, F=2048, E=256, y=False, dim1=True),
        # MoE-16B's width with few rows, a recomputed slice of a batch: row direction and checkpoint alone
        dict(name="swiglu_fwd_slice", op="swiglu_fwd", M=416, F=1408, E=5, y=False, dim1=False),
        # MoE-16B's routed batch backward, both directions of the gradient, the activation for the weight gradient
        dict(name="swiglu_bwd_moe16b", op="swiglu_bwd", M=51136, F=1408, E=64, y=False, dim1=True, act=True),
        # a small batch: gradients as bf16 rows and both directions
        dict(name="swiglu_bwd_small", op="swiglu_bwd", M=480, F=2048, E=16, y=True, dim1=True, act=True),
        # the Llama4-Scout layer's norm backward, with the gradient that comes along the residual stream
        dict(name="norm_bwd_scout", op="norm_bwd", T=16384, H=5120, stream=True, w32=False),
        # Llama3-8B rows, a batch cut short by one token
        dict(name="norm_bwd_ragged", op="norm_bwd", T=8191, H=4096, stream=False, w32=True),
        # the combine's weights of DeepSeek-V3's batch: every routed row against its token's gradient
        dict(name="weight_grad_dsv3", op="weight_grad", T=4096, N=7168, k=8),
        # MoE-16B's batch, cut short
        dict(name="weight_grad_moe16b", op="weight_grad", T=8189, N=2048, k=6),
    ]


def _logsize(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "swiglu_fwd", "swiglu_bwd", "norm_bwd", "weight_grad"])
    flag = lambda p=0.5: rng.random() < p  # noqa: E731
    if op == "decode":
        H, F = 32 * _logsize(rng, 8, 256), 32 * _logsize(rng, 4, 256)
        E = rng.choice([4, 8, 16, 60, 64, 100, 128, 160, 256])
        E = max(2, min(E, 2_000_000_000 // (3 * H * F)))
        k = rng.randint(1, min(E, 8))
        T = _logsize(rng, 1, max(1, min(96, 8_000_000_000 // (3 * H * F * k))))
        return dict(op=op, T=T, H=H, F=F, E=E, k=k, masked=rng.choice([0, 0, T // 3]), away=rng.choice([0.0, 0.0, 0.3]))
    if op in ("swiglu_fwd", "swiglu_bwd"):
        F = 32 * _logsize(rng, 4, 200)
        rows = 32 * _logsize(rng, 1, 50_000_000 // F // 32)
        c = dict(op=op, M=rows, F=F, E=min(_logsize(rng, 1, 256), rows // 32), y=flag(0.3), dim1=flag(0.7))
        return dict(c, act=flag(0.7)) if op == "swiglu_bwd" else c
    if op == "norm_bwd":
        H = 32 * _logsize(rng, 8, 256)
        return dict(op=op, T=_logsize(rng, 1, min(40000, 80_000_000 // H)), H=H, stream=flag(), w32=flag())
    N, k = 32 * _logsize(rng, 4, 256), rng.randint(1, 8)
    return dict(op=op, T=_logsize(rng, 1, 230_000_000 // (N * (k + 1))), N=N, k=k)


# ---------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------

def _up(a, b):
    return (a + b - 1) // b * b


MX = 1 + 1 / 32      # bytes of an MXFP8 element


def work(case):
    op = case["op"]
    if op == "decode":
        T, H, F, E, k = (case[n] for n in "THFEk")
        pairs = (T - case["masked"]) * k * (1.0 - case["away"])
        live = E * (1.0 - (1.0 - min(1.0, pairs / max(T, 1) / E)) ** T)   # experts that some token meets, on average
        return {"bytes": live * 3 * H * F * MX + T * (4 * H + 8 * k), "flops": 6 * pairs * H * F}
    if op == "norm_bwd":
        T, H = case["T"], case["H"]
        return {"bytes": T * (H * (4 + MX + (2 if case["stream"] else 0)) + 4) + H * ((4 if case["w32"] else 2) + 4),
                "flops": 13 * T * H}
    if op == "weight_grad":
        T, N, k = case["T"], case["N"], case["k"]
        return {"bytes": T * (N * (2 + MX * k) + 8 * k), "flops": 3 * T * N * k}
    M, F = case["M"], case["F"]
    dirs = 2 if case["dim1"] else 1
    if op == "swiglu_fwd":
        return {"bytes": M * F * (4 + 2 * MX + dirs * MX + (2 if case["y"] else 0)), "flops": M * F * 11}
    return {"bytes": M * F * (2 + 2 * MX + 2 * dirs * MX + (MX if case["act"] else 0) + (4 if case["y"] else 0)),
            "flops": M * F * 24}


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


def _offsets(gen, M, E):
    """Cumulative ends of E ragged groups of whole 32-row blocks, some empty."""
    share = torch.rand(E, device=DEV, generator=gen).pow(3)
    cum = share.cumsum(0) / share.sum()
    ends = (cum * (M // 32)).round().to(torch.int32) * 32
    ends[-1] = M
    return ends


def _pack(v):
    """MXFP8 of v [R, C] (bytes): codes [R, C], e8m0 scales [R, C / 32]; in pieces of rows."""
    R, C = v.shape
    q = torch.empty(R, C, dtype=torch.uint8, device=DEV)
    s = torch.empty(R, C // 32, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // C)
    for r in range(0, R, step):
        codes, scale = _mx(v[r:r + step].float())
        q[r:r + step], s[r:r + step] = codes.view(torch.uint8), scale
    return q, s


def _weights(gen, E, N, K):
    """[E, N, K] weights as MXFP8 codes, and their scales in 128x4 tiles."""
    q = torch.empty(E, N, K, dtype=torch.uint8, device=DEV)
    per = _up(N, 128) * _up(K // 32, 4)
    s = torch.zeros(E, per, dtype=torch.uint8, device=DEV)
    at = _tile_index(torch.arange(N, device=DEV), torch.arange(K // 32, device=DEV), _up(K // 32, 4)).reshape(-1)
    for e in range(E):
        codes, scale = _mx(torch.randn(N, K, device=DEV, generator=gen) * K ** -0.5)
        q[e] = codes.view(torch.uint8)
        s[e, at] = scale.reshape(-1)
    return q, s.reshape(-1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, s = case["op"], dict(case)
    p = s["plan"] = {}
    if op == "decode":
        T, H, F, E, k = (case[n] for n in "THFEk")
        s["x"] = _rows(gen, T, H)
        s["idx"] = torch.rand(T, E, device=DEV, generator=gen).topk(k, dim=1)[1].to(torch.int32)
        w = torch.rand(T, k, device=DEV, generator=gen) + 0.1
        s["w"] = w / w.sum(1, keepdim=True)
        if case["masked"]:      # rows that are no token: the router gives them weight 0
            s["w"][torch.randperm(T, device=DEV, generator=gen)[:case["masked"]]] = 0.0
        if case["away"]:        # experts that another device holds
            s["idx"][torch.rand(T, k, device=DEV, generator=gen) < case["away"]] = -1
        s["w1"], s["s1"] = _weights(gen, E, 2 * F, H)
        s["w2"], s["s2"] = _weights(gen, E, H, F)
        p["out"] = torch.empty(T, H, dtype=BF16, device=DEV)
        if own:
            import mxfp8_moe_quantization_gb300 as fp8moe
            p["workspace"] = torch.empty(fp8moe.fp8moe_mxfp8_moe_decode_workspace_bytes(T, k, E, H, F), dtype=torch.uint8,
                                         device=DEV)
    elif op == "norm_bwd":
        T, H = case["T"], case["H"]
        h = _rows(gen, T, H)
        s["w"] = _randn(gen, H, dtype=F32, scale=0.2).add_(1.0).to(F32 if case["w32"] else BF16)
        s["hq"], s["hs"] = _pack(h)
        s["rstd"] = torch.rsqrt(h.float().square().mean(1) + EPS)
        s["dy"] = _randn(gen, T, H)
        s["dh"] = _randn(gen, T, H) if case["stream"] else None
    elif op == "weight_grad":
        T, N, k = case["T"], case["N"], case["k"]
        rows = _up(T * k + 32, 32)
        s["yq"], s["ys"] = _pack(_randn(gen, rows, N))
        s["dout"] = _randn(gen, T, N)
        s["row_of"] = torch.randperm(rows, device=DEV, generator=gen)[:T * k].reshape(T, k).to(torch.int32)
    else:
        M, F, E = case["M"], case["F"], case["E"]
        h = _randn(gen, M, 2 * F, scale=1.5)
        s["offs"] = _offsets(gen, M, E)
        if op == "swiglu_fwd":
            s["h"], width = h, F
            p["hq"] = torch.empty(M, 2 * F, dtype=torch.uint8, device=DEV)
            p["hs"] = torch.empty(M, 2 * F // 32, dtype=torch.uint8, device=DEV)
        else:
            (s["hq"], s["hs"]), width = _pack(h), 2 * F
            s["dout"] = _randn(gen, M, F)
        # the output buffers that a program keeps from step to step
        cols = _up(M // 32, 4) + 4 * E
        p["out"] = torch.empty(M, width, dtype=BF16, device=DEV) if case["y"] else None
        p["q0"] = torch.empty(M, width, dtype=torch.uint8, device=DEV)
        p["s0"] = torch.zeros((_up(M, 128) // 128 + E) * 128 * _up(width // 32, 4), dtype=torch.uint8, device=DEV)
        if case["dim1"]:
            p["q1"] = torch.empty(width, M, dtype=torch.uint8, device=DEV)
            p["s1"] = torch.zeros(_up(width, 128) * cols, dtype=torch.uint8, device=DEV)
        if op == "swiglu_bwd" and case["act"]:
            p["aq1"] = torch.empty(F, M, dtype=torch.uint8, device=DEV)
            p["as1"] = torch.zeros(_up(F, 128) * cols, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


# --- plain forms ------------------------------------------------------------

def _mx(v):
    """[.., C] fp32 -> (e4m3 codes, e8m0 bytes [.., C / 32])."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    field = (b.abs().amax(-1).view(torch.int32) >> 23) & 0xFF
    byte = field.clamp(min=8) - 8
    inv = ((254 - byte) << 23).view(F32)                      # 2^-(byte - 127)
    q = (b * inv[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    return q.reshape(v.shape), byte.to(torch.uint8)


def _power(byte):
    """2^(byte - 127) in fp32."""
    return torch.exp2(byte.to(F32) - 127.0)


def _unpack(q, byte):
    """fp32 values of codes [.., C] with row-major scale bytes [.., C / 32]."""
    v = q.view(E4M3).to(F32)
    return (v.reshape(*byte.shape, 32) * _power(byte)[..., None]).reshape(v.shape)


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


def _plain_decode(s):
    T, H, F, E = (s[n] for n in "THFE")
    t1 = _tile_index(torch.arange(2 * F, device=DEV), torch.arange(H // 32, device=DEV), _up(H // 32, 4))
    t2 = _tile_index(torch.arange(H, device=DEV), torch.arange(F // 32, device=DEV), _up(F // 32, 4))
    s1, s2 = s["s1"].view(E, -1), s["s2"].view(E, -1)
    live = (s["idx"] >= 0) & (s["idx"] < E) & (s["w"] != 0)
    ids = torch.where(live, s["idx"], torch.zeros_like(s["idx"])).to(torch.int64)
    out = torch.empty(T, H, dtype=F32, device=DEV)
    for t in range(T):      # a token at a time: its experts' weights fit in 32 bits
        e = ids[t]
        gu = torch.matmul(_unpack(s["w1"][e], s1[e][:, t1]), s["x"][t].float())
        g, u = gu.chunk(2, dim=1)
        a = g / (1.0 + torch.exp(-g)) * u
        y = torch.matmul(_unpack(s["w2"][e], s2[e][:, t2]), a[:, :, None])[:, :, 0]
        y = torch.where(live[t][:, None], y * s["w"][t][:, None], torch.zeros_like(y))
        out[t] = y.sum(0)
    return [out.to(BF16)]


def _plain_quant(s, v):
    M, width = v.shape
    out = [v.to(BF16)] if s["y"] else []
    rows = _padded_rows(s["offs"], M)
    q, b = _mx(v)
    out += [q, _scatter_tiles(b, rows, torch.arange(width // 32, device=DEV), _up(width // 32, 4),
                              s["plan"]["s0"].numel()).view(E8M0)]
    return out + (_plain_columns(s, v, s["plan"]["s1"].numel()) if s["dim1"] else [])


def _plain_columns(s, v, total):
    M, width = v.shape
    q, b = _mx(v.t().contiguous())
    return [q, _scatter_tiles(b, torch.arange(width, device=DEV), _padded_rows(s["offs"], M)[::32] // 32,
                              _up(M // 32, 4) + 4 * s["E"], total).view(E8M0)]


def _plain_swiglu_fwd(s):
    h = s["h"].float()
    g, u = h.chunk(2, dim=1)
    q, b = _mx(h)
    return _plain_quant(s, g / (1.0 + torch.exp(-g)) * u) + [q, b.view(E8M0)]


def _plain_swiglu_bwd(s):
    g, u = _unpack(s["hq"], s["hs"]).chunk(2, dim=1)
    d = s["dout"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    out = _plain_quant(s, torch.cat([d * u * sig * (1.0 + g * (1.0 - sig)), d * g * sig], dim=1))
    return out + (_plain_columns(s, g * sig * u, s["plan"]["as1"].numel()) if s["act"] else [])


def _plain_norm_bwd(s):
    dy, xh = s["dy"].float(), _unpack(s["hq"], s["hs"]) * s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return [dx.to(BF16), (dy * xh).sum(0)]


def _plain_weight_grad(s):
    y, at = _unpack(s["yq"], s["ys"]), s["row_of"].to(torch.int64)
    return [(y[at] * s["dout"].float()[:, None, :]).sum(-1)]


_plain = {"decode": _plain_decode, "swiglu_fwd": _plain_swiglu_fwd, "swiglu_bwd": _plain_swiglu_bwd,
          "norm_bwd": _plain_norm_bwd, "weight_grad": _plain_weight_grad}


# --- the framework's operators ------------------------------------------------

def _own_decode(s):
    import mxfp8_moe_quantization_gb300 as F
    return [F.fp8moe_mxfp8_moe_decode(s["x"], s["idx"], s["w"], s["w1"], s["s1"], s["w2"], s["s2"], **s["plan"])]


def _own_mx(pairs):
    out = []
    for q, scale in pairs:
        out += [q.view(E4M3), scale.view(E8M0)] if q is not None else []
    return out


def _own_swiglu_fwd(s):
    import mxfp8_moe_quantization_gb300 as F
    out, q0, s0, q1, s1, hq, hs = F.fp8moe_swiglu_fwd_ckpt(
        s["h"], s["offs"], F.GROUP_ROWS, F.GROUP_COLS, need_out=s["y"], dim0=True, dim1=s["dim1"], **s["plan"])
    return ([out] if out is not None else []) + _own_mx([(q0, s0), (q1, s1), (hq, hs)])


def _own_swiglu_bwd(s):
    import mxfp8_moe_quantization_gb300 as F
    out, q0, s0, q1, s1, aq1, as1 = F.fp8moe_swiglu_bwd_ckpt(
        s["dout"], s["hq"], s["hs"], s["offs"], F.GROUP_ROWS, F.GROUP_COLS, need_dh=s["y"], dim0=True, dim1=s["dim1"],
        act1=s["act"], **s["plan"])
    return ([out] if out is not None else []) + _own_mx([(q0, s0), (q1, s1), (aq1, as1)])


def _own_norm_bwd(s):
    import mxfp8_moe_quantization_gb300 as F
    return list(F.fp8moe_add_rmsnorm_bwd_ckpt(s["dy"], s["hq"], s["hs"], s["rstd"], s["w"], s["dh"]))


def _own_weight_grad(s):
    import mxfp8_moe_quantization_gb300 as F
    return [F.fp8moe_route_weight_grad_ckpt(s["dout"], s["yq"], s["ys"], s["row_of"])]


_own = {"decode": _own_decode, "swiglu_fwd": _own_swiglu_fwd, "swiglu_bwd": _own_swiglu_bwd, "norm_bwd": _own_norm_bwd,
        "weight_grad": _own_weight_grad}


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


def _value_64(q, scale):
    """float64 values of codes [R, C] whose scales [R, C / 32] are bytes."""
    return (q.view(E4M3).to(F64).unflatten(1, (-1, 32)) * torch.ldexp(torch.ones_like(scale, dtype=F64),
                                                                       scale.to(torch.int32) - 127)[..., None]).flatten(1)


def _tile_order(full):
    """A padded [128 i, 4 j] matrix in the byte order of the 128x4 tiles."""
    R, C = full.shape
    return full.reshape(R // 128, 4, 32, C // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _from_tiles(flat, R, C):
    """The [R, C] matrix that a 128x4 buffer holds."""
    i, j = _up(R, 128) // 128, _up(C, 4) // 4
    return flat.reshape(i, j, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(i * 128, j * 4)[:R, :C]


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


def _exact_columns(s, v):
    M, width = v.shape
    q, sc = _mx_64(v.t().contiguous())
    return [q, _place(sc, torch.arange(width, device=DEV), _group_rows_64(s["offs"]).reshape(-1, 32)[:, 0] // 32,
                      (_up(width, 128), _up(M // 32, 4) + 4 * s["E"]))]


def _exact_quant(s, v):
    M, width = v.shape
    out = [v] if s["y"] else []
    q, sc = _mx_64(v)
    out += [q, _place(sc, _group_rows_64(s["offs"]), torch.arange(width // 32, device=DEV),
                      ((_up(M, 128) // 128 + s["E"]) * 128, _up(width // 32, 4)))]
    return out + (_exact_columns(s, v) if s["dim1"] else [])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "decode":
        T, H, F, E, k = (case[n] for n in "THFEk")
        out = torch.zeros(T, H, dtype=F64, device=DEV)
        idx, w, x = s["idx"].tolist(), s["w"].to(F64), s["x"].to(F64)
        # an expert at a time, for every token that chose it
        for e in range(E):
            of = [(t, j) for t in range(T) for j in range(k) if idx[t][j] == e and float(w[t, j]) != 0.0]
            if not of:
                continue
            t, j = (torch.tensor(v, device=DEV) for v in zip(*of))
            w1 = _value_64(s["w1"][e], _from_tiles(s["s1"].view(E, -1)[e], 2 * F, H // 32))
            w2 = _value_64(s["w2"][e], _from_tiles(s["s2"].view(E, -1)[e], H, F // 32))
            gate, up = x[t] @ w1[:F].t(), x[t] @ w1[F:].t()
            out.index_add_(0, t, w[t, j][:, None] * ((gate * torch.sigmoid(gate) * up) @ w2.t()))
        return [out]
    if op == "norm_bwd":
        h, dy, w, rstd = _value_64(s["hq"], s["hs"]), s["dy"].to(F64), s["w"].to(F64), s["rstd"].to(F64)
        c = (dy * w * h).sum(1) * rstd.pow(3) / case["H"]
        dx = dy * w * rstd[:, None] - h * c[:, None]
        return [dx + s["dh"].to(F64) if case["stream"] else dx, torch.einsum("th,th,t->h", dy, h, rstd)]
    if op == "weight_grad":
        d, at = s["dout"].to(F64), s["row_of"].long()
        return [torch.stack([(_value_64(s["yq"][at[:, j]], s["ys"][at[:, j]]) * d).sum(1) for j in range(case["k"])], 1)]
    if op == "swiglu_fwd":
        h = s["h"].to(F64)
        g, u = h[:, :case["F"]], h[:, case["F"]:]
        return _exact_quant(s, g * torch.sigmoid(g) * u) + list(_mx_64(h))
    h, d = _value_64(s["hq"], s["hs"]), s["dout"].to(F64)
    g, u = h[:, :case["F"]], h[:, case["F"]:]
    sig = torch.sigmoid(g)
    out = _exact_quant(s, torch.cat([d * u * (sig + g * sig * (1.0 - sig)), d * g * sig], 1))
    return out + (_exact_columns(s, g * sig * u) if case["act"] else [])
