"""The FP4, gated-norm and rotary operators of libh3dit: what is timed, on which inputs, in plain form and through the library.

The four operators sit around the linears of a DiT block whose matrices are kept in 4 bits:

  quantize  a bf16 or fp32 matrix to 4-bit floating point (E2M1) with one scale per 32 (MXFP4, E8M0) or per 16 (NVFP4,
            E4M3 and one fp32 tensor scale taken from the matrix), and back to bf16
  linear    the product of two such matrices, with a bias and the epilogues the block's linears have
  norm      x' = r x + gate * RMSNorm(branch); RMSNorm(x') (1 + scale) + shift, the row handed on as bf16 or as FP4
  rope      RMSNorm of each query and key head, then the rotation by positions on three axes (frame, row, column)

Sizes come from the model this package runs (hidden 5376, 56 heads of 96 or 128, FFN 14336; 256 + 32, 4096 + 512,
16384 + 512 and 20480 + 256 tokens) and from its small block (hidden 768, 8 heads, FFN 2048).

FP4 matrices are held as users hold them: two codes per byte (even column in the low half) and the scale bytes in blocks
of 128 rows x 4 scales; the scale of row r and block s of a row with S blocks is byte
((r / 128) * ceil(S / 4) + s / 4) * 512 + (r % 32) * 16 + (r / 32 % 4) * 4 + s % 4.
"""
import functools
import math

import numpy as np
import torch

own = False

EPS = 1e-6  # of every norm; the library's default
THETA = 10000.0
BLOCK = {"mx": 32, "nv": 16}


# ---------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # the input of a 4096^2 FFN2 made FP4 on the spot: the largest activation quantisation outside a fused epilogue
        dict(name="quantize nv 16896x5376", op="quantize", fmt="nv", src="bf16", rows=16896, k=5376),
        # the small block's tokens: a call of a few hundred KB, where the launch counts
        dict(name="quantize mx 288x768", op="quantize", fmt="mx", src="bf16", rows=288, k=768),
        # one row against a tall matrix: the AdaLN projection of a block (6 x hidden outputs), bound by reading the weights
        dict(name="linear nv 1 row adaln", op="linear", fmt="nv", epi="store", bias=True, m=1, n=32256, k=5376),
        # the small block's QKV product
        dict(name="linear mx 288x2304x768", op="linear", fmt="mx", epi="store", bias=False, m=288, n=2304, k=768),
        # FFN2 of the 2048^2 canvas into the fp32 residual stream, the longest sum
        dict(name="linear nv 4608 ffn2 gated", op="linear", fmt="nv", epi="gated", bias=True, m=4608, n=5376, k=14336),
        # FFN1 with GELU of the 4096^2 canvas, the largest product of a step
        dict(name="linear mx 16896 ffn1 gelu", op="linear", fmt="mx", epi="gelu", bias=False, m=16896, n=14336, k=5376),
        # one token, the norm's latency
        dict(name="norm 1x768", op="norm", rows=1, d=768, groups=1, post=True, branch="bf16", out="bf16"),
        # the 4096^2 canvas between two branches of a block
        dict(name="norm 16896x5376", op="norm", rows=16896, d=5376, groups=1, post=True, branch="bf16", out="bf16"),
        # two images of one batch, each with its own modulation, the row handed to an FP4 QKV product of the 2048^2 canvas
        dict(name="norm to fp4 qkv 4608", op="norm", rows=4608, d=5376, groups=2, post=False, branch="bf16", out="nv", n=16128),
        # the small block's queries and keys
        dict(name="rope 288 heads 8x96", op="rope", n=288, hq=8, hk=8, dh=96, s0=16, s1=16, s2=16, inter=False, norm=True, io="bf16"),
        # the 4096^2 canvas: 128 x 128 patches and the text
        dict(name="rope 16896 heads 56x96", op="rope", n=16896, hq=56, hk=56, dh=96, s0=16, s1=16, s2=16, inter=False, norm=True, io="bf16"),
        # reference editing: the target, four reference images (a frame each) and the text; adjacent pairs, shared key heads
        dict(name="rope 20736 heads 56:8x128", op="rope", n=20736, hq=56, hk=8, dh=128, s0=16, s1=24, s2=24, inter=True, norm=True, io="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(v, m):
    return max(m, v // m * m)


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "norm", "rope"])
    if op == "quantize":
        return dict(op=op, fmt=rng.choice(["mx", "nv"]), src=rng.choice(["bf16", "bf16", "f32"]), rows=_log(rng, 1, 16896), k=_mult(_log(rng, 64, 5376), 64))
    if op == "linear":
        m, n, k = _log(rng, 1, 16896), _mult(_log(rng, 64, 14336), 32), _mult(_log(rng, 256, 5376), 64)
        return dict(op=op, fmt=rng.choice(["mx", "nv"]), epi=rng.choice(["store", "gelu", "gated"]), bias=rng.random() < 0.5, m=m, n=n, k=k)
    if op == "norm":
        rows, out = _log(rng, 1, 16896), rng.choice(["bf16", "bf16", "mx", "nv"])
        c = dict(op=op, rows=rows, d=_mult(_log(rng, 256, 5376), 64), groups=rng.choice([1, 1, 2, 3]), post=rng.random() < 0.5, branch=rng.choice(["bf16", "f32"]), out=out)
        if out != "bf16":
            c["n"] = _mult(_log(rng, 64, 5376), 32)
        return c
    dh, s, inter = rng.choice([(64, (8, 12, 12), True), (96, (16, 16, 16), False), (96, (8, 16, 16), False), (128, (16, 24, 24), False),
                               (128, (22, 21, 21), True)])
    hq = rng.choice([4, 8, 24, 40, 56])
    hk = rng.choice([hq, hq, 4])
    return dict(op="rope", n=_log(rng, 1, 16896), hq=hq, hk=hk, dh=dh, s0=s[0], s1=s[1], s2=s[2], inter=inter, norm=rng.random() < 0.6,
                io=rng.choice(["bf16", "bf16", "f32"]))


def _fp4_bytes(fmt, rows, k):
    return rows * k / 2 + rows * (k // BLOCK[fmt])


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["k"]
        return {"bytes": n * (2 if c["src"] == "bf16" else 4) + 2 * n, "flops": 4 * n}
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        out = m * n * (8 if c["epi"] == "gated" else 2)
        return {"bytes": _fp4_bytes(c["fmt"], m, k) + _fp4_bytes(c["fmt"], n, k) + out + (4 * n if c["bias"] else 0), "flops": 2 * m * n * k}
    if c["op"] == "norm":
        n, d = c["rows"], c["d"]
        b = n * d * (8 + (2 if c["branch"] == "bf16" else 4)) + 4 * d * (3 * c["groups"] + (1 if c["post"] else 0))
        if c["out"] == "bf16":
            return {"bytes": b + 2 * n * d, "flops": 12 * n * d}
        return {"bytes": b + _fp4_bytes(c["out"], c["n"], d) + 2 * n * c["n"], "flops": 12 * n * d + 2 * n * d * c["n"]}
    e = 2 if c["io"] == "bf16" else 4
    n = c["n"] * (c["hq"] + c["hk"]) * c["dh"]
    return {"bytes": 2 * e * n + 12 * c["n"], "flops": 8 * n}


# --------------------------------------------------------------------------------- 4-bit matrices, elementary torch operations

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _code(y):
    """E2M1 codes of fp32 values: nearest, ties to the even code, at most 6 in size."""
    a = y.abs()
    c = (a > 0.25).to(torch.uint8)
    for edge, tie in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += (a >= edge) if tie else (a > edge)
    return c | ((y < 0).to(torch.uint8) << 3)


def _scales(fmt, x, tensor_scale):
    """What each block of x (fp32 [rows, blocks, size]) is divided by: the scale's byte, and 1 / (the scale it stands for)."""
    amax = x.abs().amax(-1)
    if fmt == "mx":  # 2^(floor(log2 amax) - 2), at least 2^-127
        byte = ((amax.view(torch.int32) >> 23) - 2).clamp_(min=0)
        return byte.to(torch.uint8), torch.ldexp(torch.ones_like(amax), 127 - byte)
    r = 1.0 / (6.0 * tensor_scale)
    s = (amax * r).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float() * tensor_scale
    return s.view(torch.uint8), torch.where(d >= 2.0 ** -126, 1.0 / d, torch.zeros_like(d))


def _tensor_scale(x):
    """fp32 tensor scale of an NVFP4 matrix: its largest element over 6 * 448."""
    a = x.abs().amax().float()
    # a tensor as the divisor: torch multiplies by the reciprocal of a number, which is not the quotient's rounding
    return torch.where(a > 0, a / torch.full_like(a, 2688.0), torch.ones_like(a))


def _sf_index(rows, blocks, device):
    r = torch.arange(rows, device=device)[:, None]
    s = torch.arange(blocks, device=device)[None]
    return ((r // 128) * (-(-blocks // 4)) + s // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + s % 4


def _sf_bytes(fmt, rows, k):
    return -(-rows // 128) * (-(-k // (4 * BLOCK[fmt]))) * 512


def _encode(fmt, x, tensor_scale):
    """x fp32 [rows, k] -> packed codes [rows, k / 2], scale bytes in their layout."""
    rows, k = x.shape
    blocks = x.view(rows, k // BLOCK[fmt], BLOCK[fmt])
    byte, inv = _scales(fmt, blocks, tensor_scale)
    c = _code(blocks * inv[..., None]).view(rows, k // 2, 2)
    sf = torch.zeros(_sf_bytes(fmt, rows, k), dtype=torch.uint8, device=x.device)
    sf[_sf_index(rows, k // BLOCK[fmt], x.device)] = byte
    return c[..., 0] | (c[..., 1] << 4), sf


def _decode(fmt, q, sf, k, tensor_scale=None):
    """The fp32 values of a packed matrix."""
    rows = q.shape[0]
    table = torch.tensor(E2M1, device=q.device)
    v = torch.stack((table[(q & 15).int()], table[(q >> 4).int()]), -1).view(rows, k // BLOCK[fmt], BLOCK[fmt])
    byte = sf[_sf_index(rows, k // BLOCK[fmt], q.device)]
    s = torch.ldexp(torch.ones((), device=q.device), byte.int() - 127) if fmt == "mx" else byte.view(torch.float8_e4m3fn).float()
    if tensor_scale is not None:
        s = s * tensor_scale
    return (v * s[..., None]).view(rows, k)


# ------------------------------------------------------------------------------------------------------------- the inputs

def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return lambda *shape: torch.randn(*shape, generator=g, device="cuda")


def _activations(rand, rows, k):
    """Tokens with a spread of sizes over the channels, as a trained network's have."""
    return rand(rows, k) * torch.exp(0.7 * rand(k))


def _fp4_matrix(fmt, x):
    t = _tensor_scale(x) if fmt == "nv" else None
    q, sf = _encode(fmt, x, t)
    return {"q": q, "sf": sf, "t": t}


def prepare(case, seed):
    c, rand = case, _rng(seed)
    op = c["op"]
    st = {"case": dict(c)}
    if op == "quantize":
        x = _activations(rand, c["rows"], c["k"])
        st["x"] = x.bfloat16() if c["src"] == "bf16" else x
        # buffers a program allocates once
        st["q"] = torch.empty(c["rows"], c["k"] // 2, dtype=torch.uint8, device="cuda")
        st["sf"] = torch.empty(_sf_bytes(c["fmt"], c["rows"], c["k"]), dtype=torch.uint8, device="cuda")
        st["t"] = torch.empty(1, device="cuda")
        st["out"] = torch.empty(c["rows"], c["k"], dtype=torch.bfloat16, device="cuda")
    elif op == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        st["a"] = _fp4_matrix(c["fmt"], _activations(rand, m, k).bfloat16().float())
        st["w"] = _fp4_matrix(c["fmt"], (0.02 * rand(n, k)).bfloat16().float())
        st["bias"] = 0.1 * rand(n) if c["bias"] else None
        if c["epi"] == "gated":
            st["x"], st["gate"] = rand(m, n), rand(n)
        st["out"] = torch.empty(m, n, dtype=torch.float32 if c["epi"] == "gated" else torch.bfloat16, device="cuda")
    elif op == "norm":
        n, d, g = c["rows"], c["d"], c["groups"]
        st["x"] = _activations(rand, n, d)
        y = rand(n, d)
        st["y"] = y.bfloat16() if c["branch"] == "bf16" else y
        mod = 0.5 * rand(g, 3, d)  # of each image: gate, shift, scale
        st["mod"] = mod
        st["post"] = 1.0 + 0.1 * rand(d) if c["post"] else None
        st["per"] = -(-n // g)
        st["x_out"] = torch.empty(n, d, device="cuda")
        if c["out"] == "bf16":
            st["out"] = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
        else:
            st["w"] = _fp4_matrix(c["out"], (0.02 * rand(c["n"], d)).bfloat16().float())
            # the activations' tensor scale, calibrated: a row of the norm stays below 64
            st["t"] = torch.full((1,), 64.0 / 2688.0, device="cuda") if c["out"] == "nv" else None
            st["out"] = torch.empty(n, c["n"], dtype=torch.bfloat16, device="cuda")
            st["q"] = torch.empty(n, d // 2, dtype=torch.uint8, device="cuda")
            st["sf"] = torch.empty(_sf_bytes(c["out"], n, d), dtype=torch.uint8, device="cuda")
    else:
        n, dh = c["n"], c["dh"]
        dt = torch.bfloat16 if c["io"] == "bf16" else torch.float32
        # q and k are column ranges of the Q|K|V rows a product wrote
        st["qkv"] = rand(n, (c["hq"] + 2 * c["hk"]) * dh).to(dt)
        # a target and its references: a frame index, then the rows and columns of each grid
        side = max(1, int(math.sqrt(min(n, 16384))))
        i = torch.arange(n, device="cuda")
        st["pos"] = torch.stack((i // (side * side), i // side % side, i % side), -1).float()
        st["pos"][:, 1:] += 2.0 * torch.rand(2, generator=torch.Generator().manual_seed(int(seed))).cuda()  # a crop's offset
        if c["norm"]:
            st["wq"], st["wk"] = 1.0 + 0.1 * rand(dh), 1.0 + 0.1 * rand(dh)
        st["q_out"] = torch.empty(n, c["hq"] * dh, dtype=dt, device="cuda")
        st["k_out"] = torch.empty(n, c["hk"] * dh, dtype=dt, device="cuda")
    return st


# ------------------------------------------------------------------------------------------------------- through the library

@functools.lru_cache(maxsize=None)
def _handle(hidden):
    """The library's context a program keeps, by the width its norms run at."""
    from image_generation_b200 import h3dit as H

    cfg = H.make_config(hidden, 8, 96, 64, 1, 1, norm_eps=EPS)
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    b = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    blk = dict(w_qkv=b(3 * 768, hidden), w_o=b(hidden, 768), w_ff1=b(64, hidden), w_ff2=b(hidden, 64), w_ada=b(6 * hidden, hidden), b_ada=f(6 * hidden))
    return H.Context(cfg, dict(w_t1=f(hidden, 256), b_t1=f(hidden), w_t2=f(hidden, hidden), b_t2=f(hidden)), [blk])


def _own(st):
    from image_generation_b200 import h3dit as H

    c = st["case"]
    op = c["op"]
    fmt = lambda f: H.H3DIT_FP4_MX if f == "mx" else H.H3DIT_FP4_NV  # noqa: E731
    if op == "quantize":
        h, t = _handle(768), None
        if c["fmt"] == "nv":
            t = st["t"]
            h.fp4_tensor_scale(st["x"], t)
        h.fp4_quantize(fmt(c["fmt"]), st["x"], st["q"], st["sf"], tensor_scale=t)
        h.fp4_dequantize(fmt(c["fmt"]), st["q"], st["sf"], st["out"], tensor_scale=t)
        return st["out"]
    if op == "linear":
        a, w = st["a"], st["w"]
        epi = {"store": H.H3DIT_EPI_STORE, "gelu": H.H3DIT_EPI_GELU, "gated": H.H3DIT_EPI_GATED_RESIDUAL}[c["epi"]]
        _handle(768).linear_fp4(fmt(c["fmt"]), epi, a["q"], a["sf"], w["q"], w["sf"], st["out"], a_scale=a["t"], w_scale=w["t"], bias=st["bias"],
                                gate=st.get("gate"), resid=st.get("x"))
        return st["out"]
    if op == "norm":
        h = _handle(c["d"])
        gate, shift, scale = st["mod"][:, 0], st["mod"][:, 1], st["mod"][:, 2]
        kw = dict(branch=st["y"], gate=gate, shift=shift, scale=scale, rows_per_group=st["per"], post_norm=c["post"], post_weight=st["post"], residual_scale=0.75)
        if c["out"] == "bf16":
            h.gated_norm(st["x"], st["x_out"], H.H3DIT_NORM_OUT_BF16, st["out"], **kw)
        else:
            kind = H.H3DIT_NORM_OUT_FP4_MX if c["out"] == "mx" else H.H3DIT_NORM_OUT_FP4_NV
            h.gated_norm(st["x"], st["x_out"], kind, st["q"], out_sf=st["sf"], out_scale=st["t"], **kw)
            w = st["w"]
            h.linear_fp4(fmt(c["out"]), H.H3DIT_EPI_STORE, st["q"], st["sf"], w["q"], w["sf"], st["out"], a_scale=st["t"], w_scale=w["t"])
        return st["x_out"], st["out"]
    spec = H.make_rope_spec(c["dh"], (c["s0"], c["s1"], c["s2"]), THETA, interleaved=c["inter"])
    q, k = st["qkv"][:, : c["hq"] * c["dh"]], st["qkv"][:, c["hq"] * c["dh"] : (c["hq"] + c["hk"]) * c["dh"]]
    _handle(768).rope_axes(spec, st["pos"], q, st["q_out"], c["hq"], k, st["k_out"], c["hk"], q_weight=st.get("wq"), k_weight=st.get("wk"))
    return st["q_out"], st["k_out"]


# ------------------------------------------------------------------------------------------------------------- plain forms

def _rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _gelu(x):
    return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))


def _rotate(x, cos, sin, case):
    """x fp32 [n, heads, dh]; the first 2 (s0 + s1 + s2) columns rotate."""
    secs, out, col, pair = (case["s0"], case["s1"], case["s2"]), [], 0, 0
    for s in secs:  # the three axes
        u, c, sn = x[..., col : col + 2 * s], cos[:, None, pair : pair + s], sin[:, None, pair : pair + s]
        a, b = (u[..., 0::2], u[..., 1::2]) if case["inter"] else (u[..., :s], u[..., s:])
        r = (a * c - b * sn, b * c + a * sn)
        out.append(torch.stack(r, -1).flatten(-2) if case["inter"] else torch.cat(r, -1))
        col, pair = col + 2 * s, pair + s
    return torch.cat(out + [x[..., col:]], -1)


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "quantize":
        x = st["x"].float()
        t = _tensor_scale(x) if c["fmt"] == "nv" else None
        q, sf = _encode(c["fmt"], x, t)
        return _decode(c["fmt"], q, sf, c["k"], t).bfloat16()
    if op == "linear":
        a, w = st["a"], st["w"]
        acc = _decode(c["fmt"], a["q"], a["sf"], c["k"]) @ _decode(c["fmt"], w["q"], w["sf"], c["k"]).T
        if c["fmt"] == "nv":
            acc = acc * (a["t"] * w["t"])
        if st["bias"] is not None:
            acc = acc + st["bias"]
        if c["epi"] == "gated":
            return st["x"] + st["gate"] * acc
        return (_gelu(acc) if c["epi"] == "gelu" else acc).bfloat16()
    if op == "norm":
        group = torch.arange(c["rows"], device="cuda") // st["per"]
        gate, shift, scale = st["mod"][group].unbind(1)
        y = st["y"].float()
        if c["post"]:
            y = _rms(y) * st["post"]
        x = 0.75 * st["x"] + gate * y
        v = _rms(x) * (1.0 + scale) + shift
        if c["out"] == "bf16":
            return x, v.bfloat16()
        q, sf = _encode(c["out"], v, st["t"])
        w = st["w"]
        acc = _decode(c["out"], q, sf, c["d"]) @ _decode(c["out"], w["q"], w["sf"], c["d"]).T
        if c["out"] == "nv":
            acc = acc * (st["t"] * w["t"])
        return x, acc.bfloat16()
    n, dh = c["n"], c["dh"]
    pos = st["pos"].double()
    ang = torch.cat([pos[:, i, None] * THETA ** (-torch.arange(s, device="cuda", dtype=torch.float64) / s) for i, s in enumerate((c["s0"], c["s1"], c["s2"]))], -1)
    cos, sin = ang.cos().float(), ang.sin().float()
    q = st["qkv"][:, : c["hq"] * dh].float().view(n, c["hq"], dh)
    k = st["qkv"][:, c["hq"] * dh : (c["hq"] + c["hk"]) * dh].float().view(n, c["hk"], dh)
    if c["norm"]:
        q, k = _rms(q) * st["wq"], _rms(k) * st["wk"]
    dt = st["qkv"].dtype
    return _rotate(q, cos, sin, c).to(dt).view(n, -1), _rotate(k, cos, sin, c).to(dt).view(n, -1)


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------------------------- from the definitions, in 64 bits

def _exact_values(fmt, q, sf, t=None):
    """fp64 values of a packed matrix, from the bits of its codes and scales."""
    rows, half = q.shape
    bs = BLOCK[fmt]
    code = torch.empty(rows, 2 * half, dtype=torch.int16, device=q.device)
    code[:, 0::2], code[:, 1::2] = (q % 16).to(torch.int16), (q // 16).to(torch.int16)
    e, m, neg = (code >> 1) & 3, (code & 1).double(), (code >= 8)
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
    v = torch.where(neg, -v, v)
    # undo the scales' layout by its own axes: row / 128, block / 4, row % 32, row / 32 % 4, block % 4
    cols = -(-(2 * half) // (4 * bs))
    b = sf.view(-1, cols, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * cols)[:rows, : 2 * half // bs].int()
    if fmt == "mx":
        s = torch.exp2(b.double() - 127)
    else:
        ex, man = b >> 3, (b & 7).double()
        s = torch.where(ex == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.exp2(ex.double() - 7))
    if t is not None:
        s = s * t.double()
    return v * s.repeat_interleave(bs, 1)


def _nearest(y):
    """E2M1 values nearest to fp64 y, by distance; between two as near, the one whose last bit is 0."""
    grid = torch.tensor([0.0, 1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0], dtype=torch.float64, device=y.device)  # even codes first: argmin takes them
    near = torch.full_like(y, math.inf)
    best = torch.zeros_like(y)
    for v in grid:
        d = (y.abs() - v).abs()
        best, near = torch.where(d < near, v, best), torch.minimum(d, near)
    return torch.copysign(best, y)


def _exact_quantized(fmt, x, t):
    """fp64 values that x (fp32 values) is given as. The scales are defined by single-precision steps, taken as such."""
    rows, k = x.shape
    bs = BLOCK[fmt]
    b = x.double().view(rows, k // bs, bs)
    amax = b.abs().amax(-1)
    if fmt == "mx":
        s = torch.where(amax > 0, torch.exp2((torch.frexp(amax)[1] - 3).clamp(min=-127).double()), 2.0 ** -127 * torch.ones_like(amax))
        return (_nearest(b / s[..., None]) * s[..., None]).view(rows, k)
    one = np.float32(1.0)
    tf = np.float32(t.item())
    want = (amax.float() * float(one / (np.float32(6.0) * tf))).double().clamp(max=448.0)  # in fp32, as defined
    ex = torch.floor(torch.log2(want.clamp(min=2.0 ** -6)))
    ulp = torch.exp2(ex - 3)
    s = torch.round(want / ulp) * ulp  # to E4M3, halves to even
    d32 = (s.float() * float(tf))
    inv = torch.where(d32 >= 2.0 ** -126, 1.0 / d32, torch.zeros_like(d32))
    y = (b.float() * inv[..., None]).double()
    return (_nearest(y) * (s * float(tf))[..., None]).view(rows, k)


def exact(case, seed):
    st, c = prepare(case, seed), case
    op = c["op"]
    if op == "quantize":
        x = st["x"].float()
        t = None
        if c["fmt"] == "nv":
            a = np.float32(x.abs().max().item())
            t = torch.tensor(a / np.float32(2688.0) if a > 0 else np.float32(1.0))
        rows = max(1, (1 << 24) // c["k"])
        return torch.cat([_exact_quantized(c["fmt"], p, t) for p in x.split(rows)])
    if op == "linear":
        a, w = st["a"], st["w"]
        acc = _exact_values(c["fmt"], a["q"], a["sf"], a["t"]) @ _exact_values(c["fmt"], w["q"], w["sf"], w["t"]).T
        if st["bias"] is not None:
            acc += st["bias"].double()
        if c["epi"] == "gated":
            return st["x"].double() + st["gate"].double() * acc
        return acc * 0.5 * torch.erfc(-acc / math.sqrt(2.0)) if c["epi"] == "gelu" else acc
    if op == "norm":
        x, y = st["x"].double(), st["y"].double()
        if c["post"]:
            y = y / (y.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * st["post"].double()
        mod = st["mod"].double().repeat_interleave(st["per"], 0)[: c["rows"]]
        x = 0.75 * x + mod[:, 0] * y
        v = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * (1 + mod[:, 2]) + mod[:, 1]
        if c["out"] == "bf16":
            return x, v
        v = torch.cat([_exact_quantized(c["out"], p, st["t"]) for p in v.float().split(max(1, (1 << 24) // c["d"]))])
        return x, v @ _exact_values(c["out"], st["w"]["q"], st["w"]["sf"], st["w"]["t"]).T
    n, dh, outs = c["n"], c["dh"], []
    # each axis turns its pairs by exp(i * position * theta^(-j / s)), in complex numbers
    turn = [torch.exp(1j * st["pos"][:, i, None].double() * torch.exp(torch.arange(s, device="cuda").double() * (-math.log(THETA) / s)))
            for i, s in enumerate((c["s0"], c["s1"], c["s2"]))]
    for first, heads, wt in ((0, c["hq"], st.get("wq")), (c["hq"], c["hk"], st.get("wk"))):
        u = st["qkv"][:, first * dh : (first + heads) * dh].double().reshape(n, heads, dh)
        if c["norm"]:
            u = u / (u.pow(2).sum(-1, keepdim=True) / dh + EPS).sqrt() * wt.double()
        u = u.clone()
        col = 0
        for t in turn:
            s = t.shape[1]
            at = torch.arange(s, device="cuda")
            i, j = (col + 2 * at, col + 2 * at + 1) if c["inter"] else (col + at, col + s + at)
            z = torch.complex(u[..., i], u[..., j]) * t[:, None]
            u[..., i], u[..., j] = z.real, z.imag
            col += 2 * s
        outs.append(u.view(n, heads * dh))
    return tuple(outs)
