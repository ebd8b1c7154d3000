"""The FP4 operators against their definitions in 64 bits: quantization and its
inverse bit for bit, the product exactly where fp32 holds every partial sum and
within a derived bound elsewhere, refusals, and bytes that must stay untouched."""
import numpy as np
import pytest

from image_generation_b200 import synth
from tests import operators_ref as R
from tests.helpers import block_tensors, time_tensors, to_np
from tests.test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FMTS = pytest.mark.parametrize("fmt", [R.MX, R.NV], ids=["mx", "nv"])


def make_ctx(hidden=768, **kw):
    from image_generation_b200 import h3dit as H

    d = synth.Dims(hidden, 8, 96, 64)
    cfg = H.make_config(d.hidden, d.heads, d.head_dim, d.ffn, 1, 64, **kw)
    return H.Context(cfg, time_tensors(synth.time_weights(d, 0)),
                     [block_tensors(synth.block_weights(d, 0))])


@pytest.fixture(scope="module")
def ctx():
    return make_ctx()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(a):
    """float -> the bf16 value nearest to it, as float64."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16().double().numpy()


def ok(ctx):
    torch.cuda.synchronize()
    assert ctx.sync_status() == 0


def source(rows, k, seed, f32):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, k)) * np.exp(0.7 * g.standard_normal(k))
    x[0, :32] = 0.0
    if rows > 1:
        x[1, :16] = 3e-39 if f32 else 2.0 ** -126      # subnormal, and the smallest normal
        x[rows // 2, 40] = 300.0                       # an outlier
        x[rows - 1, 48:64] = np.resize([6, -6, 5, 2.5, -0.25, 0.75, 3.5, 1.75], 16)  # ties
    x = x.astype(np.float32)
    return x if f32 else bf16(x).astype(np.float32)


def src_tensor(x, f32, pad=0):
    t = dev(np.pad(x, ((0, 0), (0, pad)), constant_values=7.0))
    t = t if f32 else t.bfloat16()
    return t[:, : x.shape[1]]


# ------------------------------------------------------------------- quantization

@FMTS
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,k,pad", [(1, 64, 0), (300, 768, 0), (129, 448, 16), (37, 5376, 8)])
def test_quantize_is_bit_exact(ctx, fmt, f32, rows, k, pad):
    x = source(rows, k, rows + k, f32)
    xt = src_tensor(x, f32, pad)
    t = None
    g = None
    if fmt == R.NV:
        tg = Guarded((1,), torch.float32)
        ctx.fp4_tensor_scale(xt, tg.t)
        tg.check("tensor scale")
        g = R.tensor_scale(x)
        assert tg.t.item() == float(g)
        t = tg.t
    q, sf = Guarded((rows, k // 2), torch.uint8), Guarded((R.sf_bytes(fmt, rows, k),), torch.uint8)
    sf.t.fill_(0xEE)
    ctx.fp4_quantize(fmt, xt, q.t, sf.t, tensor_scale=t)
    out = Guarded((rows, k), torch.bfloat16)
    ctx.fp4_dequantize(fmt, q.t, sf.t, out.t, tensor_scale=t)
    ok(ctx)
    for b, w in ((q, "codes"), (sf, "scales"), (out, "values")):
        b.check(w)
    codes, byte = R.quantize(fmt, x, g)
    want = R.sf_layout(byte, fill=0xEE)
    blocks = byte.shape[1]
    full = -(-blocks // 4) * 4
    want[R.sf_index(rows, full)[:, blocks:]] = 0   # the rest of a row's last group of four
    assert np.array_equal(sf.t.cpu().numpy(), want)
    got = R.unpack(q.t.cpu().numpy())
    same = (got == codes) | (((got | codes) & 7) == 0)  # the sign of a zero is free
    assert same.all(), np.argwhere(~same)[:4]
    d = (R.scale_values(fmt, byte).astype(np.float32) * np.float32(1 if g is None else g)).astype(np.float32)
    v = (R.values(fmt, codes, np.full_like(byte, 127 if fmt == R.MX else 0x38)).astype(np.float32)
         * np.repeat(d, R.BLOCK[fmt], 1)).astype(np.float32)
    assert np.array_equal(to_np(out.t), bf16(v))


@FMTS
def test_quantize_non_finite_and_extreme_blocks(ctx, fmt):
    x = source(8, 256, 3, True)
    x[0, 5], x[1, 40], x[2, 100] = np.nan, np.inf, -np.inf
    x[3, :64] = 3.4e38
    x[4, :64] = 1e-45
    x[5] = 0
    g = np.float32(0.02)
    xt, t = dev(x), dev(np.array([g], np.float32))
    q = torch.zeros(8, 128, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(R.sf_bytes(fmt, 8, 256), dtype=torch.uint8, device="cuda")
    out = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    ts = t if fmt == R.NV else None
    ctx.fp4_quantize(fmt, xt, q, sf, tensor_scale=ts)
    ctx.fp4_dequantize(fmt, q, sf, out, tensor_scale=ts)
    ok(ctx)
    codes, byte = R.quantize(fmt, x, g)
    assert np.array_equal(sf.cpu().numpy()[R.sf_index(8, byte.shape[1])], byte)
    ref = R.values(fmt, codes, byte, g if fmt == R.NV else None)
    got = to_np(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fin = np.isfinite(ref)
    assert np.all(np.abs(got[fin] - ref[fin]) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(ref[fin]) + 1e-40)


def test_tensor_scale_skips_non_finite_and_repeats(ctx):
    x = np.zeros((5, 192), np.float32)
    t = torch.empty(1, device="cuda")
    ctx.fp4_tensor_scale(dev(x), t)
    assert t.item() == 1.0
    x[2, 7], x[3, 3], x[4, 191] = np.inf, np.nan, -5.5
    for _ in range(3):
        ctx.fp4_tensor_scale(dev(x), t)
        assert t.item() == float(np.float32(5.5) / np.float32(2688))
    big = source(3000, 768, 1, False)  # more units than one pass of the grid
    ctx.fp4_tensor_scale(src_tensor(big, False), t)
    assert t.item() == float(R.tensor_scale(big))
    bad = torch.tensor([0.0], device="cuda")  # an unusable tensor scale: every block is NaN
    q = torch.zeros(5, 96, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(R.sf_bytes(R.NV, 5, 192), dtype=torch.uint8, device="cuda")
    ctx.fp4_quantize(R.NV, dev(np.ones((5, 192), np.float32)), q, sf, tensor_scale=bad)
    assert np.all(sf.cpu().numpy()[R.sf_index(5, 12)] == 0x7f)
    ok(ctx)


@pytest.mark.parametrize("f32", [True, False], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -149, 2.0 ** -140, 1.8e-42, 2e-42, 1e-40, 1e-38])
def test_tiny_matrices_stay_finite(ctx, size, f32):
    """Magnitudes down to the smallest: the tensor scale is never 0, and what the
    matrix stands for, alone and in a product, is finite (zeros at the lowest)."""
    from image_generation_b200 import h3dit as H

    x = np.zeros((3, 128), np.float32)
    x[0, 5], x[1, 64:] = size, -size
    x = x if f32 else bf16(x).astype(np.float32)
    g = R.tensor_scale(x)
    assert g > 0
    t = torch.full((1,), -1.0, device="cuda")
    ctx.fp4_tensor_scale(src_tensor(x, f32), t)
    assert t.item() == float(g)
    q = torch.zeros(3, 64, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(R.sf_bytes(R.NV, 3, 128), dtype=torch.uint8, device="cuda")
    out, prod = (torch.full((3, n), float("nan"), dtype=torch.bfloat16, device="cuda") for n in (128, 32))
    ctx.fp4_quantize(R.NV, src_tensor(x, f32), q, sf, tensor_scale=t)
    ctx.fp4_dequantize(R.NV, q, sf, out, tensor_scale=t)
    w, wsf, _ = operand(R.NV, 32, 128, 1, True)
    ctx.linear_fp4(R.NV, H.H3DIT_EPI_STORE, q, sf, w, wsf, prod, a_scale=t)
    ok(ctx)
    codes, byte = R.quantize(R.NV, x, g)
    ref = R.values(R.NV, codes, byte, g)
    # two fp32 products, one of them perhaps subnormal (2^-150), and one bf16 rounding (2^-134)
    assert np.all(np.abs(to_np(out) - ref) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref) + 2.0 ** -133)
    assert torch.isfinite(prod).all()


@FMTS
def test_values_of_every_scale(ctx, fmt):
    """All 256 scale bytes under tensor scales small, ordinary and large: values that
    bf16 holds are those, what passes it is infinite, zeros are zeros."""
    bs = R.BLOCK[fmt]
    blocks = 256 if fmt == R.MX else 128                  # E4M3 scales carry no sign
    byte = np.arange(blocks, dtype=np.uint8)[None]
    codes = np.resize(np.arange(16, dtype=np.uint8), (1, blocks * bs))
    q, sf = dev(R.pack(codes)), dev(R.sf_layout(byte))
    for g in (None, 2.0 ** -149, 1e-30, 0.7, 2.0, 3.0, 4.0, 1e20, 1e36, 3e38):
        out = torch.full((1, blocks * bs), 9.0, dtype=torch.bfloat16, device="cuda")
        t = None if g is None else dev(np.array([g], np.float32))
        ctx.fp4_dequantize(fmt, q, sf, out, tensor_scale=t)
        ok(ctx)
        g32 = np.float32(1 if g is None else g)
        ref, got = R.values(fmt, codes, byte, g32), to_np(out)
        assert np.array_equal(np.isnan(got), np.isnan(ref)), g
        fin, top = ~np.isnan(ref), (2 - 2.0 ** -8) * 2.0 ** 127  # from here on bf16 rounds to infinity
        with np.errstate(invalid="ignore"):
            big = np.abs(ref) >= top * (1 + 2.0 ** -22)
            # two fp32 products, either perhaps subnormal (the scale's 2^-150 grows up to six
            # times), then bf16's own rounding, perhaps subnormal too
            err = (2.0 ** -8 + 2.0 ** -22) * np.abs(ref) + 2.0 ** -134 + 7 * 2.0 ** -150
            near = fin & (np.abs(ref) < top * (1 - 2.0 ** -22))
            assert np.all(np.abs(got - ref)[near] <= err[near]), g
        assert np.all(np.isinf(got[fin & big])), g
        assert not got[fin & (ref == 0)].any(), g


def test_tensor_scale_needs_nothing_of_its_scratch():
    """Whatever an earlier call, or an overlap that the rules forbid, left in the
    workspace: the scale is right, eagerly and replayed."""
    c = make_ctx()
    x = source(3000, 768, 1, False)
    xt, t = src_tensor(x, False), torch.full((1,), -1.0, device="cuda")
    graph = torch.cuda.CUDAGraph()
    c.fp4_tensor_scale(xt, t)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.fp4_tensor_scale(xt, t)
    for byte in (0, 1, 0x5A, 0xFF):
        for go in (lambda: c.fp4_tensor_scale(xt, t), graph.replay):
            c.workspace[256:].fill_(byte)   # all but the status word
            t.fill_(-1.0)
            go()
            ok(c)
            assert t.item() == float(R.tensor_scale(x)), byte
    # fewer blocks after more, and more after fewer
    for rows in (1, 3000, 5, 700):
        c.fp4_tensor_scale(xt[:rows], t)
        assert t.item() == float(R.tensor_scale(x[:rows]))
    ok(c)


# ------------------------------------------------------------------------ product

def operand(fmt, rows, k, seed, exact, g=None):
    """An FP4 matrix: device codes and scales (padding filled with NaN scales) and
    its float64 values without g. exact: scales from a few values whose products
    and sums over k <= 16384 terms fit fp32's 24 bits."""
    r = np.random.default_rng(seed)
    codes = r.integers(0, 16, (rows, k)).astype(np.uint8)
    blocks = k // R.BLOCK[fmt]
    if fmt == R.MX:
        byte = r.integers(126, 129, (rows, blocks)) if exact else r.integers(115, 135, (rows, blocks))
    else:  # 0.5, 1, 1.5, 2
        byte = r.choice([0x30, 0x38, 0x3c, 0x40], (rows, blocks)) if exact else r.integers(8, 120, (rows, blocks))
    byte = byte.astype(np.uint8)
    sf = R.sf_layout(byte, fill=0xff if fmt == R.MX else 0x7f)
    return dev(R.pack(codes)), dev(sf), R.values(fmt, codes, byte)


SHAPES = [(1, 32, 64), (1, 64, 128), (3, 96, 192), (128, 128, 256), (129, 160, 320), (200, 768, 832),
          (127, 2304, 768), (288, 2304, 768), (257, 416, 5376), (640, 1056, 448),
          (3, 256, 1088), (17, 416, 2112), (128, 64, 4160),
          # k shared by clusters of 3, 5, 7 and 8 CTAs: even and uneven shares, rows fewer and more than CTAs
          (2, 5376, 3328), (9, 3200, 3328), (90, 2656, 7104), (1, 96, 5376), (100, 160, 7104), (7, 32, 3904),
          # pairs of CTAs: ragged rows (one in the last tile, none in a pair's second CTA) and columns
          (1300, 2112, 320), (2049, 1184, 832), (150, 9632, 192), (2304, 1376, 64)]


@FMTS
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear_is_exact_where_fp32_is(ctx, fmt, m, n, k):
    from image_generation_b200 import h3dit as H

    a, asf, av = operand(fmt, m, k, m + n, True)
    w, wsf, wv = operand(fmt, n, k, m + n + 1, True)
    ref = av @ wv.T
    # every product is a multiple of 2^-4 and no partial sum reaches 2^20: fp32 has them all
    assert np.abs(av).max() ** 2 * k < 2.0 ** 20
    out = Guarded((m, n), torch.bfloat16)
    ctx.linear_fp4(fmt, H.H3DIT_EPI_STORE, a, asf, w, wsf, out.t)
    g = np.random.default_rng(5)
    x = g.integers(-8, 8, (m, n)).astype(np.float32)
    gate = g.choice([0.0, 1.0, -1.0, 0.5], n).astype(np.float32)
    o2 = Guarded((m, n), torch.float32)
    ctx.linear_fp4(fmt, H.H3DIT_EPI_GATED_RESIDUAL, a, asf, w, wsf, o2.t, gate=dev(gate), resid=dev(x))
    o3 = Guarded((m, n), torch.float32, init=dev(x))
    ctx.linear_fp4(fmt, H.H3DIT_EPI_GATED_RESIDUAL, a, asf, w, wsf, o3.t, gate=dev(gate))
    ok(ctx)
    for o in (out, o2, o3):
        o.check("linear")
    assert np.array_equal(to_np(out.t), bf16(ref))
    assert np.array_equal(to_np(o2.t), x + gate * ref)
    assert np.array_equal(to_np(o3.t), x + gate * ref)


def sum_bound(av, wv, k):
    """Error of an fp32 accumulation of k products in any order: each is rounded
    or cut once at 2^-23 of a partial sum no larger than sum |a w|."""
    return k * 2.0 ** -23 * (np.abs(av) @ np.abs(wv).T)


@FMTS
@pytest.mark.parametrize("gelu_tanh", [False, True], ids=["erf", "tanh"])
@pytest.mark.parametrize("m,n,k", [(1, 64, 256), (5, 128, 704), (300, 320, 768), (385, 1024, 320), (6, 192, 6144),
                                   (1301, 2112, 704), (1301, 2112, 2368)])
def test_linear_epilogues(ctx, fmt, gelu_tanh, m, n, k):
    from image_generation_b200 import h3dit as H

    c = make_ctx(gelu_tanh=True) if gelu_tanh else ctx
    ga, gw = np.float32(0.003), np.float32(0.011)
    a, asf, av = operand(fmt, m, k, m, True)
    w, wsf, wv = operand(fmt, n, k, n, True)
    g = np.random.default_rng(2)
    bias, gate = g.standard_normal(n).astype(np.float32), g.standard_normal(n).astype(np.float32)
    x = g.standard_normal((m, n)).astype(np.float32)
    al = float(ga) * float(gw)
    ref = al * (av @ wv.T) + bias
    kw = dict(a_scale=dev(np.array([ga])), w_scale=dev(np.array([gw])), bias=dev(bias))
    err = al * sum_bound(av, wv, k) + 4 * 2.0 ** -24 * (np.abs(ref) + np.abs(bias))
    st, ge = (torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gr = torch.empty(m, n, device="cuda")
    c.linear_fp4(fmt, H.H3DIT_EPI_STORE, a, asf, w, wsf, st, **kw)
    c.linear_fp4(fmt, H.H3DIT_EPI_GELU, a, asf, w, wsf, ge, **kw)
    c.linear_fp4(fmt, H.H3DIT_EPI_GATED_RESIDUAL, a, asf, w, wsf, gr, gate=dev(gate), resid=dev(x), **kw)
    # GELU to FP4, under a tensor scale that the values fit
    y = R.gelu(ref) if not gelu_tanh else 0.5 * ref * (1 + np.tanh(0.7978845608028654 * (ref + 0.044715 * ref ** 3)))
    t = np.float32(np.abs(y).max() / 2688 * 1.01)
    q, sf = Guarded((m, n // 2), torch.uint8), Guarded((R.sf_bytes(fmt, m, n),), torch.uint8)
    c.linear_fp4(fmt, H.H3DIT_EPI_GELU, a, asf, w, wsf, q.t, out_sf=sf.t,
                 out_scale=dev(np.array([t])) if fmt == R.NV else None, **kw)
    ok(c)
    q.check("gelu codes")
    sf.check("gelu scales")
    half = 2.0 ** -8
    assert np.all(np.abs(to_np(st) - ref) <= half * np.abs(ref) + 1.01 * err)
    # GELU's slope is below 1.13; its erf is good to 1.5e-7 (tanh: 2^-21)
    gerr = 1.13 * err + 5e-7 * np.abs(ref) + 1e-9
    assert np.all(np.abs(to_np(ge) - y) <= half * np.abs(y) + 1.01 * gerr)
    assert np.all(np.abs(to_np(gr) - (x + gate * ref)) <=
                  np.abs(gate) * err + 2 * 2.0 ** -24 * (np.abs(x) + np.abs(gate * ref)))
    assert_quantized(fmt, q.t, sf.t, y, t)


def assert_quantized(fmt, q, sf, y, g, flips=2e-3):
    """An FP4 output is the reference's quantization but for values that fp32's
    last bits put across a rounding border: rare, and then one step apart."""
    rows, k = y.shape
    codes, byte = R.quantize(fmt, y.astype(np.float32), g)
    got_c, got_b = R.unpack(q.cpu().numpy()), sf.cpu().numpy()[R.sf_index(rows, byte.shape[1])]
    assert np.mean(got_b != byte) <= flips + 1.5 / byte.size, np.mean(got_b != byte)
    assert np.abs(got_b.astype(int) - byte).max() <= 1
    same = np.repeat(got_b == byte, R.BLOCK[fmt], 1)
    step = np.abs((got_c & 7).astype(int) - (codes & 7))[same]
    assert step.max() <= 1 and np.mean(step) <= flips + 1.5 / step.size, np.mean(step)
    sign = ((got_c ^ codes) & 8 != 0) & ((got_c & 7) > 0)
    assert not sign.any()


@FMTS
@pytest.mark.parametrize("m,n,k", [(5, 192, 704), (6, 192, 6144), (140, 192, 6144), (129, 2112, 192), (1301, 2112, 704),
                                   (1301, 2176, 704)])
def test_scales_of_an_fp4_output(ctx, fmt, m, n, k):
    """One part of k, several, and pairs: a row's last group of four scales is whole,
    with zeros past the row's end, and bytes of no row are left as they were."""
    from image_generation_b200 import h3dit as H

    a, asf, av = operand(fmt, m, k, 1, True)
    w, wsf, wv = operand(fmt, n, k, 2, True)
    q = torch.zeros(m, n // 2, dtype=torch.uint8, device="cuda")
    sf = torch.full((R.sf_bytes(fmt, m, n),), 0xEE, dtype=torch.uint8, device="cuda")
    s = torch.full((1,), 0.01, device="cuda")
    t = np.float32(0.01)
    ctx.linear_fp4(fmt, H.H3DIT_EPI_GELU, a, asf, w, wsf, q, out_sf=sf, a_scale=s,
                   out_scale=dev(np.array([t])) if fmt == R.NV else None)
    ok(ctx)
    assert_quantized(fmt, q, sf, R.gelu(float(np.float32(0.01)) * (av @ wv.T)), t)
    blocks = n // R.BLOCK[fmt]
    full = -(-blocks // 4) * 4
    got, at = sf.cpu().numpy(), R.sf_index(m, full)
    assert not got[at[:, blocks:]].any()
    rest = np.ones(got.size, bool)
    rest[at] = False
    assert np.all(got[rest] == 0xEE)


@FMTS
@pytest.mark.parametrize("m,n,k", [(77, 256, 1024), (300, 384, 5376)])
def test_linear_over_the_scales_range(ctx, fmt, m, n, k):
    from image_generation_b200 import h3dit as H

    a, asf, av = operand(fmt, m, k, 1, False)
    w, wsf, wv = operand(fmt, n, k, 2, False)
    out = torch.empty(m, n, device="cuda")
    ctx.linear_fp4(fmt, H.H3DIT_EPI_GATED_RESIDUAL, a, asf, w, wsf, out, gate=torch.ones(n, device="cuda"),
                   resid=torch.zeros(m, n, device="cuda"))
    ok(ctx)
    ref = av @ wv.T
    assert np.all(np.abs(to_np(out) - ref) <= sum_bound(av, wv, k))
    # and not only within the worst case: a random sum's error is near sqrt(k) steps
    assert np.linalg.norm(to_np(out) - ref) <= 2.0 ** -23 * np.sqrt(k) * np.linalg.norm(ref) * 4


@FMTS
def test_linear_many_tiles_and_tensor_scales_out_of_range(ctx, fmt):
    """Several tiles per CTA, and a product of tensor scales below fp32's range."""
    from image_generation_b200 import h3dit as H

    m, n, k = 2600, 2080, 320
    a, asf, av = operand(fmt, m, k, 1, True)
    w, wsf, wv = operand(fmt, n, k, 2, True)
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    ctx.linear_fp4(fmt, H.H3DIT_EPI_STORE, a, asf, w, wsf, out)
    ok(ctx)
    ref = av @ wv.T
    assert np.array_equal(to_np(out), bf16(ref))
    s = torch.tensor([1e-22], device="cuda")
    o = torch.zeros(m, n, device="cuda")
    ctx.linear_fp4(fmt, H.H3DIT_EPI_GATED_RESIDUAL, a, asf, w, wsf, o, a_scale=s, w_scale=s,
                   gate=torch.full((n,), 1e30, device="cuda"))
    ok(ctx)
    want = float(s.item()) ** 2 * ref
    # v itself is subnormal or nearly so: half a step of 2^-149 and one product's rounding each
    assert np.all(np.abs(to_np(o) / 1e30 - want) <= 2.0 ** -148 + 2.0 ** -22 * np.abs(want))


@FMTS
@pytest.mark.parametrize("m", [3, 1300], ids=["few_rows", "pairs"])
def test_tensor_scales_below_the_normal_range(ctx, fmt, m):
    """A sum of 1.5 under 2^22 and 2^-149, either of them A's: 1.5 * 2^-127, which
    fp32 holds; and under 2^100 and 2^30: past fp32, but not with a sum of 2^-20."""
    from image_generation_b200 import h3dit as H

    n, k = 2112, 64
    a, w = np.zeros((m, k), np.uint8), np.zeros((n, k), np.uint8)
    a[:, 0], w[:, 0] = 3, 2                               # 1.5 and 1
    unit = 127 if fmt == R.MX else 0x38
    asf, wsf = (dev(R.sf_layout(np.full((r, k // R.BLOCK[fmt]), unit, np.uint8))) for r in (m, n))
    a, w = dev(R.pack(a)), dev(R.pack(w))
    s = lambda v: torch.full((1,), v, device="cuda")  # noqa: E731
    for x, y in ((2.0 ** 22, 2.0 ** -149), (2.0 ** -149, 2.0 ** 22)):
        out = torch.zeros(m, n, device="cuda")
        ctx.linear_fp4(fmt, H.H3DIT_EPI_GATED_RESIDUAL, a, asf, w, wsf, out, a_scale=s(x), w_scale=s(y),
                       gate=torch.full((n,), 2.0 ** 100, device="cuda"))
        ok(ctx)
        assert torch.all(out == 1.5 * 2.0 ** -27), (x, y, out[0, 0].item())
    # sums that are small by their scales: 1.5 * 2^-20 (E8M0) or 1.5 * 2^-18 (E4M3: 2^-9 each)
    low, total = (117, -20) if fmt == R.MX else (1, -18)
    asf, wsf = (dev(R.sf_layout(np.full((r, k // R.BLOCK[fmt]), low, np.uint8))) for r in (m, n))
    for x, y in ((2.0 ** 100, 2.0 ** 30), (2.0 ** 30, 2.0 ** 100)):
        out = torch.zeros(m, n, device="cuda")
        ctx.linear_fp4(fmt, H.H3DIT_EPI_GATED_RESIDUAL, a, asf, w, wsf, out, a_scale=s(x), w_scale=s(y),
                       gate=torch.ones(n, device="cuda"))
        ok(ctx)
        assert torch.all(out == 1.5 * 2.0 ** (130 + total)), (x, y, out[0, 0].item())


@FMTS
def test_nan_scales_reach_their_rows_only(ctx, fmt):
    from image_generation_b200 import h3dit as H

    m, n, k = 140, 96, 256
    a, asf, av = operand(fmt, m, k, 1, True)
    w, wsf, wv = operand(fmt, n, k, 2, True)
    asf = asf.clone()
    asf[int(R.sf_index(m, k // R.BLOCK[fmt])[133, 3])] = 0xff if fmt == R.MX else 0x7f
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    ctx.linear_fp4(fmt, H.H3DIT_EPI_STORE, a, asf, w, wsf, out)
    ok(ctx)
    got, ref = to_np(out), bf16(av @ wv.T)
    assert np.isnan(got[133]).all()
    keep = np.arange(m) != 133
    assert np.array_equal(got[keep], ref[keep])


@pytest.mark.parametrize("m", [3, 1300], ids=["few_rows", "pairs"])
def test_sums_past_fp32_and_their_gelu(ctx, m):
    """Scales so large that sums leave fp32: infinities as fp32 has them, GELU of
    plus infinity is itself and of minus infinity 0, other rows as ever."""
    from image_generation_b200 import h3dit as H

    n, k = 2112, 128
    codes = np.full((m, k), 2, np.uint8)                  # ones
    byte = np.full((m, k // 32), 127, np.uint8)
    byte[1], byte[2] = 250, 250
    codes[2] = 10                                         # minus ones
    w = dev(R.pack(np.full((n, k), 2, np.uint8)))
    wsf = dev(R.sf_layout(np.full((n, k // 32), 135, np.uint8)))
    a, asf = dev(R.pack(codes)), dev(R.sf_layout(byte))
    for epi, want in ((H.H3DIT_EPI_STORE, [np.inf, -np.inf]), (H.H3DIT_EPI_GELU, [np.inf, 0.0])):
        out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        ctx.linear_fp4(R.MX, epi, a, asf, w, wsf, out)
        ok(ctx)
        got = to_np(out)
        assert np.all(got[0] == 32768) and np.all(got[3:] == 32768)
        assert np.all(got[1] == want[0]) and np.all(got[2] == want[1])


@FMTS
@pytest.mark.parametrize("gelu_tanh", [False, True], ids=["erf", "tanh"])
@pytest.mark.parametrize("m", [3, 1300], ids=["few_rows", "pairs"])
def test_gelu_of_sums_past_fp32(ctx, fmt, gelu_tanh, m):
    """GELU in either form, to bf16 and to FP4: of minus infinity 0, of plus infinity
    itself (to FP4 a NaN block), of a NaN a NaN, other rows as ever."""
    from image_generation_b200 import h3dit as H

    c = make_ctx(gelu_tanh=True) if gelu_tanh else ctx
    n, k = 2112, 128
    codes = np.full((m, k), 2, np.uint8)                  # ones, then minus ones
    codes[2] = 10
    unit = 127 if fmt == R.MX else 0x38
    byte = np.full((m, k // R.BLOCK[fmt]), unit, np.uint8)
    byte[0] = 255 if fmt == R.MX else 127
    wb = np.full((n, k // R.BLOCK[fmt]), unit, np.uint8)
    bias = np.zeros(n, np.float32)
    w, wsf = dev(R.pack(np.full((n, k), 2, np.uint8))), dev(R.sf_layout(wb))
    # a_scale: sums of 128 past fp32 in rows 1 and 2; the others are 0 times that
    codes[3:] = 0
    kw = dict(a_scale=dev(np.array([3e38], np.float32)), bias=dev(bias))
    a, asf = dev(R.pack(codes)), dev(R.sf_layout(byte))
    out = torch.full((m, n), 9.0, dtype=torch.bfloat16, device="cuda")
    c.linear_fp4(fmt, H.H3DIT_EPI_GELU, a, asf, w, wsf, out, **kw)
    q = torch.zeros(m, n // 2, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(R.sf_bytes(fmt, m, n), dtype=torch.uint8, device="cuda")
    c.linear_fp4(fmt, H.H3DIT_EPI_GELU, a, asf, w, wsf, q, out_sf=sf, **kw)
    vals = torch.full((m, n), 9.0, dtype=torch.bfloat16, device="cuda")
    c.fp4_dequantize(fmt, q, sf, vals)
    ok(c)
    for got, inf in ((to_np(out), np.inf), (to_np(vals), np.nan)):
        assert np.isnan(got[0]).all()
        assert np.array_equal(got[1], np.full(n, inf), equal_nan=True)
        assert not got[2:].any()


def test_offsets_past_31_bits(ctx):
    """More than 2^31 elements in and out: the last rows as when they come alone."""
    from image_generation_b200 import h3dit as H

    rows, k, last = 430_080, 5056, 200                    # 2.17e9 elements
    x = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda").normal_()
    q = torch.empty(rows, k // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(R.sf_bytes(R.NV, rows, k), dtype=torch.uint8, device="cuda")
    t = torch.full((1,), 6.0 / 2688, device="cuda")
    ctx.fp4_quantize(R.NV, x, q, sf, tensor_scale=t)
    out = torch.empty_like(x)
    ctx.fp4_dequantize(R.NV, q, sf, out, tensor_scale=t)
    alone = x[-last:].clone()
    q1 = torch.empty(last, k // 2, dtype=torch.uint8, device="cuda")
    sf1 = torch.empty(R.sf_bytes(R.NV, last, k), dtype=torch.uint8, device="cuda")
    o1 = torch.empty_like(alone)
    ctx.fp4_quantize(R.NV, alone, q1, sf1, tensor_scale=t)
    ctx.fp4_dequantize(R.NV, q1, sf1, o1, tensor_scale=t)
    ok(ctx)
    assert torch.equal(q[-last:], q1) and torch.equal(out[-last:], o1)
    amax = torch.empty(1, device="cuda")
    x[-1, -1] = 2 * x.abs().max()
    ctx.fp4_tensor_scale(x, amax)
    # numpy's quotient: torch multiplies by the reciprocal of a number
    assert amax.item() == float(np.float32(x[-1, -1].item()) / np.float32(2688))
    del x, out
    # the product: 430080 x 5056 outputs; codes of a k of 64
    a = q.view(-1)[: rows * 32].view(rows, 32)
    w, wsf, _ = operand(R.NV, 5056, 64, 3, True)
    asf = torch.full((R.sf_bytes(R.NV, rows, 64),), 0x38, dtype=torch.uint8, device="cuda")
    for epi, dt in ((H.H3DIT_EPI_STORE, torch.bfloat16), (H.H3DIT_EPI_GATED_RESIDUAL, torch.float32)):
        kw = {} if dt == torch.bfloat16 else dict(gate=torch.ones(5056, device="cuda"))
        big = torch.ones(rows, 5056, dtype=dt, device="cuda")
        small = torch.ones(last, 5056, dtype=dt, device="cuda")
        ctx.linear_fp4(R.NV, epi, a, asf, w, wsf, big, **kw)
        ctx.linear_fp4(R.NV, epi, a[-last:].clone(), asf[: R.sf_bytes(R.NV, last, 64)].clone(), w, wsf, small, **kw)
        ok(ctx)
        assert torch.equal(big[-last:], small)
        del big


def test_graph_replay_and_side_stream(ctx):
    from image_generation_b200 import h3dit as H

    m, n, k = 300, 768, 768
    x = torch.randn(m, k, device="cuda").bfloat16()
    w, wsf, wv = operand(R.NV, n, k, 2, True)
    q = torch.empty(m, k // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(R.sf_bytes(R.NV, m, k), dtype=torch.uint8, device="cuda")
    t, out = torch.empty(1, device="cuda"), torch.empty(m, n, dtype=torch.bfloat16, device="cuda")

    def go():
        ctx.fp4_tensor_scale(x, t)
        ctx.fp4_quantize(R.NV, x, q, sf, tensor_scale=t)
        ctx.linear_fp4(R.NV, H.H3DIT_EPI_STORE, q, sf, w, wsf, out, a_scale=t)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for scale in (1.0, 8.0):  # powers of two: the codes stay, the result scales
        x.mul_(scale)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, (want.float() * scale).bfloat16())
    assert ctx.sync_status() == 0


# ----------------------------------------------------------------------- refusals

def test_refusals(ctx):
    from image_generation_b200 import h3dit as H

    n0 = ctx.launch_count()
    e = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    f = lambda *s: e(*s, dt=torch.float32)  # noqa: E731
    b = lambda *s: e(*s, dt=torch.bfloat16)  # noqa: E731
    q, sf, ST = e(4, 64), e(2048), H.H3DIT_EPI_STORE
    lin = lambda **k: ctx.linear_fp4(**{**dict(fmt=0, epilogue=ST, a=q, a_sf=sf, w=e(32, 64), w_sf=sf, out=b(4, 32)), **k})  # noqa: E731
    bad = [
        lambda: ctx.fp4_quantize(2, b(4, 128), q, sf),                       # no such format
        lambda: ctx.fp4_quantize(0, b(4, 96), e(4, 48), sf),                 # k not a multiple of 64
        lambda: ctx.fp4_quantize(0, b(4, 128).double(), q, sf),              # type
        lambda: ctx.fp4_quantize(0, b(4, 128), q, sf[:16]),                  # too few scale bytes
        lambda: ctx.fp4_quantize(0, b(4, 128), q, sf, tensor_scale=f(1)),    # MXFP4 has none
        lambda: ctx.fp4_quantize(1, b(4, 132)[:, :128], q, e(8192)),         # row stride not 16 bytes
        lambda: ctx.fp4_quantize(0, b(4, 136)[:, 4:132], q, sf),             # address not 16 bytes
        lambda: ctx.fp4_quantize(0, b(128, 4).t(), q, sf),                   # columns not consecutive
        lambda: ctx.fp4_quantize(0, b(4, 128).cpu(), q, sf),                 # host memory
        lambda: ctx.fp4_quantize(0, b(4, 128), e(4, 65)[:, :64], sf),        # codes not contiguous
        lambda: ctx.fp4_tensor_scale(b(4, 128), f(2)),
        lambda: ctx.fp4_dequantize(0, q, sf, b(4, 130)),
        lambda: lin(epilogue=H.H3DIT_EPI_QKV_ROPE),
        lambda: lin(epilogue=9),
        lambda: lin(fmt=7),
        lambda: lin(out=b(4, 64)),
        lambda: lin(out=f(4, 32)),
        lambda: lin(w=e(40, 64), out=b(4, 40)),                              # n not a multiple of 32
        lambda: lin(w=e(32, 96)),                                            # another k
        lambda: lin(a_scale=f(2)),
        lambda: lin(bias=f(31)),
        lambda: lin(gate=f(32)),                                             # gate without its epilogue
        lambda: lin(epilogue=H.H3DIT_EPI_GATED_RESIDUAL, out=f(4, 32)),      # no gate
        lambda: lin(epilogue=H.H3DIT_EPI_GATED_RESIDUAL, out=f(4, 32), gate=f(32), resid=f(4, 33)),
        lambda: lin(out=e(4, 16), out_sf=sf),                                # STORE writes no FP4
        lambda: lin(epilogue=H.H3DIT_EPI_GELU, out=e(4, 16), out_sf=sf),     # n not a multiple of 64
        lambda: lin(epilogue=H.H3DIT_EPI_GELU, out_scale=f(1)),              # bf16 out has no scale
    ]
    for i, call in enumerate(bad):
        with pytest.raises(H.H3DitError) as err:
            call()
        assert err.value.status in (H.H3DIT_ERR_INVALID_ARG, H.H3DIT_ERR_UNSUPPORTED), i
    # no rows: nothing runs, nothing is examined
    ctx.fp4_quantize(0, b(0, 128), e(0, 64), e(0))
    ctx.fp4_dequantize(0, e(0, 64), e(0), b(0, 128))
    ctx.fp4_tensor_scale(b(0, 128), f(1))
    lin(a=e(0, 64), a_sf=e(0), out=b(0, 32))
    assert ctx.launch_count() == n0
    ok(ctx)


def test_linear_refuses_what_its_indexes_cannot_reach(ctx):
    """Row and column counts whose last tile ends past 31 bits, and too many tiles:
    refused on the host, before any pointer is followed."""
    from image_generation_b200 import h3dit as H

    n0 = ctx.launch_count()
    p = torch.zeros(4096, dtype=torch.uint8, device="cuda").data_ptr()
    top = 2 ** 31 - 1
    for m, n in ((top, 32), (top - 254, 64), (4, top - 31), (4, top // 32 * 32), (2 ** 30, 2 ** 14)):
        assert H.lib.h3dit_linear_fp4(ctx.handle, 0, H.H3DIT_EPI_STORE, p, p, None, p, p, None, m, n, 64, p, None,
                                      None, None, None, None, None) == H.H3DIT_ERR_UNSUPPORTED, (m, n)
    assert ctx.launch_count() == n0
