"""h3dit_gated_norm against its definition in 64 bits: every output kind, with and
without each optional part, one row to many, images with their own modulation."""
import numpy as np
import pytest

from tests import operators_ref as R
from tests.helpers import to_np
from tests.test_gpu_fp4 import assert_quantized, bf16, dev, make_ctx, ok
from tests.test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24  # half a step of fp32, relative


@pytest.fixture(scope="module")
def ctxs():
    return {}


def ctx_for(ctxs, d):
    if d not in ctxs:
        ctxs[d] = make_ctx(d)
    return ctxs[d]


def inputs(n, d, groups, seed, branch_f32):
    g = np.random.default_rng(seed)
    y = g.standard_normal((n, d)).astype(np.float32)
    return dict(x=(g.standard_normal((n, d)) * np.exp(0.7 * g.standard_normal(d))).astype(np.float32),
                y=y if branch_f32 else bf16(y).astype(np.float32),
                mod=(0.5 * g.standard_normal((groups, 3, d))).astype(np.float32),
                post=(1 + 0.1 * g.standard_normal(d)).astype(np.float32),
                pre=(1 + 0.1 * g.standard_normal(d)).astype(np.float32))


def run(ctx, i, n, d, groups, post, branch_f32, kind, use, r=0.75, t=None, in_place=False):
    """One call with the parts named in `use`; returns (x_out, out, out_sf), the
    float64 reference and the sizes its error bounds are made of."""
    from image_generation_b200 import h3dit as H

    per = -(-n // groups)
    mod = dev(i["mod"])
    part = {"gate": mod[:, 0], "shift": mod[:, 1], "scale": mod[:, 2]}
    kw = {k: part[k] for k in part if k in use}
    ref_kw = {k: i["mod"][:, j] for j, k in enumerate(("gate", "shift", "scale")) if k in use}
    if "branch" in use:
        yt = dev(i["y"])
        kw.update(branch=yt if branch_f32 else yt.bfloat16(), post_norm=post)
        ref_kw.update(branch=i["y"], post_norm=post)
        if post and "post" in use:
            kw["post_weight"], ref_kw["post_weight"] = dev(i["post"]), i["post"]
    if "pre" in use:
        kw["pre_weight"], ref_kw["pre_weight"] = dev(i["pre"]), i["pre"]
    xo = Guarded((n, d), torch.float32, init=dev(i["x"]))
    x = xo.t if in_place else dev(i["x"])
    sf = None
    if kind == H.H3DIT_NORM_OUT_BF16:
        out = Guarded((n, d), torch.bfloat16)
    elif kind == H.H3DIT_NORM_OUT_MXFP8:
        out, sf = Guarded((n * d,), torch.uint8), Guarded((H.mx_scale_bytes(n, d),), torch.uint8)
    else:
        fmt = R.MX if kind == H.H3DIT_NORM_OUT_FP4_MX else R.NV
        out, sf = Guarded((n, d // 2), torch.uint8), Guarded((R.sf_bytes(fmt, n, d),), torch.uint8)
    ctx.gated_norm(x, xo.t, kind, out.t, out_sf=None if sf is None else sf.t,
                   out_scale=None if t is None else dev(np.array([t], np.float32)),
                   rows_per_group=per if groups > 1 else 0, residual_scale=r, **kw)
    ok(ctx)
    for b in (xo, out) + (() if sf is None else (sf,)):
        b.check("gated norm")
    ref_kw["per"] = per if groups > 1 else 0
    rx, rv = R.gated_norm(i["x"], r=r, **ref_kw)
    return xo.t, out.t, None if sf is None else sf.t, rx, rv, ref_kw


def check_x(got, x, rx, r, d):
    """x' = r x + gate y: a row's sum of squares in any order is good to d/2 + 2
    roundings at the very worst (units that a thread adds one by one, then a
    tree of threads: at most 32 + 5 + 8 here), 4 for 1/sqrt, 4 for the products."""
    branch = np.abs(rx - r * x.astype(np.float64))
    err = 60 * U * branch + 3 * U * (np.abs(r * x) + branch)
    assert np.all(np.abs(to_np(got) - rx) <= err + 1e-40)
    return err


def out_error(rx, rv, shift, err_x):
    """Error of RMSNorm(x') (1 + scale) + shift before its rounding: x' off by
    err_x (its row's norm no more than that, relative), then the same roundings."""
    rel = np.max(err_x, 1, keepdims=True) / np.sqrt((rx * rx).mean(1, keepdims=True) + 1e-12)
    v = np.abs(rv) + np.abs(shift)
    point = np.where(np.abs(rx) > 0, err_x / np.maximum(np.abs(rx), 1e-30), 0)
    return (60 * U + rel + point) * v + 4 * U * v + 1e-12


ALL = ("branch", "gate", "shift", "scale", "post", "pre")
CASES = [(1, 768, 1), (1, 64, 1), (3, 5376, 1), (257, 768, 2), (130, 448, 3), (65, 2112, 1), (40, 4160, 2),
         (33, 8192, 1), (2, 256, 2)]


@pytest.mark.parametrize("post", [False, True], ids=["plain", "post"])
@pytest.mark.parametrize("branch_f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,d,groups", CASES)
def test_bf16_output(ctxs, n, d, groups, post, branch_f32):
    ctx = ctx_for(ctxs, d)
    i = inputs(n, d, groups, n + d, branch_f32)
    xo, out, _, rx, rv, kw = run(ctx, i, n, d, groups, post, branch_f32, 0, ALL)
    ex = check_x(xo, i["x"], rx, 0.75, d)
    g = np.arange(n) // (kw["per"] or n)
    ev = out_error(rx, rv, i["mod"][g, 1], ex)
    assert np.all(np.abs(to_np(out) - rv) <= 2.0 ** -8 * np.abs(rv) + 1.01 * ev)


@pytest.mark.parametrize("use", [(), ("branch",), ("branch", "gate"), ("scale",), ("shift", "pre"),
                                 ("branch", "shift"), ("branch", "post", "scale")],
                         ids=lambda u: "+".join(u) or "none")
@pytest.mark.parametrize("in_place", [False, True], ids=["out", "in_place"])
def test_each_part_may_be_left_out(ctxs, use, in_place):
    n, d = 37, 768
    ctx = ctx_for(ctxs, d)
    i = inputs(n, d, 1, 9, False)
    xo, out, _, rx, rv, kw = run(ctx, i, n, d, 1, "post" in use, False, 0, use, r=1.0, in_place=in_place)
    ex = check_x(xo, i["x"], rx, 1.0, d)
    ev = out_error(rx, rv, i["mod"][0, 1] if "shift" in use else 0 * rv, ex)
    assert np.all(np.abs(to_np(out) - rv) <= 2.0 ** -8 * np.abs(rv) + 1.01 * ev)


@pytest.mark.parametrize("kind", [2, 3], ids=["mxfp4", "nvfp4"])
@pytest.mark.parametrize("n,d,groups", [(1, 64, 1), (130, 768, 2), (33, 448, 1), (7, 5376, 3), (5, 8192, 1)])
def test_fp4_output(ctxs, kind, n, d, groups):
    ctx = ctx_for(ctxs, d)
    i = inputs(n, d, groups, n + d, False)
    fmt = R.MX if kind == 2 else R.NV
    t = np.float32(64.0 / 2688) if fmt == R.NV else None
    xo, q, sf, rx, rv, _ = run(ctx, i, n, d, groups, True, False, kind, ALL, t=t)
    check_x(xo, i["x"], rx, 0.75, d)
    assert_quantized(fmt, q, sf, rv, t)
    blocks = d // R.BLOCK[fmt]
    full = -(-blocks // 4) * 4
    assert np.all(sf.cpu().numpy()[R.sf_index(n, full)[:, blocks:]] == (0 if fmt == R.MX else 0))


def test_mxfp8_output_is_the_modulated_norms(ctxs):
    """With no branch the call is h3dit_rmsnorm_modulate_mx."""
    n, d = 140, 768
    ctx = ctx_for(ctxs, d)
    i = inputs(n, d, 1, 4, False)
    _, q, sf, _, _, _ = run(ctx, i, n, d, 1, False, False, 1, ("shift", "scale"), r=1.0)
    from image_generation_b200 import h3dit as H

    q2 = torch.zeros(n * d, dtype=torch.uint8, device="cuda")
    sf2 = torch.full((H.mx_scale_bytes(n, d),), 255, dtype=torch.uint8, device="cuda")
    ctx.rmsnorm_modulate_mx(dev(i["x"]), dev(i["mod"][0, 1]), dev(i["mod"][0, 2]), q2, sf2)
    ok(ctx)
    # the two sum a row's squares in different orders: a last bit may move a rounding
    assert (q != q2).float().mean().item() <= 2e-3 and (sf != sf2).sum().item() <= 2
    assert (q.int() - q2.int()).abs().max().item() <= 1 or (sf != sf2).any()


def test_mxfp8_codes_block_by_block(ctxs):
    """Beside h3dit_rmsnorm_modulate_mx, in every block under the same scale no code is
    more than a step off and few are; blocks under another scale are a step of it off."""
    from image_generation_b200 import h3dit as H

    n, d = 300, 5376
    ctx = ctx_for(ctxs, d)
    i = inputs(n, d, 1, 14, False)
    _, q, sf, _, _, _ = run(ctx, i, n, d, 1, False, False, 1, ("shift", "scale"), r=1.0)
    q2 = torch.zeros(n * d, dtype=torch.uint8, device="cuda")
    sf2 = torch.zeros(H.mx_scale_bytes(n, d), dtype=torch.uint8, device="cuda")
    ctx.rmsnorm_modulate_mx(dev(i["x"]), dev(i["mod"][0, 1]), dev(i["mod"][0, 2]), q2, sf2)
    ok(ctx)
    at = R.sf_index(n, d // 32)
    a, b = (s.cpu().numpy()[at].astype(int) for s in (sf, sf2))
    assert np.abs(a - b).max() <= 1 and np.mean(a != b) <= 1e-4
    order = lambda t: np.where(t < 128, t, 128 - t)  # noqa: E731  codes in the order of their values
    step = np.abs(order(to_np(q).astype(int)) - order(to_np(q2).astype(int))).reshape(n, d // 32, 32)[a == b]
    assert step.max() <= 1 and np.mean(step) <= 2e-3


def test_zero_rows_and_nan_rows(ctxs):
    n, d = 6, 768
    ctx = ctx_for(ctxs, d)
    i = inputs(n, d, 1, 4, True)
    i["x"][1] = 0
    i["y"][1] = 0
    i["x"][3, 17] = np.nan
    i["x"][4] = 1e-30
    i["y"][4] = 0
    xo, out, _, rx, rv, _ = run(ctx, i, n, d, 1, True, True, 0, ALL)
    got, gx = to_np(out), to_np(xo)
    assert np.isnan(got[3]).all() and np.isnan(gx[3, 17]) and np.isfinite(np.delete(gx[3], 17)).all()
    keep = [0, 1, 2, 4, 5]
    assert np.all(np.abs(got[keep] - rv[keep]) <= (2.0 ** -8 + 1e-4) * np.abs(rv[keep]) + 1e-4)
    assert np.all(gx[1] == 0)
    # an FP4 row with a NaN: every scale of it is the format's NaN
    _, _, sf, _, _, _ = run(ctx, i, n, d, 1, True, True, 3, ALL, t=np.float32(0.02))
    b = sf.cpu().numpy()[R.sf_index(n, d // 16)]
    assert np.all(b[3] == 0x7f) and not np.any(b[keep] == 0x7f)


@pytest.mark.parametrize("kind", [0, 1, 2, 3], ids=["bf16", "mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("post", [False, True], ids=["plain", "post"])
@pytest.mark.parametrize("where", ["x", "branch"])
def test_where_a_nan_goes(ctxs, where, post, kind):
    """x' is NaN where x or the branch is, all along the row if a normed branch has
    one; out all along the row in any case; other rows know nothing of it."""
    n, d, row, col = 5, 768, 2, 333
    ctx = ctx_for(ctxs, d)
    i = inputs(n, d, 1, 21, True)
    clean = run(ctx, i, n, d, 1, post, True, kind, ALL, t=np.float32(0.02) if kind == 3 else None)
    i["x" if where == "x" else "y"][row, col] = np.nan
    xo, out, sf, *_ = run(ctx, i, n, d, 1, post, True, kind, ALL, t=np.float32(0.02) if kind == 3 else None)
    nan = torch.isnan(xo)
    want = torch.zeros_like(nan)
    want[row, slice(None) if where == "branch" and post else col] = True
    assert torch.equal(nan, want)
    keep = [r for r in range(n) if r != row]
    assert torch.equal(xo[keep], clean[0][keep])
    if kind == 0:
        assert torch.isnan(out[row]).all() and torch.equal(out[keep], clean[1][keep])
    elif kind == 1:
        assert (out.view(n, d)[row] & 127 == 127).all()   # E4M3 NaN
        assert torch.equal(out.view(n, d)[keep], clean[1].view(n, d)[keep])
    else:
        at = R.sf_index(n, d // (32 if kind == 2 else 16))
        got, ref = (s.cpu().numpy()[at] for s in (sf, clean[2]))
        assert np.all(got[row] == (255 if kind == 2 else 127))
        assert np.array_equal(got[keep], ref[keep]) and torch.equal(out[keep], clean[1][keep])


def test_more_rows_than_ctas_match_alone(ctxs):
    """A row's result does not depend on the rows beside it or on the launch."""
    n, d = 6000, 768
    ctx = ctx_for(ctxs, d)
    i = inputs(n, d, 1, 11, False)
    xo, out, *_ = run(ctx, i, n, d, 1, True, False, 0, ALL)
    for row in (0, 2999, n - 1):
        j = dict(i, x=i["x"][row:row + 1], y=i["y"][row:row + 1])
        xo1, out1, *_ = run(ctx, j, 1, d, 1, True, False, 0, ALL)
        assert torch.equal(xo1[0], xo[row]) and torch.equal(out1[0], out[row])


def test_offsets_past_31_bits(ctxs):
    n, d = 262_200, 8192                                  # 2.15e9 elements
    ctx = ctx_for(ctxs, d)
    x = torch.empty(n, d, device="cuda").normal_()
    y = torch.empty(n, d, dtype=torch.bfloat16, device="cuda").normal_()
    out = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
    x1, y1 = x[-3:].clone(), y[-3:].clone()
    o1 = torch.empty(3, d, dtype=torch.bfloat16, device="cuda")
    g = torch.randn(d, device="cuda")
    for a, b, o in ((x, y, out), (x1, y1, o1)):
        ctx.gated_norm(a, a, 0, o, branch=b, gate=g, post_norm=True)
    ok(ctx)
    assert torch.equal(x[-3:], x1) and torch.equal(out[-3:], o1)


def test_refusals(ctxs):
    from image_generation_b200 import h3dit as H

    ctx = ctx_for(ctxs, 768)
    odd = ctx_for(ctxs, 448)
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    b = lambda *s: f(*s).bfloat16()  # noqa: E731
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    n0 = ctx.launch_count()
    x, o = f(4, 768), b(4, 768)
    call = lambda c=ctx, **k: c.gated_norm(**{**dict(x=x, x_out=f(4, 768), out_kind=0, out=o), **k})  # noqa: E731
    bad = [
        lambda: call(out_kind=4),
        lambda: call(x=f(4, 770)),
        lambda: call(x=b(4, 768)),
        lambda: call(x_out=f(3, 768)),
        lambda: call(out=f(4, 768)),
        lambda: call(out_sf=u(65536)),                              # bf16 has no scales
        lambda: call(out_kind=2, out=u(4, 384)),                    # FP4 needs them
        lambda: call(out_kind=2, out=u(4, 384), out_sf=u(16)),
        lambda: call(out_kind=2, out=u(4, 384), out_sf=u(65536), out_scale=f(1)),
        lambda: call(post_norm=True),                               # no branch
        lambda: call(gate=f(768)),                                  # no branch
        lambda: call(branch=o, post_weight=f(768)),                 # no post norm
        lambda: call(branch=o.half()),
        lambda: call(branch=b(5, 768)),
        lambda: call(branch=o, gate=f(1, 768), rows_per_group=2),   # one row, two groups
        lambda: call(branch=o, gate=f(2, 768), shift=f(2, 2, 768)[:, 0], rows_per_group=2),  # strides
        lambda: call(rows_per_group=-1),
        lambda: call(scale=f(770)[2:]),                             # address not 16 bytes
        lambda: call(c=odd, x=f(4, 448), x_out=None, out_kind=1, out=u(4 * 448), out_sf=u(65536)),
    ]
    for j, c in enumerate(bad):
        with pytest.raises(H.H3DitError) as err:
            c()
        assert err.value.status in (H.H3DIT_ERR_INVALID_ARG, H.H3DIT_ERR_UNSUPPORTED), j
    call(x=f(0, 768), x_out=f(0, 768), out=b(0, 768))
    assert ctx.launch_count() == n0
    ok(ctx)
