"""h3dit_rope_axes against its definition in 64 bits: both pair orders, shared key
heads, sections of any size, partial rotation, far positions, strides, the
inverse as the rotation's gradient."""
import numpy as np
import pytest

from tests import operators_ref as R
from tests.helpers import to_np
from tests.test_gpu_fp4 import bf16, dev, make_ctx, ok
from tests.test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# an angle is off by 2^-25 half turns and its sine by 2 steps (under 3e-7 in all), two
# products and a sum by 3 * 2^-24; the norm by 30 * 2^-24
TURN, NORM = 3e-7 + 3 * 2.0 ** -24, 30 * 2.0 ** -24


@pytest.fixture(scope="module")
def ctx():
    return make_ctx()


def rows(n, width, seed, f32, pad):
    x = np.random.default_rng(seed).standard_normal((n, width)).astype(np.float32)
    x = x if f32 else bf16(x).astype(np.float32)
    t = dev(np.pad(x, ((0, 0), (0, pad)), constant_values=9.0))
    return x, (t if f32 else t.bfloat16())[:, :width]


def positions(n, seed, far=False):
    g = np.random.default_rng(seed)
    p = np.stack([np.arange(n) // 64, np.arange(n) // 8 % 8, np.arange(n) % 8], -1) + g.random(3)
    return (p * (12345.678 if far else 1) - (7 if not far else 0)).astype(np.float32)


SPECS = [(64, (8, 12, 12), True), (64, (8, 12, 12), False), (96, (16, 16, 16), False), (96, (8, 16, 16), False),
         (128, (16, 24, 24), False), (128, (22, 21, 21), True), (128, (22, 21, 21), False), (16, (2, 3, 3), False),
         (256, (40, 40, 40), False), (240, (1, 0, 31), True), (48, (0, 0, 0), False), (112, (8, 0, 24), False),
         (80, (5, 7, 9), False)]


def bound(ref, size, f32, norm):
    e = (TURN + (NORM if norm else 0)) * size
    return e if f32 else 2.0 ** -8 * np.abs(ref) + 1.01 * e


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
@pytest.mark.parametrize("dh,sec,inter", SPECS, ids=str)
def test_heads(ctx, dh, sec, inter, norm, f32):
    from image_generation_b200 import h3dit as H

    n, hq, hk = 133, 8, 3
    spec = H.make_rope_spec(dh, sec, 10000.0, interleaved=inter)
    pos = positions(n, dh)
    q, qt = rows(n, hq * dh, 1, f32, 16)
    k, kt = rows(n, hk * dh, 2, f32, 32)
    g = np.random.default_rng(3)
    wq, wk = ((1 + 0.1 * g.standard_normal(dh)).astype(np.float32) for _ in range(2))
    dt = torch.float32 if f32 else torch.bfloat16
    qo, ko = Guarded((n, hq * dh), dt), Guarded((n, hk * dh), dt)
    ctx.rope_axes(spec, dev(pos), qt, qo.t, hq, kt, ko.t, hk, q_weight=dev(wq) if norm else None,
                  k_weight=dev(wk) if norm else None)
    ok(ctx)
    qo.check("q")
    ko.check("k")
    for x, o, h, w in ((q, qo, hq, wq), (k, ko, hk, wk)):
        ref, size = R.rope(x.reshape(n, h, dh), pos, sec, 10000.0, inter, w, norm)
        assert np.all(np.abs(to_np(o.t).reshape(n, h, dh) - ref) <= bound(ref, size, f32, norm) + 1e-30)


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("dh,sec,inter", [(96, (16, 16, 16), False), (128, (22, 21, 21), True), (80, (5, 7, 9), False),
                                          (112, (8, 0, 24), False), (112, (9, 0, 24), False), (240, (1, 0, 31), True)],
                         ids=str)
def test_one_weight_norms_both(ctx, dh, sec, inter, which):
    """With a weight for Q or K alone both are normalised, the other by 1, also where the
    lane in which the rotation ends reads its weights again."""
    from image_generation_b200 import h3dit as H

    n, hq, hk = 41, 5, 2
    pos = positions(n, dh)
    q, qt = rows(n, hq * dh, 1, True, 0)
    k, kt = rows(n, hk * dh, 2, True, 0)
    wt = (1 + 0.3 * np.random.default_rng(3).standard_normal(dh)).astype(np.float32)
    qo, ko = torch.empty_like(qt), torch.empty_like(kt)
    ctx.rope_axes(H.make_rope_spec(dh, sec, interleaved=inter), dev(pos), qt, qo, hq, kt, ko, hk,
                  **{which + "_weight": dev(wt)})
    ok(ctx)
    for name, x, o, h in (("q", q, qo, hq), ("k", k, ko, hk)):
        ref, size = R.rope(x.reshape(n, h, dh), pos, sec, 10000.0, inter, wt if name == which else None, True)
        assert np.all(np.abs(to_np(o).reshape(n, h, dh) - ref) <= bound(ref, size, True, True) + 1e-30), name


@pytest.mark.parametrize("n", [1, 2, 700, 5000])
def test_token_counts(ctx, n):
    """One token to several per CTA, with a ragged end; only keys, only queries."""
    from image_generation_b200 import h3dit as H

    dh, sec = 96, (16, 16, 16)
    spec = H.make_rope_spec(dh, sec, 10000.0)
    pos = positions(n, n)
    q, qt = rows(n, 5 * dh, 1, False, 0)
    qo = Guarded((n, 5 * dh), torch.bfloat16)
    ctx.rope_axes(spec, dev(pos), qt, qo.t, 5)
    ko = Guarded((n, 5 * dh), torch.bfloat16)
    ctx.rope_axes(spec, dev(pos), None, None, 0, qt, ko.t, 5)
    ok(ctx)
    qo.check("q")
    ref, size = R.rope(q.reshape(n, 5, dh), pos, sec, 10000.0, False)
    assert np.all(np.abs(to_np(qo.t).reshape(n, 5, dh) - ref) <= bound(ref, size, False, False))
    assert torch.equal(qo.t, ko.t)


def test_far_positions_and_the_table_of_the_block(ctx):
    from image_generation_b200 import h3dit as H

    n, dh, sec = 300, 96, (16, 16, 16)
    spec = H.make_rope_spec(dh, sec, 10000.0)
    q, qt = rows(n, 2 * dh, 1, True, 0)
    pos = positions(n, 1, far=True)
    assert pos.max() > 5e4
    qo = torch.empty_like(qt)
    ctx.rope_axes(spec, dev(pos), qt, qo, 2)
    ok(ctx)
    ref, size = R.rope(q.reshape(n, 2, dh), pos, sec, 10000.0, False)
    assert np.all(np.abs(to_np(qo).reshape(n, 2, dh) - ref) <= bound(ref, size, True, False))
    # the angles of h3dit_rope_table's grids
    grids, n_txt = [(0, 9, 11), (1, 5, 6)], 4
    m = n_txt + 99 + 30
    table = torch.empty(m, dh // 2, 2, device="cuda")
    ctx.rope_table(grids, n_txt, table)
    p = [(0, 0, 0)] * n_txt + [(f, r, c) for f, h, w in grids for r in range(h) for c in range(w)]
    one = torch.zeros(m, dh, device="cuda")
    for s in range(3):
        one[:, 32 * s:32 * s + 16] = 1.0   # every pair (1, 0) turns into (cos, sin)
    o = torch.empty_like(one)
    ctx.rope_axes(spec, dev(np.array(p, np.float32)), one, o, 1)
    ok(ctx)
    got = torch.stack([o.view(m, 3, 2, 16)[:, :, i] for i in (0, 1)], -1).reshape(m, 48, 2)
    assert (got - table).abs().max().item() <= 4e-7


@pytest.mark.parametrize("theta", [1.0, 1e4, 2.0 ** 100, 3e38])
def test_positions_up_to_a_million(ctx, theta):
    """The angle's promise over the bases: its frequency is good to 2.2e-14, so at 1e6
    it is off by 2.2e-8 beside the 9.4e-8 of its last rounding: within TURN."""
    from image_generation_b200 import h3dit as H

    n, dh, sec = 64, 256, (43, 42, 43)
    pos = np.random.default_rng(6).uniform(-1e6, 1e6, (n, 3)).astype(np.float32)
    q, qt = rows(n, 2 * dh, 1, True, 0)
    for inter in (False, True):
        out = torch.empty_like(qt)
        ctx.rope_axes(H.make_rope_spec(dh, sec, theta, interleaved=inter), dev(pos), qt, out, 2)
        ok(ctx)
        t = float(np.float32(theta))
        ref, size = R.rope(q.reshape(n, 2, dh), pos, sec, t, inter)
        assert np.all(np.abs(to_np(out).reshape(n, 2, dh) - ref) <= bound(ref, size, True, False))


@pytest.mark.parametrize("inter,sec", [(False, (16, 16, 16)), (True, (16, 16, 16)), (False, (5, 7, 9))])
def test_in_place_and_inverse_is_the_gradient(ctx, inter, sec):
    from image_generation_b200 import h3dit as H

    n, h, dh = 70, 4, 96
    spec = H.make_rope_spec(dh, sec, 500.0, interleaved=inter)
    pos = positions(n, 5)
    x, xt = rows(n, h * dh, 1, True, 0)
    d, dt = rows(n, h * dh, 2, True, 0)
    y, grad = torch.empty_like(xt), torch.empty_like(xt)
    ctx.rope_axes(spec, dev(pos), xt, y, h)
    ctx.rope_axes(spec, dev(pos), dt, grad, h, inverse=True)
    ip = xt.clone()
    ctx.rope_axes(spec, dev(pos), ip, ip, h)
    ok(ctx)
    assert torch.equal(ip, y)
    gref, size = R.rope(d.reshape(n, h, dh), pos, sec, 500.0, inter, inverse=True)
    assert np.all(np.abs(to_np(grad).reshape(n, h, dh) - gref) <= bound(gref, size, True, False))
    # d/dx of <rope(x), d> by differences of the float64 definition (linear: any step will do)
    f = lambda v: float((R.rope(v.reshape(n, h, dh), pos, sec, 500.0, inter)[0] * d.reshape(n, h, dh)).sum())  # noqa: E731
    g = np.random.default_rng(8)
    for _ in range(3):
        e = g.standard_normal(x.shape)
        num = (f(x + 0.5 * e) - f(x - 0.5 * e))
        ana = float((to_np(grad) * e).sum())
        # |grad| is off by 1e-6 of itself at most, element by element
        assert abs(num - ana) <= 1e-6 * float((np.abs(size.reshape(x.shape)) * np.abs(e)).sum())
    back = torch.empty_like(y)
    ctx.rope_axes(spec, dev(pos), y, back, h, inverse=True)
    ok(ctx)
    assert np.all(np.abs(to_np(back) - x) <= 4 * TURN * (size.reshape(x.shape) * 0 + np.abs(x).max() * 2))


def test_zero_and_extreme_heads(ctx):
    from image_generation_b200 import h3dit as H

    n, h, dh, sec = 3, 4, 96, (16, 16, 16)
    spec = H.make_rope_spec(dh, sec)
    x = np.random.default_rng(0).standard_normal((n, h, dh)).astype(np.float32)
    x[0, 1] = 0
    x[1, 2, 5] = np.nan
    x[2, 3] = 1e-25
    xt = dev(x.reshape(n, -1))
    o = torch.empty_like(xt)
    ctx.rope_axes(spec, dev(positions(n, 1)), xt, o, h, q_weight=torch.ones(dh, device="cuda"))
    ok(ctx)
    got = to_np(o).reshape(n, h, dh)
    assert np.all(got[0, 1] == 0) and np.isnan(got[1, 2]).all()
    ref, size = R.rope(x, positions(n, 1), sec, 1e4, False, 1.0, True)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isfinite(got), fin)
    assert np.all(np.abs(got - ref)[fin] <= bound(ref, size, True, True)[fin])


@pytest.mark.parametrize("sec", [(8, 0, 24), (5, 7, 9), (0, 0, 0)])
@pytest.mark.parametrize("inter", [False, True], ids=["split", "interleaved"])
def test_what_passes_through_keeps_to_itself(ctx, sec, inter):
    """Infinities and NaN in the part that does not turn come out where they went in."""
    from image_generation_b200 import h3dit as H

    n, h, dh, turning = 9, 3, 112, 2 * sum(sec)
    x = np.random.default_rng(4).standard_normal((n, h, dh)).astype(np.float32)
    x[2, 1, turning + 1], x[3, 0, dh - 1], x[4, 2, turning] = np.inf, np.nan, -np.inf
    xt = dev(x.reshape(n, -1))
    o = torch.empty_like(xt)
    ctx.rope_axes(H.make_rope_spec(dh, sec, interleaved=inter), dev(positions(n, 1)), xt, o, h)
    ok(ctx)
    assert np.array_equal(to_np(o).reshape(n, h, dh)[..., turning:], x[..., turning:].astype(np.float64),
                          equal_nan=True)
    assert np.isfinite(to_np(o).reshape(n, h, dh)[..., :turning]).all()


def test_offsets_past_31_bits(ctx):
    from image_generation_b200 import h3dit as H

    n, h, dh = 300_100, 56, 128                           # 2.15e9 elements, in place
    spec = H.make_rope_spec(dh, (16, 24, 24))
    x = torch.empty(n, h * dh, dtype=torch.bfloat16, device="cuda").normal_()
    pos = dev(positions(n, 2))
    x1 = x[-5:].clone()
    ctx.rope_axes(spec, pos, x, x, h)
    ctx.rope_axes(spec, pos[-5:].clone(), x1, x1, h)
    ok(ctx)
    assert torch.equal(x[-5:], x1)


def test_refusals(ctx):
    from image_generation_b200 import h3dit as H

    b = lambda *s: torch.zeros(*s, device="cuda").bfloat16()  # noqa: E731
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    n0 = ctx.launch_count()
    spec = H.make_rope_spec(96, (16, 16, 16))
    q, p = b(4, 192), f(4, 3)
    call = lambda **k: ctx.rope_axes(**{**dict(spec=spec, positions=p, q=q, q_out=b(4, 192), heads_q=2), **k})  # noqa: E731
    big = b(4, 400)
    bad = [
        lambda: call(spec=H.make_rope_spec(100, (16, 16, 16)), q=b(4, 200), q_out=b(4, 200)),
        lambda: call(spec=H.make_rope_spec(272, (16, 16, 16)), q=b(4, 544), q_out=b(4, 544)),
        lambda: call(spec=H.make_rope_spec(96, (16, 16, 17))),
        lambda: call(spec=H.make_rope_spec(96, (-1, 16, 16))),
        lambda: call(spec=H.make_rope_spec(96, (16, 16, 16), theta=0.0)),
        lambda: call(spec=H.make_rope_spec(96, (16, 16, 16), theta=float("inf"))),
        lambda: call(positions=f(5, 3)),
        lambda: call(positions=f(4, 2)),
        lambda: call(positions=p.double()),
        lambda: call(q=q.half()),
        lambda: call(q_out=f(4, 192)),
        lambda: call(heads_q=3),
        lambda: call(heads_q=-1),
        lambda: call(q=b(4, 196)[:, :192]),                            # stride not 16 bytes
        lambda: call(q=big[:, 4:196]),                                 # address not 16 bytes
        lambda: call(q=big[:, :192], q_out=big.view(-1)[:768].view(4, 192)),  # in place, two strides
        lambda: call(q=big[:1, :192].expand(4, 192)),                  # rows that overlap
        lambda: call(k=f(4, 96), k_out=f(4, 96), heads_k=1),           # two types
        lambda: call(q_weight=f(95)),
        lambda: call(q_weight=f(96), inverse=True),
    ]
    for j, c in enumerate(bad):
        with pytest.raises(H.H3DitError) as err:
            c()
        assert err.value.status in (H.H3DIT_ERR_INVALID_ARG, H.H3DIT_ERR_UNSUPPORTED), j
    call(positions=f(0, 3), q=b(0, 192), q_out=b(0, 192))
    call(q=None, q_out=None, heads_q=0)
    assert ctx.launch_count() == n0
    ok(ctx)
