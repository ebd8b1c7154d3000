"""The FP4, gated-norm and rotary operators run together as one DiT block with
4-bit linears: norm (FP4 rows out) -> QKV -> norm and rotation of the heads ->
attention -> FP4 -> out-projection -> norm across the residual -> FFN1 with GELU
(FP4 rows out) -> FFN2 -> the next norm. Two images of a batch with their own
modulation share the row-wise steps; the attention is per image.

Each step is held to its own definition in 64 bits on what the library's step
before it wrote, with that operator's bound: a run's end compared with a 64-bit
run's end would say less, since the attention's bf16 probabilities move values
across FP4's borders, a third of the value at a time."""
import numpy as np
import pytest

from image_generation_b200 import synth
from oracle import dit_block as O
from tests import operators_ref as R
from tests.helpers import assert_attention_bound, to_np
from tests.test_gpu_fp4 import FMTS, assert_quantized, bf16, dev, make_ctx, ok, sum_bound
from tests.test_gpu_gated_norm import check_x, out_error
from tests.test_gpu_rope_axes import bound as rope_bound

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D, HEADS, DH, FFN, N = 768, 8, 96, 2048, 150  # N tokens of each of two images
I = HEADS * DH
SEC = (16, 16, 16)


def weights(seed):
    g = np.random.default_rng(seed)
    w = {k: bf16(0.02 * g.standard_normal(s)) for k, s in
         (("qkv", (3 * I, D)), ("o", (D, I)), ("ff1", (FFN, D)), ("ff2", (D, FFN)))}
    w["mod"] = (0.3 * g.standard_normal((2, 6, D))).astype(np.float32)
    w["post1"], w["post2"] = ((1 + 0.1 * g.standard_normal(D)).astype(np.float32) for _ in range(2))
    w["wq"], w["wk"] = ((1 + 0.1 * g.standard_normal(DH)).astype(np.float32) for _ in range(2))
    w["b1"] = (0.1 * g.standard_normal(FFN)).astype(np.float32)
    return w


# what an activation's tensor scale is calibrated to: its largest element over 2688
SCALES = {"xn": 8.0, "attn": 4.0, "u": 4.0}


class Library:
    """The block through the library, every buffer made once."""

    def __init__(self, fmt, w, pos):
        from image_generation_b200 import h3dit as H

        self.H, self.fmt, self.ctx = H, fmt, make_ctx(D)
        rows = 2 * N
        e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        fp4 = lambda r, k: (e(r, k // 2, dt=torch.uint8), e(R.sf_bytes(fmt, r, k), dt=torch.uint8))  # noqa: E731
        self.w = {}
        for k in ("qkv", "o", "ff1", "ff2"):
            t = dev(w[k].astype(np.float32)).bfloat16()
            s = torch.empty(1, device="cuda") if fmt == R.NV else None
            if s is not None:
                self.ctx.fp4_tensor_scale(t, s)
            q, sf = fp4(*w[k].shape)
            self.ctx.fp4_quantize(fmt, t, q, sf, tensor_scale=s)
            self.w[k] = (q, sf, s)
        self.v = {k: dev(w[k]) for k in ("mod", "post1", "post2", "wq", "wk", "b1")}
        self.t = {k: torch.full((1,), v / 2688, device="cuda") if fmt == R.NV else None
                  for k, v in SCALES.items()}
        self.pos = dev(np.concatenate([pos, pos]).astype(np.float32))
        self.spec = H.make_rope_spec(DH, SEC)
        self.x, self.out = e(rows, D, dt=torch.float32), e(rows, D)
        self.xn, self.an, self.un = fp4(rows, D), fp4(rows, I), fp4(rows, FFN)
        self.qkv, self.qk, self.attn = e(rows, 3 * I), e(rows, 2 * I), e(rows, I)
        self.branch = e(rows, D)

    def __call__(self, x_in):
        H, c, fmt, v, t, w = self.H, self.ctx, self.fmt, self.v, self.t, self.w
        kind = H.H3DIT_NORM_OUT_FP4_NV if fmt == R.NV else H.H3DIT_NORM_OUT_FP4_MX
        seen = self.seen = {}
        keep = lambda k, *ts: seen.update({k: [z.clone() for z in ts]})  # noqa: E731
        m = lambda i: v["mod"][:, i]  # noqa: E731
        lin = lambda epi, a, ts, k, out, **kw: c.linear_fp4(fmt, epi, *a, *w[k][:2], out, a_scale=ts, w_scale=w[k][2], **kw)  # noqa: E731
        c.gated_norm(x_in, None, kind, *self.xn, out_scale=t["xn"], shift=m(0), scale=m(1), rows_per_group=N)
        keep("xn1", *self.xn)
        lin(H.H3DIT_EPI_STORE, self.xn, t["xn"], "qkv", self.qkv)
        keep("qkv", self.qkv)
        c.rope_axes(self.spec, self.pos, self.qkv[:, :I], self.qk[:, :I], HEADS, self.qkv[:, I:2 * I],
                    self.qk[:, I:], HEADS, q_weight=v["wq"], k_weight=v["wk"])
        keep("qk", self.qk)
        self.qkv[:, :2 * I] = self.qk  # the attention takes one row stride
        c.attention_batched(self.qkv[:, :I], self.qkv[:, I:2 * I], self.qkv[:, 2 * I:], 3 * I, self.attn, I, N, 2)
        c.fp4_quantize(fmt, self.attn, *self.an, tensor_scale=t["attn"])
        keep("attn", self.attn, *self.an)
        lin(H.H3DIT_EPI_STORE, self.an, t["attn"], "o", self.branch)
        keep("branch1", self.branch)
        c.gated_norm(x_in, self.x, kind, *self.xn, out_scale=t["xn"], branch=self.branch, post_norm=True,
                     post_weight=v["post1"], gate=m(2), shift=m(3), scale=m(4), rows_per_group=N)
        keep("x1", self.x, *self.xn)
        lin(H.H3DIT_EPI_GELU, self.xn, t["xn"], "ff1", self.un[0], out_sf=self.un[1], out_scale=t["u"], bias=v["b1"])
        keep("u", *self.un)
        lin(H.H3DIT_EPI_STORE, self.un, t["u"], "ff2", self.branch)
        keep("branch2", self.branch)
        c.gated_norm(self.x, self.x, H.H3DIT_NORM_OUT_BF16, self.out, branch=self.branch, post_norm=True,
                     post_weight=v["post2"], gate=m(5), rows_per_group=N)
        return self.x, self.out


def setup(fmt):
    w = weights(3)
    grid = np.stack([np.zeros(N), np.arange(N) // 15, np.arange(N) % 15], -1)
    x = synth.normal_f32((2 * N, D), 1.0, 5, "x")
    return w, grid, x


@FMTS
def test_block_with_4_bit_linears(fmt):
    w, pos, x = setup(fmt)
    lib = Library(fmt, w, pos)
    xg, og = lib(dev(x))
    ok(lib.ctx)
    s = lib.seen
    t = {k: np.float32(v / 2688) if fmt == R.NV else None for k, v in SCALES.items()}
    m = lambda i: w["mod"][:, i]  # noqa: E731

    def given(pair, k, g):  # what an FP4 matrix of the library stands for
        q, sf = pair
        byte = sf.cpu().numpy()[R.sf_index(q.shape[0], k // R.BLOCK[fmt])]
        return R.values(fmt, R.unpack(q.cpu().numpy()), byte, g)

    def weight(k):
        g = R.tensor_scale(w[k]) if fmt == R.NV else None
        return R.values(fmt, *R.quantize(fmt, w[k].astype(np.float32), g), g)

    def product(a, wv, got, what):
        ref = a @ wv.T
        err = sum_bound(a, wv, a.shape[1]) + 2 * 2.0 ** -24 * np.abs(ref)
        assert np.all(np.abs(to_np(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * err), what
        return ref, err

    # norm -> QKV -> heads
    _, v = R.gated_norm(x, shift=m(0), scale=m(1), per=N)
    assert_quantized(fmt, *s["xn1"], v, t["xn"])
    product(given(s["xn1"], D, t["xn"]), weight("qkv"), s["qkv"][0], "qkv")
    qkv, qk = to_np(s["qkv"][0]), to_np(s["qk"][0])
    p2 = np.concatenate([pos, pos])
    for j, wt in ((0, w["wq"]), (1, w["wk"])):
        ref, size = R.rope(qkv[:, j * I:(j + 1) * I].reshape(-1, HEADS, DH), p2, SEC, 1e4, False, wt, True)
        got = qk[:, j * I:(j + 1) * I].reshape(-1, HEADS, DH)
        assert np.all(np.abs(got - ref) <= rope_bound(ref, size, False, True)), j
    # attention -> FP4, bit for bit -> out-projection
    h = lambda a, i: a[i * N:(i + 1) * N].reshape(N, HEADS, DH)  # noqa: E731
    attn = to_np(s["attn"][0])
    for i in range(2):
        q, k, vv = h(qk[:, :I], i), h(qk[:, I:], i), h(qkv[:, 2 * I:], i)
        assert_attention_bound(attn[i * N:(i + 1) * N], O.attention(q, k, vv).reshape(N, I),
                               np.abs(vv).max(), f"image {i}")
    codes, byte = R.quantize(fmt, attn.astype(np.float32), t["attn"])
    assert np.array_equal(s["attn"][2].cpu().numpy()[R.sf_index(2 * N, byte.shape[1])], byte)
    got = R.unpack(s["attn"][1].cpu().numpy())
    assert np.all((got == codes) | (((got | codes) & 7) == 0))
    product(given(s["attn"][1:], I, t["attn"]), weight("o"), s["branch1"][0], "out-projection")
    # across the residual -> FFN1 -> FFN2
    rx, v = R.gated_norm(x, to_np(s["branch1"][0]), m(2), m(3), m(4), N, True, w["post1"])
    check_x(s["x1"][0], x, rx, 1.0, D)
    assert_quantized(fmt, *s["x1"][1:], v, t["xn"])
    pre = given(s["x1"][1:], D, t["xn"]) @ weight("ff1").T + w["b1"]
    assert_quantized(fmt, *s["u"], R.gelu(pre), t["u"])
    product(given(s["u"], FFN, t["u"]), weight("ff2"), s["branch2"][0], "ffn2")
    x1 = to_np(s["x1"][0])
    rx, rv = R.gated_norm(x1, to_np(s["branch2"][0]), m(5), None, None, N, True, w["post2"])
    ex = check_x(xg, x1, rx, 1.0, D)
    assert np.all(np.abs(to_np(og) - rv) <= 2.0 ** -8 * np.abs(rv) + 1.01 * out_error(rx, rv, 0 * rv, ex))


@FMTS
def test_images_do_not_see_each_other(fmt):
    """The two images in the other order, with their modulations: the same rows."""
    w, pos, x = setup(fmt)
    lib = Library(fmt, w, pos)
    first = [z.clone() for z in lib(dev(x))]
    lib.v["mod"] = lib.v["mod"].flip(0).contiguous()
    for a, b in zip(first, lib(dev(np.concatenate([x[N:], x[:N]])))):
        assert torch.equal(a[:N], b[N:]) and torch.equal(a[N:], b[:N])
    ok(lib.ctx)


@FMTS
def test_block_repeats_and_replays(fmt):
    """Run to run the same bits, and the same from a captured graph with new inputs."""
    w, pos, x = setup(fmt)
    lib = Library(fmt, w, pos)
    xt = dev(x)
    first = [t.clone() for t in lib(xt)]
    second = [t.clone() for t in lib(xt)]
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib(xt)
    xt.copy_(dev(x[::-1].copy()))
    graph.replay()
    got = [t.clone() for t in (lib.x, lib.out)]
    ok(lib.ctx)
    want = lib(xt)
    ok(lib.ctx)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_decoder_context_takes_the_calls():
    """The decoder's context has them too, its width for the norm."""
    from image_generation_b200 import h3dit as H
    from tests.test_gpu_vae import _decoder

    v = synth.VAE_SMALL
    ctx, _ = _decoder(v, 2048)
    n, k = 40, v.width
    x = synth.normal_f32((n, k), 1.0, 1, "x")
    q = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(R.sf_bytes(R.NV, n, k), dtype=torch.uint8, device="cuda")
    t, out = torch.empty(1, device="cuda"), torch.ones(n, 32, dtype=torch.bfloat16, device="cuda")
    ctx.gated_norm(dev(x), None, H.H3DIT_NORM_OUT_FP4_NV, q, out_sf=sf)
    _, v64 = R.gated_norm(x)
    ok(ctx)
    assert_quantized(R.NV, q, sf, v64, np.float32(1))
    ctx.fp4_tensor_scale(dev(x), t)
    assert t.item() == float(R.tensor_scale(x))
    w = torch.zeros(32, k // 2, dtype=torch.uint8, device="cuda")
    wsf = torch.zeros(R.sf_bytes(R.NV, 32, k), dtype=torch.uint8, device="cuda")
    ctx.linear_fp4(R.NV, H.H3DIT_EPI_STORE, q, sf, w, wsf, out)
    ok(ctx)
    assert not out.any()


@FMTS
def test_two_contexts_on_two_streams(fmt):
    """Each on its own stream, their calls among one another's: as alone."""
    w, pos, x = setup(fmt)
    libs = [Library(fmt, w, pos) for _ in range(2)]
    xs = [dev(x), dev(np.ascontiguousarray(x[::-1]))]
    want = [[z.clone() for z in lib(v)] for lib, v in zip(libs, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = libs[i](xs[i])
    for i in range(2):
        ok(libs[i].ctx)
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


@FMTS
def test_calls_allocate_nothing(fmt):
    """Repeated calls take nothing of the device's memory, nor of torch's."""
    from image_generation_b200 import h3dit as H

    c = make_ctx(D)
    e = lambda *s, dt=torch.bfloat16: torch.ones(*s, dtype=dt, device="cuda")  # noqa: E731
    x, xo, y, out = e(N, D, dt=torch.float32), e(N, D, dt=torch.float32), e(N, D), e(N, D)
    q, sf = e(N, D // 2, dt=torch.uint8), e(R.sf_bytes(fmt, N, D), dt=torch.uint8)
    w, wsf = e(D, D // 2, dt=torch.uint8), e(R.sf_bytes(fmt, D, D), dt=torch.uint8)
    t, pos = e(1, dt=torch.float32), e(N, 3, dt=torch.float32)
    kind = H.H3DIT_NORM_OUT_FP4_NV if fmt == R.NV else H.H3DIT_NORM_OUT_FP4_MX
    ts, spec = (t if fmt == R.NV else None), H.make_rope_spec(DH, SEC)

    def go():
        c.gated_norm(x, xo, kind, q, out_sf=sf, out_scale=ts, branch=y)
        c.linear_fp4(fmt, H.H3DIT_EPI_STORE, q, sf, w, wsf, out, a_scale=ts)
        c.rope_axes(spec, pos, out, out, HEADS)
        c.fp4_tensor_scale(out, t)
        c.fp4_quantize(fmt, out, q, sf, tensor_scale=ts)
        c.fp4_dequantize(fmt, q, sf, y, tensor_scale=ts)

    go()
    ok(c)
    held, free = torch.cuda.memory_allocated(), torch.cuda.mem_get_info()[0]
    for _ in range(20):
        go()
    ok(c)
    assert torch.cuda.memory_allocated() == held and torch.cuda.mem_get_info()[0] >= free
