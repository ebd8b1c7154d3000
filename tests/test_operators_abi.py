"""The FP4, gated-norm and rotary calls without a GPU: sizes, refusals that come
before the device is touched, and the reference's own pins."""
import ctypes as C

import numpy as np
import pytest

from image_generation_b200 import h3dit as H
from tests import operators_ref as R

torch = pytest.importorskip("torch")


def test_null_context_is_rejected():
    p = 0x10000
    bad = H.H3DIT_ERR_INVALID_ARG
    assert H.lib.h3dit_fp4_tensor_scale(None, p, 0, 64, 4, 64, p, None) == bad
    assert H.lib.h3dit_fp4_quantize(None, 0, p, 0, 64, 4, 64, None, p, p, None) == bad
    assert H.lib.h3dit_fp4_dequantize(None, 0, p, p, None, 4, 64, p, None) == bad
    assert H.lib.h3dit_linear_fp4(None, 0, 0, p, p, None, p, p, None, 4, 32, 64, p, None, None, None,
                                  None, None, None) == bad
    args = H.h3dit_norm_args()
    assert H.lib.h3dit_gated_norm(None, C.byref(args), None) == bad
    spec = H.make_rope_spec(96, (16, 16, 16))
    assert H.lib.h3dit_rope_axes(None, C.byref(spec), p, 4, 0, p, 96, p, 96, 1, None, 0, None, 0, 0,
                                 None, None, 0, None) == bad


def test_scale_bytes():
    assert H.fp4_scale_bytes(H.H3DIT_FP4_MX, 128, 128) == 512
    assert H.fp4_scale_bytes(H.H3DIT_FP4_NV, 128, 64) == 512
    assert H.fp4_scale_bytes(H.H3DIT_FP4_MX, 129, 192) == 2 * 2 * 512
    assert H.fp4_scale_bytes(H.H3DIT_FP4_NV, 16896, 5376) == 132 * 84 * 512
    for fmt, rows, k in ((0, 0, 64), (0, 4, 96), (1, 4, 0), (2, 4, 64), (-1, 4, 64)):
        assert H.fp4_scale_bytes(fmt, rows, k) == 0
    for fmt in (R.MX, R.NV):
        for rows, k in ((1, 64), (300, 448), (128, 5376)):
            assert H.fp4_scale_bytes(fmt, rows, k) == R.sf_bytes(fmt, rows, k)
            at = R.sf_index(rows, k // R.BLOCK[fmt])
            assert len(np.unique(at)) == at.size and at.max() < R.sf_bytes(fmt, rows, k)


def test_structs_have_the_headers_layout():
    """Offsets a C compiler gives the two argument structs of include/h3dit.h."""
    import os
    import shutil
    import subprocess
    import tempfile

    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    src = '#include <stdio.h>\n#include "h3dit.h"\nint main(void) {\n'
    for st in (H.h3dit_norm_args, H.h3dit_rope_spec):
        for f in st._fields_:
            src += f'printf("%zu\\n", offsetof({st.__name__}, {f[0]}));\n'
        src += f'printf("%zu\\n", sizeof({st.__name__}));\n'
    with tempfile.TemporaryDirectory() as d:
        path = os.path.join(d, "t.c")
        with open(path, "w") as fh:
            fh.write(src + "return 0; }\n")
        exe = os.path.join(d, "t")
        subprocess.run([cc, "-I", os.path.dirname(H.HEADER), path, "-o", exe], check=True)
        got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for st in (H.h3dit_norm_args, H.h3dit_rope_spec):
        want += [getattr(st, f[0]).offset for f in st._fields_] + [C.sizeof(st)]
    assert got == want


@pytest.fixture
def host_ctx():
    """A context object without a library context on a device that is not there:
    whatever the binding lets through ends as the library's refusal of NULL."""
    ctx = H.Context.__new__(H.Context)
    ctx.cfg = H.make_config(768, 8, 96, 64, 1, 1)
    ctx.workspace = torch.empty(0, device="meta")
    ctx.handle = None
    return ctx


def test_binding_refuses_other_devices_and_shapes(host_ctx):
    c, m = host_ctx, dict(device="meta")
    u8, f32, bf = (dict(dtype=t, **m) for t in (torch.uint8, torch.float32, torch.bfloat16))
    q, sf, x = torch.empty(4, 64, **u8), torch.empty(2048, **u8), torch.empty(4, 128, **bf)
    spec = H.make_rope_spec(96, (16, 16, 16))
    calls = [
        (lambda: c.fp4_quantize(0, x.new_empty(4, 128, device="cpu"), q, sf), "is on cpu"),
        (lambda: c.fp4_quantize(0, x, q[:, :63], sf), "shape"),
        (lambda: c.fp4_quantize(0, x, q, sf[:100]), "needed"),
        (lambda: c.fp4_quantize(5, x, q, sf), "format"),
        (lambda: c.fp4_quantize(0, x.float().int(), q, sf), "dtype"),
        (lambda: c.fp4_tensor_scale(x, torch.empty(2, **f32)), "one number"),
        (lambda: c.linear_fp4(0, 0, q, sf, torch.empty(32, 32, **u8), sf, torch.empty(4, 32, **bf)), "shape"),
        (lambda: c.linear_fp4(0, 0, q, None, torch.empty(32, 64, **u8), sf, torch.empty(4, 32, **bf)), "needed"),
        (lambda: c.gated_norm(torch.empty(4, 768, **f32), None, 0, None), "needed"),
        (lambda: c.gated_norm(torch.empty(4, 770, **f32), None, 0, x), "shape"),
        (lambda: c.rope_axes(spec, None, x, x, 1), "positions is needed"),
        (lambda: c.rope_axes(spec, torch.empty(4, 3, **f32), x, x, 2), "shape"),
        (lambda: c.rope_axes(spec, torch.empty(4, 3, **f32), None, None, 2), "needed"),
    ]
    for call, words in calls:
        with pytest.raises(H.H3DitError, match=words):
            call()


def test_reference_quantization_pins():
    """Hand-computed blocks of both formats."""
    x = np.zeros((1, 64), np.float32)
    x[0, :8] = [6, -6, 5, 2.5, 0.25, 0.75, -1.25, 3.5]
    c, b = R.quantize(R.MX, x)
    assert b.tolist() == [[127, 0]]
    # ties go to the even code: 5 -> 4, 2.5 -> 2, 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 3.5 -> 4
    assert c[0, :8].tolist() == [7, 15, 6, 4, 0, 2, 10, 6]
    assert np.allclose(R.values(R.MX, c, b)[0, :8], [6, -6, 4, 2, 0, 1, -1, 4])
    g = R.tensor_scale(x)
    assert g == np.float32(6) / np.float32(2688)
    c, b = R.quantize(R.NV, x, g)
    assert b[0, 0] == R.e4m3_code(448.0) == 0x7e and not b[0, 1:].any()
    assert R.e4m3_code(np.array([0, 2.0 ** -10, 2.0 ** -9, 1.0625, 1.1875, 460])).tolist() == \
        [0, 0, 1, 0x38, 0x3a, 0x7e]
    assert R.e2m1_code(np.array([0.0, -0.0, 100, -100, 1.75])).tolist() == [0, 8, 7, 15, 4]
    assert np.array_equal(R.unpack(R.pack(c)), c)


def test_reference_rope_is_a_rotation():
    g = np.random.default_rng(0)
    h, pos = g.standard_normal((5, 2, 96)), g.standard_normal((5, 3)) * 50
    for inter in (False, True):
        y, _ = R.rope(h, pos, (16, 8, 20), 1e4, inter)
        back, _ = R.rope(y, pos, (16, 8, 20), 1e4, inter, inverse=True)
        assert np.allclose(back, h) and np.allclose((y * y).sum(-1), (h * h).sum(-1))
        assert np.array_equal(y[..., 88:], h[..., 88:])
