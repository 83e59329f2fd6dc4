"""One workspace, as large as the largest batch needs, serves every smaller one, and nothing is written past it."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import fp8_ref as R  # noqa: E402

E, K, H, I = 12, 2, 272, 128
GUARD = 1 << 16


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_moe_quantize_gb300 import _lib, build
    build.build()
    return _lib.load()


def buffers(n):
    buf = torch.full((n + GUARD + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    skip = -buf.data_ptr() % 256
    return buf[skip:skip + n], buf[skip + n:]


# one token, one slot each, tiles of 16, of 32, and of 256
SIZES = [1, 3, 20, 72, 73, 300, 312, 313, 400]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("most", [312, 400, 2000])
def test_layer(lib, dt, most):
    import bit_quantized_moe_quantize_gb300 as ft
    g = R.gen(most)
    w13, s13 = R.weights(g, E, 2 * I, H)
    w2, s2 = R.weights(g, E, H, I)
    n = lib.ft_moe_layer_fp8_workspace_bytes(most, K, E, H, I)
    ws, guard = buffers(n)
    for T in [t for t in SIZES if t <= most] + [most]:
        x = R.rows(g, T, H, dt)
        logits = torch.randn(T, E, generator=g, device="cuda")
        want = ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, K)
        y, ids = torch.empty_like(x), torch.empty_like(want[1])
        w = torch.empty_like(want[2])
        st = lib.ft_moe_layer_fp8(x.data_ptr(), 1 if dt == torch.float16 else 2, logits.data_ptr(), 0, E, None, w13.data_ptr(),
                                  s13.data_ptr(), w2.data_ptr(), s2.data_ptr(), y.data_ptr(), ids.data_ptr(), w.data_ptr(),
                                  T, E, K, H, I, 0, 1, 1, 1, 1, 1.0, 0, ws.data_ptr(), n,
                                  torch.cuda.current_stream().cuda_stream)
        assert st == 0, (T, lib.ft_last_error())
        assert torch.equal(y, want[0]) and torch.equal(ids, want[1]) and torch.equal(w, want[2])
        assert (guard == 0xA5).all()


@pytest.mark.parametrize("most", [312, 400, 2000])
def test_product(lib, most):
    import bit_quantized_moe_quantize_gb300 as ft
    g = R.gen(most)
    wt, sw = R.weights(g, E, I, H)
    n = lib.ft_moe_fp8_workspace_bytes(most, K, E, H)
    ws, guard = buffers(n)
    for T in [t for t in SIZES if t <= most] + [most]:
        q, s = R.codes(g, T, H)
        ids = R.ids(g, T, E, K, 0.1)
        out = torch.empty(T, K, I, device="cuda")
        st = lib.ft_moe_fp8_fp8(wt.data_ptr(), sw.data_ptr(), q.data_ptr(), s.data_ptr(), ids.data_ptr(), out.data_ptr(), 0, T, K,
                                E, I, H, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
        assert st == 0, (T, lib.ft_last_error())
        assert torch.equal(out, ft.moe_fp8_fp8(wt, sw, q, s, ids)) and (guard == 0xA5).all()
