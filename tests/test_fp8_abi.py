"""The FP8 entry points reject bad arguments on the host, before any CUDA call (CPU only)."""

import ctypes

import pytest

ARG, SIZE, ALIGN, WORKSPACE = 1, 2, 3, 5
P = [0x10000 * (i + 1) for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_moe_quantize_gb300 import _lib, build
    build.build()
    return _lib.load()


def gate(lib, **kw):
    a = dict(logits=P[0], dtype=0, stride=8, bias=None, ids=P[1], w=P[2], T=4, E=8, k=2, score=0, G=1, TG=1, GT=1,
             renorm=1, scale=1.0)
    a.update(kw)
    return lib.ft_moe_gate(a["logits"], a["dtype"], a["stride"], a["bias"], a["ids"], a["w"], a["T"], a["E"], a["k"],
                           a["score"], a["G"], a["TG"], a["GT"], a["renorm"], a["scale"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(E=0), ARG), (dict(E=5000, stride=5000), ARG), (dict(k=0), ARG), (dict(k=9), ARG),
    (dict(dtype=7), ARG), (dict(score=2), ARG), (dict(G=3), ARG), (dict(G=0), ARG), (dict(G=4, TG=5), ARG),
    (dict(G=4, TG=0), ARG), (dict(GT=3), ARG), (dict(GT=0), ARG), (dict(G=8, TG=8, GT=2), ARG),
    (dict(G=4, TG=1, k=3), ARG), (dict(stride=7), ARG), (dict(T=1 << 31), SIZE), (dict(logits=None), ARG),
    (dict(ids=None), ARG), (dict(w=None), ARG), (dict(logits=P[0] + 2), ALIGN), (dict(w=P[2] + 1), ALIGN),
    (dict(T=0, logits=None), 0),
])
def test_gate_refuses(lib, kw, status):
    assert gate(lib, **kw) == status, lib.ft_last_error()


def test_quantizers_refuse(lib):
    f = lib.ft_quantize_fp8
    assert f(P[0], 0, P[1], P[2], -1, 128, None) == ARG
    assert f(P[0], 0, P[1], P[2], 4, 24, None) == ARG and b"multiple of 16" in lib.ft_last_error()
    assert f(P[0], 0, P[1], P[2], 4, 0, None) == ARG
    assert f(P[0], 3, P[1], P[2], 4, 128, None) == ARG
    assert f(P[0], 0, P[1], P[2], 1 << 58, 128, None) == SIZE
    assert f(None, 0, P[1], P[2], 4, 128, None) == ARG
    assert f(P[0] + 8, 0, P[1], P[2], 4, 128, None) == ALIGN
    assert f(P[0], 0, P[1] + 2, P[2], 4, 128, None) == ALIGN
    assert f(None, 0, None, None, 0, 128, None) == 0
    g = lib.ft_act_mul_quantize_fp8
    assert g(P[0], 0, P[1], P[2], 4, 128, 5, None) == ARG
    assert g(P[0], 0, P[1], P[2], 4, 100, 0, None) == ARG


def product(lib, dense=False, **kw):
    a = dict(w=P[0], ws=P[1], a=P[2], s=P[3], ids=P[4], out=P[5], dt=0, T=4, k=2, E=8, N=128, K=256, work=P[6],
             n=1 << 40)
    a.update(kw)
    if dense:
        return lib.ft_matmul_fp8_fp8(a["w"], a["ws"], a["a"], a["s"], a["out"], a["dt"], a["T"], a["N"], a["K"], None)
    got = {f(a["w"], a["ws"], a["a"], a["s"], a["ids"], a["out"], a["dt"], a["T"], a["k"], a["E"], a["N"], a["K"],
             a["work"], a["n"], None) for f in (lib.ft_moe_fp8_fp8, lib.ft_moe_fp8_fp8_slots)}
    assert len(got) == 1
    return got.pop()


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(N=0), ARG), (dict(K=8), ARG), (dict(K=264), ARG), (dict(K=1 << 20), SIZE),
    (dict(N=1 << 31), SIZE), (dict(dt=1), ARG), (dict(T=1 << 31), SIZE), (dict(w=None), ARG), (dict(ws=None), ARG),
    (dict(a=None), ARG), (dict(s=None), ARG), (dict(out=None), ARG), (dict(w=P[0] + 8), ALIGN),
    (dict(a=P[2] + 8), ALIGN), (dict(s=P[3] + 2), ALIGN), (dict(out=P[5] + 2), ALIGN), (dict(T=0, w=None), 0),
])
def test_products_refuse(lib, dense, kw, status):
    assert product(lib, dense, **kw) == status, lib.ft_last_error()


def test_routed_products_refuse(lib):
    assert product(lib, E=0) == ARG and product(lib, k=9) == ARG and product(lib, ids=None) == ARG
    assert product(lib, E=4096, N=1 << 20) == SIZE and product(lib, ids=P[4] + 2) == ALIGN
    need = lib.ft_moe_fp8_workspace_bytes(4, 2, 8, 256)
    if need:
        assert product(lib, n=need - 1) == WORKSPACE and product(lib, work=None) == WORKSPACE
        assert product(lib, work=P[6] + 16) == ALIGN
    assert lib.ft_moe_fp8_workspace_bytes(4, 9, 8, 256) == 0 and lib.ft_moe_fp8_workspace_bytes(4, 2, 8, 100) == 0


def test_combine_refuses(lib):
    f = lib.ft_moe_combine
    assert f(P[0], 0, P[1], None, P[2], 0, -1, 2, 64, None) == ARG
    assert f(P[0], 0, P[1], None, P[2], 0, 4, 0, 64, None) == ARG
    assert f(P[0], 0, P[1], None, P[2], 0, 4, 2, 0, None) == ARG
    assert f(P[0], 1, P[1], None, P[2], 0, 4, 2, 64, None) == ARG       # fp16 rows
    assert f(P[0], 0, P[1], None, P[2], 9, 4, 2, 64, None) == ARG
    assert f(P[0], 0, P[1], None, P[2], 0, 1 << 30, 2, 64, None) == SIZE
    assert f(P[0], 0, None, None, P[2], 0, 4, 2, 64, None) == ARG
    assert f(P[0] + 2, 0, P[1], None, P[2], 0, 4, 2, 64, None) == ALIGN
    assert f(None, 0, None, None, None, 0, 0, 2, 64, None) == 0


def test_layer_refuses(lib):
    def call(**kw):
        a = dict(x=P[0], xdt=2, logits=P[1], ldt=0, stride=8, bias=None, w13=P[2], s13=P[3], w2=P[4], s2=P[5], y=P[6],
                 ids=P[7], w=P[8], T=4, E=8, k=2, H=256, I=128, score=0, G=1, TG=1, GT=1, renorm=1, scale=1.0, act=0,
                 work=P[9], n=1 << 40)
        a.update(kw)
        return lib.ft_moe_layer_fp8(a["x"], a["xdt"], a["logits"], a["ldt"], a["stride"], a["bias"], a["w13"], a["s13"],
                                    a["w2"], a["s2"], a["y"], a["ids"], a["w"], a["T"], a["E"], a["k"], a["H"], a["I"],
                                    a["score"], a["G"], a["TG"], a["GT"], a["renorm"], a["scale"], a["act"], a["work"],
                                    a["n"], None)
    assert call(xdt=0) == ARG and call(H=100) == ARG and call(I=0) == ARG and call(act=2) == ARG and call(k=0) == ARG
    assert call(H=1 << 20) == SIZE and call(I=1 << 20) == SIZE and call(T=1 << 31) == SIZE
    for name in ("x", "logits", "w13", "s13", "w2", "s2", "y", "ids", "w"):
        assert call(**{name: None}) == ARG, name
    assert call(x=P[0] + 2) == ALIGN and call(w2=P[4] + 4) == ALIGN and call(y=P[6] + 1) == ALIGN
    need = lib.ft_moe_layer_fp8_workspace_bytes(4, 2, 8, 256, 128)
    assert need > 0 and call(n=need - 1) == WORKSPACE and call(work=None) == WORKSPACE
    assert call(work=P[9] + 8) == ALIGN
    assert lib.ft_moe_layer_fp8_workspace_bytes(4, 2, 8, 100, 128) == 0
    assert call(T=0, x=None) == 0
