"""The entry points that adapt a layer reject bad arguments on the host, before any CUDA call (CPU only)."""

import pytest

ARG, SIZE, ALIGN, WORKSPACE = 1, 2, 3, 5
P = [0x10000 * (i + 1) for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_moe_quantize_gb300 import _lib, build
    build.build()
    return _lib.load()


def balance(lib, **kw):
    a = dict(x=P[0], dt=0, stride=8, ids=P[1], off=None, loss=P[2], counts=P[3], scale=P[4], T=4, E=8, k=2, score=0, S=1,
             work=P[5], n=1 << 30)
    a.update(kw)
    return lib.ft_moe_balance_loss(a["x"], a["dt"], a["stride"], a["ids"], a["off"], a["loss"], a["counts"], a["scale"], a["T"],
                                   a["E"], a["k"], a["score"], a["S"], a["work"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(E=0), ARG), (dict(E=5000, stride=5000), ARG), (dict(k=0), ARG), (dict(k=9), ARG), (dict(dt=3), ARG),
    (dict(score=2), ARG), (dict(stride=7), ARG), (dict(S=0), ARG), (dict(S=2), ARG), (dict(S=0, off=P[6]), ARG),
    (dict(T=1 << 31), SIZE), (dict(x=None), ARG), (dict(ids=None), ARG), (dict(loss=None), ARG), (dict(counts=None), ARG),
    (dict(scale=None), ARG), (dict(x=P[0] + 2), ALIGN), (dict(ids=P[1] + 1), ALIGN), (dict(off=P[6] + 2), ALIGN),
    (dict(work=None), WORKSPACE), (dict(n=64), WORKSPACE), (dict(work=P[5] + 16), ALIGN),
])
def test_balance_refuses(lib, kw, status):
    if status in (WORKSPACE,) or "work" in kw:      # more sequences than a call without a workspace takes
        kw = dict(kw, S=9, off=P[6])
    assert balance(lib, **kw) == status, lib.ft_last_error()


def test_balance_workspace(lib):
    f = lib.ft_moe_balance_workspace_bytes
    assert f(-1, 8, 1) == 0 and f(4, 0, 1) == 0 and f(4, 5000, 1) == 0 and f(4, 8, 0) == 0
    for E in (1, 8, 100, 128, 300, 4096):
        for S in (1, 9, 1000):
            sizes = [f(T, E, S) for T in (0, 1, 7, 64, 65, 1000, 1001, 40000, 10 ** 7)]
            assert sizes == sorted(sizes) and sizes[-1] > 0 and (sizes[0] == 0) == (S <= 8)


def gate(lib, **kw):
    a = dict(x=P[0], dt=0, stride=8, ids=P[1], gw=P[2], counts=P[3], scale=P[4], gl=P[5], off=None, out=P[6], T=4, E=8, k=2,
             score=0, S=1)
    a.update(kw)
    return lib.ft_moe_gate_backward(a["x"], a["dt"], a["stride"], a["ids"], a["gw"], a["counts"], a["scale"], a["gl"], a["off"],
                                    a["out"], a["T"], a["E"], a["k"], a["score"], 1, 1.0, a["S"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(E=0), ARG), (dict(k=0), ARG), (dict(k=9), ARG), (dict(dt=3), ARG), (dict(score=2), ARG),
    (dict(stride=7), ARG), (dict(S=2), ARG), (dict(T=1 << 31), SIZE), (dict(x=None), ARG), (dict(ids=None), ARG),
    (dict(out=None), ARG), (dict(counts=None), ARG), (dict(scale=None), ARG), (dict(gl=None), ARG),
    (dict(gw=None, counts=None, scale=None, gl=None), ARG), (dict(x=P[0] + 2), ALIGN), (dict(out=P[6] + 1), ALIGN),
    (dict(gw=P[2] + 2), ALIGN), (dict(T=0, x=None), 0),
])
def test_gate_backward_refuses(lib, kw, status):
    assert gate(lib, **kw) == status, lib.ft_last_error()


def test_combine_backward_refuses(lib):
    f = lib.ft_moe_combine_backward
    assert f(P[0], 0, P[1], 0, P[2], P[3], P[4], -1, 2, 64, None) == ARG
    assert f(P[0], 0, P[1], 0, P[2], P[3], P[4], 4, 0, 64, None) == ARG
    assert f(P[0], 0, P[1], 0, P[2], P[3], P[4], 4, 2, 0, None) == ARG
    assert f(P[0], 5, P[1], 0, P[2], P[3], P[4], 4, 2, 64, None) == ARG
    assert f(P[0], 0, P[1], 1, P[2], P[3], P[4], 4, 2, 64, None) == ARG       # fp16 rows
    assert f(P[0], 0, P[1], 0, P[2], None, None, 4, 2, 64, None) == ARG
    assert f(None, 0, P[1], 0, P[2], P[3], P[4], 4, 2, 64, None) == ARG
    assert f(P[0], 0, P[1], 0, P[2], P[3], P[4], 1 << 30, 2, 64, None) == SIZE
    assert f(P[0], 0, P[1] + 2, 0, P[2], P[3], P[4], 4, 2, 64, None) == ALIGN
    assert f(None, 0, None, 0, None, P[3], P[4], 0, 2, 64, None) == 0


def lora(lib, **kw):
    a = dict(x=P[0], dt=2, a=P[1], b=P[2], scales=P[3], ids=P[4], add=P[5], out=P[6], odt=0, T=4, k=2, ps=0, L=3, R=16, K=64,
             N=128, work=P[7], n=1 << 40)
    a.update(kw)
    return lib.ft_lora_add(a["x"], a["dt"], a["a"], a["b"], a["scales"], a["ids"], a["add"], a["out"], a["odt"], a["T"], a["k"],
                           a["ps"], a["L"], a["R"], a["K"], a["N"], a["work"], a["n"], None)


def lora_back(lib, **kw):
    a = dict(g=P[8], x=P[0], dt=2, a=P[1], b=P[2], scales=P[3], ids=P[4], add=P[5], gx=P[6], ga=P[9], gb=P[10], T=4, k=2, ps=0,
             L=3, R=16, K=64, N=128, work=P[7], n=1 << 40)
    a.update(kw)
    return lib.ft_lora_backward(a["g"], a["x"], a["dt"], a["a"], a["b"], a["scales"], a["ids"], a["add"], a["gx"], a["ga"],
                                a["gb"], a["T"], a["k"], a["ps"], a["L"], a["R"], a["K"], a["N"], a["work"], a["n"], None)


@pytest.mark.parametrize("f", [lora, lora_back])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(k=0), ARG), (dict(L=0), ARG), (dict(L=5000), ARG), (dict(R=0), ARG), (dict(R=12), ARG),
    (dict(R=136), ARG), (dict(K=0), ARG), (dict(K=60), ARG), (dict(N=60), ARG), (dict(N=0), ARG), (dict(dt=0), ARG),
    (dict(K=1 << 17), SIZE), (dict(N=1 << 17), SIZE), (dict(T=1 << 31), SIZE), (dict(T=1 << 30, k=2), SIZE),
    (dict(x=None), ARG), (dict(a=None), ARG), (dict(b=None), ARG), (dict(ids=None), ARG), (dict(x=P[0] + 8), ALIGN),
    (dict(a=P[1] + 8), ALIGN), (dict(b=P[2] + 2), ALIGN), (dict(add=P[5] + 8), ALIGN), (dict(scales=P[3] + 2), ALIGN),
    (dict(ids=P[4] + 2), ALIGN), (dict(work=None), WORKSPACE), (dict(n=16), WORKSPACE), (dict(work=P[7] + 16), ALIGN),
])
def test_lora_refuses(lib, f, kw, status):
    if "work" in kw or "n" in kw:
        kw = dict(kw, T=200)      # more slots than a call without a workspace takes
    assert f(lib, **kw) == status, lib.ft_last_error()


def test_lora_outputs_refused(lib):
    assert lora(lib, out=None) == ARG and lora(lib, odt=1) == ARG and lora(lib, out=P[6] + 8) == ALIGN
    assert lora(lib, T=0, x=None) == 0
    assert lora_back(lib, g=None) == ARG and lora_back(lib, gx=None, ga=None, gb=None) == ARG
    assert lora_back(lib, ga=P[9] + 4) == ALIGN and lora_back(lib, g=P[8] + 8) == ALIGN
    assert lora_back(lib, T=0, gx=None, ga=None, gb=None) == 0


def test_lora_workspace(lib):
    f = lib.ft_lora_workspace_bytes
    assert f(-1, 1, 1, 16, 64, 64, 0) == 0 and f(4, 1, 1, 12, 64, 64, 0) == 0 and f(4, 1, 1, 16, 64, 60, 1) == 0
    tokens = sorted({int(1.13 ** i) for i in range(120)} | {255, 256, 257, 1023, 1024, 1025, 32767, 32768, 32769, 262144, 262145})
    for k in (1, 3, 8):
        for L in (1, 7, 64, 1100):
            for R in (8, 64, 128):
                for back in (0, 1):
                    sizes = [f(T, k, L, R, 512, 1024, back) for T in tokens]
                    assert sizes == sorted(sizes) and sizes[-1] > 0 and (sizes[0] > 0) == bool(back)
