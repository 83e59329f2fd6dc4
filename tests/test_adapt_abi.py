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
    assert balance(lib, **kw) == status, lib.ft_last_error()


def test_balance_workspace(lib):
    f = lib.ft_moe_balance_workspace_bytes
    assert f(-1, 8, 1) == 0 and f(4, 0, 1) == 0 and f(4, 5000, 1) == 0 and f(4, 8, 0) == 0
    for E in (1, 8, 100, 128, 300, 4096):
        for S in (1, 9, 1000):
            sizes = [f(T, E, S) for T in (0, 1, 7, 64, 65, 1000, 1001, 40000, 10 ** 7)]
            assert sizes == sorted(sizes) and sizes[0] > 0


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
