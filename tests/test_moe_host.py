"""The operators of a whole prompt's experts refuse bad arguments on the host,
before any CUDA call: the addresses below are never dereferenced."""

import ctypes

import pytest
import torch

OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
P = 0x10000  # a 16-byte aligned address
BF16, FP16, FP32 = 0, 1, 2


@pytest.fixture(scope="module")
def M():
    from moe_decode_step_persistent_gb300 import build as B
    import moe_decode_step_persistent_gb300 as mod
    B.build()
    mod.load_library()
    return mod


@pytest.fixture(scope="module")
def lib(M):
    return M.load_library()


@pytest.mark.parametrize("change,status", [
    (dict(tokens=0), OK), (dict(tokens=0, logits=None), OK), (dict(tokens=-1), INVALID), (dict(dt=3), INVALID), (dict(dt=-1), INVALID),
    (dict(E=0), SHAPE), (dict(E=1025, ld=2000), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(k=5, E=4), SHAPE),
    (dict(tokens=1 << 29), SHAPE), (dict(logits=None), INVALID), (dict(experts=None), INVALID), (dict(gates=None), INVALID),
    (dict(ld=63), INVALID), (dict(logits=P + 2), ALIGN), (dict(logits=P + 1, dt=BF16), ALIGN), (dict(bias=P + 2), ALIGN),
    (dict(experts=P + 1), ALIGN), (dict(gates=P + 2), ALIGN)])
def test_route(lib, change, status):
    a = dict(logits=P, dt=FP32, tokens=5, E=64, ld=64, bias=P, k=8, experts=P, gates=P)
    a.update(change)
    assert lib.msk_moe_route(a["logits"], a["dt"], a["tokens"], a["E"], a["ld"], a["bias"], a["k"], a["experts"], a["gates"],
                             None) == status


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), INVALID), (dict(n=(1 << 30) + 1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(experts=None), INVALID),
    (dict(offsets=None), INVALID), (dict(offsets=None, n=0), INVALID), (dict(slots=None), INVALID), (dict(places=None), INVALID),
    (dict(experts=P + 2), ALIGN), (dict(offsets=P + 1), ALIGN), (dict(slots=P + 2), ALIGN), (dict(places=P + 3), ALIGN)])
def test_sort(lib, change, status):
    a = dict(experts=P, n=100, E=64, offsets=P, slots=P, places=P)
    a.update(change)
    assert lib.msk_moe_sort(a["experts"], a["n"], a["E"], a["offsets"], a["slots"], a["places"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=0), OK), (dict(rows=-1), INVALID), (dict(dt=7), INVALID), (dict(cols=0), SHAPE), (dict(cols=24, stride=24), SHAPE),
    (dict(cols=1 << 25, stride=1 << 25), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(rows=1 << 30, cols=1024, stride=1024), SHAPE),
    (dict(ts=0.0), INVALID), (dict(ts=-1.0), INVALID), (dict(ts=float("nan")), INVALID), (dict(ts=float("inf")), INVALID),
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(stride=-64), INVALID),
    (dict(x=P + 8), ALIGN), (dict(stride=66), ALIGN), (dict(stride=68), ALIGN), (dict(codes=P + 8), ALIGN), (dict(scales=P + 4), ALIGN)])
def test_quantize(lib, change, status):
    a = dict(x=P, dt=BF16, rows=5, cols=64, stride=64, ts=1.0, codes=P, scales=P)
    a.update(change)
    assert lib.msk_quantize_fp4(a["x"], a["dt"], a["rows"], a["cols"], a["stride"], a["ts"], a["codes"], a["scales"], None) == status
    assert lib.msk_dequantize_fp4(a["codes"], a["scales"], a["ts"], a["rows"], a["cols"], a["x"], a["dt"], a["stride"], None) == status


def test_rows_that_overlap_are_not_written(lib):
    for stride in (0, 48):
        assert lib.msk_dequantize_fp4(P, P, 1.0, 5, 64, P, BF16, stride, None) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(n=0), OK), (dict(rows=0), OK), (dict(n=-1), INVALID), (dict(ydt=3), INVALID), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(rows=-1), SHAPE), (dict(rows=(1 << 24) + 1, E=1), SHAPE), (dict(rows=1 << 24, E=128), SHAPE), (dict(cols=96), SHAPE),
    (dict(cols=0), SHAPE), (dict(cols=131136), SHAPE), (dict(n=(1 << 30) + 1), SHAPE), (dict(xrows=(1 << 30) + 1), SHAPE),
    (dict(xrows=-1), SHAPE), (dict(xcols=64), INVALID), (dict(up_rows=127), INVALID), (dict(up_cols=64), INVALID), (dict(up_E=3), INVALID),
    (dict(slots=None, xrows=99), INVALID), (dict(k=0), INVALID), (dict(xrows=0), INVALID), (dict(x=None), INVALID), (dict(xs=None), INVALID),
    (dict(offsets=None), INVALID), (dict(w=None), INVALID), (dict(ws=None), INVALID), (dict(up=None), INVALID), (dict(ups=None), INVALID),
    (dict(y=None), INVALID), (dict(ys=127), INVALID), (dict(x=P + 8), ALIGN), (dict(xs=P + 8), ALIGN), (dict(w=P + 8), ALIGN),
    (dict(ws=P + 4), ALIGN), (dict(up=P + 8), ALIGN), (dict(ups=P + 1), ALIGN), (dict(y=P + 1), ALIGN), (dict(slots=P + 2), ALIGN),
    (dict(offsets=P + 2), ALIGN), (dict(ts=P + 2), ALIGN), (dict(up_ts=P + 1), ALIGN)])
def test_experts(M, lib, change, status):
    a = dict(x=P, xs=P, xrows=50, xcols=128, slots=P, k=2, n=100, offsets=P, w=P, ws=P, ts=P, E=4, rows=128, cols=128, up=P, ups=P, up_ts=None,
             y=P, ydt=BF16, ys=1 << 25)
    a.update(change)
    if "cols" in change:
        a["xcols"] = a["cols"]
    x = ctypes.pointer(M.Nvfp4Desc(a["x"], a["xs"], 1.0, a["xrows"], a["xcols"]))
    w = ctypes.pointer(M.Fp4ExpertsC(a["w"], a["ws"], a["ts"], a["E"], a["rows"], a["cols"]))
    up = ctypes.pointer(M.Fp4ExpertsC(a["up"], a["ups"], a["up_ts"], a.get("up_E", a["E"]), a.get("up_rows", a["rows"]),
                                      a.get("up_cols", a["cols"])))
    call = lib.msk_experts_fp4
    assert call(x, a["slots"], a["k"], a["n"], a["offsets"], w, up, a["y"], a["ydt"], a["ys"], None) == status
    assert call(None, P, 2, 100, P, w, None, P, BF16, 128, None) == INVALID
    assert call(x, P, 2, 100, P, None, None, P, BF16, 128, None) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(w=None), INVALID), (dict(ws=None), INVALID), (dict(maps=None), INVALID), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(rows=0), SHAPE), (dict(cols=96), SHAPE), (dict(w=P + 8), ALIGN), (dict(ws=P + 8), ALIGN), (dict(maps=P + 32), ALIGN)])
def test_experts_maps(M, lib, change, status):
    a = dict(w=P, ws=P, E=4, rows=128, cols=128, maps=P)
    a.update(change)
    w = ctypes.pointer(M.Fp4ExpertsC(a["w"], a["ws"], None, a["E"], a["rows"], a["cols"], None))
    assert lib.msk_fp4_experts_maps(w, a["maps"]) == status
    assert lib.msk_fp4_experts_maps(None, P) == INVALID
    # an address of maps that is not aligned is refused before it is read
    x = ctypes.pointer(M.Nvfp4Desc(P, P, 1.0, 50, 128))
    w = ctypes.pointer(M.Fp4ExpertsC(P, P, None, 4, 128, 128, P + 8))
    assert lib.msk_experts_fp4(x, P, 2, 100, P, w, None, P, BF16, 128, None) == ALIGN


@pytest.mark.parametrize("change,status", [
    (dict(tokens=0), OK), (dict(cols=0), OK), (dict(tokens=-1), INVALID), (dict(ydt=3), INVALID), (dict(odt=9), INVALID),
    (dict(rows=-1), INVALID), (dict(k=0), SHAPE), (dict(cols=-1), SHAPE), (dict(tokens=1 << 30), SHAPE),
    (dict(tokens=1 << 20, cols=1 << 19, k=1, ys=1 << 20, os=1 << 20), SHAPE), (dict(y=None), INVALID), (dict(places=None), INVALID),
    (dict(out=None), INVALID), (dict(ys=63), INVALID), (dict(os=63), INVALID), (dict(y=P + 1), ALIGN), (dict(out=P + 1), ALIGN),
    (dict(places=P + 2), ALIGN), (dict(gates=P + 2), ALIGN)])
def test_combine(lib, change, status):
    a = dict(y=P, ydt=BF16, rows=40, ys=64, places=P, gates=P, tokens=5, k=8, cols=64, out=P, odt=BF16, os=64)
    a.update(change)
    assert lib.msk_moe_combine(a["y"], a["ydt"], a["rows"], a["ys"], a["places"], a["gates"], a["tokens"], a["k"], a["cols"],
                               a["out"], a["odt"], a["os"], None) == status


def test_binding_refuses_on_the_host(M):
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    p, s = torch.zeros(2, 8, 64, dtype=u8), torch.zeros(2, 8, 8, dtype=u8)
    for bad in ((p, s), (p.float(), s), (p[0], s[0]), (p, s[:, :7]), (p, s, torch.zeros(3)), (p, s, torch.zeros(2, dtype=torch.float64))):
        with pytest.raises(ValueError):
            M.Fp4Experts(*bad)

    class W:  # (nothing of it is reached)
        n_experts, rows, cols = 2, 8, 128
    class X:
        rows, cols = 5, 128
    class Narrow:
        rows, cols = 5, 96
    class Up:
        n_experts, rows, cols = 2, 9, 128
    off = torch.zeros(3, dtype=i32)
    for kw in (dict(offsets=off[:2]), dict(offsets=off.long()), dict(x=Narrow), dict(up=Up), dict(slots=torch.zeros(4, dtype=torch.int64)),
               dict(slots=torch.zeros(4, dtype=i32), top_k=0), dict(out=torch.zeros(5, 9)), dict(out=torch.zeros(4, 8)),
               dict(out_dtype=i32)):
        args = dict(x=X, experts=W, offsets=off)
        args.update(kw)
        with pytest.raises(ValueError):
            M.msk_experts_fp4(**args)
    for args in ((torch.zeros(4), 1), (torch.zeros(4, 8), 9), (torch.zeros(4, 8), 0), (torch.zeros(4, 40), 33),
                 (torch.zeros(4, 8, dtype=i32), 1), (torch.zeros(8, 4).t(), 1), (torch.zeros(4, 8), 1, torch.zeros(7)),
                 (torch.zeros(4, 8), 1, torch.zeros(8, dtype=torch.float64))):
        with pytest.raises(ValueError):
            M.msk_moe_route(*args)
    for args in ((torch.zeros(4, dtype=torch.int64), 4), (torch.zeros(4, dtype=i32), 0), (torch.zeros(4, dtype=i32), 1025),
                 (torch.zeros(4, 4, dtype=i32).t()[:, 1:], 4)):
        with pytest.raises(ValueError):
            M.msk_moe_sort(*args)
    for x in (torch.zeros(4, 24), torch.zeros(16), torch.zeros(4, 16, dtype=torch.float64), torch.zeros(16, 32).t(), torch.zeros(4, 0)):
        with pytest.raises(ValueError):
            M.msk_quantize_fp4(x)
    y, places = torch.zeros(8, 16), torch.zeros(4, 2, dtype=i32)
    for args, kw in (((y[0], places), {}), ((y, places.long()), {}), ((y, places[0]), {}), ((y, places, torch.zeros(4, 3)), {}),
                     ((y, places), dict(out=torch.zeros(4, 15))), ((y, places), dict(out_dtype=i32)), ((y.t(), places), {})):
        with pytest.raises(ValueError):
            M.msk_moe_combine(*args, **kw)
