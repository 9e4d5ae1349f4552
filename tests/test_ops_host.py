"""The operators beside the step refuse bad arguments on the host, before any
CUDA call: the addresses below are never dereferenced."""

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


def cache(M, codes=P, scales=P, heads=8, d=128, max_seq=1024, ks=1.0, vs=1.0):
    return ctypes.pointer(M.Kv4Desc(codes, scales, heads, d, max_seq, ks, vs))


BAD_CACHES = [(dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(d=96), SHAPE), (dict(heads=0), SHAPE),
              (dict(max_seq=0), SHAPE), (dict(ks=0.0), INVALID), (dict(vs=-1.0), INVALID),
              (dict(ks=float("nan")), INVALID), (dict(vs=float("inf")), INVALID), (dict(codes=P + 8), ALIGN),
              (dict(scales=P + 4), ALIGN), (dict(max_seq=(1 << 30) + 1), SHAPE)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_cache(M, lib, bad, status):
    c = cache(M, **bad)
    assert lib.msk_kv4_write(c, P, P, BF16, 4, 1024, 128, 0, None, None) == status
    assert lib.msk_kv4_read(c, 0, 4, P, P, BF16, 1024, 128, None) == status
    assert lib.msk_attention_kv4(P, BF16, 4096, c, 4, 32, 100, None, None, 0, 0.0, P, P, 1 << 30, None) == status


@pytest.mark.parametrize("args,status", [
    ((P, P, BF16, 0, 1024, 128, 0), OK), ((None, P, BF16, 4, 1024, 128, 0), INVALID),
    ((P, None, BF16, 4, 1024, 128, 0), INVALID), ((P, P, 3, 4, 1024, 128, 0), INVALID),
    ((P, P, BF16, -1, 1024, 128, 0), INVALID), ((P, P, BF16, 4, -1024, 128, 0), INVALID),
    ((P, P, BF16, 4, 1024, 128, -1), INVALID), ((P, P, BF16, 4, 1024, 128, 1021), INVALID),
    ((P, P, BF16, 1025, 1024, 128, 0), INVALID), ((P + 2, P, BF16, 4, 1024, 128, 0), ALIGN),
    ((P, P, BF16, 4, 1028, 128, 0), ALIGN), ((P, P, FP32, 4, 1024, 130, 0), ALIGN)])
def test_rows(M, lib, args, status):
    k, v, dt, tokens, ts, hs, pos = args
    assert lib.msk_kv4_write(cache(M), k, v, dt, tokens, ts, hs, pos, None, None) == status
    assert lib.msk_kv4_read(cache(M), pos, tokens, k, v, dt, ts, hs, None) == status


def test_rows_that_overlap_are_not_written(M, lib):
    for strides in ((0, 128), (1024, 0)):
        assert lib.msk_kv4_read(cache(M), 0, 4, P, P, BF16, *strides, None) == INVALID


def test_no_cache(lib):
    assert lib.msk_kv4_write(None, P, P, BF16, 4, 1024, 128, 0, None, None) == INVALID
    assert lib.msk_kv4_read(None, 0, 4, P, P, BF16, 1024, 128, None) == INVALID
    assert lib.msk_attention_kv4(P, BF16, 4096, None, 4, 32, 0, None, None, 0, 0.0, P, P, 1 << 30, None) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(dt=FP32), INVALID), (dict(tokens=0), SHAPE),
    (dict(tokens=17), SHAPE), (dict(hq=0), SHAPE), (dict(hq=30), SHAPE), (dict(window=-1), INVALID),
    (dict(length=-1), INVALID), (dict(length=1021), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(qs=4088), INVALID), (dict(q=P + 8), ALIGN), (dict(out=P + 2), ALIGN),
    (dict(ws=P + 8), ALIGN), (dict(qs=4100), ALIGN), (dict(parents=[-1, 1, 0, 0]), INVALID),
    (dict(parents=[-2, 0, 0, 0]), INVALID), (dict(ws=None, rows=100000, length=90000), INVALID),
    (dict(nbytes=16, rows=100000, length=90000), INVALID)])
def test_attention(M, lib, change, status):
    a = dict(q=P, dt=BF16, qs=4096, tokens=4, hq=32, length=100, parents=None, window=0, scale=0.0, out=P, ws=P,
             nbytes=1 << 40, rows=1024)
    a.update(change)
    par = None if a["parents"] is None else (ctypes.c_int32 * 4)(*a["parents"])
    assert lib.msk_attention_kv4(a["q"], a["dt"], a["qs"], cache(M, max_seq=a["rows"]), a["tokens"], a["hq"], a["length"], None, par,
                                 a["window"], a["scale"], a["out"], a["ws"], a["nbytes"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(tokens=0), OK), (dict(rows=0), OK), (dict(tokens=17), SHAPE), (dict(tokens=-1), SHAPE),
    (dict(cols=192), SHAPE), (dict(cols=0), SHAPE), (dict(cols=32896), SHAPE), (dict(rows=-1), SHAPE),
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(packed=None), INVALID), (dict(scales=None), INVALID),
    (dict(xdt=FP32), INVALID), (dict(ydt=7), INVALID), (dict(xs=248), INVALID), (dict(ys=99), INVALID),
    (dict(x=P + 8), ALIGN), (dict(xs=260), ALIGN), (dict(packed=P + 8), ALIGN), (dict(scales=P + 1), ALIGN),
    (dict(y=P + 1), ALIGN)])
def test_linear(M, lib, change, status):
    a = dict(x=P, xdt=BF16, xs=256, packed=P, scales=P, rows=100, cols=256, tokens=4, y=P, ydt=BF16, ys=100)
    a.update(change)
    w = ctypes.pointer(M.Nvfp4Desc(a["packed"], a["scales"], 1.0, a["rows"], a["cols"]))
    assert lib.msk_linear_fp4(a["x"], a["xdt"], a["xs"], w, a["tokens"], a["y"], a["ydt"], a["ys"], None) == status
    assert lib.msk_linear_fp4(P, BF16, 256, None, 4, P, BF16, 100, None) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(rows=0), OK), (dict(logits=None), INVALID), (dict(dt=5), INVALID), (dict(rows=-1), INVALID),
    (dict(t=0.0), INVALID), (dict(t=-1.0), INVALID), (dict(t=float("nan")), INVALID), (dict(t=float("inf")), INVALID),
    (dict(vocab=0), SHAPE), (dict(vocab=1 << 31), SHAPE), (dict(top=33), SHAPE), (dict(top=-1), SHAPE),
    (dict(vocab=4, top=5), INVALID), (dict(ld=999), INVALID), (dict(tokens=None), INVALID),
    (dict(logits=P + 2), ALIGN), (dict(tokens=P + 2), ALIGN), (dict(lp=P + 1), ALIGN)])
def test_logprobs(lib, change, status):
    a = dict(logits=P, dt=FP32, rows=3, vocab=1000, ld=1000, tokens=P, t=1.0, top=2, lp=P)
    a.update(change)
    assert lib.msk_token_logprobs(a["logits"], a["dt"], a["rows"], a["vocab"], a["ld"], a["tokens"], a["t"], a["top"],
                                  a["lp"], P, P, P, P, None) == status


def test_workspace_sizes(lib):
    size = lib.msk_attention_kv4_workspace
    assert size(16, 32, 8, 128, 0, 100000) > 0
    assert size(16, 32, 8, 128, 2048, 100000) == 0 and size(16, 32, 8, 128, 0, 100) == 0
    most = 2 ** 31 - 1  # (no overflow; a shorter cache or window never needs more)
    assert size(16, 32, 8, 128, 0, most) >= size(16, 32, 8, 128, 0, 10 ** 6) >= size(16, 32, 8, 128, 0, 10 ** 5)
    assert size(16, 32, 8, 128, most, most) == size(16, 32, 8, 128, 0, most)
    for bad in ((0, 32, 8, 128, 0, 10), (17, 32, 8, 128, 0, 10), (16, 30, 8, 128, 0, 10), (16, 32, 0, 128, 0, 10),
                (16, 32, 8, 128, -1, 10), (16, 32, 8, 128, 0, -1)):
        assert size(*bad) == 0


def test_binding_refuses_on_the_host(M):
    cpu = torch.zeros(2, 2, 8, 64, dtype=torch.uint8)
    sc = torch.zeros(2, 2, 8, 8, dtype=torch.uint8)
    with pytest.raises(ValueError):
        M.Kv4Cache(cpu, sc)  # not on a GPU
    with pytest.raises(ValueError):
        M.Kv4Cache(cpu.float(), sc)
    with pytest.raises(ValueError):
        M.Kv4Cache(cpu, sc[:, :1])
    with pytest.raises(ValueError):
        M.Fp4Weight(cpu[0, 0], sc[0, 0])
    with pytest.raises(ValueError):
        M.Fp4Weight(cpu[0, 0], sc[0, 0, :, :3])


@pytest.mark.parametrize("k_scale,scale,status", [(1e20, 1e20, INVALID), (3e38, 2.0, INVALID), (3e38, 0.0, None), (1e-30, 1e30, None)])
def test_attention_scales_that_leave_the_range_together(M, lib, k_scale, scale, status):
    got = lib.msk_attention_kv4(P, BF16, 4096, cache(M, ks=k_scale), 0 if status is None else 4, 32, 100, None, None, 0, scale, P, P,
                                1 << 30, None)
    assert got == (SHAPE if status is None else status)  # (no tokens: refused for that alone)


def test_binding_refuses_numbers_that_do_not_fit(M):
    """2^32 is not row 0, and a window of 2^32 not a global one: refused, and not cut to 32 bits."""
    class Cache:  # (nothing of it is reached)
        n_kv_heads, head_dim, max_seq = 2, 64, 16
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    q, out = k.new_zeros(3, 4, 64), k.new_zeros(3, 256)
    for big in (1 << 32, (1 << 32) + 5, 1 << 31, -(1 << 31) - 1, -(1 << 32)):
        with pytest.raises(ValueError, match="32 bits"):
            M.msk_kv4_write(Cache, k, k, big)
        with pytest.raises(ValueError, match="32 bits"):
            M.msk_attention_kv4(q, Cache, big, out=out)
        with pytest.raises(ValueError, match="32 bits"):
            M.msk_attention_kv4(q, Cache, 5, window=big, out=out)
        with pytest.raises(ValueError, match="32 bits"):
            M.msk_attention_kv4_workspace(3, 4, 2, 64, 0, big)
        with pytest.raises(ValueError, match="32 bits"):
            M._positions([-1, 0, big])
