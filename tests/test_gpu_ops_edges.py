"""The operators beside the step at the ends of their ranges, against their
definitions in 64 bits with the tolerances of test_gpu_ops.py."""

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import formats as F
from tests.test_gpu_ops import DT, M, check_attention, check_linear, filled_cache, gen, pack, random_fp4, randn  # noqa: F401

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------
# rows with one element far above the rest
# ----------------------------------------------------------------------------


def small_elements(seed, *shape):
    """bf16 numbers of all significands, 2^-31 up to 2^-30."""
    s = torch.randint(128, 256, shape, generator=gen(seed)).float() * 2.0 ** -38
    return s * (1 - 2.0 * torch.randint(0, 2, shape, generator=gen(seed + 1)))


@pytest.mark.parametrize("T,N,K", [(1, 130, 512), (5, 300, 4096), (16, 77, 1024)])
def test_linear_with_one_element_far_above_the_rest(M, T, N, K):
    """Elements down to 2^-31 of their row's greatest enter without rounding: with
    weights of 0 for the greatest only they are left."""
    packed, scales = random_fp4(201, N, K)
    packed[:, 0] &= 0xF0
    x = small_elements(202, T, K)
    x[:, 0] = 255 / 128
    x = x.bfloat16().cuda()
    y = M.msk_linear_fp4(x, M.Fp4Weight(packed.cuda(), scales.cuda()), out_dtype=torch.float32)
    check_linear(y, x, packed, scales, 1.0)


@pytest.mark.parametrize("T,hq,d", [(1, 4, 64), (4, 4, 128), (16, 4, 128)])
def test_attention_with_one_element_far_above_the_rest(M, T, hq, d):
    cache = filled_cache(M, 203, 1, 300, d)
    cache.codes[0, :, :, 0] &= 0xF0
    q = small_elements(204, T, hq, d)
    q[..., 0] = 255 / 128
    q = q.bfloat16().cuda()
    scale = 2.0 ** 30 / math.sqrt(d)
    check_attention(M, M.msk_attention_kv4(q, cache, 280, softmax_scale=scale), q, cache, 280, 0, None, scale)


# ----------------------------------------------------------------------------
# results in range whose parts are not
# ----------------------------------------------------------------------------


@pytest.mark.parametrize("T,N,K", [(2, 48, 1024), (16, 20000, 256), (3, 40, 8192)])
@pytest.mark.parametrize("xt,yt,size,ts", [
    ("bf16", "fp32", 2e36, 4.4e-5), ("bf16", "bf16", 3e37, 1e-38), ("bf16", "fp32", 1e-36, 1e36), ("bf16", "fp32", 1e-38, 3e38),
    ("fp16", "fp32", 6e4, 1e-38), ("fp16", "fp32", 6e-5, 1e35)])
def test_linear_of_far_apart_scales(M, T, N, K, xt, yt, size, ts):
    """Rows and tensor scales at the two ends of their types: the products of one
    alone with the weights (up to 2688) pass fp32's range, the result does not."""
    packed, scales = random_fp4(211, N, K)
    scales[:] = 0x7E - scales % 16  # block scales of 112 to 448
    x = randn(212, T, K).clamp(-3, 3) / 3
    x = (x.double() * size).to(DT[xt]).cuda()
    y = M.msk_linear_fp4(x, M.Fp4Weight(packed.cuda(), scales.cuda(), ts), out_dtype=DT[yt])
    assert torch.isfinite(y).all()
    check_linear(y, x, packed, scales, ts)


@pytest.mark.parametrize("ts", [0.0, -0.75, float("inf"), float("nan")])
def test_linear_of_any_tensor_scale(M, ts):
    packed, scales = random_fp4(213, 40, 256)
    x = randn(214, 2, 256).bfloat16().cuda()
    y = M.msk_linear_fp4(x, M.Fp4Weight(packed.cuda(), scales.cuda(), ts), out_dtype=torch.float32)
    if math.isfinite(ts):
        check_linear(y, x, packed, scales, ts)
    else:
        assert not torch.isfinite(y).any()


# ----------------------------------------------------------------------------
# signs of zeros in the cache
# ----------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("scales", [(1.0, 0.37), (2.5, 1.0), (1e-20, 1e20)])
def test_write_keeps_the_signs_of_zeros(M, dtype, scales):
    """Codes and scales bit for bit the oracle's where elements are -0, among others, among
    elements that round to 0, among saturating ones and alone."""
    x = randn(221, 2, 6, 1, 64)
    x[:, :, :, ::3] = -0.0
    x[:, :, :, 1::7] *= -1e-3
    x[:, 1] = -0.0
    x[:, 2, 0, 17] = 6e4
    x[:, 3, 0, ::2] = 0.0
    if scales[0] < 1e-10 and dtype != "fp16":
        x[0] *= scales[0]
        x[1] *= scales[1]
    x = x.to(DT[dtype])
    cache = M.Kv4Cache.empty(1, 6, 64, *scales)
    M.msk_kv4_write(cache, x[0].cuda(), x[1].cuda(), 0)
    for i in (0, 1):
        y = (x[i].float() / torch.tensor(scales[i], dtype=torch.float32)).transpose(0, 1)
        codes, sc, _ = F.q4(y.double().numpy())
        assert np.array_equal(cache.codes[i].cpu().numpy(), pack(codes).numpy())
        assert np.array_equal(cache.scales[i].cpu().numpy(), sc)
        assert ((codes == 8) & (y.numpy() == 0)).any() or not sc.any()


# ----------------------------------------------------------------------------
# errors of other calls
# ----------------------------------------------------------------------------

AFTER_AN_ERROR = """
import ctypes
import torch
import moe_decode_step_persistent_gb300 as M
c = M.Kv4Cache.empty(2, 32, 64)
x = torch.ones(4, 2, 64, device="cuda").bfloat16()
torch.cuda.synchronize()
side, cuda, graph = torch.cuda.Stream(), ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p()
assert cuda.cuStreamBeginCapture_v2(ctypes.c_void_p(side.cuda_stream), 2) == 0
try:
    M.msk_ops_check(side)  # (it synchronises, which a capture refuses)
    raise SystemExit("not refused")
except M.MskError:
    pass
cuda.cuStreamEndCapture(ctypes.c_void_p(side.cuda_stream), ctypes.byref(graph))
M.msk_kv4_write(c, x, x, 3)
k, v = M.msk_kv4_read(c, 3, 4)
# 1 / 6 = 1.333 * 2^-3 takes the block scale 1.375 * 2^-3, and 1 / 0.171875 = 5.8 the code of 6
assert (k == 6 * 0.171875).all() and (v == 6 * 0.171875).all()
print("written")
"""


def test_rows_do_not_report_the_errors_of_other_calls(M):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", AFTER_AN_ERROR], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "written" in run.stdout, run.stderr[-2000:]


# ----------------------------------------------------------------------------
# first calls from several threads
# ----------------------------------------------------------------------------

FIRST_FROM_THREADS = """
import threading
import torch
import moe_decode_step_persistent_gb300 as M
caches = [M.Kv4Cache.empty(2, 20000, 128) for _ in range(8)]
q = torch.randn(16, 8, 128, device="cuda").bfloat16()
kv = torch.randn(16000, 2, 128, device="cuda").bfloat16()
w = M.Fp4Weight(torch.full((1000, 512), 0x23, dtype=torch.uint8, device="cuda"),
                torch.full((1000, 64), 0x38, dtype=torch.uint8, device="cuda"))
x = torch.randn(16, 1024, device="cuda").bfloat16()
torch.cuda.synchronize()
outs, go = [None] * 8, threading.Barrier(8)

def calls(i):
    s, c = torch.cuda.Stream(), caches[i]
    go.wait()
    M.msk_kv4_write(c, kv, kv, 0, stream=s)
    got = [M.msk_attention_kv4(q[:t], c, n, stream=s) for t in (1, 3, 16) for n in (100, 15000)]
    got += [M.msk_linear_fp4(x[:t], w, stream=s) for t in (1, 16)]
    got += [M.msk_token_logprobs(got[-1], top=3, stream=s)[4]]
    s.synchronize()
    outs[i] = got

threads = [threading.Thread(target=calls, args=(i,)) for i in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
assert all(torch.equal(a, b) for o in outs for a, b in zip(o, outs[0]))
M.msk_ops_check()
print("the same")
"""


def test_first_calls_from_several_threads(M):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_FROM_THREADS], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "the same" in run.stdout, run.stderr[-2000:]
