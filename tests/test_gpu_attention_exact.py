"""Attention over the 4-bit cache where single keys and the weights' last bits
show: caches whose values are set one by one, against the definition in 64 bits.

Tolerance, from the arithmetic (h: half a rounding step of the output's type).
  A score of m nonzero terms is an fp32 sum of exact products, off by at most
    (m + 8) 2^-23 of its terms' magnitudes (sums that truncate, the scale's and the
    maximum's roundings with it).
  A weight: 2^-22 for the exponential, 2^-22 for its two fp16 parts, 2^-20 for the
    rounding of its exponent (up to 16): 2^-18 in all; below the parts' range
    2^-32 of the greatest weight with the same reference.
  Sums of n keys, 16 an addition and up to 32 more where parts are joined, numerator
    and denominator: 2 (n / 16 + 32) 2^-23.
  out: h |o| + (2 score + 2^-18 + 2 (n / 16 + 32) 2^-23) sum p |v| + 2^-32 floor,
    floor: sum |v| over the keys, over the sum of weights relative to the greatest."""

import math

import pytest
import torch

from tests.test_gpu_ops import DT, M, filled_cache, gen, half_step, randn, tree_parents, values64, visible  # noqa: F401

pytestmark = pytest.mark.gpu

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def coded(M, k, v, k_scale=1.0, v_scale=1.0):
    """A cache of these E2M1 values ([heads][rows][d]), all block scales 1."""
    x = torch.stack((k, v))
    code = torch.searchsorted(E2M1, x.abs().contiguous())
    assert torch.equal(E2M1[code], x.abs())
    code = (code + 8 * (x < 0)).to(torch.uint8)
    c = M.Kv4Cache.empty(x.shape[1], x.shape[2], x.shape[3], k_scale, v_scale)
    c.codes.copy_(code[..., 0::2] | (code[..., 1::2] << 4))
    c.scales.fill_(0x38)
    return c


def check(out, q, k, v, length, window=0, parents=None, terms=None, k_scale=1.0, v_scale=1.0, least=1.0):
    """out against the definition; k, v: values of at least length + T rows
    without the tensors' scales; least: the least sum of weights relative to the greatest."""
    T, hq, d = q.shape
    n = length + T
    k, v = (x[:, :n].cuda().double() * torch.tensor(s, dtype=torch.float32).double().item()
            for x, s in ((k, k_scale), (v, v_scale)))
    hkv, scale = k.shape[0], 1 / math.sqrt(d)
    qq = q.cuda().double().view(T, hkv, hq // hkv, d)
    see = visible(T, length, window, parents).cuda()[:, None, None, :]
    s = (torch.einsum("thgd,hnd->thgn", qq, k) * scale).masked_fill(~see, float("-inf"))
    p = torch.softmax(s, -1)
    o, mag = torch.einsum("thgn,hnd->thgd", p, v), torch.einsum("thgn,hnd->thgd", p, v.abs())
    size = (torch.einsum("thgd,hnd->thgn", qq.abs(), k.abs()) * scale).masked_fill(~see, 0).amax(-1)
    ds = ((d if terms is None else terms) + 8) * 2.0 ** -23 * size.unsqueeze(-1)
    floor = torch.einsum("thgn,hnd->thgd", see.double().expand(T, hkv, hq // hkv, n), v.abs()) / least
    h = half_step(q.dtype)
    tol = h * o.abs() + (2 * ds + 2.0 ** -18 + (n / 16 + 32) * 2.0 ** -22) * mag + 2.0 ** -32 * floor + 1e-30
    if q.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = (out.double().view_as(o) - o).abs()
    worst = (err / tol).max().item()
    assert worst <= 1.0, f"error up to {worst:.2f} of the tolerance (max error {err.max().item():.3e})"


@pytest.mark.parametrize("T,hq,hkv,d,pairs,dtype", [
    (1, 4, 1, 64, 3, "fp16"), (1, 8, 2, 128, 6, "bf16"), (2, 8, 2, 128, 90, "fp16"), (4, 8, 2, 128, 6, "fp16"),
    (4, 8, 2, 64, 40, "bf16"), (8, 8, 2, 128, 5, "fp16"), (16, 8, 2, 128, 6, "bf16"), (16, 8, 2, 64, 100, "fp16")])
def test_weights_keep_their_bits(M, T, hq, hkv, d, pairs, dtype):
    """Pairs of keys whose weights are 3 to 2 and whose values are 2 to -3, so
    that what is left of the sum is the weights' rounding."""
    n = 2 * pairs + T
    k, v = torch.zeros(hkv, n, d), torch.zeros(hkv, n, d)
    first, second = slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)
    k[:, first, 0] = 1.0
    k[:, first, 1] = k[:, second, 1] = E2M1[torch.randint(0, 6, (hkv, pairs), generator=gen(1))]
    a = torch.randint(0, 2, (hkv, pairs, d), generator=gen(2)).float() + 1
    a = a * (1 - 2.0 * torch.randint(0, 2, a.shape, generator=gen(3)))
    v[:, first], v[:, second] = 2 * a, -3 * a
    q = torch.zeros(T, hq, d)
    q[..., 0] = math.log(1.5) * math.sqrt(d)
    q[..., 1] = (torch.rand(T, hq, generator=gen(4)) * 2 - 1) * math.sqrt(d)
    q = q.to(DT[dtype]).cuda()
    out = M.msk_attention_kv4(q, coded(M, k, v), n - T)
    check(out, q, k, v, n - T, terms=2)


@pytest.mark.parametrize("T,hq,hkv,d,n,dtype", [
    (1, 4, 1, 64, 2000, "fp16"), (1, 8, 2, 128, 40000, "bf16"), (4, 8, 2, 128, 4000, "fp16"), (8, 8, 2, 128, 2000, "bf16"),
    (16, 8, 2, 128, 2000, "fp16"), (16, 8, 2, 64, 30000, "bf16")])
def test_keys_far_below_the_greatest_count(M, T, hq, hkv, d, n, dtype):
    """One key of 16 is 17 nats above the rest and has no values: all that
    comes out is the rest's."""
    k, v = torch.zeros(hkv, n, d), torch.zeros(hkv, n, d)
    v[:] = E2M1[torch.arange(d) % 7 + 1]
    k[:, 5::16, 0], v[:, 5::16] = 6.0, 0.0
    q = torch.zeros(T, hq, d)
    q[..., 0] = 24.42 * math.log(2) * math.sqrt(d) / 6
    q = q.to(DT[dtype]).cuda()
    out = M.msk_attention_kv4(q, coded(M, k, v, v_scale=1e6), n - T)
    check(out, q, k, v, n - T, terms=1, v_scale=1e6, least=(n - T) // 16)
