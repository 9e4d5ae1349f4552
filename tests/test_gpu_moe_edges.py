"""The operators of a whole prompt's experts where test_gpu_moe.py does not go:
signals that stay away, kernels for many elements, sizes and scales at the ends
of their ranges.  Tolerances are those of test_gpu_moe.py."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from tests.test_gpu_moe import (DT, M, gen, half_step, make_experts, no_wait_ran_out, products_ref, randn,  # noqa: F401
                                random_fp4, run_products, sort_ref_many, strided, tiny, values64)

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------
# signals that stay away
# ----------------------------------------------------------------------------


def products_of(M, counts, rows, cols, glu, gather, top_k=2):
    """A call without arguments, of fixed inputs."""
    n = sum(counts)
    w, _ = make_experts(M, 31, len(counts), rows, cols)
    up = make_experts(M, 32, len(counts), rows, cols)[0] if glu else None
    xr = (n + top_k - 1) // top_k if gather else n
    c, s = random_fp4(33, xr, cols)
    x = M.Fp4Weight(c.cuda(), s.cuda())
    slots = torch.randperm(xr * top_k, generator=gen(34))[:n].int().cuda() if gather else None
    off = torch.tensor([0] + counts).cumsum(0).int().cuda()
    return lambda: M.msk_experts_fp4(x, w, off, up=up, slots=slots, top_k=top_k)


@pytest.mark.parametrize("counts,rows,cols", [([40], 256, 256), ([5], 40, 64), ([100, 30], 300, 1344), ([256] * 40, 1030, 320)])
@pytest.mark.parametrize("glu,gather", [(False, False), (True, False), (False, True), (True, True)])
def test_a_signal_that_stays_away_is_reported(M, counts, rows, cols, glu, gather):
    """Nobody says that a pair's first tile is complete: the warps that end tiles wait for it
    in vain, long after the copies' warps have ended where the pair has no other tile.  The
    check reports it, once, and the next call is sound."""
    call = products_of(M, counts, rows, cols, glu, gather)
    want = call()
    M.msk_ops_check()
    try:
        M.msk_debug_experts_fault(0, 2_000_000)
        call()
    finally:
        M.msk_debug_experts_fault()
    with pytest.raises(M.MskError) as e:
        M.msk_ops_check()
    assert e.value.status == M.MSK_ERR_TIMEOUT
    M.msk_ops_check()
    assert torch.equal(call(), want)
    # a tile that no pair has: nothing is missed within the short limit
    try:
        M.msk_debug_experts_fault(1 << 20, 50_000_000)
        assert torch.equal(call(), want)
    finally:
        M.msk_debug_experts_fault()
    M.msk_ops_check()


# ----------------------------------------------------------------------------
# warps of which some lanes store nothing
# ----------------------------------------------------------------------------


@pytest.mark.parametrize("rows", [1, 17, 31, 33, 63, 250, 257, 290])
@pytest.mark.parametrize("counts", [[256], [250, 3, 128], [255] * 12])
@pytest.mark.parametrize("glu,gather", [(False, False), (True, True)])
def test_products_whose_last_rows_are_part_of_a_warp(M, rows, counts, glu, gather):
    """Lanes behind the last weight row go through all of a tile's chunks of 32 tokens beside those that store."""
    run_products(M, counts, rows, 192, glu, gather, out="fp32", extra=1)


@pytest.mark.parametrize("E", [1, 31, 33, 1023])
@pytest.mark.parametrize("n", [4095, 4097, 32769, 49153, 65537])
def test_sort_of_experts_that_end_inside_a_warp(M, E, n):
    """Of the block's threads as many as there are experts read the cluster's counts between its meetings."""
    e = torch.randint(-1, E + 1, (n,), generator=gen(n + E), dtype=torch.int32)
    for got, want in zip(M.msk_moe_sort(e.cuda(), E), sort_ref_many(e, E)):
        assert np.array_equal(got.cpu().numpy(), want)


# ----------------------------------------------------------------------------
# tensors' scales at the ends of their range
# ----------------------------------------------------------------------------


@pytest.mark.parametrize("x_ts,w_ts", [(1e-40, 0.02), (0.02, 1e-40), (3e-45, 5e4), (1e-39, 1e-3), (-1e-41, 0.7), (1e-42, -2e-2)])
def test_products_of_subnormal_tensor_scales(M, x_ts, w_ts):
    """The product of the two scales is far below fp32's normal numbers and loses their digits, results are not:
    block scales of 112 to 448 bring the sums to 1e5."""
    counts, rows, cols = [5, 40], 70, 64
    p, s = random_fp4(51, 2, rows, cols)
    s = 0x7E - s % 16
    t = torch.tensor([w_ts, w_ts * 0.7])
    w = M.Fp4Experts(p.cuda(), s.cuda(), t.cuda())
    wv = values64(p, s) * t.double().view(2, 1, 1)
    c, xs = random_fp4(53, 45, cols)
    xs = 0x7E - xs % 16
    x = M.Fp4Weight(c.cuda(), xs.cuda(), x_ts)
    off = torch.tensor([0, 5, 45], dtype=torch.int32, device="cuda")
    y = M.msk_experts_fp4(x, w, off, out_dtype=torch.float32)
    ref, err = products_ref(values64(c, xs, x_ts), wv, None, counts, torch.arange(45))
    assert ref.abs().max() > 2.0 ** -126
    assert ((y.cpu().double() - ref).abs() <= 2.0 ** -24 * ref.abs() + err + 2.0 ** -149).all()


# ----------------------------------------------------------------------------
# slots and top_k
# ----------------------------------------------------------------------------


def test_slots_without_top_k(M):
    """One expert a token: slots are tokens, with and without saying so; more slots than rows need it said."""
    w, _ = make_experts(M, 61, 2, 40, 128)
    c, s = random_fp4(62, 6, 128)
    x, off = M.Fp4Weight(c.cuda(), s.cuda()), torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 5, 0, 1, 2, 4], dtype=torch.int32, device="cuda")
    assert torch.equal(M.msk_experts_fp4(x, w, off, slots=slots), M.msk_experts_fp4(x, w, off, slots=slots, top_k=1))
    many = torch.tensor([4, 4, 0, 1, 4, 2, 5, 5], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="top_k"):
        M.msk_experts_fp4(x, w, off, slots=many)
    y = M.msk_experts_fp4(x, w, off, slots=many, top_k=1)
    assert torch.equal(y[:6], M.msk_experts_fp4(x, w, off, slots=many[:6].contiguous()))


# ----------------------------------------------------------------------------
# kernels for many elements
# ----------------------------------------------------------------------------


@pytest.mark.parametrize("ydt", list(DT))
@pytest.mark.parametrize("odt", list(DT))
@pytest.mark.parametrize("tokens,k,cols,extra,offset", [
    (2048, 3, 2048, 0, 0), (2047, 3, 2048, 0, 0),      # 2^22 outputs, and fewer: pieces of 32 bytes and of 16
    (2050, 9, 2064, 16, 0), (2050, 9, 2064, 32, 16),   # padded rows, more ranks than are loaded at once
    (2100, 2, 2048, 0, 8), (2100, 2, 2040, 4, 0),      # aligned to 16 bytes and not to 32: a y of 16-bit elements, rows of fp32
    (20000, 5, 240, 0, 4)])                            # a y of 16-bit elements aligned to 8
def test_combine_of_many_outputs(M, ydt, odt, tokens, k, cols, extra, offset):
    g, n = torch.Generator("cuda").manual_seed(tokens + cols), tokens * k
    wide = torch.full((n * (cols + extra) + offset + 64,), 7.0, dtype=DT[ydt], device="cuda")
    y = wide[offset:offset + n * (cols + extra)].view(n, cols + extra)[:, :cols]
    y.copy_(torch.randn(n, cols, generator=g, device="cuda"))
    places = torch.randperm(n, generator=g, device="cuda").int().view(tokens, k)
    drop = torch.rand(tokens, k, generator=g, device="cuda") < 0.1
    y[places[drop].long()] = float("nan")              # (not read)
    places[drop] = torch.tensor([-1, n, 2 ** 31 - 1, -2 ** 31], device="cuda")[torch.arange(int(drop.sum()), device="cuda") % 4].int()
    places[5] = -1
    gates = torch.rand(tokens, k, generator=g, device="cuda")
    out = torch.full((tokens, cols + extra), 5.0, dtype=DT[odt], device="cuda")
    M.msk_moe_combine(y, places, gates, out=out[:, :cols])
    ref, mag = torch.zeros(tokens, cols, dtype=torch.float64, device="cuda"), torch.zeros(tokens, cols, dtype=torch.float64, device="cuda")
    for r in range(k):
        p = places[:, r].long()
        ok = ((p >= 0) & (p < n)).unsqueeze(1)
        term = torch.where(ok, y[p.clamp(0, n - 1)].double(), 0.0) * gates[:, r:r + 1].double()
        ref += term
        mag += term.abs()
    bound = half_step(DT[odt]) * (ref.abs() + 2.0 ** -20 * mag) + k * 2.0 ** -23 * mag + tiny(DT[odt])
    assert ((out[:, :cols].double() - ref).abs() <= bound).all()
    assert (out[:, cols:] == 5.0).all() and (out[5, :cols] == 0).all()


@pytest.mark.parametrize("dtype,ts", [("bf16", 1.0), ("fp16", 0.37), ("fp32", 1.0)])
def test_quantize_of_many_elements(M, dtype, ts):
    """More blocks of 16 than run at once (8 x 256 an SM), the last pass part of one, bit for bit: contiguous rows, rows
    apart by a multiple of 32 bytes, and by one of 16 only."""
    rows, cols = 2701, 4112
    x = randn(71, rows, cols)
    x[:, ::97] *= 12.0
    x[100:103] *= 1e-4
    x = x.to(DT[dtype])
    c, s, _ = F.q4((x.float() / torch.tensor(ts, dtype=torch.float32)).double().numpy())
    c, s = torch.from_numpy(c), torch.from_numpy(s)
    packed = c[..., 0::2] | (c[..., 1::2] << 4)
    values, packed, s = values64(packed, s).float(), packed.cuda(), s.cuda()
    assert rows * cols // 16 > 2 * 8 * 256 * torch.cuda.get_device_properties(0).multi_processor_count
    for extra in (0, 16, 8):
        w = M.msk_quantize_fp4(strided(x, extra), ts)
        assert torch.equal(w.packed, packed) and torch.equal(w.scales, s)
        back = torch.full((rows, cols + extra), 3.0, dtype=DT[dtype], device="cuda")
        M.msk_dequantize_fp4(w, out=back[:, :cols])
        # two fp32 products, the second one rounding, then the type's
        assert torch.equal(back[:, :cols], (values * torch.tensor(ts, dtype=torch.float32)).to(DT[dtype]).cuda())
        assert (back[:, cols:] == 3.0).all()


@pytest.mark.parametrize("n,E", [(1 << 20, 256), (16_777_217, 1024), (50_000_003, 61)])
def test_sort_of_many_slots(M, n, E):
    """Runs of a warp far longer than what its threads hold; most slots are other clusters'."""
    g = torch.Generator("cuda").manual_seed(n)
    e = torch.randint(-1, E + 1, (n,), generator=g, dtype=torch.int32, device="cuda")
    e[n // 3:n // 2] = 1                               # (a favourite)
    offsets, slots, places = M.msk_moe_sort(e, E)
    key = torch.where((e >= 0) & (e < E), e, E)
    order = torch.sort(key, stable=True)
    kept = int((key < E).sum())
    assert torch.equal(offsets.long(), torch.searchsorted(order.values, torch.arange(E + 1, dtype=torch.int32, device="cuda")))
    assert torch.equal(slots[:kept].long(), order.indices[:kept]) and (slots[kept:] == -1).all()
    want = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    want[order.indices[:kept]] = torch.arange(kept, dtype=torch.int32, device="cuda")
    assert torch.equal(places, want)
