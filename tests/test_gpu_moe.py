"""The operators of a whole prompt's experts on the GPU, against their
definitions in 64 bits (the quantiser against the oracle's, bit for bit).

Tolerances, from the arithmetic.  h(t) = eps(t) / 2 is half a rounding step of
the output's type.
  route: a gate is e^(v - v0) over a sum of such.  v - v0 is rounded once
    (2^-24 of it), the exponential is off by 2^-22, the sum of k by k 2^-24, the
    quotient by 2^-24: relative 2 (2^-22 + max |v - v0| 2^-24) + (k + 1) 2^-24.
  products: fp32 sums of K exact products: (K + 64) 2^-23 sum |x w|, and the
    tensors' scales: three roundings of 2^-24.
  SwiGLU: s = g sigma(g), |ds / dg| <= 1.1; the exponential, sum, quotient and
    two products add 2^-20 of s u.
  combine: k fused products and sums: k 2^-23 sum |gate y|."""

import math

import numpy as np
import pytest
import torch

from oracle import formats as F

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half a step among the type's subnormal numbers."""
    return torch.finfo(t).smallest_normal * half_step(t)


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import moe_decode_step_persistent_gb300 as mod
    mod.load_library()
    return mod


@pytest.fixture(autouse=True)
def no_wait_ran_out(M):
    yield
    M.msk_ops_check()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(seed, *shape):
    return torch.randn(*shape, generator=gen(seed))


def values64(codes, scales, ts=1.0):
    cols = codes.shape[-1] * 2
    v = F.nvfp4_dequant(codes.reshape(-1, cols // 2).numpy(), scales.reshape(-1, cols // 16).numpy(), 1.0, cols)
    return torch.from_numpy(v).reshape(*codes.shape[:-1], cols) * float(np.float32(ts))


def random_fp4(seed, *shape):
    """Codes and scales as a quantiser makes them."""
    c, s, _ = F.q4(randn(seed, *shape).numpy())
    c = torch.from_numpy(c)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.from_numpy(s)


def strided(t, extra):
    """t's values in rows `extra` elements further apart."""
    if extra == 0:
        return t.cuda()
    wide = torch.full((t.shape[0], t.shape[1] + extra), 7.0, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]]


# ----------------------------------------------------------------------------
# route
# ----------------------------------------------------------------------------


def route_ref(logits, bias, k):
    """(experts, gates in 64 bits) by a loop over the ranks."""
    x = logits.float()
    if bias is not None:
        x = x + bias
    x = torch.where(torch.isnan(x), -math.inf, x)
    T, E = x.shape
    experts = torch.full((T, k), -1, dtype=torch.int32)
    vals = torch.full((T, k), -math.inf, dtype=torch.float64)
    for t in range(T):
        left = x[t].tolist()
        for r in range(k):
            best = max(range(E), key=lambda e: (left[e], -e))
            if left[best] == -math.inf:
                break
            experts[t, r], vals[t, r] = best, left[best]
            left[best] = -math.inf
    gates = torch.softmax(vals, -1)
    return experts, torch.where(experts >= 0, gates, 0.0), vals


@pytest.mark.parametrize("tokens,E,k,dtype,bias,extra", [
    (1, 16, 2, "fp32", False, 0), (16, 256, 8, "fp32", True, 0), (37, 256, 8, "bf16", True, 0), (5, 1, 1, "fp32", True, 3),
    (9, 60, 4, "fp16", False, 0), (33, 1024, 32, "bf16", True, 8), (7, 1000, 9, "fp32", False, 1), (130, 128, 5, "fp32", True, 4),
    (3, 33, 32, "bf16", False, 1), (64, 512, 8, "fp16", True, 8), (6, 200, 8, "fp32", True, 0)])
def test_route(M, tokens, E, k, dtype, bias, extra):
    logits = (randn(1, tokens, E) * 2).to(DT[dtype])
    if tokens > 4 and E > 8:
        logits[1] = 0.5                                 # all alike: the lowest indices
        logits[2, ::3] = -math.inf                      # barred experts
        logits[3] = -math.inf                           # none left
        logits[4] = -math.inf                           # fewer than k left, a NaN among the barred
        logits[4, E // 2], logits[4, 3], logits[4, 1] = 1.25, -2.0, math.nan
        logits[0, 5], logits[0, 2] = 0.0, -0.0          # two zeros are alike
    b = randn(2, E) if bias else None
    if bias:
        b[0] = -math.inf
    want, gates, vals = route_ref(logits, b, k)
    got_e, got_g = M.msk_moe_route(strided(logits, extra), k, bias=None if b is None else b.cuda())
    assert torch.equal(got_e.cpu(), want)
    spread = torch.where(want >= 0, vals[:, :1] - vals, 0.0).amax()
    tol = 2 * (2.0 ** -22 + float(spread) * 2.0 ** -24) + (k + 1) * 2.0 ** -24
    assert ((got_g.cpu().double() - gates).abs() <= tol * gates + 1e-37).all()


def test_route_of_an_infinite_logit(M):
    logits = randn(3, 4, 64)
    logits[2, 9] = math.inf
    e, g = M.msk_moe_route(logits.cuda(), 4)
    want, _, _ = route_ref(logits, None, 4)
    assert torch.equal(e.cpu(), want)
    assert torch.isnan(g[2]).all() and not torch.isnan(g[[0, 1, 3]]).any()


# ----------------------------------------------------------------------------
# sort
# ----------------------------------------------------------------------------


def sort_ref(experts, E):
    flat = experts.flatten().tolist()
    order = sorted((s for s in range(len(flat)) if 0 <= flat[s] < E), key=lambda s: (flat[s], s))
    count = np.bincount([flat[s] for s in order], minlength=E) if order else np.zeros(E, int)
    offsets = np.concatenate(([0], np.cumsum(count)))
    places = np.full(len(flat), -1)
    places[order] = np.arange(len(order))
    return offsets, np.array(order + [-1] * (len(flat) - len(order))), places.reshape(experts.shape)


def sort_ref_many(experts, E):
    """The same by a stable sort of numpy's."""
    flat = experts.flatten().numpy()
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order, kept = np.argsort(key, kind="stable"), int((key < E).sum())
    places = np.full(flat.size, -1)
    places[order[:kept]] = np.arange(kept)
    return np.concatenate(([0], np.cumsum(np.bincount(key, minlength=E + 1)[:E]))), np.where(np.arange(flat.size) < kept, order, -1), places.reshape(experts.shape)


@pytest.mark.parametrize("tokens,k,E", [(0, 8, 4), (1, 1, 1), (1, 8, 256), (16, 8, 256), (31, 5, 7), (512, 8, 60), (513, 8, 1024),
                                        (4096, 1, 256), (4097, 8, 256), (8192, 5, 1000), (20000, 8, 3), (32768, 8, 256),
                                        (70001, 5, 1024), (300000, 8, 60)])
@pytest.mark.parametrize("kind", ["mixed", "one", "dropped"])
def test_sort(M, tokens, k, E, kind):
    g = gen(tokens * 7 + E)
    e = torch.randint(-2, E + 2, (tokens, k), generator=g, dtype=torch.int32)  # (some outside: dropped)
    if kind == "one":
        e.fill_(E - 1)
    elif kind == "dropped":
        e.fill_(-1)
    offsets, slots, places = (x.cpu().numpy() for x in M.msk_moe_sort(e.cuda(), E))
    want = sort_ref(e, E) if tokens < 50000 else sort_ref_many(e, E)
    assert np.array_equal(offsets, want[0]) and np.array_equal(slots, want[1]) and np.array_equal(places, want[2])


# ----------------------------------------------------------------------------
# rows in and out
# ----------------------------------------------------------------------------


@pytest.mark.parametrize("rows,cols,dtype,ts,extra", [
    (1, 16, "bf16", 1.0, 0), (3, 48, "fp16", 1.0, 0), (16, 2048, "bf16", 1.0, 8), (130, 64, "fp32", 0.37, 4), (33, 112, "bf16", 2.5, 16),
    (5, 4096, "fp32", 4.4e-5, 0), (7, 1040, "fp16", 0.01, 8), (2, 32, "fp32", 1e-30, 0), (2, 32, "fp32", 3e30, 0)])
def test_quantize_and_back(M, rows, cols, dtype, ts, extra):
    x = randn(1, rows, cols)
    x[:, ::5] *= 40.0
    x[rows // 2, :16] = 0.0             # a block of zeros
    x[0, -16:] = 3e-4                   # a scale among E4M3's subnormals
    x[-1, -16:] *= 1e-5                 # a scale that rounds to zero
    x = x * ts if dtype == "fp32" or ts > 1e-3 else x
    if dtype != "fp16" and rows > 2:
        x[1, :16] *= 1e5                # saturates
    x = x.to(DT[dtype])
    w = M.msk_quantize_fp4(strided(x, extra), ts)
    c, s, _ = F.q4((x.float() / torch.tensor(ts, dtype=torch.float32)).double().numpy())
    c = torch.from_numpy(c)
    assert torch.equal(w.packed.cpu(), c[..., 0::2] | (c[..., 1::2] << 4))
    assert np.array_equal(w.scales.cpu().numpy(), s)
    ref = values64(w.packed.cpu(), w.scales.cpu(), ts)
    for out in DT.values():
        if out == torch.float16 and float(ref.abs().max()) > 65504:
            continue
        got = M.msk_dequantize_fp4(w, dtype=out)
        # two fp32 products, the second one rounding, then the type's
        ref32 = (values64(w.packed.cpu(), w.scales.cpu()).float() * torch.tensor(ts, dtype=torch.float32))
        assert torch.equal(got.cpu(), ref32.to(out))
    wide = torch.full((rows, cols + 8), 3.0, device="cuda")
    M.msk_dequantize_fp4(w, out=wide[:, :cols])
    assert torch.equal(wide[:, :cols], M.msk_dequantize_fp4(w, dtype=torch.float32)) and (wide[:, cols:] == 3.0).all()


def test_quantize_special_values(M):
    x = randn(5, 4, 64)
    x[0, 3], x[1, 20], x[2, 40], x[3, 0] = math.inf, -math.inf, math.nan, -0.0
    w = M.msk_quantize_fp4(x.cuda())
    v = M.msk_dequantize_fp4(w, dtype=torch.float32).cpu()
    assert v[0, 3] == 2688.0 and v[1, 20] == -2688.0
    assert torch.isfinite(v).all() and v[2, 40].abs() == 6 * values64(torch.full((1, 8), 0x22, dtype=torch.uint8), w.scales[2:3, 2:3].cpu())[0, 0]
    assert (w.packed[3, 0].item() & 15) == 8


# ----------------------------------------------------------------------------
# products
# ----------------------------------------------------------------------------


def make_experts(M, seed, E, rows, cols, ts=True):
    p, s = random_fp4(seed, E, rows, cols)
    t = 0.02 * (0.5 + torch.rand(E, generator=gen(seed))) if ts else None
    h = M.Fp4Experts(p.cuda(), s.cuda(), None if t is None else t.cuda())
    v = values64(p, s)
    return h, v if t is None else v * t.double().view(E, 1, 1)


def products_ref(x, w, up, counts, source):
    """(y, bound of the error before the output's rounding) in 64 bits."""
    K = x.shape[1]
    ys, errs, at = [], [], 0
    for e, n in enumerate(counts):
        part = x[source[at:at + n]]
        at += n
        g = part @ w[e].T
        dg = (K + 64) * 2.0 ** -23 * (part.abs() @ w[e].abs().T) + 3 * 2.0 ** -24 * g.abs()
        if up is not None:
            u = part @ up[e].T
            du = (K + 64) * 2.0 ** -23 * (part.abs() @ up[e].abs().T) + 3 * 2.0 ** -24 * u.abs()
            s = g * torch.sigmoid(g)
            ys.append(s * u)
            errs.append(s.abs() * du + (u.abs() + du) * 1.1 * dg + 2.0 ** -20 * (s * u).abs())
        else:
            ys.append(g)
            errs.append(dg)
    return torch.cat(ys), torch.cat(errs)


def run_products(M, counts, rows, cols, glu=False, gather=False, out="bf16", x_ts=1.0, seed=11, extra=0, top_k=3, ts=True):
    E, n = len(counts), sum(counts)
    w, wv = make_experts(M, seed, E, rows, cols, ts)
    up, uv = make_experts(M, seed + 1, E, rows, cols, ts) if glu else (None, None)
    g = gen(seed + 2)
    if gather:
        xr = max(1, (n + top_k - 1) // top_k)
        slots = torch.randint(0, xr * top_k, (n,), generator=g, dtype=torch.int32)  # (the same index twice, too)
        source = (slots // top_k).long()
    else:
        xr, slots, source = n, None, torch.arange(n)
    c, s = random_fp4(seed + 3, xr, cols)
    x = M.Fp4Weight(c.cuda(), s.cuda(), x_ts)
    offsets = torch.tensor([0] + counts).cumsum(0).int()
    y = torch.full((n + 3, rows + extra), 5.0, dtype=DT[out], device="cuda")
    got = M.msk_experts_fp4(x, w, offsets.cuda(), up=up, slots=None if slots is None else slots.cuda(), top_k=top_k,
                            out=y[:n, :rows])
    ref, err = products_ref(values64(c, s, x_ts), wv, uv, counts, source)
    diff = (got.cpu().double() - ref).abs()
    bound = half_step(DT[out]) * (ref.abs() + err) + err + tiny(DT[out])
    assert (diff <= bound).all(), float((diff / bound).max())
    # nothing beside the rows
    assert (y[n:] == 5.0).all() and (y[:, rows:] == 5.0).all()


@pytest.mark.parametrize("counts,rows,cols", [
    ([1], 128, 256), ([16], 128, 64), ([17], 64, 128), ([5], 1, 192), ([3], 129, 320), ([128], 256, 512), ([129], 128, 256),
    ([224], 128, 1024), ([225], 200, 256), ([700], 136, 576), ([0, 1, 0], 128, 256), ([3, 0, 40, 1, 130, 0, 300], 160, 384),
    ([2] * 40, 72, 128), ([0, 0, 0, 33], 31, 448)])
@pytest.mark.parametrize("glu,gather", [(False, False), (True, False), (False, True), (True, True)])
def test_products(M, counts, rows, cols, glu, gather):
    run_products(M, counts, rows, cols, glu, gather)


@pytest.mark.parametrize("counts,rows,cols", [
    ([3] * 300, 600, 64), ([40, 0] * 100, 520, 128), ([256] * 40, 1030, 320), ([209, 256, 208, 31, 255, 240, 1, 224] * 12, 520, 512),
    ([500, 7, 213] * 20, 600, 192)])
@pytest.mark.parametrize("glu,gather", [(False, False), (True, False), (False, True), (True, True)])
def test_products_of_many_tiles(M, counts, rows, cols, glu, gather):
    """Several tiles for a pair of blocks, of one stage and more, of few tokens and so many that accumulators overlap."""
    run_products(M, counts, rows, cols, glu, gather)


@pytest.mark.parametrize("rows", [256, 300, 302, 301, 4, 2])
@pytest.mark.parametrize("cols", [64, 128, 1984, 2880, 4032])
@pytest.mark.parametrize("glu,gather", [(False, False), (True, False), (False, True), (True, True)])
def test_products_of_columns_that_end_inside_a_stage(M, rows, cols, glu, gather):
    """Weights' scales by copies of two and four rows as one, and by loads; more stages than the ring has."""
    run_products(M, [5, 0, 130, 261], rows, cols, glu, gather)


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("glu", [False, True])
def test_products_types_and_strides(M, out, glu):
    run_products(M, [7, 0, 250, 31], 100, 256, glu, True, out, extra=5)
    run_products(M, [20, 1], 96, 4096, glu, False, out, extra=8, ts=False)


@pytest.mark.parametrize("x_ts,out", [(0.37, "bf16"), (1e-20, "fp32"), (3e18, "fp32")])
def test_products_scales(M, x_ts, out):
    run_products(M, [30, 3], 130, 256, x_ts=x_ts, out=out)


def test_products_scales_that_leave_the_range_alone(M):
    """Two tensors' scales whose product leaves fp32's range, with results in it."""
    c = torch.full((1, 32), 0x22, dtype=torch.uint8)          # ones
    s = torch.full((1, 4), 0x01, dtype=torch.uint8)           # 2^-9
    w = M.Fp4Experts(c.view(1, 1, 32).cuda(), s.view(1, 1, 4).cuda(), torch.tensor([2.0 ** 100], device="cuda"))
    x = M.Fp4Weight(c.cuda(), s.cuda(), 2.0 ** 36)
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    y = M.msk_experts_fp4(x, w, off, out_dtype=torch.float32)
    assert y.item() == 64 * 2.0 ** (-18 + 100 + 36 - 0)
    x = M.Fp4Weight(c.cuda(), torch.full((1, 4), 0x78, dtype=torch.uint8).cuda(), 2.0 ** -100)  # 256
    w = M.Fp4Experts(c.view(1, 1, 32).cuda(), torch.full((1, 1, 4), 0x78, dtype=torch.uint8).cuda(),
                     torch.tensor([2.0 ** -55], device="cuda"))
    y = M.msk_experts_fp4(x, w, off, out_dtype=torch.float32)
    assert y.item() == 2.0 ** (6 + 16 - 155)


def test_every_scale_code(M):
    """Every finite E4M3 scale on both sides: exact sums of one product."""
    codes = torch.arange(0x7F, dtype=torch.uint8)
    n = codes.numel()
    wp = torch.zeros(1, n, 128, dtype=torch.uint8)
    wp[:, :, 8 * 5] = 0x07                                       # element 80: 6
    ws = torch.zeros(1, n, 16, dtype=torch.uint8)
    ws[0, :, 5] = codes
    xp = torch.zeros(n, 128, dtype=torch.uint8)
    xp[:, 40] = 0x03                                             # 1.5
    xs = torch.zeros(n, 16, dtype=torch.uint8)
    xs[:, 5] = codes
    y = M.msk_experts_fp4(M.Fp4Weight(xp.cuda(), xs.cuda()), M.Fp4Experts(wp.cuda(), ws.cuda()),
                          torch.tensor([0, n], dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    v = values64(torch.full((n, 8), 0x22, dtype=torch.uint8), codes.view(n, 1))[:, 0]
    assert torch.equal(y.cpu().double(), 9.0 * v.view(n, 1) * v.view(1, n))


def test_nan_scales_stay_in_their_rows(M):
    counts, rows, cols = [20, 9], 70, 256
    w, _ = make_experts(M, 5, 2, rows, cols)
    c, s = random_fp4(6, 29, cols)
    off = torch.tensor([0, 20, 29], dtype=torch.int32, device="cuda")
    base = M.msk_experts_fp4(M.Fp4Weight(c.cuda(), s.cuda()), w, off)
    w.scales[0, 33, 2] = 0x7F
    s[25, 7] = 0x7F
    got = M.msk_experts_fp4(M.Fp4Weight(c.cuda(), s.cuda()), w, off)
    bad = torch.zeros(29, rows, dtype=torch.bool, device="cuda")
    bad[:20, 33] = True
    bad[25] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], base[~bad])


def test_places_of_no_expert_are_left(M):
    """Offsets that begin behind 0, end before n, or are cut off: only experts' places are written."""
    w, wv = make_experts(M, 7, 3, 40, 128)
    c, s = random_fp4(8, 50, 128)
    x = M.Fp4Weight(c.cuda(), s.cuda())
    xv = values64(c, s)
    for offsets, ranges in (([4, 10, 10, 30], [(4, 10), (10, 10), (10, 30)]), ([0, 0, 0, 0], [(0, 0)] * 3),
                            ([-5, 7, 60, 80], [(0, 7), (7, 50), (50, 50)]), ([0, 20, 10, 30], [(0, 20), (20, 20), (20, 30)])):
        y = torch.full((50, 40), 9.0, device="cuda")
        M.msk_experts_fp4(x, w, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=y)
        want = torch.full((50, 40), 9.0, dtype=torch.float64)
        for e, (a, b) in enumerate(ranges):
            want[a:b] = xv[a:b] @ wv[e].T
        assert torch.allclose(y.cpu().double(), want, rtol=1e-4, atol=1e-3)
        assert torch.equal(y.cpu() == 9.0, want == 9.0)


def test_slots_beyond_x_are_cut_off(M):
    w, wv = make_experts(M, 9, 1, 16, 64)
    c, s = random_fp4(10, 5, 64)
    slots = torch.tensor([-1, 0, 9, 10, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    y = M.msk_experts_fp4(M.Fp4Weight(c.cuda(), s.cuda()), w, torch.tensor([0, 6], dtype=torch.int32, device="cuda"),
                          slots=slots.cuda(), top_k=2, out_dtype=torch.float32)
    want = values64(c, s)[[0, 0, 4, 4, 4, 0]] @ wv[0].T
    assert torch.allclose(y.cpu().double(), want, rtol=1e-4, atol=1e-3)


# ----------------------------------------------------------------------------
# combine
# ----------------------------------------------------------------------------


@pytest.mark.parametrize("tokens,k,cols,ydt,odt,extra", [
    (1, 1, 8, "bf16", "bf16", 0), (16, 8, 2048, "bf16", "bf16", 0), (5, 2, 7, "fp16", "fp32", 0), (33, 9, 136, "fp32", "bf16", 0),
    (3, 17, 64, "bf16", "fp32", 8), (20, 4, 1000, "fp16", "fp16", 3), (7, 8, 1, "bf16", "bf16", 0), (130, 5, 24, "fp32", "fp32", 4),
    (9, 8, 64, "fp32", "fp16", 0)])
@pytest.mark.parametrize("gated", [True, False])
def test_combine(M, tokens, k, cols, ydt, odt, extra, gated):
    n = tokens * k
    y = randn(1, n, cols).to(DT[ydt])
    places = torch.randperm(n, generator=gen(2)).int().view(tokens, k)
    if n > 8:
        drop = torch.rand(tokens, k, generator=gen(3)) < 0.2
        y[places[drop].long()] = math.nan                         # (not read)
        places[drop] = torch.tensor([-1, n, 2 ** 31 - 1, -2 ** 31])[torch.arange(int(drop.sum())) % 4].int()
        places[0] = -1                                            # a token with nothing: zeros
        places[1, 0] = places[1, k - 1]                           # the same place twice
    gates = torch.rand(tokens, k, generator=gen(4)) if gated else None
    out = torch.full((tokens, cols + extra), 5.0, dtype=DT[odt], device="cuda")
    got = M.msk_moe_combine(strided(y, extra), places.cuda(), None if gates is None else gates.cuda(), out=out[:, :cols])
    ok = (places >= 0) & (places < n)
    terms = torch.where(ok.unsqueeze(-1), y[places.long().clamp(0, n - 1)].double(), 0.0)
    if gated:
        terms = terms * gates.double().unsqueeze(-1)
    ref, mag = terms.sum(1), terms.abs().sum(1)
    diff = (got.cpu().double() - ref).abs()
    assert (diff <= half_step(DT[odt]) * (ref.abs() + 2.0 ** -20 * mag) + k * 2.0 ** -23 * mag + tiny(DT[odt])).all()
    assert (out[:, cols:] == 5.0).all()


# ----------------------------------------------------------------------------
# together
# ----------------------------------------------------------------------------


def moe(M, logits, bias, x, gate, up, down, k, stream=None):
    experts, gates = M.msk_moe_route(logits, k, bias=bias, stream=stream)
    offsets, slots, places = M.msk_moe_sort(experts, gate.n_experts, stream=stream)
    xq = M.msk_quantize_fp4(x, stream=stream)
    h = M.msk_experts_fp4(xq, gate, offsets, up=up, slots=slots, top_k=k, stream=stream)
    hq = M.msk_quantize_fp4(h, stream=stream)
    y = M.msk_experts_fp4(hq, down, offsets, stream=stream)
    return M.msk_moe_combine(y, places, gates, stream=stream), (experts, gates, offsets, slots, xq, h, hq, y)


@pytest.mark.parametrize("tokens,E,k,P,I", [(1, 16, 2, 128, 128), (16, 64, 8, 256, 192), (150, 8, 3, 320, 128)])
def test_a_prompt_through_its_experts(M, tokens, E, k, P, I):
    """The operators one after the other, each stage against its definition on the stage's own input."""
    logits, bias = randn(1, tokens, E).cuda(), randn(2, E).cuda()
    x = randn(3, tokens, P).bfloat16().cuda()
    gate, gv = make_experts(M, 4, E, I, P)
    up, uv = make_experts(M, 5, E, I, P)
    down, dv = make_experts(M, 6, E, P, I)
    out, (experts, gates, offsets, slots, xq, h, hq, y) = moe(M, logits, bias, x, gate, up, down, k)
    counts = np.diff(offsets.cpu().numpy()).tolist()
    s = slots.cpu().long()
    ref, err = products_ref(values64(xq.packed.cpu(), xq.scales.cpu()), gv, uv, counts, s // k)
    assert ((h.cpu().double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + err) + err + 1e-38).all()
    c, sc, _ = F.q4(h.cpu().double().numpy())
    c = torch.from_numpy(c)
    assert torch.equal(hq.packed.cpu(), c[..., 0::2] | (c[..., 1::2] << 4)) and np.array_equal(hq.scales.cpu().numpy(), sc)
    ref, err = products_ref(values64(hq.packed.cpu(), hq.scales.cpu()), dv, None, counts, torch.arange(tokens * k))
    assert ((y.cpu().double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + err) + err + 1e-38).all()
    # back at the tokens, from the slots' own order and not from the places
    yv, total, mag = y.cpu().double(), torch.zeros(tokens, P, dtype=torch.float64), torch.zeros(tokens, P, dtype=torch.float64)
    for p in range(tokens * k):
        t, r = int(s[p]) // k, int(s[p]) % k
        total[t] += gates[t, r].item() * yv[p]
        mag[t] += abs(gates[t, r].item()) * yv[p].abs()
    assert ((out.cpu().double() - total).abs() <= 2.0 ** -8 * total.abs() + (k + 1) * 2.0 ** -23 * mag + 1e-38).all()


def test_captured_and_on_two_streams(M):
    """A captured run gives the eager one's bits for new inputs, and so do two streams at once."""
    E, k, T, P, I = 32, 4, 200, 256, 128
    gate, up, down = (make_experts(M, s, E, r, c)[0] for s, r, c in ((4, I, P), (5, I, P), (6, P, I)))
    logits, x = randn(1, T, E).cuda(), randn(3, T, P).bfloat16().cuda()
    inputs = [(randn(10 + i, T, E).cuda(), randn(20 + i, T, P).bfloat16().cuda()) for i in range(3)]
    want = [moe(M, l, None, v, gate, up, down, k)[0] for l, v in inputs]
    moe(M, logits, None, x, gate, up, down, k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = moe(M, logits, None, x, gate, up, down, k)
    for (l, v), w in zip(inputs, want):
        logits.copy_(l)
        x.copy_(v)
        graph.replay()
        assert torch.equal(out, w)
    streams = [torch.cuda.Stream() for _ in inputs]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [moe(M, l, None, v, gate, up, down, k, stream=s) for (l, v), s in zip(inputs, streams)]
        torch.cuda.synchronize()
        for (o, _), w in zip(outs, want):
            assert torch.equal(o, w)


def test_runs_repeat_bit_for_bit(M):
    E, k, T = 64, 8, 1500
    gate, _ = make_experts(M, 4, E, 128, 256)
    experts = torch.randint(0, E, (T, k), generator=gen(1), dtype=torch.int32).cuda()
    first = None
    for _ in range(10):
        offsets, slots, places = M.msk_moe_sort(experts, E)
        c, s = random_fp4(3, T, 256) if first is None else (c, s)
        y = M.msk_experts_fp4(M.Fp4Weight(c.cuda(), s.cuda()), gate, offsets, slots=slots, top_k=k)
        now = (offsets, slots, places, y)
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


FIRST_CAPTURED = """
import torch
import moe_decode_step_persistent_gb300 as M
E, k, T = 40, 4, 900
logits = torch.randn(T, E, device="cuda")
x = torch.randn(T, 256, device="cuda").bfloat16()
def weights(rows, cols):
    return M.Fp4Experts(torch.full((E, rows, cols // 2), 0x22, dtype=torch.uint8, device="cuda"),
                        torch.full((E, rows, cols // 16), 0x38, dtype=torch.uint8, device="cuda"))
gate, up, down, odd = weights(96, 256), weights(96, 256), weights(256, 96 // 32 * 64), weights(32, 320)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    experts, gates = M.msk_moe_route(logits, k)
    offsets, slots, places = M.msk_moe_sort(experts, E)
    xq = M.msk_quantize_fp4(x)
    xv = M.msk_dequantize_fp4(xq, dtype=torch.float32)
    h = M.msk_experts_fp4(xq, gate, offsets, up=up, slots=slots, top_k=k)
    p = M.msk_experts_fp4(xq, gate, offsets, slots=slots, top_k=k, out_dtype=torch.float32)
    z = M.msk_experts_fp4(M.msk_quantize_fp4(torch.cat((h, h), 1)), down, offsets)
    out = M.msk_moe_combine(z, places, gates)
g.replay()
torch.cuda.synchronize()
want = xv.sum(1)[slots.long() // k]
assert (p - want.unsqueeze(1)).abs().max() < 1e-3 * want.abs().max()
assert torch.isfinite(out).all()
M.msk_ops_check()
print("captured")
"""


def test_captured_without_a_call_before(M):
    """The process's first calls are captured ones."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]


def test_behind_an_event_of_another_stream(M):
    """Calls wait for what their stream waits for, whatever ran before them: they start early."""
    gate, _ = make_experts(M, 4, 8, 128, 256)
    k, T = 2, 300
    src = [(randn(30 + i, T, 8).cuda(), randn(40 + i, T, 256).bfloat16().cuda()) for i in range(4)]
    logits, x = torch.zeros(T, 8, device="cuda"), torch.zeros(T, 256, dtype=torch.bfloat16, device="cuda")
    big, side = torch.zeros(1 << 26, device="cuda"), torch.cuda.Stream()

    def run(l, v):
        experts, gates = M.msk_moe_route(l, k)
        offsets, slots, places = M.msk_moe_sort(experts, 8)
        y = M.msk_experts_fp4(M.msk_quantize_fp4(v), gate, offsets, slots=slots, top_k=k)
        return M.msk_moe_combine(y, places, gates)

    want = [run(l, v) for l, v in src]
    torch.cuda.synchronize()
    got = []
    for l, v in src:
        run(logits, x)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            big.add_(1.0)  # tens of microseconds, then the inputs
            logits.copy_(l)
            x.copy_(v)
        torch.cuda.current_stream().wait_stream(side)
        got.append(run(logits, x))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("counts,rows,cols,glu,gather", [
    ([2], 8, 131072, False, False), ([1, 2], 24, 16384, True, True), ([1] * 1024, 16, 64, False, True), ([1] * 1024, 40, 256, True, False)])
def test_products_of_extreme_sizes(M, counts, rows, cols, glu, gather):
    run_products(M, counts, rows, cols, glu, gather, out="fp32")


def test_maps_of_other_weights_are_refused(M):
    import ctypes
    a, _ = make_experts(M, 1, 2, 64, 128)
    b, _ = make_experts(M, 2, 2, 64, 128)
    c, s = random_fp4(3, 5, 128)
    x, off = M.Fp4Weight(c.cuda(), s.cuda()), torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    base = M.msk_experts_fp4(x, a, off)
    made = a.desc.contents.maps
    a.desc.contents.maps = None                   # made for the call instead
    assert torch.equal(M.msk_experts_fp4(x, a, off), base)
    a.desc.contents.maps = b.desc.contents.maps
    with pytest.raises(M.MskError) as e:
        M.msk_experts_fp4(x, a, off)
    assert e.value.status == M.MSK_ERR_INVALID_ARG
    with pytest.raises(M.MskError):
        M.msk_experts_fp4(x, b, off, up=a)
    a.desc.contents.maps = made


def test_quantised_weights_in_a_product_of_unquantised_rows(M):
    """An Fp4Weight made by msk_quantize_fp4 is a weight of msk_linear_fp4."""
    w, x = randn(1, 300, 512) * 0.02, randn(2, 5, 512).bfloat16()
    q = M.msk_quantize_fp4(w.cuda(), 4.4e-5)
    y = M.msk_linear_fp4(x.cuda(), q, out_dtype=torch.float32)
    v = values64(q.packed.cpu(), q.scales.cpu(), 4.4e-5)
    ref, mag = x.double() @ v.T, x.double().abs() @ v.abs().T
    assert ((y.cpu().double() - ref).abs() <= 2.0 ** -24 * ref.abs() + (512 + 64) * 2.0 ** -23 * mag).all()


def test_beside_a_launch_of_the_step(M):
    """What the step's launch does between its pooled vectors and their experts' sum, done by the operators on the same
    vectors.  Rows between the two projections are kept in fp32, as in the launch.  The experts are the same; codes of
    the rows between differ where the two exponentials and orders of summation put a value on another side of a border:
    at most one in 500 of them here, and the sums' cosine stays above 0.999 (the step's own bar)."""
    import msk_synth as S
    from tests._gpu import Setup, read_scratch, run_layers
    wl = S.scaled(S.WORKLOADS["tiny"], tokens=16, cached=64, windows=(0, 0), pooled=256, inter=256, top_k=4)
    st = Setup(wl)
    run_layers(st, st.hidden(), st.fresh_kv(), wl.positions)
    torch.cuda.synchronize()
    pooled, logits, sq_codes, m = (read_scratch(st, n) for n in ("pooled", "logits", "sq_codes", "mvec"))
    lt = st.lts_cpu[1]
    gate, up, down = (M.Fp4Experts(*(t.cuda() for t in w)) for w in (lt.gate, lt.up, lt.down))
    experts, gates = M.msk_moe_route(logits, wl.top_k)
    offsets, slots, places = M.msk_moe_sort(experts, wl.n_experts)
    h = M.msk_experts_fp4(M.msk_quantize_fp4(pooled), gate, offsets, up=up, slots=slots, top_k=wl.top_k, out_dtype=torch.float32)
    hq = M.msk_quantize_fp4(h)
    out = M.msk_moe_combine(M.msk_experts_fp4(hq, down, offsets), places, gates)
    mine = hq.packed[places.flatten().long()]                # by slot, as in the launch
    assert (mine != sq_codes).float().mean().item() <= 1 / 500
    a, b = out.double().flatten(), m.double().flatten()
    assert float(a @ b / (a.norm() * b.norm())) >= 0.999
    st.model.close()


def test_no_tokens(M):
    """A prompt of no tokens goes through all of it; experts without tokens write nothing."""
    E, k, P, I = 6, 2, 128, 64
    gate, up, down = (make_experts(M, s, E, r, c)[0] for s, r, c in ((1, I, P), (2, I, P), (3, P, I)))
    x = torch.zeros(0, P, dtype=torch.bfloat16, device="cuda")
    out, (experts, gates, offsets, slots, xq, h, hq, y) = moe(M, torch.zeros(0, E, device="cuda"), None, x, gate, up, down, k)
    assert out.shape == (0, P) and experts.shape == (0, k) and y.shape == (0, P) and hq.rows == 0
    assert offsets.tolist() == [0] * (E + 1)
    # every slot dropped: nothing is written, sums are 0
    experts = torch.full((5, k), -1, dtype=torch.int32, device="cuda")
    offsets, slots, places = M.msk_moe_sort(experts, E)
    c, s = random_fp4(4, 5, P)
    y = torch.full((5 * k, I), 4.0, device="cuda")
    M.msk_experts_fp4(M.Fp4Weight(c.cuda(), s.cuda()), gate, offsets, up=up, slots=slots, top_k=k, out=y)
    assert (y == 4.0).all() and (M.msk_moe_combine(y, places) == 0).all()


def test_rows_that_are_one_and_the_same(M):
    """A row stride of 0 is read, and refused where rows are written."""
    x = randn(1, 1, 96).bfloat16().cuda()
    w = M.msk_quantize_fp4(x.expand(7, 96))
    one = M.msk_quantize_fp4(x)
    assert torch.equal(w.packed, one.packed.expand(7, 48)) and torch.equal(w.scales, one.scales.expand(7, 6))
    flat = torch.zeros(1, 96, device="cuda").expand(7, 96)
    with pytest.raises(M.MskError):
        M.msk_dequantize_fp4(w, out=flat)
    l = randn(2, 1, 16).cuda()
    e, g = M.msk_moe_route(l.contiguous(), 3)
    gate, _ = make_experts(M, 1, 1, 16, 96 // 32 * 64)
    with pytest.raises(ValueError):
        M.msk_experts_fp4(w, gate, torch.tensor([0, 7], dtype=torch.int32, device="cuda"))
    v, vv = make_experts(M, 2, 1, 16, 128)
    c, s = random_fp4(3, 7, 128)
    with pytest.raises(M.MskError):
        M.msk_experts_fp4(M.Fp4Weight(c.cuda(), s.cuda()), v, torch.tensor([0, 7], dtype=torch.int32, device="cuda"),
                          out=torch.zeros(1, 16, device="cuda").expand(7, 16))
    with pytest.raises(M.MskError):
        M.msk_moe_combine(randn(4, 6, 16).cuda(), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), out=torch.zeros(1, 16, device="cuda").expand(3, 16))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route_of_many_tokens_with_ties(M, dtype):
    """Tokens whose logits take few values, several times what runs at once: against a stable sort."""
    T, E, k = 30000, 256, 8
    logits = (randn(7, T, E) * 2).round().div(2).to(DT[dtype]).cuda()
    order = torch.sort(logits.float(), dim=-1, descending=True, stable=True)
    e, g = M.msk_moe_route(logits, k)
    assert torch.equal(e, order.indices[:, :k].int())
    want = torch.softmax(order.values[:, :k].double(), -1)
    assert ((g.double() - want).abs() <= (2 * (2.0 ** -22 + 16 * 2.0 ** -24) + (k + 1) * 2.0 ** -24) * want).all()
