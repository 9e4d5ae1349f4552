"""The operators beside the step on the GPU, against their definitions in
64 bits (and the oracle's quantiser, bit for bit).

Tolerances, from the arithmetic.  h(t) = eps(t) / 2 is half a rounding step of
the output's type.
  attention: a softmax weight e^(s - m) carries the error of its score and its
    own rounding to fp16.  A score is an fp32 sum of d exact products, so
    off by at most (d + 8) 2^-23 sum |q k| scale, and the exponential adds
    2^-21.  The weight's rounding is 2^-11 relative above fp16's 2^-14 and
    2^-25 absolute below (relative to weights that reach 1; the sum of weights
    is at least 2^-10 of that where a reference lags behind the maximum, by
    at most 8 powers of two in any variant: 2^-25 with sums >= 1 either way).
    out: h |o| + (2^-11 + score + 2^-16) sum p |v| + 2^-25 n max |v|.
  linear: fp32 sums of exact products: h |y| + (K + 64) 2^-23 sum |x w|.
  logprobs: fp32 differences and sums: lse off by 2^-21 (1 + max |x / T|) +
    (V / 512 + 64) 2^-24 (serial partial sums of V / 512 or fewer terms, up to
    32768 logits of V / 256: no more than V / 512 + 64)."""

import math

import numpy as np
import pytest
import torch

from oracle import formats as F

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_step(t):
    return torch.finfo(t).eps / 2


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import moe_decode_step_persistent_gb300 as mod
    mod.load_library()
    return mod


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(seed, *shape):
    return torch.randn(*shape, generator=gen(seed))


def values64(codes, scales, ts):
    """Values of packed codes and scales (CPU) in 64 bits, by the oracle."""
    cols = codes.shape[-1] * 2
    v = F.nvfp4_dequant(codes.reshape(-1, cols // 2).numpy(), scales.reshape(-1, cols // 16).numpy(), 1.0, cols)
    return torch.from_numpy(v).reshape(*codes.shape[:-1], cols) * float(np.float32(ts))


def random_fp4(seed, *shape):
    """Codes and scales as a quantiser makes them."""
    c, s, _ = F.q4(randn(seed, *shape).numpy())
    c = torch.from_numpy(c)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.from_numpy(s)


def pack(codes):
    c = torch.from_numpy(codes)
    return c[..., 0::2] | (c[..., 1::2] << 4)


# ----------------------------------------------------------------------------
# rows in and out
# ----------------------------------------------------------------------------


@pytest.mark.parametrize("tokens,heads,d,pos0,dtype,layout,scales", [
    (1, 1, 64, 0, "bf16", "rows", (1.0, 1.0)), (16, 8, 128, 37, "bf16", "qkv", (1.0, 1.0)),
    (5, 3, 64, 2, "fp16", "planes", (0.37, 2.5)), (300, 2, 128, 1, "fp32", "rows", (1.0, 0.01)),
    (33, 2, 128, 0, "bf16", "planes", (1e-30, 3e30))])
def test_write_and_read(M, tokens, heads, d, pos0, dtype, layout, scales):
    max_seq = pos0 + tokens + 3
    base = randn(1, 2, tokens, heads, d)
    base[:, :, :, ::5] *= 40.0
    base[:, tokens // 2, 0, 16:32] = 0.0          # a block of zeros
    base[:, 0, 0, :16] = 3e-4                     # a scale among E4M3's subnormals
    base[:, -1, -1, 16:32] *= 1e-5                # a scale that rounds to zero
    if scales == (1e-30, 3e30):
        base[0] *= 1e-30
        base[1] *= 3e30
    if dtype != "fp16" and scales[0] == 1.0:
        base[0, 0, 0, 32:48] *= 1e5               # saturates
    src = base.to(DT[dtype])
    if layout == "qkv":     # slices of wider rows
        wide = torch.zeros(tokens, (4 + 2 * heads) * d, dtype=DT[dtype], device="cuda")
        k = wide[:, 4 * d:(4 + heads) * d].unflatten(1, (heads, d))
        v = wide[:, (4 + heads) * d:].unflatten(1, (heads, d))
        k.copy_(src[0])
        v.copy_(src[1])
    elif layout == "planes":
        k, v = (x.transpose(0, 1).contiguous().cuda().transpose(0, 1) for x in src)
    else:
        k, v = src[0].cuda(), src[1].cuda()
    cache = M.Kv4Cache.empty(heads, max_seq, d, *scales)
    cache.codes.fill_(0xA5)
    cache.scales.fill_(0x5A)
    M.msk_kv4_write(cache, k, v, pos0)
    got_c, got_s = cache.codes.cpu(), cache.scales.cpu()
    for i in (0, 1):
        x = (src[i].float() / torch.tensor(scales[i], dtype=torch.float32)).transpose(0, 1)
        c, s, _ = F.q4(x.double().numpy())
        assert np.array_equal(got_c[i, :, pos0:pos0 + tokens].numpy(), pack(c).numpy())
        assert np.array_equal(got_s[i, :, pos0:pos0 + tokens].numpy(), s)
    outside = [j for j in range(max_seq) if not pos0 <= j < pos0 + tokens]
    assert (got_c[:, :, outside] == 0xA5).all() and (got_s[:, :, outside] == 0x5A).all()
    rk, rv = M.msk_kv4_read(cache, pos0, tokens, dtype=DT[dtype])
    for i, r in enumerate((rk, rv)):
        ref = values64(got_c[i], got_s[i], scales[i])[:, pos0:pos0 + tokens].transpose(0, 1)
        # two fp32 products, the second one rounding, then the type's
        ref32 = (values64(got_c[i], got_s[i], 1.0)[:, pos0:pos0 + tokens].transpose(0, 1).float()
                 * torch.tensor(scales[i], dtype=torch.float32)).to(DT[dtype])
        assert torch.equal(r.cpu(), ref32)
        if DT[dtype] != torch.float16:
            assert torch.allclose(r.cpu().double(), ref, rtol=half_step(DT[dtype]) * 1.01, atol=0)


def test_write_of_infinities_and_nan(M):
    x = randn(3, 1, 1, 64)
    x[0, 0, 3] = float("inf")
    x[0, 0, 17] = float("-inf")
    x[0, 0, 33] = float("nan")
    x[0, 0, 48:] = float("nan")
    cache = M.Kv4Cache.empty(1, 4, 64)
    M.msk_kv4_write(cache, x.cuda(), x.cuda(), 1)
    k, _ = M.msk_kv4_read(cache, 1, 1, dtype=torch.float32)
    k = k.cpu()[0, 0]
    assert torch.isfinite(k).all()
    assert k[3] == 2688 and k[17] == -2688
    rest = torch.cat((x[0, 0, 32:33], x[0, 0, 34:48]))
    assert abs(k[33].item()) >= rest.abs().max() * 0.9 and (k[48:] == 0).all()


def test_write_at_a_device_position(M):
    k = randn(4, 5, 2, 64).cuda()
    a, b = M.Kv4Cache.empty(2, 32, 64), M.Kv4Cache.empty(2, 32, 64)
    for pos, real in ((9, 9), (-7, 0), (1000, 27)):
        a.codes.zero_(), b.codes.zero_(), a.scales.zero_(), b.scales.zero_()
        M.msk_kv4_write(a, k, k, torch.tensor([pos], dtype=torch.int32, device="cuda"))
        M.msk_kv4_write(b, k, k, real)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


# ----------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------


def visible(tokens, length, window, parents):
    par = [t - 1 for t in range(tokens)] if parents is None else parents
    depth, anc = [], []
    for t, p in enumerate(par):
        depth.append(0 if p < 0 else depth[p] + 1)
        anc.append({t} | (set() if p < 0 else anc[p]))
    see = torch.zeros(tokens, length + tokens, dtype=torch.bool)
    for t in range(tokens):
        for j in range(length):
            see[t, j] = True
        for u in anc[t]:
            see[t, length + u] = True
        if window:
            pos = torch.tensor(list(range(length)) + [length + x for x in depth])
            see[t] &= pos > length + depth[t] - window
    return see


def check_attention(M, out, q, cache, length, window, parents, scale=None):
    T, hq, d = q.shape
    n = length + T
    kc, ks = cache.codes.cpu()[:, :, :n], cache.scales.cpu()[:, :, :n]
    desc = cache.desc.contents
    k, v = values64(kc[0], ks[0], desc.k_scale), values64(kc[1], ks[1], desc.v_scale)
    hkv = k.shape[0]
    qq = q.cpu().double().view(T, hkv, hq // hkv, d)
    scale = 1 / math.sqrt(d) if scale is None else scale
    s = torch.einsum("thgd,hnd->thgn", qq, k) * scale
    see = visible(T, length, window, parents)[:, None, None, :]
    s = s.masked_fill(~see, float("-inf"))
    p = torch.softmax(s, -1)
    o = torch.einsum("thgn,hnd->thgd", p, v)
    mag = torch.einsum("thgn,hnd->thgd", p, v.abs())
    ds = (d + 8) * 2.0 ** -23 * (torch.einsum("thgd,hnd->thgn", qq.abs(), k.abs()) * scale).masked_fill(~see, 0).amax(-1)
    tol = (half_step(q.dtype) * o.abs() + (2.0 ** -11 + 2 * ds.unsqueeze(-1) + 2.0 ** -16) * mag
           + 2.0 ** -25 * n * v.abs().amax((1, 2)).view(1, hkv, 1, 1) + 1e-30)
    if q.dtype == torch.float16:
        tol += 2.0 ** -25
    err = (out.cpu().double().view(T, hkv, hq // hkv, d) - o).abs()
    worst = (err / tol).max().item()
    assert worst <= 1.0, f"error up to {worst:.2f} of the tolerance (max error {err.max().item():.3e})"


def filled_cache(M, seed, heads, max_seq, d, ks=1.0, vs=1.0):
    c = M.Kv4Cache.empty(heads, max_seq, d, ks, vs)
    codes, scales = random_fp4(seed, 2, heads, max_seq, d)
    c.codes.copy_(codes)
    c.scales.copy_(scales)
    return c


ATTN = [  # tokens, q heads, kv heads, head_dim, cached, window, tree, dtype
    (1, 4, 1, 64, 128, 0, False, "bf16"), (1, 1, 1, 64, 0, 0, False, "bf16"), (1, 8, 8, 128, 1, 0, False, "fp16"),
    (16, 32, 8, 128, 1000, 0, False, "bf16"), (16, 8, 2, 128, 517, 100, False, "bf16"),
    (16, 8, 2, 64, 333, 0, True, "bf16"), (7, 12, 4, 128, 15, 5, True, "fp16"), (3, 5, 1, 128, 4097, 1, False, "bf16"),
    (16, 4, 1, 128, 16, 4, True, "bf16"), (11, 24, 1, 128, 260, 0, True, "bf16"), (16, 64, 2, 64, 129, 64, False, "fp16"),
    (2, 32, 8, 128, 5003, 2048, False, "bf16"), (5, 3, 3, 128, 64, 0, False, "bf16"), (4, 48, 1, 128, 700, 0, False, "bf16"),
    (16, 1, 1, 64, 0, 0, True, "bf16"), (16, 16, 16, 128, 127, 300, False, "bf16"), (9, 14, 2, 128, 2049, 0, False, "fp16"),
    (1, 8, 2, 128, 9000, 0, False, "bf16"), (16, 16, 4, 128, 8500, 0, True, "bf16"), (3, 6, 1, 64, 20011, 0, False, "fp16"),
    (16, 8, 8, 64, 8193, 8190, True, "bf16"), (2, 10, 1, 128, 33000, 20000, False, "bf16"),
        (1, 8, 1, 128, 131000, 0, False, "bf16"), (16, 8, 1, 64, 70001, 0, True, "fp16"), (6, 24, 2, 128, 70002, 0, True, "bf16")]


def tree_parents(tokens, seed):
    r = gen(seed)
    return [int(torch.randint(-1, t, (1,), generator=r)) if t else -1 for t in range(tokens)]


@pytest.mark.parametrize("T,hq,hkv,d,length,window,tree,dtype", ATTN)
def test_attention(M, T, hq, hkv, d, length, window, tree, dtype):
    cache = filled_cache(M, 11, hkv, length + T + 5, d, 0.37, 1.9)
    # whatever lies behind the last row does not count: NaN scales, huge values
    cache.scales[:, :, length + T:] = 0x7F
    q = (randn(12, T, hq, d) * 2).to(DT[dtype]).cuda()
    parents = tree_parents(T, 13) if tree else None
    out = torch.full((T, hq * d), float("nan"), dtype=DT[dtype], device="cuda")
    M.msk_attention_kv4(q, cache, length, window=window, parents=parents, out=out)
    check_attention(M, out, q, cache, length, window, parents)
    again = M.msk_attention_kv4(q, cache, length, window=window, parents=parents)
    assert torch.equal(out, again)  # the same call, the same bits


def test_attention_rows_beyond_the_window_do_not_count(M):
    cache = filled_cache(M, 21, 2, 600, 128)
    cache.scales[:, :, :413] = 0x7F  # NaN scales on rows that no query sees
    q = randn(22, 4, 8, 128).bfloat16().cuda()
    out = M.msk_attention_kv4(q, cache, 512, window=100)
    assert torch.isfinite(out).all()
    cache.scales[:, :, :413] = 0
    assert torch.equal(out, M.msk_attention_kv4(q, cache, 512, window=100))


@pytest.mark.parametrize("dtype,size", [("bf16", 1e-30), ("bf16", 1e30), ("fp16", 60000.0), ("fp16", 1e-6)])
def test_attention_of_very_small_and_large_queries(M, dtype, size):
    """Rows are scaled by powers of two before they are fp16; a scale that
    brings the scores back makes the result that of ordinary queries."""
    cache = filled_cache(M, 31, 1, 300, 64)
    q = randn(32, 2, 4, 64)
    q = (q / q.abs().max() * size).to(DT[dtype]).cuda()
    scale = 0.3 / size
    out = M.msk_attention_kv4(q, cache, 290, softmax_scale=scale)
    check_attention(M, out, q, cache, 290, 0, None, float(np.float32(scale)))


def test_attention_with_steep_scores(M):
    """Maxima that rise along the cache, one key far above the rest, keys that
    underflow."""
    cache = filled_cache(M, 41, 1, 2100, 128)
    q = randn(42, 16, 4, 128).bfloat16().cuda()
    k = randn(43, 2100, 1, 128) * torch.linspace(0.1, 6, 2100).view(-1, 1, 1)
    k[1700] = q[3, 1].float().cpu() * 3
    M.msk_kv4_write(cache, k.cuda(), randn(44, 2100, 1, 128).cuda(), 0)
    for length in (2084, 1690, 40):
        check_attention(M, M.msk_attention_kv4(q, cache, length), q, cache, length, 0, None)


def test_attention_of_strided_queries_and_long_lengths(M):
    cache = filled_cache(M, 51, 1, 40, 64)
    wide = randn(52, 6, 3 * 64 + 128).bfloat16().cuda()
    q = wide[:, 64:64 + 128].unflatten(1, (2, 64))
    out = M.msk_attention_kv4(q, cache, 30)
    check_attention(M, out, q.contiguous(), cache, 30, 0, None)


def test_attention_where_offsets_pass_32_bits(M):
    """A cache whose last head lies 4 GB behind its first byte; only a window
    at its end is read."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    heads, max_seq = 8, 4_300_000  # codes: 2 * 8 * 4.3 M * 64 B = 4.4 GB, keys and values each past 2^31
    small = filled_cache(M, 61, heads, 416, 128)
    big = M.Kv4Cache(torch.empty(2, heads, max_seq, 64, dtype=torch.uint8, device="cuda"),
                     torch.empty(2, heads, max_seq, 8, dtype=torch.uint8, device="cuda"))
    big.codes[:, :, -416:] = small.codes
    big.scales[:, :, -416:] = small.scales
    q = randn(62, 16, 32, 128).bfloat16().cuda()
    got = M.msk_attention_kv4(q, big, max_seq - 16, window=300)
    check_attention(M, got, q, small, 400, 300, None)
    k, v = M.msk_kv4_read(big, max_seq - 20, 20)
    k2, v2 = M.msk_kv4_read(small, 396, 20)
    assert torch.equal(k, k2) and torch.equal(v, v2)


# ----------------------------------------------------------------------------
# products with 4-bit weights
# ----------------------------------------------------------------------------


def check_linear(y, x, packed, scales, ts):
    w = values64(packed.cpu(), scales.cpu(), ts)
    xx = x.cpu().double()
    ref, mag = xx @ w.t(), xx.abs() @ w.abs().t()
    t = y.dtype
    tol = half_step(t) * ref.abs() + (x.shape[1] + 64) * 2.0 ** -23 * mag + 1e-37
    if t == torch.float16:
        tol += 2.0 ** -25
    err = (y.cpu().double() - ref).abs()
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"error up to {worst:.2f} of the tolerance"
    # (errors of single outputs are far below their bound: the norm shows a systematic one)
    assert err.norm() <= (half_step(t) + 2.0 ** -17) * ref.norm() + 1e-30


LIN = [  # tokens, rows, cols, x type, y type
    (1, 16, 128, "bf16", "bf16"), (1, 1, 128, "bf16", "fp32"), (1, 4096, 4096, "bf16", "bf16"),
    (16, 6144, 4096, "bf16", "bf16"), (16, 1000, 4096, "bf16", "fp32"), (8, 2048, 1024, "fp16", "fp16"),
    (9, 333, 2048, "bf16", "bf16"), (5, 77, 384, "fp16", "fp32"), (16, 31, 8320, "bf16", "bf16"),
    (3, 5003, 640, "bf16", "bf16"), (2, 257, 16384, "bf16", "bf16"), (16, 65, 12288, "fp16", "fp16"),
    (16, 130, 32768, "bf16", "fp32"), (13, 40000, 256, "bf16", "bf16"), (7, 4864, 2176, "bf16", "fp32"),
    (16, 17800, 8320, "bf16", "fp32"), (1, 19600, 8576, "fp16", "bf16")]  # (clusters that take several tiles)


@pytest.mark.parametrize("T,N,K,xt,yt", LIN)
def test_linear(M, T, N, K, xt, yt):
    packed, scales = random_fp4(71, N, K)
    packed, scales = packed.cuda(), scales.cuda()
    x = randn(72, T, K)
    x[:, ::61] *= 30
    x = x.to(DT[xt]).cuda()
    w = M.Fp4Weight(packed, scales, 0.0125)
    y = torch.full((T, N), float("nan"), dtype=DT[yt], device="cuda")
    M.msk_linear_fp4(x, w, out=y)
    check_linear(y, x, packed, scales, 0.0125)
    assert torch.equal(y, M.msk_linear_fp4(x, w, out_dtype=DT[yt]))


def test_no_wait_has_run_out(M):
    """After whatever ran before in this process."""
    M.msk_ops_check()


def test_linear_strides_and_untouched_neighbours(M):
    packed, scales = random_fp4(73, 99, 256)
    w = M.Fp4Weight(packed.cuda(), scales.cuda())
    x = randn(74, 5, 2 * 256).bfloat16().cuda()[:, 256:]
    wide = torch.full((7, 120), 7.0, device="cuda")
    y = wide[1:6, 11:110]
    M.msk_linear_fp4(x, w, out=y)
    check_linear(y, x, packed, scales, 1.0)
    keep = torch.ones_like(wide, dtype=torch.bool)
    keep[1:6, 11:110] = False
    assert (wide[keep] == 7.0).all()


@pytest.mark.parametrize("xt,size", [("bf16", 1e-36), ("bf16", 1e30), ("fp16", 6e4), ("fp16", 1e-7)])
def test_linear_of_very_small_and_large_rows(M, xt, size):
    packed, scales = random_fp4(75, 48, 1024)
    x = randn(76, 4, 1024)
    x = x / x.abs().max() * size
    x[2] *= 1e-3
    x = x.to(DT[xt]).cuda()
    ts = 1.0 / size
    y = M.msk_linear_fp4(x, M.Fp4Weight(packed.cuda(), scales.cuda(), ts), out_dtype=torch.float32)
    check_linear(y, x, packed, scales, ts)


def test_linear_non_finite_rows_stay_apart(M):
    packed, scales = random_fp4(77, 64, 512)
    scales[5, 3] = 0x7F  # a NaN scale
    x = randn(78, 4, 512)
    x[1, 100] = float("inf")
    x[3, 7] = float("nan")
    x = x.bfloat16().cuda()
    y = M.msk_linear_fp4(x, M.Fp4Weight(packed.cuda(), scales.cuda()), out_dtype=torch.float32).cpu()
    assert torch.isnan(y[:, 5]).all() and torch.isnan(y[3]).all()
    assert not torch.isfinite(y[1]).any()
    ok = [r for r in range(64) if r != 5]
    assert torch.isfinite(y[0][ok]).all() and torch.isfinite(y[2][ok]).all()
    check_linear(y[[0, 2]][:, ok], x[[0, 2]], packed[ok], scales[ok], 1.0)


# ----------------------------------------------------------------------------
# log probabilities
# ----------------------------------------------------------------------------


def check_logprobs(got, logits, tokens, top, temperature):
    lp, ent, rank, ids, tlp = (None if g is None else g.cpu() for g in got)
    raw = logits.cpu().double()
    R, V = raw.shape
    x = raw / temperature
    ref = torch.log_softmax(x, -1)
    p = ref.exp()
    ent_ref = torch.special.entr(p).sum(-1)
    fin = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    slack = 2.0 ** -21 * (1 + 2 * fin) + (V / 512 + 64) * 2.0 ** -24

    def near(a, b, tol):
        a, b = a.double(), b.double()
        same = (a == b) | (torch.isnan(a) & torch.isnan(b))
        assert (same | ((a - b).abs() <= tol)).all(), f"off by {(a - b).abs()[~same].max().item():.3e}"

    # the entropy weights an error of x - lse by p and by p |x - lse|
    near(ent, ent_ref, slack * (2 + ref.masked_fill(p == 0, 0).abs().mul(p).sum(-1)))
    if tokens is not None:
        t = tokens.cpu().long()
        ok = (t >= 0) & (t < V)
        tt = t.clamp(0, V - 1).unsqueeze(1)
        near(torch.where(ok, lp, 0.0), torch.where(ok, ref.gather(1, tt).squeeze(1), 0.0), slack)
        assert (lp[~ok] == 0).all() and (rank[~ok] == -1).all()
        want = (raw > raw.gather(1, tt)).sum(-1)
        assert torch.equal(rank[ok].long(), want[ok])
    order = torch.sort(raw, dim=-1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(ids.long(), order)
    near(tlp, ref.gather(1, order), slack.unsqueeze(1))


LOGP = [  # rows, vocab, top, type, temperature
    (1, 1, 1, "fp32", 1.0), (1, 2, 0, "fp32", 0.5), (3, 1000, 5, "fp32", 1.0), (16, 131072, 8, "fp32", 0.7),
    (1, 32003, 32, "bf16", 1.0), (5, 50021, 20, "bf16", 1.3), (200, 4097, 32, "fp16", 1.0), (2, 33, 32, "bf16", 1.0),
    (700, 777, 3, "fp32", 1.0), (4, 262147, 20, "bf16", 1.0), (1, 1000003, 10, "fp32", 1.0), (320, 16384, 1, "bf16", 2.0)]


@pytest.mark.parametrize("R,V,top,dtype,temperature", LOGP)
def test_logprobs(M, R, V, top, dtype, temperature):
    x = randn(81, R, V) * 3
    x[torch.rand(R, V, generator=gen(82)) < 0.1] = float("-inf")
    x[:, V // 2] = 4.0
    x = x.to(DT[dtype])
    tokens = torch.randint(0, V, (R,), generator=gen(83), dtype=torch.int32)
    tokens[::3] = V // 2
    logits, tok = x.cuda(), tokens.cuda()
    got = M.msk_token_logprobs(logits, tok, top=top, temperature=temperature)
    check_logprobs(got, logits, tok, top, float(np.float32(temperature)))
    again = M.msk_token_logprobs(logits, tok, top=top, temperature=temperature)
    assert all(torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["constant", "rising", "falling", "steps", "two", "one", "zeros"])
def test_logprobs_of_ties_and_orders(M, kind, dtype):
    V = 40003
    i = torch.arange(V)
    x = {"constant": torch.full((V,), -3.0), "rising": i / 1000.0, "falling": -i / 1000.0,
         "steps": (i % 7).float(), "two": torch.where((i == 39999) | (i == 20001), 5.0, float("-inf")),
         "one": torch.where(i == 12345, 100.0, 0.0),
         "zeros": torch.where(i % 2 == 0, -0.0, 0.0)}[kind].to(DT[dtype]).repeat(3, 1)
    tok = torch.tensor([39999, -1, V], dtype=torch.int32).cuda()
    for R in (3, 1):
        check_logprobs(M.msk_token_logprobs(x[:R].cuda(), tok[:R], top=32), x[:R], tok[:R], 32, 1.0)


def test_logprobs_without_a_distribution(M):
    V = 3001
    x = randn(91, 6, V)
    x[1] = float("-inf")
    x[2, 7] = float("nan")
    x[3, 8] = float("inf")
    x[4, 1:] = float("-inf")
    tok = torch.tensor([3, 3, 3, 3, 0, 1], dtype=torch.int32)
    lp, ent, rank, ids, tlp = (g.cpu() for g in M.msk_token_logprobs(x.cuda(), tok.cuda(), top=4))
    for r in (1, 2, 3):
        assert torch.isnan(lp[r]) and torch.isnan(ent[r]) and torch.isnan(tlp[r]).all()
        assert ((ids[r] >= 0) & (ids[r] < V)).all()
    assert lp[4] == 0 and ent[4] == 0 and ids[4].tolist() == [0, 1, 2, 3] and tlp[4, 0] == 0 and tlp[4, 1] == float("-inf")
    check_logprobs([g[[0, 5]] for g in (lp, ent, rank, ids, tlp)], x[[0, 5]], tok[[0, 5]], 4, 1.0)


@pytest.mark.parametrize("R,V,top,dtype", [(640, 5003, 20, "bf16"), (1300, 8192, 32, "fp16"), (330, 40001, 32, "fp32"),
                                           (305, 70000, 0, "bf16"), (2500, 129, 9, "bf16"), (600, 4099, 1, "fp32"),
                                           (640, 35003, 20, "bf16"), (320, 17003, 32, "fp32"), (307, 300007, 32, "fp16")])
def test_logprobs_of_many_rows(M, R, V, top, dtype):
    x = (randn(98, R, V) * 4).to(DT[dtype])
    tokens = torch.randint(-1, V + 1, (R,), generator=gen(99), dtype=torch.int32)
    check_logprobs(M.msk_token_logprobs(x.cuda(), tokens.cuda(), top=top), x, tokens, top, 1.0)


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
@pytest.mark.parametrize("R,V", [(700, 6007), (620, 34007)])
def test_logprobs_of_many_rows_with_ties(M, dtype, R, V):
    i = torch.arange(V)
    kinds = [torch.full((V,), -3.0), i / 500.0, -i / 500.0, (i % 7).float(), (i // 100).float(),
             torch.where((i == 5999) | (i == 2001), 5.0, float("-inf")), torch.where(i == 1234, 100.0, 0.0),
             torch.where(i % 2 == 0, -0.0, 0.0), torch.where(i % 512 == 7, i / 1000.0, -9.0), randn(89, V).round()]
    x = torch.stack([kinds[r % len(kinds)] for r in range(R)]).to(DT[dtype])
    tokens = torch.randint(0, V, (R,), generator=gen(90), dtype=torch.int32)
    logits = x.cuda()
    for top in (32, 3):
        check_logprobs(M.msk_token_logprobs(logits, tokens.cuda(), top=top), x, tokens, top, 1.0)
    wide = torch.zeros(R, V + 5, dtype=DT[dtype], device="cuda")
    wide[:, 3:V + 3] = logits
    check_logprobs(M.msk_token_logprobs(wide[:, 3:V + 3], tokens.cuda(), top=32), x, tokens, 32, 1.0)


@pytest.mark.parametrize("dtype,size,temperature", [
    ("bf16", 1e6, 1.0), ("bf16", 1e6, 1e5), ("bf16", 1e37, 1.0), ("bf16", 1e-36, 1e-30), ("fp16", 2e4, 1.0), ("fp16", 2e4, 1e-5),
    ("fp16", 1e-6, 1e-7), ("fp32", 1e9, 1e-3), ("fp32", 1e20, 1e20), ("fp32", 1.0, 1e-30), ("fp32", 1.0, 1e30),
    ("bf16", 1e-3, 1e30)])
@pytest.mark.parametrize("R,V", [(2, 20011), (40, 1003), (310, 5001), (306, 34001)])
def test_logprobs_of_very_small_and_large_logits(M, dtype, size, temperature, R, V):
    x = (randn(95, R, V) * size).to(DT[dtype])
    x[:, 5::97] = float("-inf")
    x[0] -= size * 3
    tokens = torch.randint(0, V, (R,), generator=gen(96), dtype=torch.int32)
    got = M.msk_token_logprobs(x.cuda(), tokens.cuda(), top=9, temperature=temperature)
    check_logprobs(got, x, tokens, 9, float(np.float32(temperature)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R,V", [(5, 20001), (310, 34001)])
def test_logprobs_of_16_bits_without_a_distribution(M, dtype, R, V):
    x = randn(97, R, V).to(DT[dtype])
    x[1] = float("-inf")
    x[2, 7] = float("nan")
    x[3, 8] = float("inf")
    x[4, 1:] = float("-inf")
    tok = torch.zeros(R, dtype=torch.int32)
    lp, ent, rank, ids, tlp = (g.cpu() for g in M.msk_token_logprobs(x.cuda(), tok.cuda(), top=4))
    for r in (1, 2, 3):
        assert torch.isnan(lp[r]) and torch.isnan(ent[r]) and torch.isnan(tlp[r]).all()
        assert ((ids[r] >= 0) & (ids[r] < V)).all()
    assert torch.equal(rank.long(), (x > x[:, :1]).sum(-1))
    assert ids[3, 0] == 8
    assert lp[4] == 0 and ent[4] == 0 and ids[4].tolist() == [0, 1, 2, 3]


def test_logprobs_strides_and_missing_tokens(M):
    wide = randn(92, 9, 5011).cuda()
    logits = wide[1:8, 3:4999]  # rows that start off any 16-byte boundary
    got = M.msk_token_logprobs(logits, None, top=7)
    assert got[0] is None and got[2] is None
    check_logprobs(got, logits, None, 7, 1.0)
    half = randn(93, 4, 3007).bfloat16().cuda()[:, 1:]
    check_logprobs(M.msk_token_logprobs(half, None, top=5), half, None, 5, 1.0)


def test_logprobs_of_empty_batches(M):
    x = torch.empty(0, 100, device="cuda")
    lp, ent, rank, ids, tlp = M.msk_token_logprobs(x, torch.empty(0, dtype=torch.int32, device="cuda"), top=3)
    assert lp.shape == (0,) and ids.shape == (0, 3)
    packed, scales = random_fp4(94, 16, 128)
    w = M.Fp4Weight(packed.cuda(), scales.cuda())
    assert M.msk_linear_fp4(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), w).shape == (0, 16)
    cache = M.Kv4Cache.empty(1, 8, 64)
    k, v = M.msk_kv4_read(cache, 0, 0)
    M.msk_kv4_write(cache, k, v, 0)


# ----------------------------------------------------------------------------
# together, on streams, in graphs
# ----------------------------------------------------------------------------


class Tail:
    """A token block's way through the operators: new rows into the cache,
    attention, output projection, vocabulary head, log probabilities of the
    drafted tokens."""

    def __init__(self, M, T=16, hq=8, hkv=2, d=64, V=3001, max_seq=400):
        self.M, self.T = M, T
        self.cache = filled_cache(M, 101, hkv, max_seq, d)
        self.qkv = randn(102, T, (hq + 2 * hkv) * d).bfloat16().cuda()
        self.q = self.qkv[:, :hq * d].unflatten(1, (hq, d))
        self.k = self.qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        self.v = self.qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        self.w = [tuple(t.cuda() for t in random_fp4(103 + i, n, k)) for i, (n, k) in enumerate(((512, hq * d), (V, 512)))]
        self.wo, self.head = (M.Fp4Weight(p, s, 0.05) for p, s in self.w)
        self.tok = torch.randint(0, V, (T,), generator=gen(105), dtype=torch.int32).cuda()

    def run(self, pos, stream=None):
        M = self.M
        M.msk_kv4_write(self.cache, self.k, self.v, pos, stream=stream)
        o = M.msk_attention_kv4(self.q, self.cache, pos, window=100, stream=stream)
        h = M.msk_linear_fp4(o, self.wo, stream=stream)
        logits = M.msk_linear_fp4(h, self.head, out_dtype=torch.float32, stream=stream)
        return (o, h, logits) + M.msk_token_logprobs(logits, self.tok, top=4, stream=stream)

    def check(self, outs, pos):
        o, h, logits = outs[:3]
        check_attention(self.M, o, self.q.contiguous(), self.cache, pos, 100, None)
        check_linear(h, o, *self.w[0], 0.05)
        check_linear(logits, h, *self.w[1], 0.05)
        check_logprobs(outs[3:], logits, self.tok, 4, 1.0)


def test_a_run_of_them(M):
    t = Tail(M)
    for pos in (0, 200, 384):
        t.check(t.run(pos), pos)


def test_on_another_stream(M):
    t = Tail(M)
    want = t.run(250)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    junk = []
    got = t.run(250, stream=side)
    for _ in range(20):  # memory that the call let go of is not handed out under it
        junk.append(torch.full((1 << 20,), 3.0, device="cuda"))
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_captured_with_device_positions(M):
    t = Tail(M)
    pos = torch.tensor([100], dtype=torch.int32, device="cuda")
    t.run(pos)  # (first calls set attributes)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(t.run(pos))
        graphs.append(g)
    for p in (0, 37, 384):
        want = [x.clone() for x in t.run(p)]
        pos.fill_(p)
        for g, o in zip(graphs, outs):
            for x in o:
                x.zero_()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(want, o):
                assert torch.equal(a, b)


FIRST_CAPTURED = """
import torch
import moe_decode_step_persistent_gb300 as M
c = M.Kv4Cache.empty(2, 20000, 128)
kv = torch.randn(16, 2, 128, device="cuda").bfloat16()
q = torch.randn(16, 8, 128, device="cuda").bfloat16()
w = M.Fp4Weight(torch.full((1000, 512), 0x22, dtype=torch.uint8, device="cuda"),
                torch.full((1000, 64), 0x38, dtype=torch.uint8, device="cuda"))
x = torch.ones(16, 1024, device="cuda").bfloat16()
tok = torch.zeros(16, dtype=torch.int32, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    M.msk_kv4_write(c, kv, kv, 0)
    k, v = M.msk_kv4_read(c, 0, 16)
    o = [M.msk_attention_kv4(q[:t], c, n) for t in (1, 3, 16) for n in (0, 100, 15000)]
    y = [M.msk_linear_fp4(x[:t], w, out_dtype=torch.float32) for t in (1, 16)]
    lp = M.msk_token_logprobs(y[1], tok, top=4)
g.replay()
torch.cuda.synchronize()
assert all((t == 1024).all() for t in y) and (k.float() - kv.float()).abs().max() < 2
assert all(torch.isfinite(t).all() for t in o) and torch.isfinite(lp[0]).all()
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


@pytest.mark.parametrize("captured", [False, True])
def test_behind_an_event_of_another_stream(M, captured):
    """A call waits for what its stream waits for, whatever ran before it."""
    packed, scales = (t.cuda() for t in random_fp4(151, 512, 256))
    w = M.Fp4Weight(packed, scales)
    src = randn(152, 8, 16, 256).bfloat16().cuda()
    big = torch.zeros(1 << 26, device="cuda")
    x, side = torch.zeros(16, 256, dtype=torch.bfloat16, device="cuda"), torch.cuda.Stream()
    y = torch.zeros(8, 16, 512, dtype=torch.bfloat16, device="cuda")
    want = torch.stack([M.msk_linear_fp4(t, w) for t in src])
    torch.cuda.synchronize()

    def run():
        for i in range(8):
            M.msk_linear_fp4(x, w, out=y[i])  # (the kernel in front, of the same kind)
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                big.add_(1.0)  # tens of microseconds, then the input
                x.copy_(src[i])
            torch.cuda.current_stream().wait_stream(side)
            M.msk_linear_fp4(x, w, out=y[i])

    if captured:
        run()
        torch.cuda.synchronize()
        y.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        g.replay()
    else:
        run()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_around_a_step(M):
    """A verify step, its layers' bf16 caches turned into 4-bit ones and attended
    to, the step's hidden state through the head, the drafted tokens' log
    probabilities: enqueued without a wait in between."""
    import msk_synth as S
    from tests._gpu import Setup
    wl = S.scaled(S.WORKLOADS["tiny"], tokens=16, cached=300, windows=(8, 0))
    st = Setup(wl, gamma_std=0.1)
    kv, h = st.fresh_kv(), st.hidden()
    hkv, d, T = wl.n_kv_heads, wl.head_dim, wl.tokens
    q = randn(141, T, wl.n_q_heads, d).bfloat16().cuda()
    packed, scales = (t.cuda() for t in random_fp4(142, 777, wl.hidden))
    w = M.Fp4Weight(packed, scales, 0.02)
    tok = torch.randint(0, 777, (T,), generator=gen(143), dtype=torch.int32).cuda()
    st.model.decode_step(h, kv, [wl.cached + t for t in range(T)])
    outs = []
    for layer in range(wl.n_layers):
        cache = M.Kv4Cache.empty(hkv, wl.max_seq, d)
        k, v = (kv[layer, i].transpose(0, 1)[:wl.cached + T] for i in (0, 1))
        M.msk_kv4_write(cache, k, v, 0)
        outs.append((cache, M.msk_attention_kv4(q, cache, wl.cached, window=wl.windows[layer])))
    logits = M.msk_linear_fp4(h, w, out_dtype=torch.float32)
    got = M.msk_token_logprobs(logits, tok, top=5)
    for layer, (cache, out) in enumerate(outs):
        for i in (0, 1):
            c, e, _ = F.q4(kv[layer, i, :, :wl.cached + T].cpu().double().numpy())
            assert np.array_equal(cache.codes[i, :, :wl.cached + T].cpu().numpy(), pack(c).numpy())
            assert np.array_equal(cache.scales[i, :, :wl.cached + T].cpu().numpy(), e)
        check_attention(M, out, q, cache, wl.cached, wl.windows[layer], None)
    check_linear(logits, h, packed, scales, 0.02)
    check_logprobs(got, logits, tok, 5, 1.0)
    M.msk_ops_check()
    st.model.close()


@pytest.mark.parametrize("captured", [False, True])
def test_back_to_back(M, captured):
    """Kernels that start before the one in front of them has ended read and
    write as if they did not: the same buffers over and over, torch's kernels in
    between, against the same calls one at a time."""
    T, hq, hkv, d, N, V = 16, 8, 2, 64, 256, 9001
    packed, scales = (t.cuda() for t in random_fp4(131, N, hq * d))
    w = M.Fp4Weight(packed, scales, 0.03)
    packed, scales = (t.cuda() for t in random_fp4(132, V, N))
    head = M.Fp4Weight(packed, scales, 0.05)
    kv = randn(133, 6, T, hkv, d).bfloat16().cuda()
    tok = torch.randint(0, V, (T,), generator=gen(134), dtype=torch.int32).cuda()

    def chain(after):
        cache, q = filled_cache(M, 135, hkv, 9500, d), randn(136, T, hq, d).bfloat16().cuda()
        o, h = torch.zeros(T, hq * d, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
        logits = torch.zeros(T, V, device="cuda")
        start = q.clone()

        def run():
            got = []
            q.copy_(start), o.zero_(), h.zero_(), after()  # (a second run starts as the first one)
            for i in range(18):
                length = (40, 700, 9300)[i % 3]
                M.msk_kv4_write(cache, kv[i % 6], kv[(i + 1) % 6], length), after()
                M.msk_attention_kv4(q[:1 + 5 * (i % 4)], cache, length, out=o[:1 + 5 * (i % 4)]), after()
                M.msk_linear_fp4(o, w, out=h), after()
                if i % 2:
                    h.add_(1), after()
                M.msk_linear_fp4(h, head, out=logits), after()
                got += [t for t in M.msk_token_logprobs(logits, tok, top=3)]
                after()
                logits.fill_(float("nan")), after()
                q.copy_(o.view(T, hq, d)), after()
            got += [o.clone(), h.clone()]
            return got
        return run

    want = chain(torch.cuda.synchronize)()
    run = chain(lambda: None)
    if captured:
        run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run()
        g.replay(), g.replay()
    else:
        got = run()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))
    M.msk_ops_check()


def test_two_calls_at_once(M):
    """Calls on two streams, each with its own workspace, do not disturb each
    other."""
    a, b = Tail(M), Tail(M, T=5, hq=4, hkv=2, d=128, V=997)
    want = a.run(300), b.run(120)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):
        got.append((a.run(300, s1), b.run(120, s2)))
    torch.cuda.synchronize()
    for pair in got:
        for w, g in zip(want, pair):
            assert all(torch.equal(x, y) for x, y in zip(w, g))


def test_binding_refuses(M):
    cache = filled_cache(M, 111, 2, 64, 64)
    q = randn(112, 4, 4, 64).bfloat16().cuda()
    with pytest.raises(ValueError):
        M.msk_attention_kv4(q.cpu(), cache, 10)
    with pytest.raises(ValueError):
        M.msk_attention_kv4(q[..., :32], cache, 10)
    with pytest.raises(ValueError):
        M.msk_attention_kv4(q, cache, 10, parents=[-1, 0])
    with pytest.raises(ValueError):
        M.msk_attention_kv4(q, cache, 10, out=torch.empty(4, 256, device="cuda"))
    with pytest.raises(ValueError):
        M.msk_attention_kv4(q, cache, torch.tensor([10], device="cuda"))
    with pytest.raises(M.MskError):
        M.msk_attention_kv4(q, cache, 61)
    with pytest.raises(M.MskError):
        M.msk_attention_kv4(q, M.Kv4Cache.empty(2, 20000, 64), 19000,
                            workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        M.msk_kv4_write(cache, q, q, 0)
    with pytest.raises(M.MskError):
        M.msk_kv4_write(cache, q[:, :2], q[:, :2], 61)
    with pytest.raises(M.MskError):
        M.msk_kv4_read(cache, 60, 5)
    with pytest.raises(AttributeError):  # (the handle's tensors stay)
        cache.codes = cache.codes.clone()
    packed, scales = random_fp4(113, 32, 256)
    w = M.Fp4Weight(packed.cuda(), scales.cuda())
    with pytest.raises(AttributeError):
        w.packed = w.packed.clone()
    x = randn(114, 17, 256).bfloat16().cuda()
    with pytest.raises(M.MskError):
        M.msk_linear_fp4(x, w)
    with pytest.raises(ValueError):
        M.msk_linear_fp4(x[:4, :128], w)
    with pytest.raises(M.MskError):
        M.msk_linear_fp4(x[:4].float(), w)
    with pytest.raises(ValueError):
        M.msk_token_logprobs(x, torch.zeros(17, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        M.msk_token_logprobs(x, None, top=33)
    with pytest.raises(M.MskError):
        M.msk_token_logprobs(x, None, temperature=0.0)
