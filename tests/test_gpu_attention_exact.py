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

from tests.test_gpu_ops import DT, M, gen, half_step, randn, tree_parents, visible  # noqa: F401

pytestmark = pytest.mark.gpu

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def coded(M, k, v, k_scale=1.0, v_scale=1.0):
    """A cache of these E2M1 values ([heads][rows][d]), all block scales 1."""
    x = torch.stack((k, v)).cuda()
    code = torch.searchsorted(E2M1.cuda(), x.abs())
    assert torch.equal(E2M1.cuda()[code], x.abs())
    code = (code + 8 * (x < 0)).to(torch.uint8)
    c = M.Kv4Cache.empty(x.shape[1], x.shape[2], x.shape[3], k_scale, v_scale)
    c.codes.copy_(code[..., 0::2] | (code[..., 1::2] << 4))
    c.scales.fill_(0x38)
    return c


def seen_by(T, length, window, parents):
    """visible() without its loop over the cached rows."""
    see = torch.ones(T, length + T, dtype=torch.bool)
    depth = []
    own = visible(T, 0, window, parents)
    for t, p in enumerate([t - 1 for t in range(T)] if parents is None else parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        if window:
            see[t, :max(0, min(length, length + depth[t] - window + 1))] = False
        see[t, length:] = own[t]
    return see


def check(out, q, k, v, length, window=0, parents=None, terms=None, k_scale=1.0, v_scale=1.0, least=1.0):
    """out against the definition; k, v: values of at least length + T rows
    without the tensors' scales; least: the least sum of weights relative to the greatest."""
    T, hq, d = q.shape
    n = length + T
    k, v = (x[:, :n].to(out.device).double() * torch.tensor(s, dtype=torch.float32).double().item()
            for x, s in ((k, k_scale), (v, v_scale)))
    hkv, scale = k.shape[0], 1 / math.sqrt(d)
    qq = q.to(out.device).double().view(T, hkv, hq // hkv, d)
    see = seen_by(T, length, window, parents).to(out.device)[:, None, None, :]
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
    return o


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


# ----------------------------------------------------------------------------
# every visible row counts once
# ----------------------------------------------------------------------------


def counted_rows(T, hq, hkv, d, n, levels, seed, dtype):
    """q, k, v in which each 16 rows have a value of 1 in one dimension only, 16
    d rows on in the same one again, so that an output is the share of its
    dimension's rows: a row more or less of some hundred shows.  levels "flat": all
    weights equal, else scores that rise along the cache, or do not."""
    k, v = torch.zeros(hkv, n, d), torch.zeros(hkv, n, d)
    row = torch.arange(n)
    v[:, row, row // 16 % d] = 1.0
    if levels == "rising":
        k[:, :, 0] = E2M1[row * 8 // n]
    elif levels == "random":
        k[:, :, 0] = E2M1[torch.randint(0, 8, (n,), generator=gen(seed))]
    q = torch.zeros(T, hq, d)
    q[..., 0] = (torch.rand(T, hq, generator=gen(seed + 1)) * 4 - 2) * math.sqrt(d)
    return q.to(DT[dtype]), k, v


COUNT = [  # tokens, q heads, kv heads, head_dim, cached, window, tree, dtype
    (1, 4, 1, 64, 0, 0, False, "fp16"), (1, 4, 1, 64, 130, 0, False, "fp16"), (1, 8, 2, 128, 1151, 0, False, "fp16"),
    (2, 8, 2, 128, 8100, 0, False, "fp16"), (1, 4, 1, 128, 8200, 0, False, "fp16"), (1, 8, 8, 64, 30001, 0, False, "fp16"),
    (2, 32, 8, 128, 32768, 0, False, "fp16"), (1, 8, 2, 128, 65536, 0, False, "fp16"), (1, 8, 1, 128, 131000, 0, False, "fp16"),
    (1, 1, 1, 64, 131071, 0, False, "fp16"), (1, 4, 1, 128, 40000, 12345, False, "fp16"),
    (4, 8, 2, 128, 2290, 0, True, "fp16"), (4, 8, 2, 128, 2400, 0, True, "fp16"), (16, 8, 8, 64, 40003, 0, True, "fp16"),
    (8, 16, 8, 128, 16384, 3000, False, "fp16"), (16, 1, 1, 128, 70001, 0, False, "fp16"),
    (8, 8, 2, 128, 2200, 0, False, "fp16"), (16, 8, 2, 128, 2288, 0, True, "fp16"), (16, 8, 2, 128, 2500, 0, True, "fp16"),
    (16, 32, 8, 128, 16384, 2048, False, "fp16"), (7, 32, 8, 128, 33001, 0, True, "fp16"), (16, 8, 1, 64, 70001, 0, True, "fp16"),
    (6, 24, 2, 128, 70002, 0, True, "fp16"), (16, 32, 2, 64, 9001, 5000, False, "fp16"), (16, 32, 8, 128, 32768, 0, True, "bf16")]


@pytest.mark.parametrize("levels", ["flat", "rising", "random"])
@pytest.mark.parametrize("T,hq,hkv,d,length,window,tree,dtype", COUNT)
def test_every_row_counts_once(M, T, hq, hkv, d, length, window, tree, dtype, levels):
    n = length + T
    q, k, v = counted_rows(T, hq, hkv, d, n, levels, 31, dtype)
    cache = coded(M, torch.cat((k, torch.ones(hkv, 3, d)), 1), torch.cat((v, torch.ones(hkv, 3, d)), 1))
    parents = tree_parents(T, 32) if tree else None
    out = M.msk_attention_kv4(q.cuda(), cache, length, window=window, parents=parents)
    check(out, q, k, v, length, window, parents, terms=1)
    if levels == "flat":
        # weights are equal powers of two, their sums exact: the quotient and its rounding are left
        see = seen_by(T, length, window, parents).double()
        share = (see @ v[0].double()) / see.sum(-1, keepdim=True)
        err = (out.cpu().double().view(T, hq, d) - share[:, None]).abs()
        assert (err <= (half_step(q.dtype) + 2.0 ** -20) * share[:, None]).all()


def random_rows(T, hq, hkv, d, n, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def values(most):
        code = torch.randint(0, 2 * most, (hkv, n, d), generator=g, device="cuda")
        return E2M1.cuda()[code % most] * (1 - 2.0 * (code >= most))

    q = torch.randn(T, hq, d, generator=g, device="cuda") * 0.4
    return q.to(DT[dtype]), values(7), values(8)


@pytest.mark.parametrize("T,hq,hkv,d,length,tree,dtype", [
    (1, 32, 8, 128, 131071, False, "bf16"), (1, 8, 1, 128, 131000, False, "fp16"), (3, 8, 2, 64, 50001, True, "fp16"),
    (16, 8, 8, 128, 30001, False, "fp16"), (16, 8, 1, 64, 70001, True, "fp16"), (6, 24, 2, 128, 70002, True, "fp16"),
    (16, 32, 8, 128, 32768, False, "fp16")])
def test_long_caches(M, T, hq, hkv, d, length, tree, dtype):
    """Random keys and values over long caches: beside the bound of each output the norm
    of all errors, which grows with a bias but not with single roundings."""
    n = length + T
    q, k, v = random_rows(T, hq, hkv, d, n, 41, dtype)
    parents = tree_parents(T, 42) if tree else None
    out = M.msk_attention_kv4(q, coded(M, k, v), length, parents=parents)
    o = check(out, q, k, v, length, 0, parents)
    err = (out.double().view_as(o) - o).norm()
    # 2^-12: a warp's or a team's sums take up to 1100 additions, each off by 2^-23 of a part
    # of the sum; weights and scores are off by less.  (16 of 131000 rows lost: some 2^-6.)
    assert err <= (half_step(q.dtype) + 2.0 ** -12) * o.norm()


# ----------------------------------------------------------------------------
# layouts by ranges, with lengths on the device, on streams, in graphs
# ----------------------------------------------------------------------------


class Ranges:
    """A call over more keys than a cluster takes: ranges in a workspace, joined
    by a second kernel.  4, 12 or 64 query rows: each of the kernels."""

    def __init__(self, M, T, seed=51, max_seq=20000):
        self.M, self.T, self.max_seq = M, T, max_seq
        self.q, self.k, self.v = random_rows(T, 8, 2, 64, max_seq, seed, "bf16")
        self.cache = coded(M, self.k, self.v)
        self.bytes = M.msk_attention_kv4_workspace(T, 8, 2, 64, 0, max_seq - T)
        assert self.bytes > 0

    def run(self, length, **how):
        return self.M.msk_attention_kv4(self.q, self.cache, length, **how)

    def check(self, out, length):
        check(out, self.q, self.k, self.v, length)


@pytest.mark.parametrize("T", [1, 3, 16])
def test_lengths_on_the_device(M, T):
    """Most ranges are empty at short lengths; lengths out of range are clamped."""
    a = Ranges(M, T)
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    a.run(pos)
    graphs, outs = [], []
    for _ in range(2):  # (each graph has a workspace of its own)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(a.run(pos))
    ws = torch.full((a.bytes,), 0xFF, dtype=torch.uint8, device="cuda")  # (NaN whatever is read of it)
    last = a.max_seq - T
    for given, real in ((0, 0), (1, 1), (15, 15), (37, 37), (4097, 4097), (9000, 9000), (last - 1, last - 1), (last, last),
                        (-5, 0), (-2 ** 31, 0), (last + 1, last), (10 ** 6, last), (2 ** 31 - 1, last), (0, 0)):
        pos.fill_(given)
        ws.fill_(0xFF)
        eager = a.run(pos, workspace=ws)
        a.check(eager, real)
        for g, o in zip(graphs, outs):
            o.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, eager)
    a.check(a.run(9000), 9000)  # (another layout: by the length)


@pytest.mark.parametrize("window", [0, 9000])
def test_rows_behind_a_device_length_do_not_count(M, window):
    """Whatever lies behind the last row or before the window: NaN scales."""
    for T in (1, 3, 16):
        a = Ranges(M, T)
        length = 11000
        a.cache.scales[:, :, length + T:] = 0x7F
        if window:
            a.cache.scales[:, :, :length - window + 1] = 0x7F
        pos = torch.tensor([length], dtype=torch.int32, device="cuda")
        for how in (pos, length):
            check(a.run(how, window=window), a.q, a.k, a.v, length, window)


def test_ranges_on_two_streams_at_once(M):
    """Two calls with workspaces of their own, given or allocated."""
    a, b = Ranges(M, 16), Ranges(M, 3, seed=61)
    want = a.run(19000), b.run(15000)
    ws = [torch.full((x.bytes,), 0xFF, dtype=torch.uint8, device="cuda") for x in (a, b)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for i in range(20):
        given = (dict(workspace=ws[0]), dict(workspace=ws[1])) if i % 2 else ({}, {})
        got.append((a.run(19000, stream=s1, **given[0]), b.run(15000, stream=s2, **given[1])))
    torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


def test_a_call_s_workspace_is_not_handed_out_under_it(M):
    """The workspace that a call on a side stream allocates and lets go of when it
    returns: tensors of its size made meanwhile on the current stream lie elsewhere."""
    a = Ranges(M, 16)
    want = a.run(19000)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        got, junk = [], []
        for _ in range(8):
            got.append(a.run(19000, stream=side))
            for _ in range(2):
                junk.append(torch.full((a.bytes // 4,), float("nan"), device="cuda"))
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in got)
        del junk


def test_graphs_that_share_a_workspace_take_turns(M):
    """Two captured calls on one given workspace, replayed one after the other on one
    stream: nothing of a call's parts is left for the next."""
    a, b = Ranges(M, 16), Ranges(M, 1, seed=71)
    ws = torch.full((max(a.bytes, b.bytes),), 0xFF, dtype=torch.uint8, device="cuda")
    want = a.run(19000), b.run(12345)
    graphs, outs = [], []
    for x, n in ((a, 19000), (b, 12345)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(x.run(n, workspace=ws))
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
            o.zero_()
