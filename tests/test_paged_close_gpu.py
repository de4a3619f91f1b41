"""mxattn_paged_forward against the fp64 oracle, with the tolerance of tests/paged_parity.py: it knows only the keys that a
row sees, so the random bytes in the cache's unused slots (scale bytes up to 255) do not widen it."""
import numpy as np
import pytest
import torch

from mxfp4_microscaled_bit_quantize_b200 import api, build
from oracle import paged as op
from tests import paged_parity as pp
from tests import test_paged_gpu as base
from tests.test_paged_gpu import SHAPES, i32, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    return torch.device("cuda:0")


def attend(on, lens, causal, max_kv, with_lse=True):
    """(out, lse) of a call whose workspace, out and lse held something else before."""
    q, cache = on[0], on[1]
    (T, Hq, d), H, n = q.shape, cache.shape[1], max(n for _, n in lens)
    ws = torch.full((api.paged_workspace_size(T, len(lens), Hq, H, d, n, max_kv),), 0xFF, dtype=torch.uint8, device=q.device)
    out, lse = torch.full_like(q, 7.0), torch.full((T, Hq), 7.0, device=q.device) if with_lse else None
    api.mxattn_paged_forward(*on, max_new=n, max_kv=max_kv, causal=causal, workspace=ws, out=out, lse=lse)
    assert api.mxattn_check_status(ws) == 0
    return out, lse


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_shapes(dev, case):
    lens, causal, Hq, H, d, P = SHAPES[case]
    on, host = make(dev, lens, causal, Hq, H, d, P, seed=case)
    want = pp.expected(*host, causal)
    out, lse = attend(on, lens, causal, max(host[4]))
    pp.check(out, lse, want)
    assert torch.all(out[host[3][-1]:] == 7) and torch.all(lse[host[3][-1]:] == 7)       # rows of no request
    pp.check(attend(on, lens, causal, host[2].shape[1] * P, with_lse=False)[0], None, want)   # a looser bound


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,causal,Hq,H,P", [
    ([(2500, 70), (40, 70), (900, 3)], True, 4, 1, 64),      # one request in parts, the others in fewer or one
    ([(3000, 40), (7, 2)], True, 24, 2, 16),
    ([(2700, 33), (130, 33), (0, 33)], False, 6, 2, 32),
    ([(5000, 1), (37, 1), (0, 1)], True, 8, 2, 16),
    ([(2900, 4), (1500, 2)], False, 3, 3, 128)])
def test_contexts_in_parts(dev, d, lens, causal, Hq, H, P):
    on, host = make(dev, lens, causal, Hq, H, d, P, seed=d)
    n, bound = max(n for _, n in lens), max(host[4])
    assert api.paged_workspace_size(on[0].shape[0], len(lens), Hq, H, d, n, bound) > 256      # parts are laid out
    out, lse = attend(on, lens, causal, bound)
    pp.check(out, lse, pp.expected(*host, causal))
    again = attend(on, lens, causal, bound)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("n,causal", [(1, True), (3, True), (40, True), (1, False), (150, False)])
def test_bad_pages_and_lengths(dev, n, causal):
    lens = [(70 + n, n), (200, n), (40, n), (90, n)]
    on, host = make(dev, lens, True, 8, 2, 64, 16, seed=n)
    table, kv = host[2], np.array(host[4])
    table[0, 1] = -1
    table[1, :] = table.max() + 1000
    table[3, 0] = 2 ** 31 - 1
    kv[2], kv[3] = -5, 1 << 20
    out, lse = attend((on[0], on[1], i32(table, dev), on[3], i32(kv, dev)), lens, causal, 64)
    pp.check(out, lse, pp.expected(host[0], host[1], table, host[3], kv, causal, max_kv=64))


@pytest.mark.parametrize("n", [1, 2, 30])
def test_starts_outside(dev, n):
    on, host = make(dev, [(40, n + 3), (9, n + 3)], True, 4, 1, 128, 16, seed=n, tail=0)
    out = torch.full_like(on[0], 7.0)
    api.mxattn_paged_forward(on[0], on[1], on[2], i32([-4, n + 3, on[0].shape[0] + 50], dev), on[4], max_new=n, out=out)
    want, rows = pp.expected(*host, True), np.concatenate([np.arange(n), n + 3 + np.arange(n)])
    pp.check(out[rows], None, {k: x[rows] for k, x in want.items()})


@pytest.mark.parametrize("scale", [base._spread_values, base._large_values, base._small_values])
@pytest.mark.parametrize("n,Hq,H,d,P", [(1, 8, 2, 128, 16), (2, 6, 1, 64, 32), (37, 8, 2, 128, 32), (140, 2, 2, 64, 64)])
def test_value_ranges(dev, scale, n, Hq, H, d, P):
    lens = [(400, n), (65, n)]
    on, host = make(dev, lens, True, Hq, H, d, P, seed=n, scale=scale)
    pp.check(*attend(on, lens, True, 400 + n), pp.expected(*host, True))


@pytest.mark.parametrize("n,Hq,H", [(1, 64, 1), (2, 24, 1), (5, 33, 3)])
def test_large_groups(dev, n, Hq, H):
    lens = [(200, n), (17, n), (0, n)]
    on, host = make(dev, lens, True, Hq, H, 128, 32, seed=Hq)
    pp.check(*attend(on, lens, True, 200 + n), pp.expected(*host, True))


@pytest.mark.parametrize("n,bound", [(2, 512), (20, 512), (20, 5000)])
def test_replayed_for_other_lengths(dev, n, bound):
    on, host = make(dev, [(302 - n, n), (42 - n, n), (131 - n, n)], True, 8, 2, 128, 16, tail=0)
    q, cache, table, start, kv = on
    ws = torch.empty(api.paged_workspace_size(3 * n, 3, 8, 2, 128, n, bound), dtype=torch.uint8, device=dev)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=dev)

    def call():
        api.mxattn_paged_forward(q, cache, table, start, kv, max_new=n, max_kv=bound, workspace=ws, out=out, lse=lse)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for now in ([302, 42, 131], [17, 2, 100], [0, 42, 131]):
        kv.copy_(i32(now, dev))
        q.copy_(torch.randn_like(q))
        g.replay()
        torch.cuda.synchronize()
        pp.check(out, lse, pp.expected(q.cpu().double().numpy(), host[1], host[2], host[3], now, True))
    del g


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,Hq,H,exp", [
    ([(31, 1), (36, 1), (0, 1)], 4, 1, 118),                 # whole groups of 16 keys, and a partial one
    ([(31, 1), (15, 1), (700, 1)], 4, 2, 124),
    ([(29, 3), (60, 2)], 5, 1, 118),
    ([(5000, 1), (17, 1)], 8, 2, 118),                       # parts that are joined
    ([(31, 40), (80, 20)], 4, 2, 116),
    ([(700, 40)], 4, 2, 108)])
def test_values_near_the_top_of_the_range(dev, d, lens, Hq, H, exp):
    # |v| up to 2^(exp + 2): scale bytes of 241 and more from exp = 116 on
    on, host = make(dev, lens, True, Hq, H, d, 16, seed=exp, scale=lambda rng, k, v: (k, v * 2.0 ** exp))
    pp.check(*attend(on, lens, True, max(host[4])), pp.expected(*host, True))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("low,high", [(20, 120), (-100, 10), (100, 122)])
def test_values_of_far_scales_next_to_each_other(dev, d, low, high):
    # keys of two magnitudes, 2^100 or 2^22 apart, in the same groups of 16 keys and in groups of their own; the row sums
    # of the large ones alone would hide the small ones, so one request has small ones only behind its first key
    def scale(rng, k, v):
        v = v * np.exp2(np.where(rng.random(v.shape[:2] + (1,)) < 0.3, high, low))
        v[:16] *= 2.0 ** (low - high)
        return k, np.clip(v, -2.0 ** 122, 2.0 ** 122)

    lens = [(200, 2), (70, 1)]
    on, host = make(dev, lens, True, 4, 1, d, 32, seed=7, scale=scale)
    pp.check(*attend(on, lens, True, 202), pp.expected(*host, True))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 12])
@pytest.mark.parametrize("far", [5, 6, 7, 14, 60])
def test_small_probabilities_behind_an_outlier_of_v(dev, d, group, far):
    # One key dominates, a long flat tail of probabilities near 2^-16 adds up to a visible share, and one key without any
    # weight has values 2^far above all others. Many requests over the same pages, so that a context stays in one part and
    # a warp meets a quarter of the tail behind the outlier; the first 64 keys give every warp the same beginning.
    H, P, L, R = 8, 64, 2048, 300
    rng = np.random.default_rng(far)
    k, v = np.zeros((2, L, H, d))
    k[:, :, 1] = rng.choice([0, 0.5, 1, -0.5, -1], (L, H))
    v[:] = rng.choice([0.5, 1, 1.5, 1.5], (L, H, d))
    for first in (0, 16, 32, 48):
        k[first + 1, :, :2] = 3, 0                 # the dominating key, with small values of its own
        v[first + 1] *= 2.0 ** -3
        k[first + 2, :, :2] = -6, 0                # no weight
        v[first + 2] *= 2.0 ** far
    cache = np.zeros((L // P, H, 2, P, 17 * d // 32), dtype=np.uint8)
    op.append(cache, k, v, np.arange(L), 1)
    q = np.zeros((1, H * group, d))
    q[..., 0], q[..., 1] = (8 if d == 64 else 11.3125) * 3.8125, rng.choice([0.5, 1, 2], (1, H * group))
    table = np.arange(L // P)[None]
    q = torch.from_numpy(q).bfloat16()
    want = pp.expected(q.double().numpy(), cache, table, [0, 1], [L], True)
    qs = q.to(dev).expand(R, -1, -1)
    ws = torch.empty(api.paged_workspace_size(R, R, H * group, H, d, 1, L), dtype=torch.uint8, device=dev)
    assert ws.numel() == 256                       # one part
    lse = torch.zeros(R, H * group, device=dev)
    out = api.mxattn_paged_forward(qs, torch.from_numpy(cache).to(dev), i32(np.repeat(table, R, 0), dev), i32(np.arange(R + 1), dev), i32([L] * R, dev), 1,
                                   max_kv=L, workspace=ws, lse=lse)
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    pp.check(out[:1], lse[:1], want)


@pytest.mark.parametrize("lens", [[(50, 1), (20, 1), (3, 1)], [(40, 3), (9, 2)], [(90, 40), (7, 11)], [(4000, 2), (60, 2)], [(2500, 40), (30, 9)]])
def test_queries_of_nan_stay_in_their_rows(dev, lens):
    # out and lse of such a row are NaN (lse = -infinity means that a row has no key); every other row is as usual
    on, host = make(dev, lens, True, 8, 2, 128, 16, seed=3, tail=0)
    bad = [0, int(host[3][-1]) - 1]
    q = host[0].copy()
    q[bad[0], :, 5], q[bad[1]] = np.nan, np.nan
    out, lse = attend((torch.from_numpy(q).bfloat16().to(dev), *on[1:]), lens, True, max(host[4]))
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    want = pp.expected(*host, True)
    for x in want.values():
        x[bad] = np.nan
    pp.check(out, lse, want)


@pytest.mark.parametrize("lens,causal,Hq,H,d", [
    ([(1500, 100), (700, 90)], True, 8, 2, 128), ([(1400, 130)], True, 6, 6, 64), ([(900, 200)], False, 4, 2, 128),     # many rows a head
    ([(1500, 2)] * 24, True, 8, 4, 128), ([(1000, 1)] * 48, True, 8, 2, 64)])                                           # few
def test_dominating_keys_are_not_rounded(dev, lens, causal, Hq, H, d):
    # peaked rows: what the probability of the largest key costs would show in the norm of the error
    on, host = make(dev, lens, causal, Hq, H, d, 16, seed=d + Hq, scale=lambda rng, k, v: (3 * k, v))
    want = pp.expected(*host, causal)
    out, lse = attend(on, lens, causal, max(host[4]))
    pp.check(out, lse, want)
    n = int(host[3][-1])
    err = np.linalg.norm((out[:n].cpu().double().numpy() - want["out"][:n]).ravel())
    assert err <= 1.05 * pp.roundings(want), err / pp.roundings(want)


@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("exp", [-100, -60, 60, 105])
def test_keys_of_any_range(dev, n, exp):
    # |k| around 2^exp and queries around 2^-exp: ordinary scores
    lens = [(300, n), (33, n)]
    on, host = make(dev, lens, True, 8, 2, 128, 16, seed=n, tail=0, scale=lambda rng, k, v: (k * 2.0 ** exp, v))
    q = host[0] * 2.0 ** -exp
    out, lse = attend((torch.from_numpy(q).bfloat16().to(dev), *on[1:]), lens, True, 300 + n)
    pp.check(out, lse, pp.expected(q, *host[1:], True))
