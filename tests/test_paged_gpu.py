"""GPU parity of the paged MXFP4 KV cache: mxattn_cache_plan, mxattn_cache_append, mxattn_cache_read and
mxattn_paged_forward against the fp64 oracle.

Whole numbers, codes and read values have to be equal. Attention's tolerance, per element:
  |out - ref| <= 2^-8 |ref| + (2^-8 + 2 delta) sum_j p_j |v_j| + 2^-24 max|v|,
  delta = (d + 16) 2^-24 mass + 2^-19
The first term is the bf16 rounding of out (half a step, 2^-8 relative). Each p_j enters the product rounded to 8
significant bits or more (2^-8 relative, the row sum is not rounded). delta bounds the relative error of exp(s_j - m) and
of the row sum: a score of d products summed in fp32 is off by at most (d + 16) 2^-24 sum_c |q_c k_c| (mass; the d
roundings of the sum and those of the scale factors), and the exponential with its argument by 2^-19. The last term
covers probabilities below the smallest that the product's operand holds.
lse: |lse - ref| <= delta + 2^-22 |ref|.
"""
import numpy as np
import pytest
import torch

from mxfp4_microscaled_bit_quantize_b200 import _lib, api, build
from oracle import mxfp4 as mx
from oracle import paged as op

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    return torch.device("cuda:0")


def i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


# ------------------------------------------------------------------ plan

PLANS = [
    # ctx, new, width, free pages, P, max_tokens
    ([0], [1], 1, 1, 16, 1),
    ([16, 3, 47, 0, 0], [1, 2, 2, 17, 1], 3, 3, 16, 25),       # refusals: table width, then free pages
    ([5, 0, 31, 32, 33], [0, 0, 1, 1, 0], 4, 9, 32, 2),         # requests that sit out
    ([10, -1, 3], [4, 4, -2], 2, 5, 16, 20),                    # bad lengths
    ([0, 0, 0], [100, 100, 100], 20, 100, 16, 150),             # rows past max_tokens
    ([0, 17], [1 << 30, 1], 4, 10, 256, 40),
    ([2147483647, 3], [5, 5], 4, 10, 64, 40),                   # lengths whose sum passes 31 bits
    ([], [], 3, 4, 64, 5),
]


@pytest.mark.parametrize("case", range(len(PLANS)))
def test_plan(dev, case):
    ctx, new, width, n_free, P, T = PLANS[case]
    rng = np.random.default_rng(case)
    pages = rng.permutation(1000)
    table = np.full((len(ctx), width), -7)
    for r, c in enumerate(ctx):
        held = min(width, -(-max(c, 0) // P))
        table[r, :held] = pages[100 * (r + 1):100 * (r + 1) + held]
    _check_plan(dev, ctx, new, table, pages[:n_free], P, T)


def _check_plan(dev, ctx, new, table, free, P, T):
    got_table = i32(table, dev)
    start, kv, slots, info = api.mxattn_cache_plan(i32(ctx, dev), i32(new, dev), got_table, i32(free, dev), P, T)
    want = op.plan(ctx, new, table, list(free), P, T)
    for a, b, name in zip((got_table, start, kv, slots, info), want, ("table", "q_start", "kv_len", "slots", "info")):
        assert np.array_equal(a.cpu().numpy(), b), name


@pytest.mark.parametrize("R,ctx,new,P,short", [(1, 0, 1, 16, 0), (513, 300, 1, 16, 0), (1500, 40, 9, 32, 0), (1024, 100, 60, 64, 0), (700, 90, 40, 16, 800)])
def test_plan_many(dev, R, ctx, new, P, short):
    rng = np.random.default_rng(R)
    c, n = rng.integers(0, ctx + 1, R), rng.integers(0, new + 1, R)
    held, full = -(-c // P), -(-(c + n) // P)
    pool = rng.permutation(int(full.sum()) + 3)
    width = int(full.max()) + 1
    table = np.full((R, width), -1)
    for r in range(R):
        table[r, :held[r]] = pool[held[:r].sum():held[:r].sum() + held[r]]
    free = pool[held.sum():len(pool) - short]
    _check_plan(dev, c.tolist(), n.tolist(), table, free, P, int(n.sum()) + 5)


# ------------------------------------------------------------------ append and read

def rows(rng, T, H, d):
    x = rng.standard_normal((T, H, d)) * np.exp2(rng.integers(-6, 7, (T, H, 1)))
    x[rng.random(x.shape) < 0.01] *= 40
    x[rng.random((T, H)) < 0.05] = 0
    return torch.from_numpy(x).bfloat16()


@pytest.mark.parametrize("T,H,d,P,mode", [(1, 1, 64, 16, 1), (1, 8, 128, 16, 0), (77, 3, 64, 32, 1), (130, 5, 128, 64, 1), (33, 2, 128, 256, 0), (257, 7, 64, 128, 0)])
def test_append_and_read(dev, T, H, d, P, mode):
    rng = np.random.default_rng(T)
    n_pages = -(-T // P) + 2
    k, v = rows(rng, T, H, d), rows(rng, T, H, d)
    slots = rng.permutation(n_pages * P)[:T]
    slots[T // 2] = [-1, n_pages * P, -(1 << 40), 1 << 40][T % 4]      # outside: skipped
    cache = torch.from_numpy(rng.integers(0, 256, (n_pages, H, 2, P, 17 * d // 32), dtype=np.uint8))
    want = cache.numpy().copy()
    op.append(want, k.double().numpy(), v.double().numpy(), slots, mode)
    cache = cache.to(dev)
    s = torch.from_numpy(slots).to(dev)
    api.mxattn_cache_append(k.to(dev), v.to(dev), s, cache, scale_mode=mode)
    assert np.array_equal(cache.cpu().numpy(), want)                   # the other tokens' bytes included
    got = api.mxattn_cache_read(cache, s)
    for a, b in zip(got, op.read(want, slots)):
        assert np.array_equal(a.cpu().double().numpy(), b)


def test_append_from_strided_rows(dev):
    # K and V inside one projection's rows, V not 16-byte aligned: [T, (Hq + 2 Hkv) d + 3]
    rng = np.random.default_rng(4)
    T, H, d, P = 19, 2, 128, 16
    x = torch.from_numpy(rng.standard_normal((T, 6 * d + 8))).bfloat16().to(dev)
    k = x[:, 2 * d:4 * d].unflatten(1, (H, d))
    v = x[:, 4 * d + 3:6 * d + 3].unflatten(1, (H, d))
    cache = api.cache_alloc(2, H, d, P, dev)
    slots = torch.arange(5, 5 + T, device=dev)
    api.mxattn_cache_append(k, v, slots, cache)
    want = np.zeros(tuple(cache.shape), dtype=np.uint8)
    op.append(want, k.cpu().double().numpy(), v.cpu().double().numpy(), slots.cpu().numpy(), 1)
    assert np.array_equal(cache.cpu().numpy(), want)
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)                # heads before tokens
    api.mxattn_cache_append(kt, v, slots, cache)
    assert np.array_equal(cache.cpu().numpy(), want)


def test_append_extreme_values(dev):
    # the smallest and largest bf16 blocks: subnormals, the top binade, and zeros of both signs
    H, d, P = 1, 64, 16
    x = torch.zeros(6, H, d)
    x[0, 0, 0] = 2.0 ** -133
    x[1] = 2.0 ** -126
    x[2, 0, 5] = 3.0e38
    x[3] = -0.0
    x[4, 0, :32] = 3e38 * torch.linspace(-1, 1, 32)      # not linspace(-3e38, 3e38): its range overflows to infinity
    x[5, 0, 32:] = torch.linspace(-1e-38, 1e-38, 32)
    x = x.bfloat16()
    for mode in (0, 1):
        cache = api.cache_alloc(1, H, d, P, dev)
        slots = torch.arange(6, device=dev)
        api.mxattn_cache_append(x.to(dev), x.to(dev), slots, cache, scale_mode=mode)
        want = np.zeros(tuple(cache.shape), dtype=np.uint8)
        op.append(want, x.double().numpy(), x.double().numpy(), slots.cpu().numpy(), mode)
        assert np.array_equal(cache.cpu().numpy(), want)
        k, v = api.mxattn_cache_read(cache, slots)
        ref = torch.from_numpy(op.read(want, slots.cpu().numpy())[0]).bfloat16()
        assert torch.equal(k.cpu(), ref) and torch.equal(v.cpu(), ref)


def test_cache_past_32_bit_offsets(dev):
    # 4.6 GB of pages: the last pages lie past 2^32 bytes
    H, d, P = 8, 128, 256
    n_pages = (46 << 28) // 10 * 4 // (H * 2 * P * 68)
    cache = torch.empty(n_pages, H, 2, P, 68, dtype=torch.uint8, device=dev)
    assert cache.numel() > 1 << 32
    rng = np.random.default_rng(6)
    T = 300
    k, v = rows(rng, T, H, d), rows(rng, T, H, d)
    first = (n_pages - 2) * P
    slots = torch.arange(first, first + T, device=dev)
    api.mxattn_cache_append(k.to(dev), v.to(dev), slots, cache)
    small = np.zeros((2, H, 2, P, 68), dtype=np.uint8)
    op.append(small, k.double().numpy(), v.double().numpy(), np.arange(T), 1)
    for a, b in zip(api.mxattn_cache_read(cache, slots), op.read(small, np.arange(T))):
        assert np.array_equal(a.cpu().double().numpy(), b)
    q = torch.from_numpy(rng.standard_normal((1, 2 * H, d))).bfloat16()
    out = api.mxattn_paged_forward(q.to(dev), cache, i32([[n_pages - 2, n_pages - 1]], dev), i32([0, 1], dev), i32([T], dev), 1)
    _close(out, None, op.attention(q.double().numpy(), small, np.array([[0, 1]]), [0, 1], [T], True), q, small)


# ------------------------------------------------------------------ attention

def _close(out, lse, want, q, cache):
    ref, ref_lse, spread, mass = want
    d = ref.shape[-1]
    vmax = np.abs(op.read(cache, np.arange(cache.shape[0] * cache.shape[3]))[1]).max(initial=0)
    rows = ~np.isnan(ref[:, 0, 0])
    delta = (d + 16) * 2.0 ** -24 * mass + 2.0 ** -19
    got = out.cpu().double().numpy()
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * delta[..., None]) * spread + 2.0 ** -24 * vmax
    err = np.abs(got - ref)[rows]
    assert np.all(err <= tol[rows]), (float(err.max()), float((err / np.maximum(tol[rows], 1e-300)).max()))
    if lse is not None:
        got = lse.cpu().double().numpy()[rows]
        empty = np.isneginf(ref_lse[rows])
        assert np.array_equal(empty, np.isneginf(got))
        err = np.abs(got[~empty] - ref_lse[rows][~empty])
        lim = (delta + 2.0 ** -22 * np.abs(np.where(np.isfinite(ref_lse), ref_lse, 0)))[rows][~empty]
        assert np.all(err <= lim), float((err / lim).max())


def make(dev, lens, causal, Hq, H, d, P, seed=0, garbage=True, scale=None, extra=2, tail=3):
    """Inputs of one call: (q, cache, table, q_start, kv_len) on the device, and their numpy forms. The cache's unused
    slots hold random bytes, the rows behind the last request random values."""
    rng = np.random.default_rng(seed)
    total = [c + n if causal else c for c, n in lens]
    count = [-(-t // P) for t in total]
    width = max(max(count), 1) + extra
    n_pages = sum(count) + 4
    pool = rng.permutation(n_pages)
    cache = rng.integers(0, 256, (n_pages, H, 2, P, 17 * d // 32), dtype=np.uint8) if garbage else np.zeros((n_pages, H, 2, P, 17 * d // 32), dtype=np.uint8)
    table = rng.integers(-3, n_pages + 3, (len(lens), width))
    for r, t in enumerate(total):
        mine = pool[sum(count[:r]):sum(count[:r + 1])]
        table[r, :count[r]] = mine
        pos = np.arange(t)
        k, v = rng.standard_normal((2, t, H, d))
        if scale is not None:
            k, v = scale(rng, k, v)
        k, v = (torch.from_numpy(x).bfloat16().double().numpy() for x in (k, v))
        op.append(cache, k, v, mine[pos // P] * P + pos % P, 1)
    new = [n for _, n in lens]
    start = np.concatenate([[0], np.cumsum(new)])
    q = torch.from_numpy(rng.standard_normal((int(start[-1]) + tail, Hq, d)) * 1.5).bfloat16()
    on = (q.to(dev), torch.from_numpy(cache).to(dev), i32(table, dev), i32(start, dev), i32(total, dev))
    return on, (q.double().numpy(), cache, table, start, total)


SHAPES = [
    # (context, new) of each request, causal, Hq, Hkv, d, P
    ([(0, 1)], True, 1, 1, 64, 16),
    ([(0, 1)], True, 8, 1, 128, 16),
    ([(15, 1), (16, 1), (17, 1), (0, 1)], True, 4, 2, 128, 16),
    ([(1000, 1)], True, 32, 8, 128, 16),
    ([(63, 1), (300, 1), (0, 0), (511, 1)], True, 5, 1, 64, 32),
    ([(700, 1), (33, 1)], True, 14, 2, 128, 128),
    ([(100, 1), (2000, 1)], True, 48, 3, 64, 256),              # 16 heads a group
    ([(90, 4), (1, 3), (0, 2), (255, 4)], True, 8, 2, 128, 64),
    ([(90, 7), (12, 0), (40, 5)], True, 6, 6, 64, 16),
    ([(500, 17), (130, 33), (0, 40)], True, 8, 2, 128, 16),
    ([(0, 129)], True, 4, 1, 128, 32),
    ([(257, 200), (0, 1), (31, 77)], True, 15, 3, 64, 64),
    ([(0, 300)], True, 2, 2, 128, 128),
    ([(77, 50), (1, 50), (0, 50), (128, 50)], False, 3, 3, 64, 16),
    ([(512, 260)], False, 2, 2, 128, 64),
    ([(3, 1), (40, 1)], False, 4, 1, 128, 32),
    ([(300, 9), (129, 130)], False, 7, 1, 128, 16),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_paged_forward(dev, case):
    lens, causal, Hq, H, d, P = SHAPES[case]
    on, host = make(dev, lens, causal, Hq, H, d, P, seed=case)
    T = on[0].shape[0]
    out = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((T, Hq), 7.0, device=dev)
    max_new, max_kv = max(n for _, n in lens), max(host[4])
    ws = torch.full((api.paged_workspace_size(T, len(lens), Hq, H, d, max_new, max_kv),), 0xFF, dtype=torch.uint8, device=dev)
    api.mxattn_paged_forward(*on, max_new=max_new, max_kv=max_kv, causal=causal, workspace=ws, out=out, lse=lse)
    assert api.mxattn_check_status(ws) == 0
    _close(out, lse, op.attention(*host, causal), on[0], host[1])
    assert torch.all(out[host[3][-1]:] == 7) and torch.all(lse[host[3][-1]:] == 7)       # rows of no request
    again = api.mxattn_paged_forward(*on, max_new=max_new, causal=causal)                # bounds from the table, no lse
    _close(again, None, op.attention(*host, causal), on[0], host[1])


@pytest.mark.parametrize("n,causal", [(1, True), (3, True), (40, True), (1, False), (150, False)])
def test_paged_bad_pages_and_lengths(dev, n, causal):
    # pages that are not there (outside the pool) are no keys; lengths past the table or max_kv are cut; a negative one is 0
    lens = [(70 + n, n), (200, n), (40, n), (90, n)]
    on, host = make(dev, lens, True, 8, 2, 64, 16, seed=n)
    table = host[2]
    table[0, 1] = -1
    table[1, :] = table.max() + 1000
    table[3, 0] = 2 ** 31 - 1
    kv = np.array(host[4])
    kv[2] = -5
    kv[3] = 1 << 20
    on = (on[0], on[1], i32(table, dev), on[3], i32(kv, dev))
    cut = 64
    lse = torch.zeros(on[0].shape[:2], device=dev)
    out = api.mxattn_paged_forward(*on, max_new=n, max_kv=cut, causal=causal, lse=lse)
    want = op.attention(host[0], host[1], table, host[3], kv, causal, max_kv=cut)
    _close(out, lse, want, on[0], host[1])
    assert torch.all(out[int(host[3][1]):int(host[3][3])] == 0)


@pytest.mark.parametrize("n", [1, 2, 30])
def test_paged_starts_outside(dev, n):
    # q_start values outside [0, T] are clamped, and rows past max_new are left as they were
    on, host = make(dev, [(40, n + 3), (9, n + 3)], True, 4, 1, 128, 16, seed=n, tail=0)
    T = on[0].shape[0]
    start = np.array([-4, n + 3, T + 50])
    out = torch.full((T, 4, 128), 7.0, dtype=torch.bfloat16, device=dev)
    api.mxattn_paged_forward(on[0], on[1], on[2], i32(start, dev), on[4], max_new=n, out=out)
    full = op.attention(*host, True)
    rows = np.concatenate([np.arange(n), n + 3 + np.arange(n)])
    _close(out[rows], None, [x[rows] for x in full], on[0], host[1])
    rest = np.setdiff1d(np.arange(T), rows)
    assert torch.all(out[rest] == 7)


def _spread_values(rng, k, v):
    # block scales of V over 2^20 and of K over 2^12 within a request, some K rows that dominate, some zero rows
    k = k * np.exp2(rng.integers(-8, 5, k.shape[:2] + (1,)))
    v = v * np.exp2(rng.integers(-10, 11, v.shape[:2] + (1,)))
    v[rng.random(v.shape[:2]) < 0.1] = 0
    k[rng.random(k.shape[:2]) < 0.1] = 0
    return k, v


def _large_values(rng, k, v):
    return k * 2.0 ** -40, v * 2.0 ** 60


def _small_values(rng, k, v):
    return k * 2.0 ** 12, v * 2.0 ** -70


@pytest.mark.parametrize("scale", [_spread_values, _large_values, _small_values])
@pytest.mark.parametrize("n,Hq,H,d,P", [(1, 8, 2, 128, 16), (2, 6, 1, 64, 32), (37, 8, 2, 128, 32), (140, 2, 2, 64, 64)])
def test_paged_value_ranges(dev, scale, n, Hq, H, d, P):
    on, host = make(dev, [(400, n), (65, n)], True, Hq, H, d, P, seed=n, scale=scale)
    out = api.mxattn_paged_forward(*on, max_new=n)
    _close(out, None, op.attention(*host, True), on[0], host[1])


def test_paged_strided_queries(dev):
    on, host = make(dev, [(100, 3), (37, 2)], True, 6, 2, 128, 16, tail=0)
    qkv = torch.randn(5, 6 * 128 + 2 * 2 * 128 + 8, dtype=torch.bfloat16, device=dev)
    qkv[:, 8:8 + 768] = on[0].flatten(1)
    q = qkv[:, 8:8 + 768].unflatten(1, (6, 128))
    want = api.mxattn_paged_forward(*on, max_new=3)
    assert torch.equal(api.mxattn_paged_forward(q, *on[1:], max_new=3), want)
    qt = on[0].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(api.mxattn_paged_forward(qt, *on[1:], max_new=3), want)


@pytest.mark.parametrize("lens,Hq,H", [([(5000, 1), (37, 1)], 8, 2), ([(3000, 2)], 4, 4), ([(2500, 70)], 4, 1)])
def test_paged_long_contexts_are_repeatable(dev, lens, Hq, H):
    # contexts long enough to be split over many blocks: within tolerance, and the same bits every time
    on, host = make(dev, lens, True, Hq, H, 128, 64, seed=9, garbage=False)
    n = max(x for _, x in lens)
    lse = torch.zeros(on[0].shape[:2], device=dev)
    out = api.mxattn_paged_forward(*on, max_new=n, max_kv=max(host[4]), lse=lse)
    _close(out, lse, op.attention(*host, True), on[0], host[1])
    rows = int(host[3][-1])
    for _ in range(5):
        assert torch.equal(api.mxattn_paged_forward(*on, max_new=n, max_kv=max(host[4]))[:rows], out[:rows])


@pytest.mark.parametrize("n,bound", [(2, 512), (20, 512), (20, 5000)])
def test_paged_captured_calls_share_a_workspace(dev, n, bound):
    # two graphs over one workspace, replayed in turn for lengths and queries that changed after the capture
    lens = [(302 - n, n), (42 - n, n), (131 - n, n)]
    on, host = make(dev, lens, True, 8, 2, 128, 16, tail=0)
    q, cache, table, start, kv = on
    ws = torch.empty(api.paged_workspace_size(3 * n, 3, 8, 2, 128, n, bound), dtype=torch.uint8, device=dev)
    outs = [torch.zeros_like(q) for _ in range(2)]
    graphs = []
    for i, causal in enumerate((True, False)):
        api.mxattn_paged_forward(q, cache, table, start, kv, max_new=n, max_kv=bound, causal=causal, workspace=ws, out=outs[i])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.mxattn_paged_forward(q, cache, table, start, kv, max_new=n, max_kv=bound, causal=causal, workspace=ws, out=outs[i])
        graphs.append(g)
    for kv_now in ([302, 42, 131], [17, 2, 100], [0, 42, 131]):
        kv.copy_(i32(kv_now, dev))
        q.copy_(torch.randn_like(q))
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        for causal, out in zip((True, False), outs):
            _close(out, None, op.attention(q.cpu().double().numpy(), host[1], host[2], host[3], kv_now, causal), q, host[1])
    del graphs


def test_paged_on_another_stream(dev):
    on, host = make(dev, [(600, 1), (90, 1)], True, 8, 2, 64, 16, tail=0)
    st = torch.cuda.Stream(dev)
    st.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(st):
        out = api.mxattn_paged_forward(*on, max_new=1)
    st.synchronize()
    _close(out, None, op.attention(*host, True), on[0], host[1])


@pytest.mark.parametrize("n,Hq,H", [(1, 64, 1), (2, 24, 1), (5, 33, 3)])
def test_paged_large_groups(dev, n, Hq, H):
    # 64, 48 and 55 rows a KV head: few tokens, but more rows than the small kernel takes
    on, host = make(dev, [(200, n), (17, n), (0, n)], True, Hq, H, 128, 32, seed=Hq)
    _close(api.mxattn_paged_forward(*on, max_new=n), None, op.attention(*host, True), on[0], host[1])


@pytest.mark.parametrize("n", [1, 60])
def test_paged_two_calls_at_once(dev, n):
    # two streams, a workspace each: the same bits as one after the other
    calls = [make(dev, [(1500, n), (90, n)], True, 8, 2, 128, 16, seed=s, garbage=False, tail=0)[0] for s in (1, 2)]
    want = [api.mxattn_paged_forward(*on, max_new=n) for on in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in calls]
    got = []
    for st, on in zip(streams, calls):
        with torch.cuda.stream(st):
            got.append([api.mxattn_paged_forward(*on, max_new=n) for _ in range(8)])
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert all(torch.equal(o, w) for o in outs)


@pytest.mark.parametrize("n", [1, 24])
def test_result_is_there_for_the_next_launch(dev, n):
    # a bound on the lengths that plans for splits, and lengths that need none: the joining launch has nothing to do
    # and must not let the stream go on before the parts' launch has ended
    R, H, Hq, P, L = 16, 2, 8, 64, 6000
    g = torch.Generator(device=dev).manual_seed(1)
    pages = R * -(-L // P)
    cache = torch.randint(0, 256, (pages, H, 2, P * 68), generator=g, device=dev, dtype=torch.uint8)
    cache[..., P * 64:] = 126
    cache = cache.view(pages, H, 2, P, 68)
    table = torch.arange(pages, dtype=torch.int32, device=dev).view(R, -1)
    q = torch.randn(R * n, Hq, 128, generator=g, device=dev).bfloat16()
    start, kv = torch.arange(0, R * n + 1, n, dtype=torch.int32, device=dev), torch.full((R,), L, dtype=torch.int32, device=dev)
    ws = torch.empty(api.paged_workspace_size(R * n, R, Hq, H, 128, n, 1 << 20), dtype=torch.uint8, device=dev)
    assert ws.numel() > 256
    for _ in range(20):
        out = torch.zeros_like(q)
        api.mxattn_paged_forward(q, cache, table, start, kv, max_new=n, max_kv=1 << 20, workspace=ws, out=out)
        seen = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(seen, out) and bool((out != 0).any())


def test_empty_calls(dev):
    cache = api.cache_alloc(3, 2, 64, 16, dev)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=dev)
    slots = torch.empty(0, dtype=torch.int64, device=dev)
    api.mxattn_cache_append(none, none, slots, cache)
    assert api.mxattn_cache_read(cache, slots)[0].shape == (0, 2, 64)
    table = torch.zeros(0, 4, dtype=torch.int32, device=dev)
    start, kv, sl, info = api.mxattn_cache_plan(i32([], dev), i32([], dev), table, i32([1], dev), 16, 0)
    assert start.tolist() == [0] and info.tolist() == [0, 0, 0, 0] and sl.numel() == 0
    assert api.mxattn_paged_forward(none, cache, table, start, kv, max_new=0).shape == (0, 2, 64)
    # a pool without pages and a table without columns: no keys, zeros
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device=dev)
    for n in (1, 3):
        for c, tab in ((cache[:0], torch.zeros(1, 4, dtype=torch.int32, device=dev)), (cache, torch.zeros(1, 0, dtype=torch.int32, device=dev))):
            out = api.mxattn_paged_forward(q[:n], c, tab, i32([0, n], dev), i32([40], dev), max_new=n)
            assert torch.all(out == 0)


def test_captured_step_for_changing_batches(dev):
    # plan, append and attend captured once with padded rows, replayed for batches that change on the device
    H, Hq, d, P, width, T = 2, 8, 64, 16, 8, 6
    rng = np.random.default_rng(3)
    cache = api.cache_alloc(30, H, d, P, dev)
    ctx, new = torch.zeros(3, dtype=torch.int32, device=dev), torch.ones(3, dtype=torch.int32, device=dev)
    table = torch.full((3, width), -1, dtype=torch.int32, device=dev)
    free = i32(rng.permutation(30), dev)
    outs = (torch.zeros(4, dtype=torch.int32, device=dev), torch.zeros(3, dtype=torch.int32, device=dev),
            torch.zeros(T, dtype=torch.int64, device=dev), torch.zeros(4, dtype=torch.int32, device=dev))
    qkv = torch.zeros(T, Hq + 2 * H, d, dtype=torch.bfloat16, device=dev)
    out = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=dev)
    ws = torch.empty(api.paged_workspace_size(T, 3, Hq, H, d, 2, width * P), dtype=torch.uint8, device=dev)

    def step():
        api.mxattn_cache_plan(ctx, new, table, free, P, T, out=outs)
        api.mxattn_cache_append(qkv[:, Hq:Hq + H], qkv[:, Hq + H:], outs[2], cache)
        api.mxattn_paged_forward(qkv[:, :Hq], cache, table, outs[0], outs[1], max_new=2, max_kv=width * P, workspace=ws, out=out)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    cache.zero_()
    table.fill_(-1)
    host, host_table, pages, lens = np.zeros(tuple(cache.shape), dtype=np.uint8), np.full((3, width), -1), rng.permutation(30), [0, 0, 0]
    for n in ([2, 1, 2], [1, 0, 2], [2, 2, 2], [0, 1, 0]) * 5:
        ctx.copy_(i32(lens, dev))
        new.copy_(i32(n, dev))
        free.copy_(i32(np.concatenate([pages, np.full(30 - len(pages), -1)]), dev))
        x = torch.from_numpy(rng.standard_normal(tuple(qkv.shape))).bfloat16()
        qkv.copy_(x)
        g.replay()
        host_table, start, kv, slots, info = op.plan(lens, n, host_table, list(pages), P, T)
        assert np.array_equal(outs[2].cpu().numpy(), slots) and np.array_equal(table.cpu().numpy(), host_table)
        op.append(host, x[:, Hq:Hq + H].double().numpy(), x[:, Hq + H:].double().numpy(), slots, 1)
        assert np.array_equal(cache.cpu().numpy(), host)
        _close(out, None, op.attention(x[:, :Hq].double().numpy(), host, host_table, start, kv, True), None, host)
        pages, lens = pages[int(info[1]):], kv.tolist()
    del g


def test_serving_steps_together(dev):
    # plan, append and attend as a server runs them: two prompts in chunks, then decoding, then a third request joins
    H, Hq, d, P, width, n_pages = 2, 8, 128, 16, 12, 40
    rng = np.random.default_rng(12)
    cache = api.cache_alloc(n_pages, H, d, P, dev)
    host = np.zeros(tuple(cache.shape), dtype=np.uint8)
    table = torch.full((3, width), -1, dtype=torch.int32, device=dev)
    host_table = np.full((3, width), -1)
    free = rng.permutation(n_pages)
    ctx = [0, 0, 0]
    for new in ([50, 21, 0], [30, 21, 0], [1, 1, 0], [1, 1, 40], [1, 1, 1], [2, 0, 3]):
        T = sum(new) + 2                                                  # two padded rows
        start, kv, slots, info = api.mxattn_cache_plan(i32(ctx, dev), i32(new, dev), table, i32(free, dev), P, T)
        host_table, hstart, hkv, hslots, hinfo = op.plan(ctx, new, host_table, list(free), P, T)
        assert np.array_equal(slots.cpu().numpy(), hslots) and np.array_equal(table.cpu().numpy(), host_table)
        qkv = torch.from_numpy(rng.standard_normal((T, Hq + 2 * H, d))).bfloat16()
        on = qkv.to(dev)
        api.mxattn_cache_append(on[:, Hq:Hq + H], on[:, Hq + H:], slots, cache)
        op.append(host, qkv[:, Hq:Hq + H].double().numpy(), qkv[:, Hq + H:].double().numpy(), hslots, 1)
        assert np.array_equal(cache.cpu().numpy(), host)
        out = api.mxattn_paged_forward(on[:, :Hq], cache, table, start, kv, max_new=max(new))
        _close(out, None, op.attention(qkv[:, :Hq].double().numpy(), host, host_table, hstart, hkv, True), None, host)
        free = free[int(hinfo[1]):]
        ctx = hkv.tolist()


def test_python_checks(dev):
    on, _ = make(dev, [(20, 2)], True, 4, 2, 64, 16)
    q, cache, table, start, kv = on
    slots = torch.arange(2, device=dev)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=dev)
    bad = [
        lambda: api.mxattn_paged_forward(q.float(), cache, table, start, kv, 2),
        lambda: api.mxattn_paged_forward(q.cpu(), cache, table, start, kv, 2),
        lambda: api.mxattn_paged_forward(q[..., ::2], cache, table, start, kv, 2),
        lambda: api.mxattn_paged_forward(q, cache[..., :-1], table, start, kv, 2),
        lambda: api.mxattn_paged_forward(q, cache, table.long(), start, kv, 2),
        lambda: api.mxattn_paged_forward(q, cache, table, start[:-1], kv, 2),
        lambda: api.mxattn_paged_forward(q, cache, table, start, kv, 2, out=torch.empty_like(q)[1:]),
        lambda: api.mxattn_paged_forward(q, cache, table, start, kv, 2, lse=torch.empty(1, device=dev)),
        lambda: api.mxattn_paged_forward(q[:, :3], cache, table, start, kv, 2),
        lambda: api.mxattn_cache_append(k[:, :1], k, slots, cache),
        lambda: api.mxattn_cache_append(k, k, slots.int(), cache),
        lambda: api.mxattn_cache_append(k, k, slots[:1], cache),
        lambda: api.mxattn_cache_read(cache, slots[None]),
        lambda: api.mxattn_cache_plan(kv, kv, table[:0], kv, 16, 4),
        lambda: api.cache_alloc(2, 2, 96, 16, dev),
        lambda: api.cache_alloc(2, 2, 64, 24, dev),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, _lib.MxattnError)):
            call()
            pytest.fail(f"call {i} was not refused")
