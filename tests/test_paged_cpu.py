"""Host-side checks of the paged KV cache: the argument checks of its entry points (returned before anything is
launched), and pins of its oracle against closed forms."""
import numpy as np
import pytest

from mxfp4_microscaled_bit_quantize_b200 import _lib, build
from oracle import mxfp4 as mx
from oracle import paged as op

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x100000  # aligned non-null address; never dereferenced by the host-side checks


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_page_bytes(lib):
    for d in (64, 128):
        for P in (16, 32, 64, 128, 256):
            assert lib.mxattn_cache_page_bytes(3, P, d) == 3 * 2 * P * (d // 2 + d // 32)
    for bad in ((0, 16, 64), (1, 8, 64), (1, 24, 64), (1, 512, 64), (1, 16, 96), (1, 0, 64), (1, -16, 64)):
        assert lib.mxattn_cache_page_bytes(*bad) == 0


PLAN = dict(ctx=FAKE, new=FAKE, R=3, table=FAKE, width=4, free=FAKE, n_free=9, page=16, start=FAKE, kv=FAKE, slots=FAKE, tokens=7, info=FAKE)


@pytest.mark.parametrize("change,status", [
    (dict(ctx=None), INVALID), (dict(new=None), INVALID), (dict(R=-1), INVALID), (dict(table=None), INVALID), (dict(width=-1), INVALID),
    (dict(free=None), INVALID), (dict(n_free=-1), INVALID), (dict(page=0), INVALID), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(page=512), UNSUPPORTED), (dict(start=None), INVALID), (dict(kv=None), INVALID), (dict(slots=None), INVALID), (dict(slots=FAKE + 4), INVALID),
    (dict(tokens=-1), INVALID), (dict(tokens=1 << 31), UNSUPPORTED), (dict(info=None), INVALID), (dict(ctx=FAKE + 2), INVALID), (dict(info=FAKE + 1), INVALID)])
def test_plan_refusals(lib, change, status):
    a = {**PLAN, **change}
    assert lib.mxattn_cache_plan(a["ctx"], a["new"], a["R"], a["table"], a["width"], a["free"], a["n_free"], a["page"], a["start"], a["kv"], a["slots"],
                                 a["tokens"], a["info"], None) == status


APPEND = dict(k=FAKE, kt=512, kh=128, v=FAKE, vt=512, vh=128, slots=FAKE, T=5, H=4, d=128, page=16, pages=8, mode=1, cache=FAKE)


@pytest.mark.parametrize("change,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=FAKE + 1), INVALID), (dict(v=FAKE + 1), INVALID), (dict(slots=None), INVALID),
    (dict(slots=FAKE + 4), INVALID), (dict(kt=-1), INVALID), (dict(kh=-1), INVALID), (dict(vt=-8), INVALID), (dict(vh=-8), INVALID), (dict(T=-1), INVALID),
    (dict(T=1 << 31), UNSUPPORTED), (dict(H=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=0), INVALID), (dict(page=20), UNSUPPORTED),
    (dict(pages=-1), INVALID), (dict(pages=1 << 31), UNSUPPORTED), (dict(mode=2), INVALID), (dict(mode=-1), INVALID), (dict(cache=None), INVALID),
    (dict(cache=FAKE + 8), INVALID), (dict(T=0, k=None, v=None, slots=None), OK)])
def test_append_refusals(lib, change, status):
    a = {**APPEND, **change}
    assert lib.mxattn_cache_append(a["k"], a["kt"], a["kh"], a["v"], a["vt"], a["vh"], a["slots"], a["T"], a["H"], a["d"], a["page"], a["pages"], a["mode"],
                                   a["cache"], None) == status


READ = dict(cache=FAKE, slots=FAKE, T=5, H=4, d=64, page=32, pages=8, k=FAKE, v=FAKE)


@pytest.mark.parametrize("change,status", [
    (dict(cache=None), INVALID), (dict(cache=FAKE + 4), INVALID), (dict(slots=None), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(T=-1), INVALID),
    (dict(H=0), INVALID), (dict(d=32), UNSUPPORTED), (dict(page=33), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=FAKE + 8), INVALID),
    (dict(v=FAKE + 2), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(T=0, slots=None, k=None, v=None), OK)])
def test_read_refusals(lib, change, status):
    a = {**READ, **change}
    assert lib.mxattn_cache_read(a["cache"], a["slots"], a["T"], a["H"], a["d"], a["page"], a["pages"], a["k"], a["v"], None) == status


PAGED = dict(q=FAKE, qt=512, qh=128, cache=FAKE, table=FAKE, width=4, start=FAKE, kv=FAKE, out=FAKE, lse=None, T=5, R=2, Hq=4, H=2, d=128, page=16, pages=8,
             new=4, max_kv=64, causal=1, ws=FAKE, ws_bytes=1 << 40)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(qt=-8), INVALID), (dict(qt=4), INVALID), (dict(qh=4), INVALID), (dict(qh=-8), INVALID),
    (dict(cache=None), INVALID), (dict(cache=FAKE + 8), INVALID), (dict(table=None), INVALID), (dict(width=-1), INVALID), (dict(start=None), INVALID),
    (dict(kv=None), INVALID), (dict(out=None), INVALID), (dict(out=FAKE + 2), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(T=-1), INVALID),
    (dict(T=1 << 31), UNSUPPORTED), (dict(R=-1), INVALID), (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(H=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(page=100), UNSUPPORTED), (dict(pages=-1), INVALID), (dict(new=-1), INVALID), (dict(max_kv=-1), INVALID), (dict(ws=None), INVALID),
    (dict(ws=FAKE + 64), INVALID), (dict(ws_bytes=0), WORKSPACE), (dict(new=1 << 30), UNSUPPORTED), (dict(R=1 << 20, new=1 << 10), UNSUPPORTED), (dict(T=0), OK), (dict(R=0), OK), (dict(new=0), OK)])
def test_paged_refusals(lib, change, status):
    a = {**PAGED, **change}
    assert lib.mxattn_paged_forward(a["q"], a["qt"], a["qh"], a["cache"], a["table"], a["width"], a["start"], a["kv"], a["out"], a["lse"], a["T"], a["R"],
                                    a["Hq"], a["H"], a["d"], a["page"], a["pages"], a["new"], a["max_kv"], a["causal"], a["ws"], a["ws_bytes"], None) == status


def test_paged_workspace_size(lib):
    assert lib.mxattn_paged_workspace_size(64, 64, 32, 8, 128, 1, 8192) >= 256
    # it follows the requests, not the rows of a padded batch
    assert lib.mxattn_paged_workspace_size(1 << 20, 4, 32, 8, 128, 1, 131072) == lib.mxattn_paged_workspace_size(4, 4, 32, 8, 128, 1, 131072) < 64 << 20
    assert lib.mxattn_paged_workspace_size(4096, 1, 32, 8, 128, 4096, 131072) < 256 << 20
    assert lib.mxattn_paged_workspace_size(4, 4, 32, 8, 128, 1, 1 << 62) < 64 << 20
    for bad in ((-1, 1, 4, 2, 128, 1, 9), (1, -1, 4, 2, 128, 1, 9), (1, 1, 3, 2, 128, 1, 9), (1, 1, 4, 2, 96, 1, 9), (1, 1, 4, 2, 128, -1, 9),
                (1, 1, 4, 2, 128, 1, -9), (1, 1, 4, 0, 128, 1, 9), (1, 1, 4, 2, 128, 1 << 30, 9),
                (1, 1 << 20, 4, 2, 128, 1 << 10, 9)):
        assert lib.mxattn_paged_workspace_size(*bad) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_oracle_places_are_permutations(d):
    for which in (0, 1):
        assert sorted(op.byte_of(x, d, which) for x in range(d // 2)) == list(range(d // 2))
        assert sorted(op.scale_row(i, which) for i in range(16)) == list(range(16))


@pytest.mark.parametrize("mode", [mx.SCALE_OCP, mx.SCALE_UOS])
def test_oracle_append_then_read_is_the_quantizer(mode):
    rng = np.random.default_rng(1)
    cache = rng.integers(0, 256, (5, 2, 2, 16, 68), dtype=np.uint8)
    before = cache.copy()
    k, v = rng.standard_normal((7, 2, 128)), rng.standard_normal((7, 2, 128))
    slots = np.array([3, 79, -1, 16, 80, 40, 41])
    op.append(cache, k, v, slots, mode)
    kr, vr = op.read(cache, slots)
    for x, got in ((k, kr), (v, vr)):
        codes, scales = mx.quantize_rows(x, mode)
        want = np.empty_like(x)
        want[..., 0::2], want[..., 1::2] = mx.e2m1_decode(codes & 15), mx.e2m1_decode(codes >> 4)
        want *= np.repeat(np.exp2(scales.astype(float) - 127), 32, axis=-1)
        want[[2, 4]] = 0
        assert np.array_equal(got, want)
    assert np.array_equal(cache[3, ...], before[3, ...])             # a page with no slot keeps its bytes


def test_oracle_plan_by_hand():
    # pages of 16; request 0 grows into page 2 of its row, 1 fits, 2 does not fit its row, 3 takes two pages, 4 finds none
    table = [[7, -1, -1], [8, -1, -1], [1, 2, 3], [-1, -1, -1], [-1, -1, -1]]
    t, start, kv, slots, info = op.plan([16, 3, 47, 0, 0], [1, 2, 2, 17, 1], table, [20, 21, 22], 16, 25)
    assert t.tolist() == [[7, 20, -1], [8, -1, -1], [1, 2, 3], [21, 22, -1], [-1, -1, -1]]
    assert start.tolist() == [0, 1, 3, 5, 22, 23] and kv.tolist() == [17, 5, 47, 17, 0]
    assert slots.tolist() == [320, 131, 132, -1, -1] + list(range(336, 352)) + [352, -1, -1, -1]
    assert info.tolist() == [23, 3, 2, 0]


def test_oracle_attention_of_one_key_is_its_value():
    rng = np.random.default_rng(2)
    cache = np.zeros((2, 1, 2, 16, 34), dtype=np.uint8)
    k, v = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    op.append(cache, k, v, [16], mx.SCALE_UOS)
    q = rng.standard_normal((3, 2, 64))
    out, lse, _, _ = op.attention(q, cache, np.array([[1], [0]]), [0, 1, 2], [1, 0], True)
    kr, vr = op.read(cache, [16])
    assert np.allclose(out[0], vr[0]) and np.allclose(lse[0], q[0] @ kr[0, 0] / 8)
    assert np.array_equal(out[1], np.zeros((2, 64))) and np.all(np.isneginf(lse[1])) and np.all(np.isnan(out[2]))
