"""Into how many parts the tcgen05 kernel of paged attention cuts a context, seen through the size of the workspace: 256
bytes, and d + 1 floats for each partial row where there are two parts or more."""
import pytest

from mxfp4_microscaled_bit_quantize_b200 import _lib, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def parts_of(lib, R, Hq, H, d, new, kv):
    size = lib.mxattn_paged_workspace_size(R * new, R, Hq, H, d, new, kv) - 256
    assert size >= 0 and size % (4 * (d + 1) * R * new * Hq) == 0
    return max(1, size // (4 * (d + 1) * R * new * Hq))


def rule(units, kv):
    """Waves of 148 CTAs times the tiles of 128 keys of a part and four more, and four for the joining; the fewest parts
    of the lowest cost, where that gains a tenth on one part."""
    tiles = -(-kv // 128)
    waves = lambda n: -(-units * n // 148)  # noqa: E731
    whole = waves(1) * (4 + tiles)
    most = max(1, min(128, tiles // 2, 1184 // units))
    cost, n = min(((waves(n) * (4 + -(-tiles // n)) + 4, n) for n in range(2, most + 1)), default=(whole, 1))
    if 10 * cost >= 9 * whole:
        n = 1
    chunk = -(-tiles // n) * 128
    return -(-kv // chunk)


@pytest.mark.parametrize("args,parts", [
    # R, Hq, Hkv, d, new tokens, keys
    ((1, 32, 8, 128, 2048, 32768), 1), ((1, 32, 8, 128, 2048, 16384), 1), ((1, 32, 8, 128, 800, 8192), 1),
    ((7, 15, 3, 64, 777, 3778), 1), ((2, 32, 8, 128, 100, 8100), 4), ((1, 32, 8, 128, 8, 100008), 18)])
def test_parts_of_known_calls(lib, args, parts):
    assert parts_of(lib, *args) == parts


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tiles", [1, 2, 3, 5, 16, 64, 127, 256, 518])
def test_parts_follow_the_rule(lib, d, tiles):
    for units in [*range(1, 40), *range(100, 160), *range(290, 302), 443, 444, 445, 591, 592, 593, 1183, 1184, 1185, 5120]:
        for kv in (tiles * 128, tiles * 128 - 77):
            got = parts_of(lib, units, 1, 1, d, 200, kv)
            assert got == rule(units, kv), (units, kv)
            assert got == 1 or units * got <= 1184
