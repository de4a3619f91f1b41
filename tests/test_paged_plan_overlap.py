"""mxattn_cache_plan with buffers that overlap: lengths advanced in place are a call like any other, everything else is
refused."""
import numpy as np
import pytest
import torch

from mxfp4_microscaled_bit_quantize_b200 import _lib, api, build
from oracle import paged as op

INVALID = 1
APART = {"ctx": 0x1000000, "new": 0x2000000, "table": 0x3000000, "free": 0x4000000, "start": 0x5000000, "kv": 0x6000000, "slots": 0x7000000, "info": 0x8000000}
SIZE = {"ctx": 12, "new": 12, "table": 48, "free": 36, "start": 16, "kv": 12, "slots": 56, "info": 16}     # R 3, width 4, 9 free pages, 7 tokens
OUTPUTS = ("table", "start", "kv", "slots", "info")


@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("other", sorted(APART))
def test_overlaps_are_refused(out, other):
    # never launched: the addresses do not exist
    build.build()
    lib = _lib.load()
    step = 8 if "slots" in (out, other) else 4
    for shift in (0, SIZE[other] // step * step - step, -(SIZE[out] // step * step - step)):
        if out == other or (out, other, shift) == ("kv", "ctx", 0):
            continue
        a = {**APART, out: APART[other] + shift}
        assert lib.mxattn_cache_plan(a["ctx"], a["new"], 3, a["table"], 4, a["free"], 9, 16, a["start"], a["kv"], a["slots"], 7, a["info"], None) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("R,ctx,new,T", [(5, 100, 40, 0), (64, 0, 2048, 0), (700, 90, 40, 3), (1500, 40, 9, 700)])
def test_lengths_advanced_in_place(R, ctx, new, T):
    # more than 512 rows of tokens (several CTAs), more than 512 requests (several chunks); T rows behind the last request
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    dev, P = torch.device("cuda:0"), 32
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    rng = np.random.default_rng(R)
    c = rng.integers(0, ctx + 1, R)
    width = -(-(ctx + 8 * new) // P)
    pool = rng.permutation(R * width)
    held = -(-c // P)
    table = np.full((R, width), -1)
    for r in range(R):
        table[r, :held[r]] = pool[held[:r].sum():held[:r].sum() + held[r]]
    free, lens, got_table = pool[held.sum():], i32(c), i32(table)
    for _ in range(6):
        n = rng.integers(0, new + 1, R)
        rows = int(n.sum()) + T
        outs = (torch.empty(R + 1, dtype=torch.int32, device=dev), lens, torch.empty(rows, dtype=torch.int64, device=dev),
                torch.empty(4, dtype=torch.int32, device=dev))
        api.mxattn_cache_plan(lens, i32(n), got_table, i32(free), P, rows, out=outs)
        table, start, c, slots, info = op.plan(c.tolist(), n.tolist(), table, list(free), P, rows)
        for a, b, name in zip((got_table, *outs), (table, start, c, slots, info), ("table", "q_start", "kv_len", "slots", "info")):
            assert np.array_equal(a.cpu().numpy(), b), name
        free = free[int(info[1]):]


@pytest.mark.gpu
def test_captured_step_that_advances_lengths_in_place():
    # one graph, replayed: every replay appends `new` tokens to each request, 8 CTAs in a cluster (more than 512 rows)
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    dev, P, R = torch.device("cuda:0"), 16, 40
    rng = np.random.default_rng(1)
    c, n = rng.integers(0, 50, R), rng.integers(10, 40, R)
    rows, width = int(n.sum()) + 7, 20
    assert rows > 512
    pool = rng.permutation(R * width)
    held = -(-c // P)
    table = np.full((R, width), -1)
    for r in range(R):
        table[r, :held[r]] = pool[held[:r].sum():held[:r].sum() + held[r]]
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    lens, new, got_table, free = i32(c), i32(n), i32(table), i32(np.zeros(R * width))
    outs = (torch.empty(R + 1, dtype=torch.int32, device=dev), lens, torch.empty(rows, dtype=torch.int64, device=dev),
            torch.empty(4, dtype=torch.int32, device=dev))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.mxattn_cache_plan(lens, new, got_table, free, P, rows, out=outs)
    left = pool[held.sum():]
    for _ in range(6):
        free.zero_()
        free[:len(left)] = i32(left)
        g.replay()
        # the captured call was told of R * width free pages: the ones behind `left` are page 0, which no request reaches
        table, start, c, slots, info = op.plan(c.tolist(), n.tolist(), table, list(left) + [0] * (R * width - len(left)), P, rows)
        for a, b, name in zip((got_table, *outs), (table, start, c, slots, info), ("table", "q_start", "kv_len", "slots", "info")):
            assert np.array_equal(a.cpu().numpy(), b), name
        left = left[int(info[1]):]
    del g
