"""The comparison of the paged attention tests: it accepts the oracle's rows rounded to bf16, and nothing that is
visibly something else, for the very inputs that the GPU tests use."""
import numpy as np
import pytest
import torch

from tests import paged_parity as pp
from tests import test_paged_gpu as gpu

CASES = [(*s, None) for s in gpu.SHAPES]
CASES += [([(400, n), (65, n)], True, Hq, H, d, P, scale) for scale in (gpu._spread_values, gpu._large_values, gpu._small_values)
          for n, Hq, H, d, P in ((1, 8, 2, 128, 16), (2, 6, 1, 64, 32), (37, 8, 2, 128, 32))]


def bf16(x):
    return torch.from_numpy(x).bfloat16().double().numpy()


@pytest.mark.parametrize("case", range(len(CASES)))
def test_comparison_tells_results_apart(case):
    lens, causal, Hq, H, d, P, scale = CASES[case]
    _, (q, cache, table, start, total) = gpu.make(torch.device("cpu"), lens, causal, Hq, H, d, P, seed=case, scale=scale)
    want = pp.expected(q, cache, table, start, total, causal)
    ref, lse = want["out"], want["lse"]
    assert pp.problems(bf16(ref), lse, want) == []
    rows = ~np.isnan(ref[:, 0, 0])
    live = rows & np.isfinite(np.where(rows[:, None], lse, -np.inf)).any(axis=1)
    if not live.any():
        return
    typical = np.abs(ref[live]).max()
    for wrong in (np.zeros_like(ref), np.full_like(ref, 1e6 * typical), -ref, np.roll(ref, 1, axis=2), ref * (1 + 2.0 ** -4), np.where(ref > 0, np.nan, ref)):
        assert pp.problems(wrong, lse, want) != []
    one = bf16(ref)                                    # one wrong row, by a quarter of its size
    r = int(np.flatnonzero(live)[-1])
    one[r, 0] += 0.25 * np.abs(ref[r, 0]).max() + 2 * want["most"][r, 0].max()
    assert pp.problems(one, lse, want) != []
    assert pp.problems(bf16(ref), np.where(np.isfinite(lse), lse + 0.01 + 4 * want["lse_most"], lse), want) != []


def test_comparison_sees_a_key_that_is_missing():
    # eight keys, one of them left out: every row that gave it weight is off by more than roundings
    _, (q, cache, table, start, total) = gpu.make(torch.device("cpu"), [(8, 4)], False, 2, 1, 64, 16, seed=5)
    want = pp.expected(q, cache, table, start, total, False)
    assert pp.problems(bf16(pp.expected(q, cache, table, start, [7], False)["out"]), None, want) != []
