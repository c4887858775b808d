"""Appends that break a bound: what is left out, and that everything else of the cache is right."""
import numpy as np
import pytest
import torch

from test_serve8 import Layer, append_reference, gen, host, i32, ss  # noqa: F401 (ss: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int", "fp8"])
@pytest.mark.parametrize("starts", [[9, 8, 12], [-1, 8, 12], [4, 3, 12], [8, 8, 13]])
def test_append_leaves_out_sequences_whose_rows_are_out_of_order(ss, fmt, starts):  # noqa: F811
    """A sequence whose starts fall, lie below 0 or beyond the tokens changes nothing; the other one is written."""
    x = torch.randn(12, 1, 64, generator=gen(5), device="cuda").bfloat16()
    layer = Layer(ss, fmt, 64, 16, 1, 32, 2, seed=6).fill([32, 32])
    lens = [20, 9]
    ws = ss.Workspace()
    before = host(layer.cache)
    ss.kv_append(layer.cache, x, x, layer.table(lens), i32(starts), i32(lens), max_new=9, ws=ws)
    assert ws.error() == 17
    after = host(layer.cache)
    good = [s for s in range(2) if 0 <= starts[s] <= starts[s + 1] <= 12 and starts[s + 1] - starts[s] <= 9]
    rows, at = [], [0]
    for s in range(2):
        if s in good:
            rows.append(x[starts[s]:starts[s + 1]].float().cpu().numpy())
        at.append(at[-1] + (len(rows[-1]) if s in good else 0))
    t = np.concatenate(rows) if rows else np.zeros((0, 1, 64), np.float32)
    for n in ("k", "v"):
        codes, scales = append_reference(layer, before, t, at, [lens[s] if s in good else 0 for s in range(2)], n)
        assert np.array_equal(after[n].view(np.uint8), codes.view(np.uint8))
        assert np.array_equal(after[n + "_scales"].view(np.int32), scales.view(np.int32))
