"""GPU tests of the alternatives of rows that hold NaN and infinities."""
import math

import pytest
import torch

from fp8_block_scaled_quantize_gb300 import rlq
from test_gpu_logprobs import DEV, DTYPES, check_forward, gen, logits_of

pytestmark = pytest.mark.gpu


def alternatives(row, top):
    """Tokens of the largest logits that are no NaN, among equal ones the lowest first, -1 past the last."""
    row = row.float().cpu()
    at = torch.nonzero(~torch.isnan(row))[:, 0]
    at = at[torch.sort(row[at], descending=True, stable=True)[1]][:top].tolist()
    return at + [-1] * (top - len(at))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(14, 70), (14, 700), (14, 5000), (14, 40000), (14, 128256), (700, 9000)])
def test_alternatives_of_rows_with_nan_and_infinities(T, V, dtype):
    """Sizes of one CTA a row and of clusters; the NaN alone, in whole units and threads, all but a few
    tokens, beside masks of -inf, and as the target."""
    g = gen(V)
    x, targets = logits_of(g, T, V, dtype)
    nan, inf = math.nan, math.inf
    x[0, V // 3] = nan
    x[1, V // 2] = inf
    x[2] = nan
    x[3] = nan
    x[3, [1, V // 2, V - 1]] = torch.tensor([1.0, 3.0, 2.0], dtype=x.dtype, device=DEV)
    x[4] = -inf
    x[4, ::2] = nan
    x[4, [5, V - 1 - V % 2]] = 1.0
    x[5, :V - 5] = nan
    x[5, V - 5:] = -inf
    x[6, targets[6]] = nan
    x[7, [3, V - 2]] = inf
    x[7, 10:30] = -inf
    x[8, : V // 2] = nan  # (whole parts of a cluster, whole threads of a CTA)
    x[9, V // 2:] = nan
    x[10] = 0.5
    x[10, ::3] = nan
    x[11] = -inf
    x[11, 7] = nan
    x[12] = torch.finfo(x.dtype).min
    x[12, 1::2] = nan
    for top in (1, 6, 20, 64):
        lp, lse, H, ids, top_lp = got = rlq.token_logprobs_top(x, targets, top=top)
        assert bool(torch.isnan(torch.stack((lp, lse, H))[:, :13]).all())
        assert bool(torch.isnan(top_lp[:13]).all())
        for r in range(13):
            assert ids[r].tolist() == alternatives(x[r], top), f"row {r}, {top} alternatives"
        check_forward(x, targets, top, 1.0, got, torch.arange(13, T, device=DEV))
