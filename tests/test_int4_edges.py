"""4-bit group-scaled weights and 8-bit checkpoints at the edges of their formulas.  Formats, references and
bounds as in test_int4.py."""
import numpy as np
import pytest
import torch

from dit_weight_compression_tile_b200 import binding as B
from test_int4 import BF, HF, case, check, pack_ref, scale_grad_ref, store


def same_infinities(got, want):
    """NaN where the formula (in float64) is NaN, and its infinities; returns where it is finite"""
    got, want = got.double().cpu().numpy(), np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), np.argwhere(np.isnan(got) != np.isnan(want))[:8]
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], want[inf])
    return np.isfinite(want)


# one CTA a tile, the contraction split over a cluster, pairs of CTAs; k ends inside a group, a word, a tile
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,group", [(3, 150, 129, 128), (20, 150, 33, 32), (40, 130, 200, 64), (100, 140, 100, 128),
                                         (600, 150, 70, 32), (1100, 40, 1, 64), (130, 2304, 1089, 64),
                                         (300, 2304, 1230, 128)])
def test_scale_grad_of_infinite_gradients(m, n, k, group, dtype):
    """infinite gradients meet the real inputs only, not the zeros behind the last"""
    q, _, _, x = case(n, k, group, dtype, 2, m)
    q[5:9] = np.abs(q[5:9]) + 1 - 9 * (q[5:9] == 8)
    q[5:9] = np.where(q[5:9] == 0, 1, np.minimum(np.abs(q[5:9]), 7))
    x = x.abs() + 0.5  # no code is 0
    dy = torch.from_numpy(np.random.default_rng(m).normal(size=(m, n))).to(dtype)
    dy[0, 5] = dy[m - 1, 12] = float("inf")  # feature 12: codes of both signs and zeros
    dy[m // 2, 6] = float("-inf")
    dy[0, 7], dy[m - 1, 7] = float("inf"), float("-inf")
    dy[1, 8] = float("nan")
    c, a = pack_ref(x)
    assert (c[:, :k] > 0).all()
    ds = B.int4_scale_grad(dy.cuda(), torch.from_numpy(c).cuda(), torch.from_numpy(a).cuda(), store(q).cuda(), k,
                           group=group).cpu()
    with np.errstate(invalid="ignore"):
        ref, mag, sub = scale_grad_ref(dy, c, a, q, k, group)
    assert (ref[5] == np.inf).all() and (ref[6] == -np.inf).all() and np.isnan(ref[7:9]).all()
    fine = same_infinities(ds, ref)
    rows = fine.all(1)
    assert rows.sum() == n - 5
    check(ds[torch.from_numpy(rows)], ref[rows], mag[rows], sub[rows], m + group, dtype)
