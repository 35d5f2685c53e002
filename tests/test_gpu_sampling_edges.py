"""GPU parity of the sampler and the walk at the edges of their values: low temperatures, cuts among values near 0,
ties at the top, at every number of CTAs per row.

The bounds are test_gpu_sampling's: tokens equal, log-probabilities within 2^-24 |ref| + 4e-9.  A decision on a border
may go either way, but how many did is counted, and none may unless a test says so."""
import math

import numpy as np
import pytest
import torch

import eagle_tree_verification_dynamic_b200 as et
from oracle import sampling as S

from test_gpu_sampling import DT, check_rows, f32, run_walk, sampling_of, walk_case

pytestmark = pytest.mark.gpu
INF = math.inf


def walks_that_differ(c, prm, wo, got):
    """Walks unlike the oracle's, those with a decision on a border among them; the form holds for every one."""
    t64, d64 = c["target"].double().numpy(), c["draft"].double().numpy()
    V, differ, near = t64.shape[-1], 0, 0
    for b in range(t64.shape[0]):
        kw = {name: a[b].item() for name, a in zip(("temperature", "top_k", "top_p", "min_p"), prm)}
        ref = S.accept_sampling(t64[b], d64[b], c["tokens"][b], c["parents"][b], c["draft_row"][b], c["u"][b], c["depth"],
                                without_replacement=wo, **kw)
        length, path, bonus = int(got[0][b]), got[1][b].tolist(), int(got[2][b])
        assert 0 <= length <= c["depth"] and path[length:] == [-1] * (c["depth"] - length) and -1 <= bonus < V
        at = 0
        for node in path[:length]:
            assert c["parents"][b][node - 1] == at
            at = node
        near += ref["near"]
        differ += (length, path, bonus) != (ref["accepted_len"], ref["path"], ref["bonus"])
    return differ, near


# rows per launch: 16 CTAs a row, 3, and 1 (on a B200's 148 SMs)
LAUNCHES = [(12, 20000), (98, 5000), (300, 700)]


def low_rows(rows, V, rng):
    """fp32 rows whose largest values weigh, at low temperatures, far more than their bins' other places do."""
    x = np.empty((rows, V))
    for r in range(rows):
        kind = r % 6
        if kind == 0:                                     # one token, negative
            x[r] = -INF
            x[r, V // 2] = -7.5
        elif kind == 1:                                   # a negative top at its bin's upper end
            x[r] = -300.0 - rng.random(V) * 5
            x[r, 7] = -300.0
        elif kind == 2:                                   # two tokens of one positive bin
            x[r] = 0.0
            x[r, [3, V - 4]] = 10.0, 10.05
        elif kind == 3:                                   # ties at a negative top
            x[r] = -8.0 - rng.random(V)
            x[r, rng.permutation(V)[:7]] = -7.9
        elif kind == 4:                                   # negative, near 0
            x[r] = -1e-3 - rng.random(V) * 1e-3
        else:
            x[r] = rng.standard_normal(V) * 3 - 20
    return x.astype(np.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", LAUNCHES)
def test_top_p_at_low_temperatures(rows, V, dtype):
    """At these the estimated weight of a whole row may round to nothing, its top included."""
    rng = np.random.default_rng(rows)
    host = torch.from_numpy(low_rows(rows, V, rng)).to(DT[dtype])
    x = host.double().numpy()
    for T, k in ((1e-2, 0), (5e-4, 0), (1e-6, 0), (1e-30, 0), (1e-4, 40)):
        t, p = [T] * rows, rng.choice([0.3, 0.6, 0.93], rows).astype(np.float32)
        u = rng.random(rows, dtype=np.float32)
        check_rows(x, u, t, [k] * rows, p, None, et.sample(host.cuda(), f32(u), sampling_of(t, [k] * rows, p)))


@pytest.mark.parametrize("wo", [False, True])
@pytest.mark.parametrize("B,V,n,depth,k", [(3, 20003, 8, 3, 3), (98, 5000, 4, 2, 2), (300, 700, 6, 2, 3)])
def test_walk_under_top_p_at_low_temperatures(B, V, n, depth, k, wo):
    c = walk_case(21, B, V, n, depth, k, "f32")
    c["target"] = c["target"] * 0.01 - 300               # every target negative, its top alone at T <= 1e-2
    rng = np.random.default_rng(B)
    prm = (rng.choice([1e-2, 5e-4, 1e-6], B).astype(np.float32), rng.choice([0, 0, 40], B).astype(np.int32),
           rng.choice([0.3, 0.6, 0.93], B).astype(np.float32), np.zeros(B, np.float32))
    differ, near = walks_that_differ(c, prm, wo, run_walk(c, sampling_of(*prm), wo))
    assert differ == 0 and near <= B // 4
