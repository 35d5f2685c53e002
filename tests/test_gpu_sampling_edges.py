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

from test_gpu_sampling import DT, check_rows, f32, params_of, run_walk, sampling_of, walk_case

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


# ------------------------------------------------- values below 2^-16 (bf16 rows count them as 0 where that cannot show)
def floor_at(top, T, at):
    """The fp32 min-p whose floor top + T ln(min_p) is next to `at`, and that floor."""
    m = np.float32(math.exp((at - top) / T))
    return m, top + T * math.log(float(m))


def near_zero_rows():
    """(row, T, min_p, u): min-p's floor, or the top, among values below 2^-16 in magnitude."""
    out = []
    m, fl = floor_at(5.0, 1.0, 5e-6)
    assert 0 < fl < 2.0 ** -17
    out.append((np.array([5.0, 1e-5]), 1.0, m, 0.999))                       # above a floor above 0: kept
    row = np.full(130, 12.0)
    row[[0, 129]] = -1.2e-5, 1e-6
    m, fl = floor_at(12.0, 1.0, -5e-6)
    assert -1.2e-5 < fl < 0
    out.append((row, 1.0, m, 0.0))                                           # below a floor below 0: not kept
    row = np.full(20001, -1.0)
    row[::2], row[9999] = 0.0, 1e-6
    out.append((row, 10.0, np.float32(1.0), 0.7))                            # the top alone
    m, _ = floor_at(0.0, 10.0, -1.0)
    while 10.0 * math.log(float(m)) > -1.0:
        m = np.nextafter(m, np.float32(0))
    row = row.copy()
    row[9999] = 1e-5                                                         # lifts the floor above -1
    out.append((row, 10.0, m, 1.0 - 2.0 ** -24))
    row = row.copy()
    row[row == 0] = -2e-5                                                    # a top below 0: lets the floor down
    row[9999] = -1e-5
    m = np.nextafter(m, np.float32(1))
    assert 10.0 * math.log(float(m)) > -1.0 > -1e-5 + 10.0 * math.log(float(m))
    out.append((row, 10.0, m, 1.0 - 2.0 ** -24))
    return out


@pytest.mark.parametrize("copies", [1, 60, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_min_p_among_values_near_zero(dtype, copies):
    for row, T, m, u in near_zero_rows():
        host = torch.from_numpy(np.tile(row.astype(np.float32), (copies, 1))).to(DT[dtype])
        full = lambda v: np.full(copies, v, np.float32)
        tok, lp = et.sample(host.cuda(), f32(full(u)), sampling_of(full(T), None, None, full(m)))
        check_rows(host[:1].double().numpy(), [u], [T], None, None, [m], (tok[:1], lp[:1]))
        assert (tok == tok[0]).all() and (lp == lp[0]).all()


@pytest.mark.parametrize("copies", [1, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_log_probability_of_a_value_near_zero(dtype, copies):
    """The drawn logit's own value counts, though the row's sums read it as 0."""
    V = 5001
    for x in (1.4e-5, -1.4e-5):
        row = np.full(V, -40.0, np.float32)
        row[100], row[V - 1] = 12.0, x
        host = torch.from_numpy(np.tile(row, (copies, 1))).to(DT[dtype])
        u = np.full(copies, 1.0 - 2.0 ** -24, np.float32)
        tok, lp = et.sample(host.cuda(), f32(u))
        check_rows(host[:1].double().numpy(), u, None, None, None, None, (tok[:1], lp[:1]))
        assert (tok == V - 1).all() and (lp == lp[0]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_child_is_accepted_by_its_own_value_near_zero(dtype):
    """p of a drafted token with logit x = +-1.4e-5 differs from that of 0 by 1.4e-5 of it; u between the two."""
    V, B, at = 1000, 2, 321
    target = np.full((B, 2, V), -40.0, np.float32)
    target[:, :, 5] = 12.0
    target[0, :, at], target[1, :, at] = 1.4e-5, -1.4e-5
    target = torch.from_numpy(target).to(DT[dtype])
    draft = np.full((B, 1, V), -40.0, np.float32)
    draft[:, 0, 5], draft[:, 0, at] = 12.0, 0.6875
    d = draft[0, 0].astype(np.float64)
    lse = math.log(np.exp(d - 12.0).sum()) + 12.0
    q = math.exp(0.6875 - lse)
    u = np.full((B, 2, 2), 0.25, np.float32)
    for b in range(B):
        t = target[b, 0].double().numpy()
        p = math.exp(t[at]) / np.exp(t).sum()
        p0 = 1.0 / np.exp(t).sum()                       # were it 0
        u[b, 0, 1] = (p + p0) / 2 / q
        assert min(p, p0) < u[b, 0, 1] * q < max(p, p0)
    c = dict(target=target, draft=torch.from_numpy(draft).to(DT[dtype]), tokens=np.full((B, 1), at, np.int32),
             parents=np.zeros((B, 1), np.int32), draft_row=np.tile(np.array([0, -1], np.int32), (B, 1)),
             lse=np.full((B, 1), lse), u=u, depth=1)
    prm = (np.ones(B, np.float32), np.zeros(B, np.int32), np.ones(B, np.float32), np.zeros(B, np.float32))
    got = run_walk(c, sampling_of(*prm), False)
    assert walks_that_differ(c, prm, False, got) == (0, 0) and got[0].tolist() == [1, 0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_argmax_of_a_row_of_values_near_zero(dtype):
    """A walk that has rejected all draft mass ends at the target's argmax, found among values near 0 too."""
    V, B = 20001, 3
    target = np.zeros((B, 2, V), np.float32)
    for b, at in enumerate((0, 777, V - 1)):
        target[b, :, at] = 1e-5
    draft = np.full((B, 1, V), -INF, np.float32)
    draft[:, 0, 55] = 2.0
    c = dict(target=torch.from_numpy(target).to(DT[dtype]), draft=torch.from_numpy(draft).to(DT[dtype]),
             tokens=np.full((B, 1), 55, np.int32), parents=np.zeros((B, 1), np.int32),
             draft_row=np.tile(np.array([0, -1], np.int32), (B, 1)), lse=np.full((B, 1), 2.0),
             u=np.full((B, 2, 2), 0.9, np.float32), depth=1)
    prm = (np.full(B, 10.0, np.float32), np.zeros(B, np.int32), np.ones(B, np.float32), np.zeros(B, np.float32))
    got = run_walk(c, sampling_of(*prm), True)
    assert walks_that_differ(c, prm, True, got) == (0, 0) and got[2].tolist() == [0, 777, V - 1]


# ------------------------------------------------------------------ many rows, wide ones, values beyond the bins
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(300, 9000), (160, 2051), (700, 2048)])
def test_wide_rows_of_one_cta_each(rows, V, dtype):
    """The draw over bf16 rows counts a row's parts again before it reads one: rows of one CTA and 256 vectors at least."""
    rng = np.random.default_rng(V)
    host = torch.from_numpy((rng.standard_normal((rows, V)) * 3).astype(np.float32)).to(DT[dtype])
    host[::7] = torch.round(host[::7])                   # many ties at any cut
    u = rng.random(rows, dtype=np.float32)
    prm = params_of(rng, rows, V)
    check_rows(host.double().numpy(), u, *prm, et.sample(host.cuda(), f32(u), sampling_of(*prm)))
    top = np.full(rows, 0.9, np.float32)
    check_rows(host.double().numpy(), u, None, None, top, None, et.sample(host.cuda(), f32(u), sampling_of(p=top)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(3, 9001), (160, 1500)])
def test_values_that_no_bin_holds(rows, V, dtype):
    """Logits of 512 and more in magnitude, NaN of either sign, more tokens around a cut than the list holds."""
    rng = np.random.default_rng(V)
    x = rng.standard_normal((rows, V)) * 3
    x[0::4] *= 200.0                                      # both ends
    x[1::4] = -600.0 - np.abs(x[1::4])                    # all below
    x[2::4, V // 3] = 700.0
    flip = rng.random((rows, V)) < 0.01
    x[flip & (np.arange(rows) % 4 == 3)[:, None]] = math.nan
    host = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
    host[3::8] = -host[3::8]                              # NaN of the other sign
    u = rng.random(rows, dtype=np.float32)
    for t, k, p, m in ((1.0, 0, 0.9, 0.0), (50.0, 0, 0.9, 0.0), (100.0, V // 2, 0.7, 0.001), (3.0, V - 3, 1.0, 0.0)):
        full = lambda v: np.full(rows, v, np.float32)
        check_rows(host.double().numpy(), u, full(t), [k] * rows, full(p), full(m),
                   et.sample(host.cuda(), f32(u), sampling_of(full(t), [k] * rows, full(p), full(m))))


@pytest.mark.parametrize("wo", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,V,n,depth,k", [(7, 50, 10, 3, 4), (20, 1001, 24, 5, 6), (3, 20003, 40, 6, 8),
                                           (2, 66000, 12, 4, 4), (200, 900, 12, 3, 4), (150, 2600, 6, 2, 3)])
def test_no_walk_differs(B, V, n, depth, k, dtype, wo):
    """Those with a decision on a border counted too: 1e-8 of a border is 10 times the weights' error."""
    c = walk_case(11, B, V, n, depth, k, dtype)
    prm = params_of(np.random.default_rng(60), B, V)
    differ, near = walks_that_differ(c, prm, wo, run_walk(c, sampling_of(*prm), wo))
    assert differ == 0 and near <= 1 + B // 50


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_an_infinite_temperature_makes_all_tokens_equally_likely(dtype):
    """min-p of 1 and below then removes nothing; top-k and top-p still go by the logits' order."""
    rng = np.random.default_rng(1)
    V, rows = 4000, 5
    host = torch.from_numpy((rng.standard_normal((rows, V)) * 3).astype(np.float32)).to(DT[dtype])
    host[:, ::2] = -INF
    alive = np.arange(1, V, 2)
    u = np.array([0.0, 0.1001, 0.5001, 0.9001, 1.0 - 2.0 ** -24], np.float32)
    full = lambda v: np.full(rows, v, np.float32)
    for m in (0.3, 1.0, 2.0):
        tok, lp = et.sample(host.cuda(), f32(u), sampling_of(full(INF), None, None, full(m)))
        assert tok.tolist() == [int(alive[int(float(v) * len(alive))]) for v in u]
        assert (lp.double().cpu() + math.log(len(alive))).abs().max().item() < 1e-6
    k = 6
    tok, lp = et.sample(host.cuda(), f32(u), sampling_of(full(INF), [k] * rows, None, full(1.0)))
    for r in range(rows):
        ids = sorted(np.argsort(-host[r].double().numpy(), kind="stable")[:k])
        assert int(tok[r]) == ids[int(float(u[r]) * k)] and abs(float(lp[r]) + math.log(k)) < 1e-6
