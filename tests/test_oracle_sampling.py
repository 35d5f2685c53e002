"""The sampling oracle on rows worked by hand and against its own definition read another way (CPU)."""
import math

import numpy as np
import pytest

import oracle
from oracle import sampling as S


def test_rows_worked_by_hand():
    x = np.log([0.4, 0.1, 0.3, 0.2])
    keep = lambda **kw: np.flatnonzero(S.filter_row(x, **kw)[1]).tolist()
    assert keep() == [0, 1, 2, 3]
    assert keep(top_k=2) == [0, 2] and keep(top_k=4) == keep(top_k=9) == [0, 1, 2, 3]
    assert keep(top_p=0.69) == [0, 2] and keep(top_p=0.72) == [0, 2, 3] and keep(top_p=0.0) == [0]
    assert keep(top_k=2, top_p=0.5) == [0]          # 0.4 / 0.7 is enough
    assert keep(top_k=2, top_p=0.6) == [0, 2]
    assert keep(min_p=0.6) == [0, 2] and keep(min_p=5.0) == [0]
    assert keep(temperature=0.0) == [0] and keep(temperature=math.nan) == [0]
    assert S.sample_row(x, 0.39)[0] == 0 and S.sample_row(x, 0.41)[0] == 1 and S.sample_row(x, 0.99)[0] == 3
    assert S.sample_row(x, 0.41, top_k=2)[0] == 0 and S.sample_row(x, 0.6, top_k=2)[0] == 2
    tok, lp, _ = S.sample_row(x, 0.6, top_k=2)
    assert lp == pytest.approx(math.log(3 / 7))


def test_ties_go_to_the_lower_id():
    x = np.zeros(10)
    assert np.flatnonzero(S.filter_row(x, top_k=3)[1]).tolist() == [0, 1, 2]
    assert np.flatnonzero(S.filter_row(x, top_p=0.45)[1]).tolist() == [0, 1, 2, 3, 4]
    assert np.flatnonzero(S.filter_row(x, temperature=0.0)[1]).tolist() == [0]


def test_masked_and_infinite_logits():
    x = np.array([-np.inf, 1.0, np.nan, 1.0])
    assert np.flatnonzero(S.filter_row(x)[1]).tolist() == [1, 3] and S.sample_row(x, 0.0)[0] == 1
    assert S.sample_row(np.full(4, -np.inf), 0.5) == (-1, -math.inf, False)
    assert np.flatnonzero(S.filter_row([1.0, np.inf, 0.0, np.inf])[1]).tolist() == [1, 3]


def test_top_p_is_the_shortest_prefix():
    rng = np.random.default_rng(0)
    for _ in range(50):
        x, p = rng.normal(size=40) * 3, rng.random()
        w = S.filter_row(x, top_p=p)[1]
        full = np.exp(x - x.max())
        assert w.sum() >= p * full.sum()
        last = min((v for v in x[w > 0]))
        assert w.sum() - math.exp(last - x.max()) < p * full.sum()


def test_the_plain_walk_is_the_walk_without_parameters():
    rng = np.random.default_rng(1)
    for seed in range(60):
        V, n = 12, 6
        parents = np.array([0, 0, 1, 1, 2, 3])
        draft = rng.normal(size=(4, V)) * 2
        draft_row = np.array([0, 1, 2, 3, -1, -1, -1])
        tokens = np.empty(n, dtype=int)
        seen = {}
        for i, p in enumerate(parents):
            tokens[i] = np.argsort(-draft[draft_row[p]])[seen.get(p, 0)]
            seen[p] = seen.get(p, 0) + 1
        target = np.stack([draft[max(r, 0)] for r in draft_row]) + rng.normal(size=(n + 1, V))
        u = rng.random((2, n + 1))
        for wo in (False, True):
            a = oracle.accept_stochastic(target, draft, tokens, parents, draft_row, u, 3, without_replacement=wo)
            b = S.accept_sampling(target, draft, tokens, parents, draft_row, u, 3, without_replacement=wo)
            assert (a["accepted_len"], a["path"], a["bonus"]) == (b["accepted_len"], b["path"], b["bonus"])


def test_greedy_parameters_give_the_greedy_walk():
    rng = np.random.default_rng(2)
    for _ in range(40):
        V = 9
        parents, tokens = np.array([0, 0, 1]), np.array([4, 2, 7])
        target, draft, u = rng.normal(size=(4, V)), rng.normal(size=(2, V)), rng.random((2, 4))
        a = oracle.accept_greedy(target, tokens, parents, 2)
        b = S.accept_sampling(target, draft, tokens, parents, np.array([0, 1, -1, -1]), u, 2, temperature=0.0)
        assert (a["accepted_len"], a["path"], a["bonus"]) == (b["accepted_len"], b["path"], b["bonus"])
