"""GPU parity: sampling of rows, and the acceptance walk, under temperature, top-k, top-p and min-p, against the fp64
oracle.

Tokens have to be equal, unless a draw or a top-p sum lies within 1e-8 of a border (the kernels' weights are off by at
most 6e-10 relative and 2^-45 of the largest).  The log-probability is fp32, rounded once: within 2^-24 |ref| + 4e-9
(the total's relative error, twice)."""
import math

import numpy as np
import pytest
import torch

import eagle_tree_verification_dynamic_b200 as et
from oracle import sampling as S
from workloads import get_config, make_target_logits, make_workload
from eagle_tree_verification_dynamic_b200.step import StepShape, VerifyStep

from gpu_helpers import i32
from serving_helpers import random_tree

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAN, INF = math.nan, math.inf


def f32(a):
    return torch.tensor(np.asarray(a, dtype=np.float32)).cuda()


def params_of(rng, rows, V):
    """Each row its own mix; every parameter off in some rows, and at its ends."""
    t = rng.choice([0.0, 0.3, 0.7, 1.0, 1.3, 3.0], rows).astype(np.float32)
    k = rng.choice([0, 0, 1, 2, 5, 50, 400, V - 1, V, V + 5], rows).astype(np.int32)
    p = rng.choice([0.0, 0.1, 0.5, 0.9, 0.99, 1.0, 1.0], rows).astype(np.float32)
    m = rng.choice([0.0, 0.0, 0.01, 0.3, 1.0], rows).astype(np.float32)
    return t, k, p, m


def sampling_of(t=None, k=None, p=None, m=None):
    return et.Sampling(None if t is None else f32(t), None if k is None else i32(k), None if p is None else f32(p),
                       None if m is None else f32(m))


def check_rows(x, u, t, k, p, m, got, max_near=0):
    """x [rows][V] fp64 values; parameters None or per row."""
    tok, lp = got[0].cpu().numpy(), got[1].double().cpu().numpy()
    near_rows = 0
    for r in range(x.shape[0]):
        kw = {}
        for name, a in (("temperature", t), ("top_k", k), ("top_p", p), ("min_p", m)):
            if a is not None:
                kw[name] = int(a[r]) if name == "top_k" else float(np.float32(a[r]))  # as the kernel reads it
        if "top_p" in kw and math.isnan(kw["top_p"]):
            kw["top_p"] = 1.0
        want, ref, near = S.sample_row(x[r], float(u[r]), **kw)
        if near and tok[r] != want:
            near_rows += 1
            continue
        assert tok[r] == want, (r, kw, float(u[r]), tok[r], want)
        if want < 0:
            assert lp[r] == -INF
        elif not near:
            assert abs(lp[r] - ref) <= 2.0 ** -24 * abs(ref) + 4e-9, (r, kw, lp[r], ref)
    assert near_rows <= max_near


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V,pad", [(1, 1, 0), (3, 2, 0), (17, 7, 0), (40, 129, 3), (33, 1000, 0), (24, 4099, 1),
                                        (9, 32003, 5), (5, 70000, 0)])
def test_rows_with_their_own_parameters(rows, V, pad, dtype):
    rng = np.random.default_rng(rows * 7 + V)
    host = torch.from_numpy((rng.standard_normal((rows, V + pad)) * 3).astype(np.float32)).to(DT[dtype])
    x = host.cuda()[:, :V]
    u = rng.random(rows, dtype=np.float32)
    prm = params_of(rng, rows, V)
    check_rows(host[:, :V].double().numpy(), u, *prm, et.sample(x, f32(u), sampling_of(*prm)))
    check_rows(host[:, :V].double().numpy(), u, None, None, None, None, et.sample(x, f32(u)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_each_parameter_alone_on_a_wide_row(dtype):
    rng = np.random.default_rng(3)
    V, rows = 40001, 12
    host = torch.from_numpy((rng.standard_normal((rows, V)) * 3).astype(np.float32)).to(DT[dtype])
    x, u = host.double().numpy(), rng.random(rows, dtype=np.float32)
    for t, k, p, m in (([0.8] * rows, None, None, None), (None, [50] * rows, None, None), (None, [5000] * rows, None, None),
                       (None, None, [0.9] * rows, None), (None, None, [0.9999] * rows, None),
                       (None, None, None, [0.05] * rows), ([1.4] * rows, [3000] * rows, [0.97] * rows, [0.001] * rows),
                       ([100.0] * rows, None, [0.5] * rows, None)):
        check_rows(x, u, t, k, p, m, et.sample(host.cuda(), f32(u), sampling_of(t, k, p, m)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [64, 3001, 20000])
def test_ties_masks_and_values_that_are_no_numbers(V, dtype):
    rng = np.random.default_rng(5)
    rows = []
    rows.append(np.zeros(V))                                             # all equal
    rows.append(np.where(np.arange(V) % 3 == 0, 1.0, 0.0))               # two values
    rows.append(np.full(V, -INF))                                        # nothing left
    one = np.full(V, -INF)
    one[V // 2] = -7.5
    rows.append(one)                                                      # one token left
    masked = rng.normal(size=V) * 3
    masked[rng.random(V) < 0.7] = -INF
    rows.append(masked)
    lowest = masked.copy()
    lowest[np.isneginf(lowest)] = float(torch.finfo(DT[dtype]).min)      # masks of the type's lowest value
    rows.append(lowest)
    nan = masked.copy()
    nan[np.isneginf(nan)] = NAN
    rows.append(nan)
    rows.append(np.full(V, NAN))
    inf = rng.normal(size=V)
    inf[[1, V - 1]] = INF
    rows.append(inf)
    rows.append(np.where(np.arange(V) == V - 1, 200.0, -200.0))          # all weight on the last
    rows.append(np.round(rng.normal(size=V) * 2))                        # few values, many ties at any cut
    rows.append(np.where(rng.random(V) < 0.5, 0.0, -0.0))                # zeros of both signs are equal
    host = torch.from_numpy(np.stack(rows).astype(np.float32)).to(DT[dtype])
    x, n = host.double().numpy(), len(rows)
    for u0 in (0.0, 0.37, 1.0 - 2.0 ** -24):
        u = np.full(n, u0, dtype=np.float32)
        for t, k, p, m in ((1.0, 0, 1.0, 0.0), (1.0, 5, 1.0, 0.0), (0.7, 0, 0.6, 0.0), (1.0, 40, 0.5, 0.0), (1.0, 0, 1.0, 0.5),
                           (0.0, 3, 0.5, 0.1), (1e-6, 0, 0.5, 0.0), (1e4, 0, 0.3, 0.0), (1.0, 1, 0.0, 2.0)):
            full = lambda v: [v] * n
            check_rows(x, u, full(t), full(k), full(p), full(m),
                       et.sample(host.cuda(), f32(u), sampling_of(full(t), full(k), full(p), full(m))))


def test_parameters_that_are_no_numbers():
    x = torch.randn(6, 500, device="cuda") * 2
    u = f32([0.2, 0.4, 0.6, 0.8, 0.1, 0.3])
    base = et.sample(x, u)[0]
    assert torch.equal(et.sample(x, u, sampling_of(p=[NAN] * 6, m=[NAN] * 6, k=[-4] * 6))[0], base)
    assert torch.equal(et.sample(x, u, sampling_of(t=[NAN] * 6))[0], x.argmax(1).int())
    assert torch.equal(et.sample(x, u, sampling_of(t=[-1.0] * 6))[0], x.argmax(1).int())
    flat = et.sample(x, u, sampling_of(t=[INF] * 6))[0].cpu()
    assert flat.tolist() == [int(v * 500) for v in u.double().cpu()]
    odd = et.sample(x, f32([NAN, -3.0, 0.0, 0.0, 0.0, -INF]))[0].cpu()
    assert odd.tolist() == [0] * 6                                       # read as u = 0
    big = et.sample(x, f32([2.0, INF, 1.0, 1.0, 1.0, 1.0]))[0].cpu()
    assert (big > 400).all()                                             # read as the largest u below 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_temperatures_near_the_smallest_float(dtype):
    """Acts as greedy where logits differ, and below 2^-100 as 2^-100: equal weights for logits 1e-37 apart (a ratio of
    1 - 1.3e-7, so that a draw in the middle of a token's share is that token's: 500 times 1.3e-7 of a share off)."""
    V = 1000
    rng = np.random.default_rng(5)
    x = torch.tensor(rng.standard_normal((4, V))).to(DT[dtype]).cuda()
    T = np.array([1.4e-45, 1e-38, 1e-30, 1e-20], dtype=np.float32)
    tok, lp = et.sample(x, f32([0.1, 0.9, 0.5, 0.0]), sampling_of(T))
    top = x.double().cpu().numpy()
    for r in range(4):
        ids = np.flatnonzero(top[r] == top[r].max())
        assert tok[r].item() == ids[int([0.1, 0.9, 0.5, 0.0][r] * len(ids))]
        assert abs(lp[r].item() + math.log(len(ids))) < 1e-6
    y = torch.zeros(3, V, dtype=DT[dtype]).cuda()
    y[:, ::2] = -1e-37
    want = [0, 501, 999]
    tok, lp = et.sample(y, f32([(i + 0.5) / V for i in want]), sampling_of([1.4e-45] * 3))
    assert tok.tolist() == want
    assert (lp.double().cpu() + math.log(V)).abs().max().item() < 2e-6


def test_the_draws_follow_the_distribution():
    """Every u of a fine grid: the tokens' shares are the kept probabilities (each within the grid's two ends)."""
    rng = np.random.default_rng(8)
    V, n = 300, 40000
    x = (rng.standard_normal(V) * 2).astype(np.float32)
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    prm = sampling_of([0.9] * n, [60] * n, [0.95] * n, [0.01] * n)
    tok = et.sample(f32(x).expand(n, V).contiguous(), f32(u), prm)[0].cpu().numpy()
    w = S.filter_row(x, float(np.float32(0.9)), 60, float(np.float32(0.95)), float(np.float32(0.01)))[1]
    assert (np.diff(tok) >= 0).all()                                     # u ascending, ids ascending
    share = np.bincount(tok, minlength=V) / n
    assert np.abs(share - w / w.sum()).max() <= 2.0 / n


def test_rows_strided_unaligned_and_out_of_order_of_size():
    rng = np.random.default_rng(9)
    big = torch.from_numpy((rng.standard_normal((6, 5, 1003)) * 3).astype(np.float32)).to(torch.bfloat16).cuda()
    x = big[:, -1]                                                       # the last position of each sequence
    u = rng.random(6, dtype=np.float32)
    check_rows(x.double().cpu().numpy(), u, None, [30] * 6, None, None, et.sample(x, f32(u), sampling_of(k=[30] * 6)))
    y = big.view(-1)[3:3 + 997][None]                                    # a row that starts 6 bytes into a vector
    check_rows(y.double().cpu().numpy(), u[:1], [0.9], None, [0.8], None, et.sample(y, f32(u[:1]), sampling_of([0.9], None, [0.8])))


def test_only_the_outputs_are_written_and_two_runs_agree():
    rng = np.random.default_rng(10)
    x = torch.from_numpy((rng.standard_normal((50, 9000)) * 3).astype(np.float32)).cuda()
    keep = x.clone()
    u = f32(rng.random(50, dtype=np.float32))
    prm = sampling_of(*params_of(rng, 50, 9000))
    tok = torch.full((60,), -9, dtype=torch.int32, device="cuda")
    lp = torch.full((60,), 5.0, device="cuda")
    et.sample_into(x, u, prm, tok[:50], lp[:50])
    assert (tok[50:] == -9).all() and (lp[50:] == 5.0).all() and torch.equal(x, keep)
    again = et.sample(x, u, prm)
    assert torch.equal(again[0], tok[:50]) and torch.equal(again[1].view(torch.int32), lp[:50].view(torch.int32))
    only = torch.empty(50, dtype=torch.int32, device="cuda")
    et.sample_into(x, u, prm, only)                                      # without log-probabilities
    assert torch.equal(only, tok[:50])


def test_on_another_stream_two_at_once_and_replayed():
    rng = np.random.default_rng(11)
    xs = [torch.from_numpy((rng.standard_normal((30, 12000)) * 3).astype(np.float32)).cuda() for _ in range(2)]
    u = f32(rng.random(30, dtype=np.float32))
    prm = sampling_of(*params_of(rng, 30, 12000))
    want = [et.sample(x, u, prm) for x in xs]
    outs = [(torch.empty_like(w[0]), torch.empty_like(w[1])) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st, x, o in zip(streams, xs, outs):
        with torch.cuda.stream(st):
            for _ in range(20):
                et.sample_into(x, u, prm, *o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        et.sample_into(xs[0], u, prm, *outs[0])
    xs[0].copy_(xs[1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], want[1][0])


def test_sample_refusals():
    x, u = torch.zeros(3, 10, device="cuda"), torch.zeros(3, device="cuda")
    for bad in (lambda: et.sample(x.half(), u), lambda: et.sample(x, u[:2]), lambda: et.sample(x, u.double()),
                lambda: et.sample(x.t(), torch.zeros(10, device="cuda")), lambda: et.sample(x[0], u),
                lambda: et.sample(x, u, sampling_of(t=[1.0])), lambda: et.sample(x, u, et.Sampling(top_k=u)),
                lambda: et.sample(x, u, et.Sampling(top_p=torch.zeros(3))), lambda: et.sample(x.cpu(), u),
                lambda: et.sample(x, u.cpu()), lambda: et.sample(x[:1].expand(3, 10), u),
                lambda: et.sample(torch.zeros(1, 262145, device="cuda"), u[:1])):
        with pytest.raises(et.EagleError):
            bad()


# ------------------------------------------------------------------- accept
def walk_case(seed, B, V, n, depth, k, dtype, sigma=0.7):
    rng = np.random.default_rng(seed)
    R = 1 + (depth - 1) * k
    draft = torch.from_numpy((rng.standard_normal((B, R, V)) * 3).astype(np.float32)).to(DT[dtype])
    d64 = draft.double().numpy()
    tokens, parents = np.zeros((B, n), np.int32), np.zeros((B, n), np.int32)
    draft_row = np.full((B, n + 1), -1, np.int32)
    for b in range(B):
        while True:
            par, _ = random_tree(rng, n, depth)
            inner = sorted({0} | set(par.tolist()))
            if len(inner) <= R and max(np.bincount(par)) <= V:
                break
        for r, j in enumerate(inner):
            draft_row[b, j] = r
        seen = np.zeros(n + 1, int)
        for i in range(n):
            order = np.argsort(-d64[b, draft_row[b, par[i]]], kind="stable")
            tokens[b, i] = order[seen[par[i]]]
            seen[par[i]] += 1
        parents[b] = par
    base = np.where((draft_row >= 0)[..., None], np.take_along_axis(d64, np.maximum(draft_row, 0)[..., None], 1),
                    rng.standard_normal((B, n + 1, V)) * 3)
    target = torch.from_numpy((base + sigma * rng.standard_normal(base.shape)).astype(np.float32)).to(DT[dtype])
    m = d64.max(-1)
    lse = np.log(np.exp(d64 - m[..., None]).sum(-1)) + m
    u = rng.random((B, 2, n + 1), dtype=np.float32)
    return dict(target=target, draft=draft, tokens=tokens, parents=parents, draft_row=draft_row, lse=lse, u=u, depth=depth)


def run_walk(c, sampling, wo):
    out = et.accept(c["target"].cuda(), i32(c["tokens"]), i32(c["parents"]), i32(c["draft_row"]), c["depth"], f32(c["u"]),
                    c["draft"].cuda(), torch.from_numpy(c["lse"]).cuda(), without_replacement=wo, sampling=sampling)
    return [o.cpu().numpy() for o in out]


def check_walk(c, prm, wo, got):
    t64, d64 = c["target"].double().numpy(), c["draft"].double().numpy()
    for b in range(t64.shape[0]):
        kw = {name: a[b].item() for name, a in zip(("temperature", "top_k", "top_p", "min_p"), prm)}
        ref = S.accept_sampling(t64[b], d64[b], c["tokens"][b], c["parents"][b], c["draft_row"][b], c["u"][b], c["depth"],
                                without_replacement=wo, **kw)
        have = (int(got[0][b]), got[1][b].tolist(), int(got[2][b]))
        assert ref["near"] or have == (ref["accepted_len"], ref["path"], ref["bonus"]), (b, kw, have, ref)


@pytest.mark.parametrize("wo", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,V,n,depth,k", [(1, 5, 1, 1, 1), (7, 50, 10, 3, 4), (20, 1001, 24, 5, 6), (3, 20003, 40, 6, 8),
                                           (2, 66000, 12, 4, 4)])
def test_walk_under_parameters(B, V, n, depth, k, dtype, wo):
    for seed in range(3 if V < 5000 else 1):
        c = walk_case(seed, B, V, n, depth, k, dtype)
        prm = params_of(np.random.default_rng(seed + 50), B, V)
        check_walk(c, prm, wo, run_walk(c, sampling_of(*prm), wo))


def test_walk_without_any_parameter_is_the_plain_walk():
    for dtype in ("f32", "bf16"):
        c = walk_case(5, 16, 3000, 30, 5, 6, dtype)
        a, b = run_walk(c, None, False), run_walk(c, et.Sampling(), False)
        for x, y in zip(a, b):
            assert (x == y).all()


def test_walk_over_masked_target_rows():
    c = walk_case(6, 8, 400, 12, 4, 4, "f32")
    t = c["target"].numpy()
    rng = np.random.default_rng(1)
    t[rng.random(t.shape) < 0.5] = -INF
    t[2] = -INF                                                          # nothing left in any row of a sequence
    t[3] = NAN
    t[4, :, 7] = INF
    prm = (np.full(8, 0.9, np.float32), np.full(8, 30, np.int32), np.full(8, 0.9, np.float32), np.zeros(8, np.float32))
    got = run_walk(c, sampling_of(*prm), False)
    check_walk(c, prm, False, got)
    assert got[2][2] == -1 and got[0][2] == 0 and got[2][3] == -1 and got[2][4] == 7


def test_walk_refusals():
    c = walk_case(7, 2, 100, 5, 2, 3, "f32")
    with pytest.raises(et.EagleError):
        run_walk(c, sampling_of(t=[1.0]), False)
    args = (c["target"].cuda(), i32(c["tokens"]), i32(c["parents"]), i32(c["draft_row"]), 2)
    with pytest.raises(et.EagleError):
        et.accept(*args, sampling=et.Sampling())                         # greedy: nothing to sample with
    with pytest.raises(et.EagleError):
        et.accept(*args, f32(c["u"]), sampling=et.Sampling())            # no draft distribution


# ------------------------------------------------------------ the whole step
@pytest.mark.parametrize("name,window,sinks", [("tiny", 50, 4), ("serve", 900, 64)])
def test_step_with_sinks_and_sampling(name, window, sinks):
    """The fused step equals its calls one after another, whose attention and walk equal the oracle's rules."""
    cfg = get_config(name, **({"B": 6} if name == "serve" else {}))
    dev = torch.device("cuda")
    w = make_workload(cfg, 1)
    tdt = DT[cfg.logits_dtype]
    lg = (lambda a: torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)) if cfg.logits_dtype == "bf16" else \
        (lambda a: torch.from_numpy(a).to(dev))
    bf = lambda a: torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)
    rng = np.random.default_rng(2)
    prm = (rng.choice([0.7, 1.0], cfg.B).astype(np.float32), rng.choice([0, 50], cfg.B).astype(np.int32),
           rng.choice([0.9, 1.0], cfg.B).astype(np.float32), np.full(cfg.B, 0.02, np.float32))
    inp = {"draft_logits": lg(w.draft_logits), "prefix_len": torch.from_numpy(w.prefix_len).to(dev), "q": bf(w.q),
           "k_cache": bf(w.k_cache), "v_cache": bf(w.v_cache), "k_tree": bf(w.k_tree), "v_tree": bf(w.v_tree),
           "uniforms": torch.from_numpy(w.uniforms).to(dev), "sampling": sampling_of(*prm)}
    shape = StepShape(B=cfg.B, Hq=cfg.Hq, Hkv=cfg.Hkv, D=cfg.D, Lmax=cfg.L, depth=cfg.depth, k=cfg.k, m=cfg.m, V=cfg.V,
                      logits_dtype=tdt, window=window, stochastic=True, sinks=sinks)
    one, sep = VerifyStep(shape, dev), VerifyStep(shape, dev)
    sep.build(inp["draft_logits"])
    torch.cuda.synchronize()
    inp["target_logits"] = lg(make_target_logits(cfg, 1, w.draft_logits, sep.tree.draft_row.cpu().numpy()))
    one.fused(inp)
    sep(inp)
    torch.cuda.synchronize()
    one.fused_attention_status()
    assert torch.equal(one.out.view(torch.int16), sep.out.view(torch.int16))
    for f in ("accepted_len", "path", "bonus"):
        assert torch.equal(getattr(one, f), getattr(sep, f)), f
    t64 = inp["target_logits"].double().cpu().numpy()
    d64 = inp["draft_logits"].double().cpu().numpy()
    got = [sep.accepted_len.cpu().numpy(), sep.path.cpu().numpy(), sep.bonus.cpu().numpy()]
    for b in range(min(cfg.B, 2)):
        kw = {k: a[b].item() for k, a in zip(("temperature", "top_k", "top_p", "min_p"), prm)}
        ref = S.accept_sampling(t64[b], d64[b], sep.tree.tokens[b].cpu().numpy(), sep.tree.parents[b].cpu().numpy(),
                                sep.tree.draft_row[b].cpu().numpy(), w.uniforms[b], cfg.depth, **kw)
        assert ref["near"] or (int(got[0][b]), got[1][b].tolist(), int(got[2][b])) == (ref["accepted_len"], ref["path"],
                                                                                        ref["bonus"])
    # the sampled continuation: the token after each sequence's stop node is the walk's own draw
    stop = torch.where(one.accepted_len > 0, one.path.gather(1, (one.accepted_len.long() - 1).clamp(min=0)[:, None])[:, 0], 0)
    for b in range(cfg.B):
        if int(one.accepted_len[b]) == cfg.depth:                        # every level accepted: a plain draw
            row = inp["target_logits"][b, int(stop[b])][None]
            u = inp["uniforms"][b, 1, int(stop[b])][None].contiguous()
            pick = lambda t: None if t is None else t[b:b + 1].contiguous()
            sm = inp["sampling"]
            tok = et.sample(row, u, et.Sampling(pick(sm.temperature), pick(sm.top_k), pick(sm.top_p), pick(sm.min_p)))[0]
            assert int(tok) == int(one.bonus[b])
