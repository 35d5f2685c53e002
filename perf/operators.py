"""What is measured of the verify step's serving operators: their cases, inputs, plain forms and exact values.

Four operators, all next to the tree-verification step of this package:

* sinks   tree attention under a sliding window with a few first tokens that stay visible (dense or paged cache)
* shared  tree attention for a batch whose sequences share a long prefix, read once for all (dense or paged cache)
* sample  a token and its log-probability from rows of logits: temperature, top-k, top-p, min-p, given uniforms
* accept  the acceptance walk of a drafted tree with the target distribution under the same sampling parameters

``run`` computes the plain form with elementary torch operations, or (``own``) makes the package's calls.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

# A weight exp((x - max) / T) below this counts as nothing: the token is never drawn.
TINY = 2.0 ** -45


# --------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one small sequence, window shorter than the prefix: latency
        dict(name="sinks_tiny", op="sinks", B=1, Hq=4, Hkv=4, D=64, L=128, L_min=128, n=10, window=64, sinks=4, page=0),
        # the long-context shape with its 2048-token window
        dict(name="sinks_long", op="sinks", B=1, Hq=32, Hkv=8, D=128, L=32768, L_min=32768, n=80, window=2048, sinks=4,
             page=0),
        # the serving mix on a paged cache: ragged prefixes, some shorter than the window; a sink block that is no tile
        dict(name="sinks_serve_paged", op="sinks", B=32, Hq=32, Hkv=8, D=128, L=4096, L_min=512, n=32, window=1000,
             sinks=100, page=16),
        # four sequences over one system prompt, every query head its own key head; own parts from nothing to a few keys
        dict(name="shared_small", op="shared", B=4, Hq=32, Hkv=32, D=128, Ls=2048, L=200, L_min=0, n=60, page=0),
        # the serving mix: a 4096-token prompt shared by 32 sequences
        dict(name="shared_serve", op="shared", B=32, Hq=32, Hkv=8, D=128, Ls=4096, L=1024, L_min=17, n=32, page=0),
        # a long shared document, paged: odd lengths, the largest trees
        dict(name="shared_long_paged", op="shared", B=16, Hq=32, Hkv=8, D=128, Ls=32763, L=1024, L_min=100, n=80, page=64),
        # one sequence's next token: latency
        dict(name="sample_one", op="sample", rows=1, V=32000, dtype="f32", pad=0, params="top_p"),
        # a decoding batch, every row with its own parameters
        dict(name="sample_batch", op="sample", rows=32, V=128256, dtype="bf16", pad=0, params="mixed"),
        # every row of the serving mix's trees
        dict(name="sample_rows", op="sample", rows=1056, V=128256, dtype="bf16", pad=0, params="top_p"),
        # an odd vocabulary in padded fp32 rows
        dict(name="sample_odd", op="sample", rows=211, V=32003, dtype="f32", pad=61, params="mixed"),
        # one sequence's walk
        dict(name="accept_7b", op="accept", B=1, V=32000, dtype="f32", n=60, depth=6, k=10, sigma=1.0, params="top_p",
             replacement=True),
        # the serving mix's walks
        dict(name="accept_serve", op="accept", B=32, V=128256, dtype="bf16", n=32, depth=5, k=4, sigma=1.0,
             params="mixed", replacement=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sinks", "shared", "sample", "accept"])
    if op == "sinks":
        Hkv = rng.choice([1, 2, 4, 8])
        L = _log_int(rng, 40, 32768)
        B = max(1, min(_log_int(rng, 1, 32), 131072 // L))
        return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 3, 4, 8]), Hkv=Hkv, D=rng.choice([64, 128]), L=L,
                    L_min=rng.choice([L, max(1, L // 8)]), n=_log_int(rng, 1, 128), window=_log_int(rng, 1, 4096),
                    sinks=_log_int(rng, 1, 300), page=rng.choice([0, 0, 16, 32, 64, 128]))
    if op == "shared":
        Hkv = rng.choice([1, 2, 4, 8])
        Ls = _log_int(rng, 50, 32768)
        L = _log_int(rng, 1, 2048)
        return dict(op=op, B=_log_int(rng, 1, 32 if Ls < 8192 else 12), Hq=Hkv * rng.choice([1, 3, 4]), Hkv=Hkv,
                    D=rng.choice([64, 128]), Ls=Ls, L=L, L_min=rng.choice([L, L // 8]), n=_log_int(rng, 1, 80),
                    page=rng.choice([0, 0, 16, 64, 128]))
    if op == "sample":
        V = _log_int(rng, 500, 128256)
        return dict(op=op, rows=_log_int(rng, 1, min(1056, 60000000 // V)), V=V, dtype=rng.choice(["f32", "bf16"]),
                    pad=rng.choice([0, 0, 5, 64]), params=rng.choice(["mixed", "top_p", "top_k", "plain"]))
    V = _log_int(rng, 500, 128256)
    k = rng.choice([2, 4, 8, 10])
    return dict(op=op, B=_log_int(rng, 1, 32), V=V, dtype=rng.choice(["f32", "bf16"]), n=_log_int(rng, 1, 80),
                depth=rng.randint(1, 8), k=k, sigma=rng.choice([0.5, 1.0]),
                params=rng.choice(["mixed", "top_p", "top_k", "plain"]), replacement=rng.choice([True, False]))


# -------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _random_tree(rng, n, depth, max_kids, max_parents):
    """Parents (1-based node ids, 0 = root) of a tree whose nodes are numbered parents first, level by level."""
    lev, kids, parents = [0], [0], []
    expandable = [0]
    for i in range(1, n + 1):
        open_ = [j for j in expandable if kids[j] < max_kids]
        if not open_:
            fresh = [j for j in range(1, i) if j not in expandable and lev[j] < depth]
            if len(expandable) < max_parents and fresh:
                expandable.append(fresh[0])
                open_ = [fresh[0]]
            else:
                open_ = [expandable[-1]]
        elif len(expandable) < max_parents and i > 2 and rng.random() < 0.5:
            fresh = [j for j in range(1, i) if j not in expandable and lev[j] < depth]
            if fresh:
                expandable.append(fresh[0])
                open_.append(fresh[0])
        p = open_[int(rng.integers(len(open_)))]
        parents.append(p)
        kids[p] += 1
        kids.append(0)
        lev.append(lev[p] + 1)
    return np.array(parents), np.array(lev[1:])


def _ancestor_words(parents):
    """[n][2] words: bit j of node i's row set iff node j+1 is node i+1 or one of its ancestors."""
    n = len(parents)
    words = np.zeros((n, 2), dtype=np.uint64)
    for i in range(n):
        if parents[i] > 0:
            words[i] = words[parents[i] - 1]
        words[i, i // 64] |= np.uint64(1 << (i % 64))
    return words.view(np.int64)


def _to_pages(cache, page, lens, order, extra):
    """[B][Hkv][L][D] -> pool [num][Hkv][page][D] with the pages in the given order, table [B][ceil(L / page)]."""
    B, Hkv, L, D = cache.shape
    per = -(-L // page)
    pad = torch.zeros(B, Hkv, per * page, D, dtype=cache.dtype, device=cache.device)
    pad[:, :, :L] = cache
    pool = torch.zeros(B * per + extra, Hkv, page, D, dtype=cache.dtype, device=cache.device)
    where = order[:B * per]
    pool[where] = pad.view(B, Hkv, per, page, D).permute(0, 2, 1, 3, 4).reshape(B * per, Hkv, page, D)
    table = where.view(B, per).to(torch.int32).clone()
    used = -(-lens // page)
    table[torch.arange(per, device=cache.device)[None, :] >= used[:, None]] = -1  # pages not allocated
    return pool, table.contiguous()


def _attention_inputs(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    B, Hq, Hkv, D, L, n = (case[x] for x in ("B", "Hq", "Hkv", "D", "L", "n"))
    s = dict(case=case)
    trees = [_random_tree(rng, n, 16, 10, 1 + n) for _ in range(B)]
    s["parents_host"] = [t[0] for t in trees]
    s["mask"] = torch.from_numpy(np.stack([_ancestor_words(t[0]) for t in trees])).cuda()
    lens = rng.integers(case["L_min"], L, size=B, endpoint=True).astype(np.int32)
    s["lens_host"] = lens
    s["prefix_len"] = torch.from_numpy(lens).cuda()
    first = lens + case.get("Ls", 0)
    s["pos_host"] = np.stack([first[b] - 1 + trees[b][1] for b in range(B)]).astype(np.int32)
    s["pos"] = torch.from_numpy(s["pos_host"]).cuda()
    s["q"] = _randn(g, B, n, Hq, D)
    s["k_tree"], s["v_tree"] = _randn(g, B, n, Hkv, D), _randn(g, B, n, Hkv, D)
    Lc = max(L, 1)
    s["k_cache"], s["v_cache"] = _randn(g, B, Hkv, Lc, D), _randn(g, B, Hkv, Lc, D)
    if case["op"] == "shared":
        s["k_shared"], s["v_shared"] = _randn(g, Hkv, case["Ls"], D), _randn(g, Hkv, case["Ls"], D)
        s["shared_len"] = torch.tensor([case["Ls"]], dtype=torch.int32, device="cuda")
    page = case["page"]
    if page:
        per = -(-Lc // page)
        sper = -(-case.get("Ls", 0) // page)
        order = torch.randperm(B * per + sper + 3, generator=g, device="cuda")
        for x in ("k", "v"):
            pool, table = _to_pages(s[x + "_cache"], page, s["prefix_len"], order, sper + 3)
            if sper:
                sh = torch.zeros(case["Hkv"], sper * page, D, dtype=torch.bfloat16, device="cuda")
                sh[:, :case["Ls"]] = s[x + "_shared"]
                pool[order[B * per:B * per + sper]] = sh.view(Hkv, sper, page, D).permute(1, 0, 2, 3)
                s["shared_table"] = order[B * per:B * per + sper].to(torch.int32).contiguous()
                del s[x + "_shared"]
            s[x + "_pages"], s["block_table"] = pool, table
            del s[x + "_cache"]
    if own:
        import eagle_tree_verification_dynamic_b200 as et
        s["out"] = torch.empty_like(s["q"])
        if case["op"] == "sinks":
            cap = s["block_table"].shape[1] * page if page else Lc
            need = et.attention_workspace_bytes(B, n, Hq, Hkv, D, cap, case["window"], case["sinks"])
        else:
            cap = s["block_table"].shape[1] * page if page else Lc
            scap = s["shared_table"].shape[0] * page if page else case["Ls"]
            need = et.shared_attention_workspace_bytes(B, n, Hq, Hkv, D, scap, cap)
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


def _sampling_params(rng, kind, rows):
    """temperature, top_k, top_p, min_p of each row (None: off for all), as requests bring them."""
    temp = rng.uniform(0.5, 1.3, rows).astype(np.float32)
    top_k = top_p = min_p = None
    if kind in ("mixed", "top_k"):
        top_k = rng.choice([20, 40, 50, 200], rows).astype(np.int32)
    if kind in ("mixed", "top_p"):
        top_p = rng.uniform(0.8, 0.98, rows).astype(np.float32)
    if kind == "mixed":
        min_p = rng.choice([0.0, 0.0, 0.02, 0.1], rows).astype(np.float32)
        temp[rng.random(rows) < 0.1] = 0.0
        top_k[rng.random(rows) < 0.4] = 0
        top_p[rng.random(rows) < 0.3] = 1.0
    put = lambda a: None if a is None else torch.from_numpy(a).cuda()
    return put(temp), put(top_k), put(top_p), put(min_p)


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _sample_inputs(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    rows, V = case["rows"], case["V"]
    s = dict(case=case)
    s["logits"] = _randn(g, rows, V + case["pad"], scale=3.0, dtype=_dtype(case))[:, :V]
    s["uniforms"] = torch.from_numpy(rng.random(rows, dtype=np.float32)).cuda()
    s["params"] = _sampling_params(rng, case["params"], rows)
    if own:
        import eagle_tree_verification_dynamic_b200 as et
        s["sampling"] = et.Sampling(*s["params"])
        s["tokens"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        s["logprob"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    return s


def _accept_inputs(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    B, V, n, depth, k = (case[x] for x in ("B", "V", "n", "depth", "k"))
    R = 1 + (depth - 1) * k
    s = dict(case=case)
    draft = _randn(g, B, R, V, scale=3.0, dtype=_dtype(case))
    best = [draft[b].float().topk(min(V, n + 1), dim=1).indices for b in range(B)]
    tokens, parents, draft_row = (np.zeros((B, x), dtype=np.int32) for x in (n, n, n + 1))
    for b in range(B):
        par, _ = _random_tree(rng, n, depth, k, R)
        row = np.full(n + 1, -1, dtype=np.int32)
        for r, j in enumerate(sorted({0} | set(par.tolist()))):
            row[j] = r
        top, seen = best[b].cpu().numpy(), np.zeros(n + 1, dtype=int)
        for i in range(n):
            tokens[b, i] = top[row[par[i]], seen[par[i]]]  # siblings: their parent's likeliest tokens in order
            seen[par[i]] += 1
        parents[b], draft_row[b] = par, row
    rows = torch.from_numpy(draft_row).cuda().long()
    base = torch.randn(B, n + 1, V, generator=g, device="cuda").mul_(3.0)
    for b in range(B):
        has = rows[b] >= 0
        base[b, has] = draft[b, rows[b, has]].float()
    base += case["sigma"] * torch.randn(B, n + 1, V, generator=g, device="cuda")
    s["target_logits"] = base.to(_dtype(case))
    s["draft_logits"] = draft
    s["draft_lse"] = torch.stack([torch.logsumexp(draft[b].double(), 1) for b in range(B)]).contiguous()
    for name, a in (("tokens", tokens), ("parents", parents), ("draft_row", draft_row)):
        s[name] = torch.from_numpy(a).cuda()
    s["uniforms"] = torch.from_numpy(rng.random((B, 2, n + 1), dtype=np.float32)).cuda()
    s["params"] = _sampling_params(rng, case["params"], B)
    if own:
        import eagle_tree_verification_dynamic_b200 as et
        s["sampling"] = et.Sampling(*s["params"])
        s["accepted_len"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["path"] = torch.empty(B, depth, dtype=torch.int32, device="cuda")
        s["bonus"] = torch.empty(B, dtype=torch.int32, device="cuda")
        code = et.F32 if case["dtype"] == "f32" else et.BF16
        s["ws"] = torch.empty(et.accept_workspace_bytes(B, n, V, code), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    if case["op"] in ("sinks", "shared"):
        return _attention_inputs(case, seed)
    return _sample_inputs(case, seed) if case["op"] == "sample" else _accept_inputs(case, seed)


# --------------------------------------------------------------------------------------------- plain forms
def _bits(mask, n):
    """[B][n][2] words -> [B][n][n] truth values."""
    j = torch.arange(n, device=mask.device)
    return ((mask[:, :, j // 64] >> (j % 64)) & 1).bool()


def _gathered(pages, table, b=None):
    """The dense [Hkv][per * page][D] keys that a table names (missing pages read as zeros)."""
    t = (table if b is None else table[b]).long()
    got = pages[t.clamp(min=0)] * (t >= 0)[:, None, None, None]
    return got.permute(1, 0, 2, 3).reshape(pages.shape[1], -1, pages.shape[3])


def _attend(q, keys, values, visible):
    """q [n][Hq][D], keys and values [Hkv][K][D], visible [n][K] -> [n][Hq][D] in fp32."""
    n, Hq, D = q.shape
    Hkv = keys.shape[0]
    qg = q.float().view(n, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
    sc = (qg @ keys.float().transpose(1, 2)) * (1.0 / math.sqrt(D))
    sc = sc.view(Hkv, Hq // Hkv, n, -1).masked_fill(~visible, float("-inf"))
    e = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = (e / e.sum(-1, keepdim=True)).view(Hkv, -1, keys.shape[1])
    return (p @ values.float()).view(Hkv, Hq // Hkv, n, D).permute(2, 0, 1, 3).reshape(n, Hq, D)


def _plain_sinks(s):
    case = s["case"]
    n, W, sinks = case["n"], case["window"], case["sinks"]
    anc, out = _bits(s["mask"], n), []
    for b in range(case["B"]):
        kc, vc = ((_gathered(s[x + "_pages"], s["block_table"], b) if case["page"] else s[x + "_cache"][b])
                  for x in ("k", "v"))
        p = torch.arange(kc.shape[1], device=kc.device)
        pos = s["pos"][b].long()
        lo = (pos - W + 1)[:, None]
        pre = (p < s["prefix_len"][b]) & ((p < sinks) | (p >= lo))
        tree = anc[b] & ((pos < sinks) | (pos >= lo))
        out.append(_attend(s["q"][b], torch.cat([kc, s["k_tree"][b].transpose(0, 1)], 1),
                           torch.cat([vc, s["v_tree"][b].transpose(0, 1)], 1), torch.cat([pre, tree], 1)))
    return torch.stack(out).to(torch.bfloat16)


def _plain_shared(s):
    case = s["case"]
    n, anc, out = case["n"], _bits(s["mask"], case["n"]), []
    ks, vs = ((_gathered(s[x + "_pages"], s["shared_table"]) if case["page"] else s[x + "_shared"]) for x in ("k", "v"))
    sh = (torch.arange(ks.shape[1], device=ks.device) < s["shared_len"]).expand(n, -1)
    for b in range(case["B"]):
        kc, vc = ((_gathered(s[x + "_pages"], s["block_table"], b) if case["page"] else s[x + "_cache"][b])
                  for x in ("k", "v"))
        pre = (torch.arange(kc.shape[1], device=kc.device) < s["prefix_len"][b]).expand(n, -1)
        out.append(_attend(s["q"][b], torch.cat([ks, kc, s["k_tree"][b].transpose(0, 1)], 1),
                           torch.cat([vs, vc, s["v_tree"][b].transpose(0, 1)], 1), torch.cat([sh, pre, anc[b]], 1)))
    return torch.stack(out).to(torch.bfloat16)


def _weights(x, temperature):
    """exp((x - max) / T) of each row in fp64 (T <= 0: 1 at the first largest, 0 elsewhere), and (x - max) / T."""
    x = x.double()
    x = torch.where(torch.isnan(x), float("-inf"), x)
    top = x.amax(1, keepdim=True)
    t = torch.ones(x.shape[0], device=x.device) if temperature is None else temperature
    t = t.double()[:, None]
    z = torch.where(x == top, 0.0, (x - top) / t)
    z = torch.where(torch.isinf(x) & (x < 0), float("-inf"), z)
    first = torch.arange(x.shape[1], device=x.device)[None, :] == (x == top).int().argmax(1, keepdim=True)
    z = torch.where(t > 0, z, torch.where(first & (x > float("-inf")), 0.0, float("-inf")))
    e = torch.exp(z)
    return torch.where(e < TINY, 0.0, e), z


def _filtered(x, params):
    """The weights kept by top-k, top-p and min-p (0 elsewhere), and z = (x - max) / T."""
    temperature, top_k, top_p, min_p = params
    e, z = _weights(x, temperature)
    if top_k is not None or top_p is not None:
        x = torch.where(torch.isnan(x), float("-inf"), x)
        order = torch.sort(x, dim=1, descending=True, stable=True).indices  # equal logits: lower ids first
        w = e.gather(1, order)
        if top_k is not None:
            k = torch.where(top_k > 0, top_k, x.shape[1])[:, None]
            w = torch.where(torch.arange(x.shape[1], device=x.device)[None, :] < k, w, 0.0)
        if top_p is not None:
            p = torch.where(torch.isnan(top_p), 1.0, top_p.double())[:, None]
            before = torch.cumsum(w, 1) - w
            keep = (before < p * w.sum(1, keepdim=True)) | (p >= 1)
            keep[:, 0] = True
            w = torch.where(keep, w, 0.0)
        e = torch.zeros_like(e).scatter(1, order, w)
    if min_p is not None:
        m = torch.where(min_p > 0, min_p.double().clamp(max=1.0), 0.0)[:, None]
        e = torch.where(e >= m, e, 0.0)
    return e, z


def _first_above(weights, u):
    """The smallest id whose cumulative weight exceeds u * total (-1: no weight at all)."""
    u = torch.where(u >= 0, u.double(), 0.0).clamp(max=1.0 - 2.0 ** -24)
    cum = torch.cumsum(weights, 1)
    total = cum[:, -1]
    above = cum > (u * total)[:, None]
    return torch.where(total > 0, above.int().argmax(1), -1)


def _plain_sample(s):
    rows, params = s["logits"], s["params"]
    e, z = _filtered(rows, params)
    tok = _first_above(e, s["uniforms"])
    at = z.gather(1, tok.clamp(min=0)[:, None])[:, 0] - torch.log(e.sum(1))
    return tok.to(torch.int32), torch.where(tok >= 0, at, float("-inf")).to(torch.float32)


def _plain_accept(s):
    case = s["case"]
    B, n, depth, V = case["B"], case["n"], case["depth"], case["V"]
    dev = s["tokens"].device
    each = torch.arange(B, device=dev)

    def target(j):
        x = s["target_logits"][each, j]
        e, _ = _filtered(x, s["params"])
        x = torch.where(torch.isnan(x), float("-inf"), x.float())
        return e / e.sum(1, keepdim=True).clamp(min=1e-300), (x == x.amax(1, keepdim=True)).int().argmax(1)

    def drafted(j):
        r = s["draft_row"][each, j].long()
        q = torch.exp(s["draft_logits"][each, r.clamp(min=0)].double() - s["draft_lse"][each, r.clamp(min=0)][:, None])
        return torch.where((r >= 0)[:, None], q, 0.0)

    node = torch.zeros(B, dtype=torch.long, device=dev)
    length = torch.zeros(B, dtype=torch.long, device=dev)
    path = torch.full((B, depth), -1, dtype=torch.int32, device=dev)
    stuck = torch.zeros(B, dtype=torch.bool, device=dev)
    p, best = target(node)
    q = drafted(node)
    for c in range(1, n + 1):
        tested = (s["parents"][:, c - 1] == node) & ~stuck & (length < depth)
        x = s["tokens"][:, c - 1].long()
        px, qx = p[each, x], q[each, x]
        take = tested & (qx > 0) & (s["uniforms"][:, 0, c].double() * qx < px)
        path[each, length.clamp(max=depth - 1)] = torch.where(take, c, path[each, length.clamp(max=depth - 1)])
        length = length + take
        node = torch.where(take, c, node)
        reject = tested & ~take
        left = (p - q).clamp(min=0.0)
        total = left.sum(1, keepdim=True)
        stuck = stuck | (reject & (total[:, 0] <= 0))
        p = torch.where(reject[:, None] & (total > 0), left / total.clamp(min=1e-300), p)
        if not case["replacement"]:
            rest = q.clone()
            rest[each, x] = 0.0
            mass = rest.sum(1, keepdim=True)
            stuck = stuck | (reject & (mass[:, 0] <= 0))
            q = torch.where(reject[:, None] & (mass > 0), rest / mass.clamp(min=1e-300), q)
        pn, bn = target(node)
        p, best = torch.where(take[:, None], pn, p), torch.where(take, bn, best)
        q = torch.where(take[:, None], drafted(node), q)
    bonus = _first_above(p, s["uniforms"][each, 1, node])
    bonus = torch.where(stuck, best, bonus)
    return length.to(torch.int32), path, bonus.to(torch.int32)


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"sinks": _plain_sinks, "shared": _plain_shared, "sample": _plain_sample, "accept": _plain_accept}[op](state)
    import eagle_tree_verification_dynamic_b200 as et
    s = state
    if op == "sinks":
        tail = (s["prefix_len"], s["k_tree"], s["v_tree"], s["mask"], s["pos"], s["out"], s["ws"])
        if case["page"]:
            et.tree_attention_paged_into(s["q"], s["k_pages"], s["v_pages"], s["block_table"], *tail,
                                         window=case["window"], sinks=case["sinks"])
        else:
            et.tree_attention_into(s["q"], s["k_cache"], s["v_cache"], *tail, window=case["window"], sinks=case["sinks"])
        return s["out"]
    if op == "shared":
        tail = (s["prefix_len"], s["k_tree"], s["v_tree"], s["mask"], s["out"], s["ws"])
        if case["page"]:
            et.tree_attention_shared_paged_into(s["q"], s["k_pages"], s["v_pages"], s["shared_table"], s["shared_len"],
                                                s["block_table"], *tail)
        else:
            et.tree_attention_shared_into(s["q"], s["k_shared"], s["v_shared"], s["shared_len"], s["k_cache"],
                                          s["v_cache"], *tail)
        return s["out"]
    if op == "sample":
        et.sample_into(s["logits"], s["uniforms"], s["sampling"], s["tokens"], s["logprob"])
        return s["tokens"], s["logprob"]
    et.accept_into(s["target_logits"], s["tokens"], s["parents"], s["draft_row"], case["depth"], s["uniforms"],
                   s["draft_logits"], s["draft_lse"], s["accepted_len"], s["path"], s["bonus"], s["ws"],
                   without_replacement=not case["replacement"], sampling=s["sampling"])
    return s["accepted_len"], s["path"], s["bonus"]


# ---------------------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("sinks", "shared"):
        B, Hq, Hkv, D, n = (case[x] for x in ("B", "Hq", "Hkv", "D", "n"))
        mean = (case["L"] + case["L_min"]) / 2
        own_keys = min(mean, case["window"] + case["sinks"]) if op == "sinks" else mean
        per_query = own_keys + case.get("Ls", 0) + min(n, 4)
        nbytes = 4 * B * n * Hq * D + 4 * B * n * Hkv * D + 4 * B * own_keys * Hkv * D + 16 * B * n
        nbytes += 4 * case.get("Ls", 0) * Hkv * D
        return {"bytes": int(nbytes), "flops": int(4 * D * B * n * Hq * per_query)}
    size = 4 if case["dtype"] == "f32" else 2
    if op == "sample":
        return {"bytes": case["rows"] * (case["V"] * size + 28), "flops": 4 * case["rows"] * case["V"]}
    # a walk reads at least the root's target row, and the draft row there unless its first child is taken;
    # taken children add rows: two target rows and one draft row a sequence stand for it
    return {"bytes": case["B"] * (3 * case["V"] * size + 28 * case["n"]), "flops": 14 * case["B"] * case["V"]}


# --------------------------------------------------------------------------------------------------- exact
def _exact_attention(case, seed):
    s = _attention_inputs(case, seed)
    B, Hq, Hkv, D, n = (case[x] for x in ("B", "Hq", "Hkv", "D", "n"))
    G, page = Hq // Hkv, case["page"]
    out = torch.empty(B, n, Hq, D, dtype=torch.float64)

    def rows_of(name, b, count):
        if not page:
            src = s[name + "_shared"] if b is None else s[name + "_cache"][b]
            return src[:, :count]
        table = (s["shared_table"] if b is None else s["block_table"][b]).cpu().numpy()
        ids = torch.tensor([int(table[i // page]) * page + i % page for i in range(count)], device="cuda").long()
        flat = s[name + "_pages"].transpose(0, 1).reshape(Hkv, -1, D)
        return flat[:, ids]

    for b in range(B):
        L = int(s["lens_host"][b])
        parents, pos = s["parents_host"][b], s["pos_host"][b]
        vis = np.zeros((n, L + n), dtype=bool)
        for i in range(n):
            lo = 0 if case["op"] == "shared" else max(0, int(pos[i]) - case["window"] + 1)
            vis[i, lo:L] = True
            vis[i, :min(L, case.get("sinks", 0))] = True
            j = i + 1
            while j > 0:
                near = case["op"] == "shared" or pos[j - 1] >= lo or pos[j - 1] < case["sinks"]
                vis[i, L + j - 1] = near
                j = int(parents[j - 1])
        seen = torch.from_numpy(vis).cuda()
        Ls = case.get("Ls", 0)
        if Ls:
            seen = torch.cat([torch.ones(n, Ls, dtype=torch.bool, device="cuda"), seen], 1)
        parts = {}
        for name in ("k", "v"):
            bits = [rows_of(name, None, Ls)] if Ls else []
            parts[name] = torch.cat(bits + [rows_of(name, b, L), s[name + "_tree"][b].transpose(0, 1)], 1)
        for g in range(Hkv):
            keys, vals = parts["k"][g].double(), parts["v"][g].double()
            for h in range(g * G, (g + 1) * G):
                sc = torch.where(seen, s["q"][b, :, h].double() @ keys.T / math.sqrt(D), float("-inf"))
                out[b, :, h] = (torch.softmax(sc, 1) @ vals).cpu()
    return out


def _exact_row(x, T, k, p, m):
    """One row by value thresholds: (z, kept weights) in fp64."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    top = x.max()
    kept = x > -np.inf
    if not kept.any():
        return x, np.zeros_like(x)
    if not T > 0:
        z = np.full_like(x, -np.inf)
        z[int(np.argmax(x))] = 0.0
        return z, (z == 0).astype(np.float64)
    with np.errstate(invalid="ignore"):
        z = np.where(x == top, 0.0, (x - top) / np.float64(T))
    z[~kept] = -np.inf

    def first(count):  # the `count` first tokens in order of (value, then id)
        vals = np.sort(x)[::-1]
        cut = vals[count - 1]
        inside = x > cut
        spare = count - int(inside.sum())
        inside[np.flatnonzero(x == cut)[:spare]] = True
        return inside

    e = np.exp(z)
    e[e < TINY] = 0.0
    V = x.shape[0]
    limit = V if not 0 < k < V else int(k)
    if p < 1:
        vals = np.sort(z)[::-1][:limit]
        w = np.exp(vals)
        w[w < TINY] = 0.0
        cum = np.cumsum(w)
        limit = 1 if p <= 0 else int(np.searchsorted(cum, np.float64(p) * cum[-1])) + 1
        limit = min(limit, V)
    if limit < V:
        e = np.where(first(limit), e, 0.0)
    if m > 0:
        e = np.where(e >= min(float(m), 1.0), e, 0.0)
    return z, e


def _row_params(params, r):
    T, k, p, m = (None if a is None else a[r].item() for a in params)
    p = 1.0 if p is None or math.isnan(p) else p
    return (1.0 if T is None else T), (0 if k is None else k), p, (0.0 if m is None else m)


def _pick(w, u):
    cum = np.cumsum(w)
    return int(np.searchsorted(cum, float(u) * cum[-1], side="right"))


def _exact_sample(case, seed):
    s = _sample_inputs(case, seed)
    x = s["logits"].float().cpu().numpy()
    u = s["uniforms"].cpu().numpy()
    params = tuple(None if a is None else a.cpu() for a in s["params"])
    tok, lp = np.zeros(case["rows"], dtype=np.int64), np.zeros(case["rows"])
    for r in range(case["rows"]):
        z, e = _exact_row(x[r], *_row_params(params, r))
        tok[r] = _pick(e, u[r])
        lp[r] = z[tok[r]] - math.log(e.sum())
    return torch.from_numpy(tok), torch.from_numpy(lp)


def _exact_accept(case, seed):
    s = _accept_inputs(case, seed)
    host = {x: s[x].cpu().numpy() for x in ("tokens", "parents", "draft_row", "uniforms", "draft_lse")}
    params = tuple(None if a is None else a.cpu() for a in s["params"])
    B, n, depth = case["B"], case["n"], case["depth"]
    length, bonus = np.zeros(B, dtype=np.int64), np.zeros(B, dtype=np.int64)
    path = np.full((B, depth), -1, dtype=np.int64)
    for b in range(B):
        args, node = _row_params(params, b), 0
        while True:
            row = s["target_logits"][b, node].float().cpu().numpy()
            e = _exact_row(row, *args)[1]
            p = e / e.sum()
            kids = [c for c in range(1, n + 1) if host["parents"][b, c - 1] == node] if length[b] < depth else []
            r = int(host["draft_row"][b, node])
            q = np.zeros_like(p) if r < 0 else np.exp(s["draft_logits"][b, r].double().cpu().numpy() - host["draft_lse"][b, r])
            moved, spent = False, False
            for c in kids:
                x = int(host["tokens"][b, c - 1])
                if q[x] > 0 and float(host["uniforms"][b, 0, c]) < p[x] / q[x]:
                    path[b, length[b]], node, moved = c, c, True
                    length[b] += 1
                    break
                left = np.maximum(p - q, 0.0)
                if left.sum() <= 0:
                    spent = True
                    break
                p = left / left.sum()
                if not case["replacement"]:
                    q = q.copy()
                    q[x] = 0.0
                    if q.sum() <= 0:
                        spent = True
                        break
                    q /= q.sum()
            if not moved:
                bonus[b] = int(np.argmax(row)) if spent else _pick(p, host["uniforms"][b, 1, node])
                break
    return torch.from_numpy(length), torch.from_numpy(path), torch.from_numpy(bonus)


def exact(case, seed):
    if case["op"] in ("sinks", "shared"):
        return _exact_attention(case, seed)
    return _exact_sample(case, seed) if case["op"] == "sample" else _exact_accept(case, seed)
