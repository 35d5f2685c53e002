"""Helpers of the tests of window attention with sinks and of shared-prefix attention: seeded inputs on the device
and the oracle's value with its rounding scale (the bound of gpu_helpers.check_attention)."""
from __future__ import annotations

import numpy as np
import torch

import oracle


def random_tree(rng, n, depth=16):
    """(parents, depth) of n nodes, parents first, no deeper than `depth`."""
    parents, lev = [], []
    for i in range(n):
        ok = [j for j in range(i + 1) if (0 if j == 0 else lev[j - 1]) < depth]
        p = int(ok[int(rng.integers(len(ok)))])
        parents.append(p)
        lev.append((0 if p == 0 else lev[p - 1]) + 1)
    return np.array(parents, dtype=np.int32), np.array(lev, dtype=np.int32)


def bf16(rng, *shape):
    """(device bf16 tensor, its fp64 values)."""
    t = torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def trees(rng, B, n, depth=16):
    """parents, depth [B][n] (host) of B random trees."""
    t = [random_tree(rng, n, depth) for _ in range(B)]
    return np.stack([a for a, _ in t]), np.stack([d for _, d in t])


def paged(dense, lens, ps, rng, spare=3, keep=None):
    """dense [B][Hkv][L][D] (device) -> pool, table: the sequences' pages shuffled; table entries past a sequence's
    length, and those `keep` (b, page) -> bool refuses, name no page (-1); the pool's other pages hold NaN."""
    B, Hkv, L, D = dense.shape
    per = max(1, -(-L // ps))
    pad = torch.full((B, Hkv, per * ps, D), float("nan"), dtype=dense.dtype, device=dense.device)
    pad[:, :, :L] = dense
    pool = torch.full((B * per + spare, Hkv, ps, D), float("nan"), dtype=dense.dtype, device=dense.device)
    order = rng.permutation(B * per + spare)[:B * per]
    pool[torch.from_numpy(order).cuda()] = pad.view(B, Hkv, per, ps, D).permute(0, 2, 1, 3, 4).reshape(-1, Hkv, ps, D)
    table = order.reshape(B, per).astype(np.int32)
    for b in range(B):
        for i in range(per):
            if i * ps >= int(lens[b]) or (keep is not None and not keep(b, i)):
                table[b, i] = -1
    return pool, torch.from_numpy(table).cuda()


def reference(q, kc, vc, L, kt, vt, parents, depth, **kw):
    """Oracle output of one sequence (fp64) and the scale sqrt(sum_j p_j^2 v_j^2) of check_attention's bound."""
    out, w = oracle.tree_attention(q, kc, vc, L, kt, vt, parents, depth, return_weights=True, **kw)
    G = q.shape[1] // kc.shape[0]
    s = np.empty_like(out)
    for h in range(q.shape[1]):
        vals = np.concatenate([vc[h // G, :L], vt[:, h // G]], axis=0)
        s[:, h] = np.sqrt((w[:, h] ** 2) @ (vals ** 2))
    return out, s
