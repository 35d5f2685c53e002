"""GPU: the serving calls on buffers whose elements lie past 2^31, each equal bit for bit to the call on a compact copy.

The buffers are not initialised but for what the calls may read; the rest may hold anything, NaN included."""
import numpy as np
import pytest
import torch

import eagle_tree_verification_dynamic_b200 as et

from gpu_helpers import i32
from serving_helpers import bf16, trees

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    yield
    torch.cuda.empty_cache()


def tree_inputs(rng, B, n, Hq, Hkv, D, lens):
    parents, depth = trees(rng, B, n)
    (q, _), (kt, _), (vt, _) = bf16(rng, B, n, Hq, D), bf16(rng, B, n, Hkv, D), bf16(rng, B, n, Hkv, D)
    plen = i32(lens)
    mask, pos = et.tree_mask(i32(parents), i32(depth), plen)
    return q, kt, vt, plen, mask, pos


def test_rows_of_logits():
    V, stride = 5000, 2_200_000_000
    for dt in (torch.bfloat16, torch.float32):
        big = torch.empty(2 * stride, dtype=dt, device="cuda").view(2, stride)
        big[:, :V] = torch.randn(2, V, device="cuda") * 3
        u = torch.tensor([0.3, 0.8], device="cuda")
        prm = et.Sampling(top_k=i32([0, 40]), top_p=torch.tensor([0.9, 0.5], device="cuda"))
        far, near = et.sample(big[:, :V], u, prm), et.sample(big[:, :V].contiguous(), u, prm)
        assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
        del big


def test_sinks_over_a_long_cache():
    """Leaving out keys that no node sees moves the window's keys and nothing else."""
    rng = np.random.default_rng(1)
    B, n, Hq, Hkv, D, W, sinks, Lmax = 2, 20, 16, 8, 128, 300, 70, 1_200_000
    lens = [Lmax, Lmax - 777]
    q, kt, vt, plen, mask, pos = tree_inputs(rng, B, n, Hq, Hkv, D, lens)
    far = [torch.empty(B, Hkv, Lmax, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    near = [torch.empty(B, Hkv, 1000, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    short = [1000, 1000 - 77]
    for x, y in zip(far, near):
        for b in range(B):
            y[b] = torch.randn(Hkv, 1000, D, device="cuda").bfloat16()
            x[b, :, :sinks] = y[b, :, :sinks]
            x[b, :, lens[b] - W:lens[b]] = y[b, :, short[b] - W:short[b]]
    out = et.tree_attention(q, *far, plen, kt, vt, mask, pos, window=W, sinks=sinks)
    shift = i32(np.array(short) - np.array(lens))
    want = et.tree_attention(q, *near, plen + shift, kt, vt, mask, pos + shift[:, None], window=W, sinks=sinks)
    assert torch.isfinite(out).all() and torch.equal(out, want)


def test_shared_prefix_in_a_large_buffer():
    rng = np.random.default_rng(2)
    B, n, Hq, Hkv, D, Ls, cap = 3, 10, 16, 8, 128, 500, 2_200_000
    q, kt, vt, plen, mask, _ = tree_inputs(rng, B, n, Hq, Hkv, D, [40, 0, 90])
    (kc, _), (vc, _) = bf16(rng, B, Hkv, 90, D), bf16(rng, B, Hkv, 90, D)
    far = [torch.empty(Hkv, cap, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    near = [torch.randn(Hkv, 1200, D, device="cuda").bfloat16() for _ in range(2)]  # (tiles for every SM, as in far)
    for x, y in zip(far, near):
        x[:, :Ls] = y[:, :Ls]
    out = et.tree_attention_shared(q, *far, i32([Ls]), kc, vc, plen, kt, vt, mask)
    want = et.tree_attention_shared(q, *near, i32([Ls]), kc, vc, plen, kt, vt, mask)
    assert torch.isfinite(out).all() and torch.equal(out, want)


@pytest.mark.parametrize("ps", [16, 64])
def test_pages_at_the_end_of_a_large_pool(ps):
    rng = np.random.default_rng(3)
    B, n, Hq, Hkv, D, W, sinks, Ls = 3, 10, 16, 8, 128, 150, 20, 300
    lens = [700, 64, 333]
    q, kt, vt, plen, mask, pos = tree_inputs(rng, B, n, Hq, Hkv, D, lens)
    per, shared = -(-max(lens) // ps), -(-Ls // ps)
    used = B * per + shared
    pages = 2_300_000_000 // (Hkv * ps * D)
    far = [torch.empty(pages, Hkv, ps, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    near = [torch.randn(used, Hkv, ps, D, device="cuda").bfloat16() for _ in range(2)]
    ids = rng.permutation(used).astype(np.int32)
    for x, y in zip(far, near):
        x[pages - used:] = y
    table, shared_table = ids[:B * per].reshape(B, per), ids[B * per:]
    off = pages - used
    out = et.tree_attention_paged(q, *far, i32(table + off), plen, kt, vt, mask, pos, window=W, sinks=sinks)
    want = et.tree_attention_paged(q, *near, i32(table), plen, kt, vt, mask, pos, window=W, sinks=sinks)
    assert torch.isfinite(out).all() and torch.equal(out, want)
    out = et.tree_attention_shared_paged(q, *far, i32(shared_table + off), i32([Ls]), i32(table + off), plen, kt, vt, mask)
    want = et.tree_attention_shared_paged(q, *near, i32(shared_table), i32([Ls]), i32(table), plen, kt, vt, mask)
    assert torch.isfinite(out).all() and torch.equal(out, want)
