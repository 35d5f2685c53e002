"""GPU parity: tree attention under a window with sinks, and over a prefix that the batch shares, against the fp64
oracle (bound of gpu_helpers.check_attention) at the lengths where the key ranges meet, end inside a tile or vanish,
with NaN in every key that no node sees, over dense and paged caches, on another stream and replayed from a graph."""
import numpy as np
import pytest
import torch

import eagle_tree_verification_dynamic_b200 as et
import oracle

from gpu_helpers import check_attention, i32
from serving_helpers import bf16, paged, reference, trees

pytestmark = pytest.mark.gpu
NAN = float("nan")


class Case:
    """Inputs of one attention, device and host; keys past each length are NaN on the device."""

    def __init__(self, seed, B, n, Hq, Hkv, D, lens, Lmax=None, Ls=0, Ls_cap=None, depth=16):
        rng = np.random.default_rng(seed)
        self.B, self.n, self.Hq, self.Hkv, self.D = B, n, Hq, Hkv, D
        self.lens, self.Ls = np.asarray(lens, dtype=np.int32), Ls
        self.Lmax = int(max(self.lens)) if Lmax is None else Lmax
        self.parents, self.depth = trees(rng, B, n, depth)
        self.q, self.qh = bf16(rng, B, n, Hq, D)
        self.kt, self.kth = bf16(rng, B, n, Hkv, D)
        self.vt, self.vth = bf16(rng, B, n, Hkv, D)
        self.kc, self.kch = bf16(rng, B, Hkv, self.Lmax, D)
        self.vc, self.vch = bf16(rng, B, Hkv, self.Lmax, D)
        for b in range(B):
            self.kc[b, :, self.lens[b]:] = NAN
            self.vc[b, :, self.lens[b]:] = NAN
        self.plen = i32(self.lens)
        self.mask, self.pos = et.tree_mask(i32(self.parents), i32(self.depth), self.plen)
        cap = Ls if Ls_cap is None else Ls_cap
        self.ks, self.ksh = bf16(rng, Hkv, cap, D)
        self.vs, self.vsh = bf16(rng, Hkv, cap, D)
        self.ks[:, Ls:] = NAN
        self.vs[:, Ls:] = NAN
        self.slen = i32([Ls])
        self.rng = rng

    def hide(self, window, sinks):
        """NaN in the prefix keys that no node of a sequence sees (depth 1 sees the most)."""
        for b in range(self.B):
            lo = max(0, int(self.lens[b]) - window + 1)
            if lo > sinks:
                self.kc[b, :, sinks:lo] = NAN
                self.vc[b, :, sinks:lo] = NAN

    def check(self, out, **kw):
        torch.cuda.synchronize()
        got = out.float().cpu().numpy()
        refs, scales = [], []
        for b in range(self.B):
            L = int(self.lens[b])
            kc = np.concatenate([self.ksh[:, :self.Ls], self.kch[b][:, :L]], axis=1)
            vc = np.concatenate([self.vsh[:, :self.Ls], self.vch[b][:, :L]], axis=1)
            r, s = reference(self.qh[b], kc, vc, self.Ls + L, self.kth[b], self.vth[b], self.parents[b], self.depth[b], **kw)
            refs.append(r)
            scales.append(s)
        check_attention(got, np.stack(refs), np.stack(scales))


# --------------------------------------------------------------------- sinks
@pytest.mark.parametrize("window,sinks", [(1, 1), (64, 4), (100, 4), (65, 64), (200, 130), (3, 63), (500, 1), (70, 1000)])
@pytest.mark.parametrize("shape", [(2, 10, 4, 4, 64), (3, 37, 8, 2, 128), (2, 128, 6, 2, 128)])
def test_sinks_dense(window, sinks, shape):
    B, n, Hq, Hkv, D = shape
    c = Case(1, B, n, Hq, Hkv, D, [0, 331, 577][:B] if B == 3 else [331, 64])
    c.hide(window, sinks)
    out = et.tree_attention(c.q, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask, c.pos, window=window, sinks=sinks)
    c.check(out, window=window, sinks=sinks)


@pytest.mark.parametrize("L", [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 192, 193, 260])
def test_sinks_where_the_ranges_meet(L):
    """One prefix length a tile apart or a key apart from sinks and window."""
    for sinks, window in ((64, 64), (4, 130), (65, 1)):
        c = Case(2, 1, 9, 4, 2, 128, [L], Lmax=max(L, 1))
        c.hide(window, sinks)
        out = et.tree_attention(c.q, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask, c.pos, window=window, sinks=sinks)
        c.check(out, window=window, sinks=sinks)


@pytest.mark.parametrize("ps", [16, 32, 64, 192])
@pytest.mark.parametrize("window,sinks", [(100, 4), (33, 100), (300, 17)])
def test_sinks_paged_with_the_hidden_pages_given_back(ps, window, sinks):
    c = Case(3, 4, 21, 8, 2, 128, [700, 5, 0, 389])
    c.hide(window, sinks)
    visible = lambda b, i: i * ps < sinks or (i + 1) * ps > int(c.lens[b]) - window + 1
    state = c.rng.bit_generator.state
    kp, table = paged(c.kc, c.lens, ps, c.rng, keep=visible)
    c.rng.bit_generator.state = state
    vp, _ = paged(c.vc, c.lens, ps, c.rng, keep=visible)
    assert (table == -1).any()
    out = et.tree_attention_paged(c.q, kp, vp, table, c.plen, c.kt, c.vt, c.mask, c.pos, window=window, sinks=sinks)
    c.check(out, window=window, sinks=sinks)
    table[0, 0] = kp.shape[0]                                     # a sink's page outside the pool
    with pytest.raises(et.EagleError, match="status 3"):
        et.tree_attention_paged(c.q, kp, vp, table, c.plen, c.kt, c.vt, c.mask, c.pos, window=window, sinks=sinks)


def test_sinks_without_effect_equal_the_call_without():
    c = Case(4, 2, 30, 8, 2, 128, [300, 77])
    args = (c.q, c.kc.nan_to_num(), c.vc.nan_to_num(), c.plen, c.kt, c.vt, c.mask, c.pos)
    assert torch.equal(et.tree_attention(*args, sinks=9), et.tree_attention(*args))
    assert torch.equal(et.tree_attention(*args, window=50, sinks=0), et.tree_attention(*args, window=50))


# ------------------------------------------------------------- shared prefix
@pytest.mark.parametrize("Ls", [0, 1, 64, 130, 515])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 64), (3, 10, 4, 4, 64), (5, 37, 8, 2, 128), (3, 128, 6, 2, 128), (2, 50, 5, 1, 64)])
def test_shared_dense(Ls, shape):
    B, n, Hq, Hkv, D = shape
    c = Case(5, B, n, Hq, Hkv, D, [70, 0, 1, 200, 64][:B], Lmax=201, Ls=Ls, Ls_cap=Ls + 70)
    out = et.tree_attention_shared(c.q, c.ks, c.vs, c.slen, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask)
    c.check(out)


def test_shared_without_own_keys_or_without_a_shared_buffer():
    c = Case(6, 4, 12, 4, 2, 128, [0, 0, 0, 0], Lmax=0, Ls=300)
    c.check(et.tree_attention_shared(c.q, c.ks, c.vs, c.slen, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask))
    c = Case(7, 4, 12, 4, 2, 128, [9, 0, 100, 64], Ls=0)
    c.check(et.tree_attention_shared(c.q, c.ks, c.vs, c.slen, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask))


def test_shared_rows_whose_mask_leaves_nothing():
    """A node whose own mask bit is clear, over no keys at all: zeros, whatever is next to it."""
    c = Case(8, 2, 6, 4, 2, 64, [0, 40], Ls=0)
    c.mask[0, 3] = 0
    out = et.tree_attention_shared(c.q, c.ks, c.vs, c.slen, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask)
    assert (out[0, 3] == 0).all() and torch.isfinite(out).all() and (out[1, 3] != 0).any()


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_shared_paged(ps):
    c = Case(9, 6, 33, 8, 2, 128, [70, 0, 1, 200, 64, 333], Ls=421)
    cap = max(c.Lmax, c.Ls)
    both = []
    state = c.rng.bit_generator.state
    for own, sh in ((c.kc, c.ks), (c.vc, c.vs)):
        c.rng.bit_generator.state = state
        dense = torch.full((c.B + 1, c.Hkv, cap, c.D), NAN, dtype=torch.bfloat16, device="cuda")
        dense[:c.B, :, :c.Lmax] = own
        dense[c.B, :, :c.Ls] = sh
        both.append(paged(dense, list(c.lens) + [c.Ls], ps, c.rng))
    (kp, table), (vp, _) = both
    own, sh = table[:c.B].contiguous(), table[c.B].contiguous()
    out = et.tree_attention_shared_paged(c.q, kp, vp, sh, c.slen, own, c.plen, c.kt, c.vt, c.mask)
    c.check(out)
    sh[2] = -5
    with pytest.raises(et.EagleError, match="status 3"):
        et.tree_attention_shared_paged(c.q, kp, vp, sh, c.slen, own, c.plen, c.kt, c.vt, c.mask)


def test_shared_equals_the_call_over_the_whole_prefix_within_rounding():
    """Against eagle_tree_attention itself on the concatenated cache: both within the oracle's bound."""
    c = Case(10, 4, 40, 8, 2, 128, [100, 300, 7, 0], Ls=640)
    kc = torch.cat([c.ks.expand(c.B, -1, -1, -1), c.kc.nan_to_num()], 2).contiguous()
    vc = torch.cat([c.vs.expand(c.B, -1, -1, -1), c.vc.nan_to_num()], 2).contiguous()
    whole = et.tree_attention(c.q, kc, vc, c.plen + c.Ls, c.kt, c.vt, c.mask)
    c.check(whole)
    c.check(et.tree_attention_shared(c.q, c.ks, c.vs, c.slen, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask))


# ------------------------------------------------ streams, graphs, workspaces
def test_on_another_stream_and_replayed_from_graphs():
    c = Case(11, 3, 20, 8, 2, 128, [500, 40, 260], Ls=200)
    c.hide(90, 5)
    shape = (c.B, c.n, c.Hq, c.Hkv, c.D)
    sink_args = (c.q, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask, c.pos)
    sh_args = (c.q, c.ks, c.vs, c.slen, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask)
    want = et.tree_attention(*sink_args, window=90, sinks=5)
    full = Case(11, 3, 20, 8, 2, 128, [500, 40, 260], Ls=200)
    sh_args = (full.q, full.ks, full.vs, full.slen, full.kc, full.vc, full.plen, full.kt, full.vt, full.mask)
    want_sh = et.tree_attention_shared(*sh_args)
    ws1 = torch.empty(et.attention_workspace_bytes(*shape, c.Lmax, 90, 5), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(et.shared_attention_workspace_bytes(*shape, 200, c.Lmax), dtype=torch.uint8, device="cuda")
    o1, o2 = torch.zeros_like(c.q), torch.zeros_like(c.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        et.tree_attention_into(*sink_args, o1, ws1, window=90, sinks=5)
        et.tree_attention_shared_into(*sh_args, o2, ws2)
    side.synchronize()
    assert torch.equal(o1, want) and torch.equal(o2, want_sh)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        et.tree_attention_into(*sink_args, o1, ws1, window=90, sinks=5)
        et.tree_attention_shared_into(*sh_args, o2, ws2)
    for _ in range(3):
        o1.zero_(), o2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, want) and torch.equal(o2, want_sh)
    for length in (30, 5):                # lengths are device data: a replay follows them
        c.plen.fill_(length)
        g.replay()
        torch.cuda.synchronize()
        again = et.tree_attention(*sink_args, window=90, sinks=5)
        assert torch.equal(o1.view(torch.int16), again.view(torch.int16))
    assert torch.isfinite(o1).all()       # 5: the sinks alone (30 also sees keys that hide() made NaN)
    et.check_attention_status(ws1)
    et.check_attention_status(ws2)


def test_a_wait_that_gives_up_is_reported_and_the_next_call_is_right():
    """The wide kernel's roles end when a bounded wait runs out (status 1); nothing stays behind."""
    c = Case(12, 3, 20, 8, 2, 128, [200, 40, 260], Ls=300)
    args = (c.q, c.ks, c.vs, c.slen, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask)
    try:
        et.attention_wait_probe(1_000_000)
        with pytest.raises(et.EagleError, match="status 1"):
            et.tree_attention_shared(*args)
    finally:
        et.attention_wait_probe(0)
    c.check(et.tree_attention_shared(*args))


def test_shared_paged_without_shared_pages():
    c = Case(13, 3, 20, 8, 2, 64, [200, 40, 260], Ls=0)
    state = c.rng.bit_generator.state
    kp, table = paged(c.kc, c.lens, 32, c.rng)
    c.rng.bit_generator.state = state
    vp, _ = paged(c.vc, c.lens, 32, c.rng)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    c.check(et.tree_attention_shared_paged(c.q, kp, vp, none, c.slen, table, c.plen, c.kt, c.vt, c.mask))


def test_shared_length_is_clamped_and_read_at_the_call():
    c = Case(14, 2, 12, 4, 2, 128, [70, 9], Ls=150)
    args = (c.q, c.ks, c.vs, c.slen, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask)
    want = et.tree_attention_shared(*args)
    c.slen.fill_(10_000)                  # past the buffer: all of it
    assert torch.equal(et.tree_attention_shared(*args), want)
    c.slen.fill_(-5)                      # none of it
    c.Ls = 0
    c.check(et.tree_attention_shared(*args))


@pytest.mark.parametrize("B,n,Hq,Hkv,D,Ls,top", [(150, 7, 6, 2, 64, 200, 90), (150, 7, 6, 2, 64, 0, 1),
                                                  (90, 3, 8, 4, 128, 70, 140), (200, 1, 4, 4, 128, 500, 60),
                                                  (33, 70, 4, 1, 64, 129, 300)])
def test_many_sequences_and_pieces(B, n, Hq, Hkv, D, Ls, top):
    """More units than CTAs, pieces of one tile after another, rows of one unit in two shared units."""
    lens = np.random.default_rng(3).integers(0, top, B)
    c = Case(15, B, n, Hq, Hkv, D, lens, Lmax=top, Ls=Ls)
    for _ in range(3):
        c.check(et.tree_attention_shared(c.q, c.ks, c.vs, c.slen, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask))


@pytest.mark.parametrize("B,n,Hq,Hkv,D,Ls,lens", [(40, 100, 12, 3, 64, 1500, 70), (12, 128, 8, 2, 128, 2100, 5),
                                                  (1, 65, 8, 2, 128, 4000, 65), (7, 43, 6, 2, 128, 700, 130)])
def test_row_blocks_full_and_in_part(B, n, Hq, Hkv, D, Ls, lens):
    """More rows a sequence than one unit holds, a last unit with a few rows of its second block or none, pieces longer
    than the ring."""
    c = Case(16, B, n, Hq, Hkv, D, np.random.default_rng(4).integers(0, lens, B), Lmax=lens, Ls=Ls)
    c.check(et.tree_attention_shared(c.q, c.ks, c.vs, c.slen, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask))


def test_attention_refusals():
    c = Case(16, 2, 6, 4, 2, 64, [20, 9], Ls=30)
    good = [c.q, c.ks, c.vs, c.slen, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask]
    for i, bad in ((0, c.q.float()), (0, c.q[0]), (1, c.ks[:1]), (2, c.vs[:, :5]), (3, c.slen.long()), (4, c.kc[:1]),
                   (5, c.vc[:, :, :, :32]), (6, c.plen[:1]), (7, c.kt[:, :3]), (8, c.vt.cpu()), (9, c.mask[:, :3])):
        args = list(good)
        args[i] = bad
        with pytest.raises(et.EagleError):
            et.tree_attention_shared(*args)
    with pytest.raises(et.EagleError):
        et.tree_attention(c.q, c.kc, c.vc, c.plen, c.kt, c.vt, c.mask, c.pos, window=8, sinks=-1)
