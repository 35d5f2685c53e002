"""Host side of window attention with sinks and of shared-prefix attention: argument checks, workspace sizes and the
oracle's visibility rule.  No GPU needed: every call here stops before anything touches a device."""
import ctypes

import numpy as np
import pytest

import eagle_tree_verification_dynamic_b200 as et
import oracle
from oracle.attention import _visible

FAKE = ctypes.c_void_p(0x1000)   # never dereferenced
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def lib():
    return et.lib()


def test_sinks_validation(lib):
    def call(**kw):
        return lib.eagle_tree_attention_with_sinks(
            kw.get("q", FAKE), kw.get("kc", FAKE), FAKE, FAKE, kw.get("Lmax", 128), FAKE, FAKE, FAKE, kw.get("pos", FAKE),
            1, kw.get("n", 10), kw.get("Hq", 4), kw.get("Hkv", 4), kw.get("D", 64), kw.get("window", 16),
            kw.get("sinks", 4), 0.0, kw.get("out", FAKE), kw.get("ws", FAKE), kw.get("wsb", 16), None)
    assert call(q=None) == 1 and call(kc=None) == 1 and call(pos=None) == 1
    assert call(sinks=-1) == 2 and call(window=-1) == 2 and call(Hq=6) == 2 and call(n=0) == 2
    assert call(D=96) == 4 and call(n=129) == 4
    assert call(out=ODD) == 6
    assert call() == 5 and call(ws=None, wsb=1 << 30) == 5      # valid but for the workspace
    paged = lambda **kw: lib.eagle_tree_attention_paged_with_sinks(
        FAKE, FAKE, FAKE, 100, kw.get("ps", 64), kw.get("bt", FAKE), 8, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 10, 32, 8, 128,
        100, kw.get("sinks", 4), 0.0, FAKE, FAKE, 16, None)
    assert paged() == 5 and paged(ps=48) == 2 and paged(bt=None) == 1 and paged(sinks=-3) == 2


def test_shared_validation(lib):
    def call(**kw):
        return lib.eagle_tree_attention_shared(
            kw.get("q", FAKE), kw.get("ks", FAKE), FAKE, kw.get("Ls", 64), kw.get("sl", FAKE), kw.get("kc", FAKE), FAKE,
            FAKE, kw.get("Lmax", 128), FAKE, FAKE, kw.get("mask", FAKE), kw.get("B", 2), kw.get("n", 10),
            kw.get("Hq", 4), kw.get("Hkv", 4), kw.get("D", 64), 0.0, FAKE, FAKE, kw.get("wsb", 16), None)
    assert call(q=None) == 1 and call(sl=None) == 1 and call(ks=None) == 1 and call(kc=None) == 1 and call(mask=None) == 1
    assert call(ks=None, Ls=0) == 5 and call(kc=None, Lmax=0) == 5   # nothing there to point at
    assert call(Ls=-1) == 2 and call(Hq=6) == 2 and call(B=0) == 2
    assert call(D=80) == 4 and call(n=129) == 4
    assert call(B=1 << 24, n=128, Hq=32, Hkv=1) == 4                   # B * n * G past int range
    assert call(ks=ODD) == 6
    def paged(**kw):
        return lib.eagle_tree_attention_shared_paged(
            FAKE, FAKE, FAKE, kw.get("num", 100), kw.get("ps", 64), kw.get("st", FAKE), kw.get("sp", 4), kw.get("sl", FAKE),
            kw.get("bt", FAKE), 8, FAKE, FAKE, FAKE, FAKE, 2, 10, 32, 8, 128, 0.0, FAKE, FAKE, 16, None)
    assert paged() == 5 and paged(st=None) == 1 and paged(sl=None) == 1 and paged(bt=None) == 1
    assert paged(st=None, sp=0) == 5 and paged(sp=-1) == 2 and paged(ps=8) == 2
    assert paged(sp=1 << 25) == 4


def test_workspaces(lib):
    plain = lib.eagle_tree_attention_workspace_bytes(2, 40, 32, 8, 128, 4096, 512)
    assert lib.eagle_tree_attention_sinks_workspace_bytes(2, 40, 32, 8, 128, 4096, 512, 0) == plain
    assert lib.eagle_tree_attention_sinks_workspace_bytes(2, 40, 32, 8, 128, 4096, 512, 4) >= plain
    assert lib.eagle_tree_attention_sinks_workspace_bytes(2, 40, 32, 8, 128, 4096, 512, -1) == 0
    one = lib.eagle_tree_attention_shared_workspace_bytes(2, 40, 32, 8, 128, 4096, 512)
    assert one % 256 == 0 and one > lib.eagle_tree_attention_workspace_bytes(2, 40, 32, 8, 128, 512, 0)
    assert lib.eagle_tree_attention_shared_workspace_bytes(2, 40, 32, 8, 128, -1, 512) == 0
    assert lib.eagle_tree_attention_shared_workspace_bytes(1 << 24, 128, 32, 1, 128, 64, 64) == 0


def test_binding_refuses_bad_shapes():
    import torch
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(et.EagleError):
        et.tree_attention_shared(z(1, 2, 4, 64), z(4, 8, 64), z(4, 8, 64), torch.zeros(1, dtype=torch.int32),
                                 z(1, 4, 8, 64), z(1, 4, 8, 64), torch.zeros(1, dtype=torch.int32), z(1, 2, 4, 64),
                                 z(1, 2, 4, 64), torch.zeros(1, 2, 2, dtype=torch.int64))


def test_oracle_sinks_are_the_rule_written_out():
    rng = np.random.default_rng(0)
    parents, depth = np.array([0, 0, 1, 3, 2]), np.array([1, 1, 2, 3, 2])
    for L, W, S in ((20, 5, 3), (3, 2, 2), (0, 1, 1), (7, 3, 9), (40, 40, 1)):
        vis = _visible(L, parents, depth, W, S)
        anc = oracle.ancestor_mask(parents)
        for i in range(5):
            pos = L - 1 + depth[i]
            for p in range(L + 5):
                at = p if p < L else L - 1 + depth[p - L]
                want = (at >= pos - W + 1 or at < S) and (p < L or bool(anc[i, p - L]))
                assert vis[i, p] == want, (L, W, S, i, p)
    assert (_visible(20, parents, depth, 0, 4) == _visible(20, parents, depth, 0)).all()
