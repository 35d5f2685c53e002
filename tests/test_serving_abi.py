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


def test_sample_validation(lib):
    def call(**kw):
        return lib.eagle_sample(kw.get("x", FAKE), kw.get("dt", 0), kw.get("rows", 4), kw.get("V", 100),
                                kw.get("stride", 100), None, kw.get("u", FAKE), kw.get("tok", FAKE), None, None)
    assert call(x=None) == 1 and call(u=None) == 1 and call(tok=None) == 1
    assert call(dt=2) == 3
    assert call(rows=0) == 2 and call(V=0) == 2 and call(stride=99) == 2
    assert call(V=262145, stride=262145) == 4 and call(rows=1 << 27) == 4
    assert call(x=ctypes.c_void_p(0x1002)) == 6 and call(x=ctypes.c_void_p(0x1001), dt=1) == 6


def test_accept_with_sampling_validation(lib):
    prm = et._lib.SamplingStruct()

    def call(**kw):
        return lib.eagle_accept_with_sampling(
            kw.get("t", FAKE), kw.get("dt", 0), kw.get("d", FAKE), kw.get("ddt", 0), kw.get("lse", FAKE), kw.get("R", 5),
            FAKE, FAKE, FAKE, kw.get("u", FAKE), kw.get("rule", 0), ctypes.byref(prm), kw.get("B", 1), kw.get("n", 10),
            kw.get("V", 1000), kw.get("depth", 3), FAKE, FAKE, FAKE, None, 0, None)
    assert call(t=None) == 1 and call(d=None) == 1 and call(lse=None) == 1 and call(u=None) == 1
    assert call(rule=2) == 2 and call(R=0) == 2 and call(B=0) == 2 and call(depth=0) == 2
    assert call(dt=4) == 3 and call(ddt=1) == 3
    assert call(n=129) == 4 and call(depth=17) == 4 and call(V=262145) == 4
    assert call(d=ctypes.c_void_p(0x1002)) == 6
    # without parameters it is eagle_accept_with_rule, which needs its workspace
    assert lib.eagle_accept_with_sampling(FAKE, 0, FAKE, 0, FAKE, 5, FAKE, FAKE, FAKE, FAKE, 0, None, 1, 10, 1000, 3, FAKE,
                                          FAKE, FAKE, None, 0, None) == 5


def test_step_options(lib):
    from eagle_tree_verification_dynamic_b200 import _lib
    fields = dict(draft_logits=FAKE, target_logits=FAKE, logits_dtype=0, B=1, V=32000, depth=6, k=10, m=60, q=FAKE,
                  k_cache=FAKE, v_cache=FAKE, prefix_len=FAKE, Lmax=2048, k_tree=FAKE, v_tree=FAKE, Hq=32, Hkv=32, D=128,
                  window=256, scale=0.0, uniforms=None, sampling_rule=0, block_table=None, page_size=0, pages_per_seq=0,
                  num_pages=0)
    step_in = lambda **kw: _lib.StepIn(*[{**fields, **kw}[name] for name, _ in _lib.StepIn._fields_])
    tree = _lib.TreeStruct(FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE)
    out = _lib.StepOut(tree, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
    call = lambda si, opt: lib.eagle_verify_step_with_options(ctypes.byref(si), opt, ctypes.byref(out), None, FAKE, 256, None)
    assert call(step_in(), None) == 5 and call(step_in(), _lib.step_options(4)) == 5
    assert call(step_in(), _lib.step_options(-1)) == 2
    assert call(step_in(), _lib.step_options(0, et.Sampling())) == 1           # sampling without uniforms
    assert call(step_in(uniforms=FAKE), _lib.step_options(0, et.Sampling())) == 5
    plain = lib.eagle_verify_step_workspace_bytes(ctypes.byref(step_in()))
    assert lib.eagle_verify_step_options_workspace_bytes(ctypes.byref(step_in()), None) == plain
    assert lib.eagle_verify_step_options_workspace_bytes(ctypes.byref(step_in()), _lib.step_options(64)) >= plain
