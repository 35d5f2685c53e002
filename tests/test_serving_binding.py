"""The binding's own checks around the serving calls, with the library and the device stood in for: nothing here
touches a GPU."""
import contextlib
import ctypes

import pytest
import torch

import eagle_tree_verification_dynamic_b200 as et
from eagle_tree_verification_dynamic_b200 import _lib
from eagle_tree_verification_dynamic_b200.step import StepShape, VerifyStep


class FakeLib:
    """Records the calls that would launch; sizes come from the real library."""

    def __init__(self, real, calls):
        self.real, self.calls = real, calls

    def __getattr__(self, name):
        if name.endswith("_bytes") or name.endswith("_offset") or name.endswith("_rows"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    """Names of the library's calls, with "+device" before and "-device" after each that a device was made current for."""
    log, real = [], et.lib()

    @contextlib.contextmanager
    def on(device):
        log.append(f"+{device}")
        yield
        log.append(f"-{device}")
    monkeypatch.setattr(_lib, "lib", lambda: FakeLib(real, log))
    monkeypatch.setattr(_lib, "_on", on)
    monkeypatch.setattr(_lib, "_stream", lambda device: ctypes.c_void_p(0))
    monkeypatch.setattr(_lib, "_need_cuda", lambda *ts: None)
    return log


SHAPE = dict(B=3, Hq=4, Hkv=2, D=64, Lmax=128, depth=2, k=2, m=4, V=50, logits_dtype=torch.float32)


def step_inputs(step, **kw):
    s = step.s
    bf = lambda *d: torch.zeros(*d, dtype=torch.bfloat16)
    return dict(draft_logits=torch.zeros(s.B, s.R, s.V), target_logits=torch.zeros(s.B, s.n + 1, s.V),
                q=bf(s.B, s.n, s.Hq, s.D), k_cache=bf(s.B, s.Hkv, s.Lmax, s.D), v_cache=bf(s.B, s.Hkv, s.Lmax, s.D),
                prefix_len=torch.zeros(s.B, dtype=torch.int32), k_tree=bf(s.B, s.n, s.Hkv, s.D),
                v_tree=bf(s.B, s.n, s.Hkv, s.D), uniforms=torch.zeros(s.B, 2, s.n + 1), **kw)


BAD = [et.Sampling(temperature=torch.ones(2)), et.Sampling(top_k=torch.ones(3)), et.Sampling(top_p=torch.ones(4)),
       et.Sampling(min_p=torch.ones(3, dtype=torch.float64)), et.Sampling(top_k=torch.ones(3, dtype=torch.int64))]


@pytest.mark.parametrize("bad", BAD)
def test_parameters_of_the_wrong_size_or_type_reach_no_launch(calls, bad):
    step = VerifyStep(StepShape(**SHAPE, stochastic=True), "cpu")
    inp = step_inputs(step, sampling=bad)
    accept = lambda: step.accept(inp["target_logits"], inp["uniforms"], inp["draft_logits"], bad)
    into = lambda: et.sample_into(torch.zeros(3, 50), torch.zeros(3), bad, torch.zeros(3, dtype=torch.int32))
    for run in (lambda: step.fused(inp), accept, into):
        with pytest.raises(et.EagleError):
            run()
    assert calls == []


def test_good_parameters_pass_and_outlive_the_callers_hold(calls):
    step = VerifyStep(StepShape(**SHAPE, stochastic=True), "cpu")
    good = et.Sampling(torch.ones(3), torch.ones(3, dtype=torch.int32), torch.ones(3), torch.zeros(3))
    step.fused(step_inputs(step, sampling=good))
    assert "eagle_verify_step_with_options" in calls
    options = et.step_options(4, good)
    at = options.sampling.contents.top_p
    good.top_p = None                                    # the options hold the tensor that they point to
    assert options.parameters.top_p.data_ptr() == at


def test_greedy_steps_refuse_sampling_parameters(calls):
    step = VerifyStep(StepShape(**SHAPE, stochastic=False), "cpu")
    inp = step_inputs(step, sampling=et.Sampling(torch.ones(3)))
    with pytest.raises(et.EagleError):
        step.fused(inp)
    with pytest.raises(et.EagleError):
        step.accept(inp["target_logits"], inp["uniforms"], inp["draft_logits"], inp["sampling"])
    assert calls == []
    step.fused(step_inputs(step))
    assert "eagle_verify_step_with_options" in calls


def test_every_launch_is_on_its_tensors_device(calls):
    i32 = lambda *d: torch.zeros(*d, dtype=torch.int32)
    bf = lambda *d: torch.zeros(*d, dtype=torch.bfloat16)
    prm = et.Sampling(torch.ones(3), None, torch.ones(3), None)
    for stochastic in (False, True):
        step = VerifyStep(StepShape(**SHAPE, stochastic=stochastic), "cpu")
        inp = step_inputs(step, **({"sampling": prm} if stochastic else {}))
        step.fused(inp)
        step(inp)
        step.draft_sweep(inp["draft_logits"])
        step.accept_sweep(inp["target_logits"])
        step.accept(inp["target_logits"], inp["uniforms"], inp["draft_logits"])
    et.row_stats(torch.zeros(3, 50), 2)
    et.tree_mask(i32(3, 4), i32(3, 4), i32(3))
    et.sample_into(torch.zeros(3, 50), torch.zeros(3), prm, i32(3))
    kt, cache = bf(3, 4, 2, 64), bf(3, 2, 128, 64)
    et.kv_compact(kt, kt, i32(3, 2), i32(3), i32(3), cache, cache)
    et.kv_compact_paged(kt, kt, i32(3, 2), i32(3), i32(3), cache, cache, i32(3, 2))
    pool, mask = bf(8, 2, 64, 64), torch.zeros(3, 4, 2, dtype=torch.int64)
    q = bf(3, 4, 4, 64)
    et.tree_attention_paged(q, pool, pool, i32(3, 2), i32(3), kt, kt, mask, check=False)
    et.tree_attention_shared(q, bf(2, 64, 64), bf(2, 64, 64), i32(1), cache, cache, i32(3), kt, kt, mask, check=False)
    et.tree_attention_shared_paged(q, pool, pool, i32(2), i32(1), i32(3, 2), i32(3), kt, kt, mask, check=False)
    et.static_tree_build(torch.zeros(3, 2, 50), [0, 1], [0, 0])
    g = et.TreeGrower(3, 50, 2, 2, torch.float32, "cpu")
    g.begin(torch.zeros(3, 50))
    g.level(torch.zeros(3, 2, 50), 2)
    g.level_width(torch.zeros(3, 1, 50), 2, 1)
    g.frontier_logv(), g.finish_widths([1, 1]), g.gains(), g.finish(2)
    launches = [i for i, name in enumerate(calls) if name.startswith("eagle_")]
    assert len({calls[i] for i in launches}) == 21
    for i in launches:
        assert calls[i - 1] == "+cpu" and calls[i + 1] == "-cpu", calls[i]
