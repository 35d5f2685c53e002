"""GPU parity: the fused step over a paged cache with a window's sinks and sampling parameters.

Equal to its calls one after another bit for bit, its attention to the oracle (bound of gpu_helpers.check_attention),
its walk to the dense step's, which does not depend on the attention."""
import numpy as np
import pytest
import torch

from eagle_tree_verification_dynamic_b200.step import StepShape, VerifyStep
from workloads import get_config, make_target_logits, make_workload

from gpu_helpers import check_attention, dec, to_dev_bf16, to_dev_logits
from serving_helpers import paged, reference
from test_gpu_sampling import DT, sampling_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,B,window,sinks,ps", [("tiny", 1, 50, 4, 16), ("tiny", 1, 50, 70, 64),
                                                     ("serve", 6, 300, 64, 16), ("serve", 6, 300, 5, 128)])
def test_paged_step_with_sinks_and_sampling(name, B, window, sinks, ps):
    cfg = get_config(name, B=B)
    dev = torch.device("cuda")
    w = make_workload(cfg, 3)
    rng = np.random.default_rng(4)
    prm = (rng.choice([0.7, 1.0], B).astype(np.float32), rng.choice([0, 50], B).astype(np.int32),
           rng.choice([0.9, 1.0], B).astype(np.float32), np.full(B, 0.02, np.float32))
    inp = {"draft_logits": to_dev_logits(w.draft_logits, cfg.logits_dtype), "q": to_dev_bf16(w.q),
           "prefix_len": torch.from_numpy(w.prefix_len).to(dev), "k_cache": to_dev_bf16(w.k_cache),
           "v_cache": to_dev_bf16(w.v_cache), "k_tree": to_dev_bf16(w.k_tree), "v_tree": to_dev_bf16(w.v_tree),
           "uniforms": torch.from_numpy(w.uniforms).to(dev), "sampling": sampling_of(*prm)}
    shape = StepShape(B=B, Hq=cfg.Hq, Hkv=cfg.Hkv, D=cfg.D, Lmax=cfg.L, depth=cfg.depth, k=cfg.k, m=cfg.m, V=cfg.V,
                      logits_dtype=DT[cfg.logits_dtype], window=window, stochastic=True, sinks=sinks)
    dense = VerifyStep(shape, dev)
    dense.build(inp["draft_logits"])
    torch.cuda.synchronize()
    inp["target_logits"] = to_dev_logits(make_target_logits(cfg, 3, w.draft_logits, dense.tree.draft_row.cpu().numpy()),
                                         cfg.logits_dtype)
    dense.fused(inp)
    # pages between the sinks and the window are gone, the pool's other pages hold NaN
    seen = lambda b, i: i * ps < sinks or (i + 1) * ps > int(w.prefix_len[b]) - window + 1
    state = rng.bit_generator.state
    kp, table = paged(inp["k_cache"], w.prefix_len, ps, rng, keep=seen)
    rng.bit_generator.state = state
    vp, _ = paged(inp["v_cache"], w.prefix_len, ps, rng, keep=seen)
    pinp = dict(inp, k_cache=kp, v_cache=vp, block_table=table)
    pshape = StepShape(**{**shape.__dict__, "paged": True, "Lmax": table.shape[1] * ps})
    one, sep = VerifyStep(pshape, dev), VerifyStep(pshape, dev)
    one.fused(pinp)
    sep(pinp)
    torch.cuda.synchronize()
    one.fused_attention_status()
    assert torch.equal(one.out.view(torch.int16), sep.out.view(torch.int16))
    for f in ("accepted_len", "path", "bonus"):
        assert torch.equal(getattr(one, f), getattr(sep, f)) and torch.equal(getattr(one, f), getattr(dense, f)), f
    for b in range(min(B, 2)):
        ref, s = reference(dec(w.q[b]), dec(w.k_cache[b]), dec(w.v_cache[b]), int(w.prefix_len[b]), dec(w.k_tree[b]),
                           dec(w.v_tree[b]), one.tree.parents[b].cpu().numpy(), one.tree.depth[b].cpu().numpy(),
                           window=window, sinks=sinks)
        check_attention(one.out[b].float().cpu().numpy(), ref, s)
    graph = torch.cuda.CUDAGraph()
    want = [t.clone() for t in (one.out, one.accepted_len, one.path, one.bonus)]
    with torch.cuda.graph(graph):
        one.fused(pinp)
    for t in (one.out, one.accepted_len, one.path, one.bonus):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for t, v in zip((one.out, one.accepted_len, one.path, one.bonus), want):
        assert torch.equal(t, v)
    table[0, 0] = -1                                     # a page of the sinks
    one.fused(pinp)
    with pytest.raises(Exception, match="status 3"):
        one.fused_attention_status()
