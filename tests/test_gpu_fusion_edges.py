"""The fused Q/K normalisation without an epsilon: rows past a chunk's end have no norm.  References and tolerances of
test_gpu_fusion."""
import pytest
import torch

from gated_delta_rule_27_gb300 import libkda
from oracle import oracle, sublayer
from tests.gpu_helpers import TOL, dev, f64, rel
from tests.test_gpu_fusion import _raw_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [[1], [63], [64, 65], [150, 77, 300]], ids=str)
@pytest.mark.parametrize("dtype,d,chunk,plan", [
    (torch.bfloat16, 128, 64, libkda.PLAN_THREE), (torch.bfloat16, 128, 64, libkda.PLAN_CHAIN), (torch.bfloat16, 128, 64, libkda.PLAN_PIPE),
    (torch.float32, 64, 32, libkda.PLAN_AUTO), (torch.bfloat16, 16, 16, libkda.PLAN_AUTO)],
    ids=["tc-three", "tc-chain", "tc-pipe", "simt-f32", "simt-bf16-d16"])
def test_norms_without_an_epsilon(lengths, dtype, d, chunk, plan):
    inp, q, k, _, _ = _raw_inputs(lengths, H=2, d=d, dtype=dtype, seed=151)
    o_ref, S_ref, _ = oracle.run(sublayer.l2norm(f64(q), 0.0), sublayer.l2norm(f64(k), 0.0), f64(inp.v), f64(inp.g), f64(inp.beta),
                                 inp.cu_seqlens.numpy(), S0=f64(inp.S0))
    x = [t.to(dev()) for t in (q, k, inp.v, inp.g, inp.beta, inp.cu_seqlens)]
    o = torch.full((inp.total_tokens, 2, d), float("nan"), dtype=dtype, device=dev())
    S = torch.full((len(lengths), 2, d, d), float("nan"), device=dev())
    libkda.testing_set_plan(plan)
    try:
        libkda.kda_prefill_chunked_ex(*x, o, S0=inp.S0.to(dev()), S_final=S, chunk_size=chunk, qk_l2norm=True, qk_eps=0.0)
        torch.cuda.synchronize()
    finally:
        libkda.testing_set_plan(libkda.PLAN_AUTO)
    assert not o.isnan().any() and not S.isnan().any()
    assert rel(o, o_ref) <= TOL[dtype] and rel(S, S_ref) <= TOL[dtype]
