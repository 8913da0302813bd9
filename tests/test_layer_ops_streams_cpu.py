"""The router, the activation and the weight gradient from 8-bit rows with `stream=`: results and workspaces come from the
launch stream's pool, and what the caller gave is kept for it (no GPU; the library is a stand-in)."""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw
from test_streams_cpu import index, watch  # noqa: F401  (a fixture)

CALLS = {
    "route": (lambda s, t: kgw.kgw_moe_route(t["scores"], 2, mask=t["mask"], stream=s), ("scores", "mask"), 1),
    "route given": (lambda s, t: kgw.kgw_moe_route(t["scores"], 2, ids=t["ids"], stream=s), ("scores", "ids"), 1),
    "route_grad": (lambda s, t: kgw.kgw_moe_route_grad(t["scores"], t["ids"], t["w"], dloss=t["one"], slope=t["slope"],
                                                       mask=t["mask"], stream=s),
                   ("scores", "ids", "w", "one", "slope", "mask"), 1),
    "act": (lambda s, t: kgw.kgw_moe_act_fp8(t["h"], offsets=t["offsets"], stream=s), ("h", "offsets"), 3),
    "act fp8": (lambda s, t: kgw.kgw_moe_act_fp8(t["h"], fp8=True, out=t["codes"], stream=s), ("h", "codes"), 3),
    "act_grad": (lambda s, t: kgw.kgw_moe_act_fp8_grad(t["dy"], t["kept"], t["ks"], offsets=t["offsets"], again=True, stream=s),
                 ("dy", "kept", "ks", "offsets"), 2),
    "act_grad fp8": (lambda s, t: kgw.kgw_moe_act_fp8_grad(t["dy"], t["kept"], t["ks"], fp8=True, again=True, y=t["codes"],
                                                           stream=s), ("dy", "kept", "ks", "codes"), 3),
    "wgrad_fp8_rows": (lambda s, t: kgw.kgw_wgrad_fp8_rows(t["codes"], t["sc"], t["dy"], t["offsets"], stream=s),
                       ("codes", "sc", "dy", "offsets"), 2),
    "wgrad_fp8_rows fp8": (lambda s, t: kgw.kgw_wgrad_fp8_rows(t["codes"], t["sc"], t["kept"], t["offsets"], sb=t["ks"],
                                                               out=t["out"], stream=s),
                           ("codes", "sc", "kept", "ks", "offsets", "out"), 1),
}


def tensors():
    bytes_ = lambda *shape: torch.zeros(shape, dtype=torch.uint8)  # noqa: E731
    return dict(scores=torch.zeros(6, 16), mask=torch.ones(6, dtype=torch.bool), ids=index(6, 2), w=torch.zeros(6, 2),
                one=torch.zeros(()), slope=torch.zeros(16), h=torch.zeros((256, 256), dtype=torch.bfloat16),
                dy=torch.zeros((256, 128), dtype=torch.bfloat16), kept=bytes_(256, 256), ks=bytes_(2, 256),
                codes=bytes_(256, 128), sc=bytes_(1, 256), offsets=torch.tensor([128, 256], dtype=torch.int32),
                out=torch.zeros((2, 128, 256)))


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_launch_stream(watch, name):  # noqa: F811
    launch, made, recorded = watch
    call, used, count = CALLS[name]
    inputs = tensors()
    call(launch, inputs)
    assert [who for who, _ in made] == ["launch"] * count
    for _, t in made:
        assert "caller" in recorded[t.untyped_storage().data_ptr()]
    for k in used:
        assert "launch" in recorded[inputs[k].untyped_storage().data_ptr()], k
