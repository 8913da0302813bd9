"""Calls with `stream=`: their results on a stream of the caller's, from memory of that stream's own pool.

The caller orders the streams with wait_stream on both sides, as the calls ask; nothing else synchronises.
"""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
TOKENS, K, E, HIDDEN = 300, 2, 8, 264


def layer_inputs():
    g = torch.Generator().manual_seed(4)
    ids = torch.rand((TOKENS, E), generator=g).topk(K, dim=1).indices.to(DEV)
    x = torch.randn((TOKENS, HIDDEN), generator=g).bfloat16().to(DEV)
    w = torch.softmax(torch.randn((TOKENS, K), generator=g), 1).to(DEV)
    return ids, x, w


def layer(ids, x, w, stream=None):
    counts, offsets, row_of, src_of = kgw.kgw_moe_sort(ids, E, stream=stream)
    rows = kgw.kgw_moe_permute(x, row_of, src_of, stream=stream)
    out = kgw.kgw_moe_unpermute(rows, row_of, w, stream=stream)
    return (counts, offsets, row_of, src_of, rows, out) + kgw.kgw_moe_unpermute_grad(x, rows, row_of, src_of, w,
                                                                                     stream=stream)


def newton(G, stream=None):
    return tuple(kgw.kgw_newton_schulz(G, out_dtype=out, stream=stream) for out in (torch.bfloat16, torch.float32))


def gradients(*shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(7)).to(DEV)


def products(a, b, rows, w, offsets, stream=None):
    q = kgw.kgw_quantize_fp8(a, 1, stream=stream) + kgw.kgw_quantize_fp8(b, 0, stream=stream)
    return (kgw.kgw_wgrad_bf16(a, b, offsets, stream=stream), kgw.kgw_wgrad_bf16_ex(a, b, offsets, stream=stream),
            kgw.kgw_mgrouped_bf16(rows, w, offsets=offsets, stream=stream), *q,
            kgw.kgw_wgrad_fp8(q[0], q[1], q[2], q[3], offsets, stream=stream),
            kgw.kgw_check_offsets(offsets, a.shape[1], 256, stream=stream))


def product_inputs():
    g = torch.Generator().manual_seed(5)
    counts = torch.tensor([4096, 0, 8192, 256])
    tokens = int(counts.sum())
    new = lambda *shape: torch.randn(shape, generator=g).bfloat16().to(DEV)  # noqa: E731
    return new(256, tokens), new(tokens, 384), new(tokens, 64), new(4, 128, 64), torch.cumsum(counts, 0).int().to(DEV)


CASES = {"products": (products, product_inputs), "layer": (layer, layer_inputs), "newton short": (newton, lambda: (gradients(2, 100, 300),)),
         "newton": (newton, lambda: (gradients(3, 200, 300),))}


@pytest.mark.parametrize("name", CASES)
def test_results_on_a_given_stream(name):
    run, make = CASES[name]
    inputs = make()
    want = run(*inputs)
    s = torch.cuda.Stream()
    for _ in range(3):
        inputs = make()                                  # written on the caller's stream ...
        s.wait_stream(torch.cuda.current_stream())
        got = run(*inputs, stream=s)
        del inputs                                       # ... let go of before the call's work is done ...
        again = make()                                   # ... and its memory written anew
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del again


@pytest.mark.parametrize("name", CASES)
def test_memory_is_the_streams_own(name):
    run, make = CASES[name]
    inputs = make()
    s = torch.cuda.Stream()
    run(*inputs)                                         # leaves blocks of every size free on the caller's stream
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    free = {b["address"] for seg in torch.cuda.memory_snapshot() if seg["stream"] == torch.cuda.current_stream().cuda_stream
            for b in seg["blocks"] if b["state"] == "inactive"}
    got = run(*inputs, stream=s)
    assert free and not free & {t.untyped_storage().data_ptr() for t in got}
    torch.cuda.current_stream().wait_stream(s)


def test_given_outputs_and_workspace():
    G = gradients(2, 200, 300)
    want = kgw.kgw_newton_schulz(G)
    need = kgw.load_library().kgw_newton_schulz_workspace_bytes(2, 200, 300, kgw.KGW_OUT_FP32)
    s = torch.cuda.Stream()
    out, ws = torch.empty_like(G), torch.empty(need, dtype=torch.uint8, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    assert kgw.kgw_newton_schulz(G, out=out, workspace=ws, stream=s) is out
    del ws
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want)
