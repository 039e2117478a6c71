"""DSMoEQ8 without a GPU: where its buffers come from (the library's calls replaced by recorders)."""
import pytest
import torch

import mixture_experts_layer_score_b200 as M
from mixture_experts_layer_score_b200 import binding as B

CFG = M.make_cfg(d_model=64, n_routed=4, top_k=2, d_ff=64, max_tokens=8)


@pytest.fixture
def calls(monkeypatch):
    """A DSMoEQ8 whose buffers are on the CPU and whose library calls are recorded."""
    seen = {"alloc": [], "rows": []}

    def empty(stream, device, shapes):
        out = [torch.empty(s, dtype=t) for s, t in shapes]
        seen["alloc"] += [stream] * len(out)
        return out

    monkeypatch.setattr(B, "_empty", empty, raising=False)
    monkeypatch.setattr(B, "dsmoe_q8_quantize", lambda h, R, C, x, q, s, stream=None: None)
    monkeypatch.setattr(B, "dsmoe_norm_q8", lambda *a: None)
    monkeypatch.setattr(B, "dsmoe_forward_q8", lambda h, T, x, xq, xs, *a: seen["rows"].append((xq, xs)))
    layer = M.DSMoEQ8.__new__(M.DSMoEQ8)
    layer.cfg, layer.device, layer.handle, layer.w, layer.q = CFG, 0, None, {}, {}
    layer.k_active, layer.range_flags, layer._weights = 2, M.DSMOE_RANGE_ADD_SHARED, M.DsmoeQ8Weights()
    seen["layer"] = layer
    return seen


def test_rows_are_kept_with_the_outputs(calls):
    """A second call with the same `out` writes the first call's 8-bit rows again; it does not let
    them go while the first call may still read them."""
    layer, x = calls["layer"], torch.zeros(3, 64, dtype=torch.bfloat16)
    out = layer.alloc_outputs(3)
    layer.forward(x, out=out, stream=5)
    layer.forward(x, out=out, stream=5)
    assert calls["rows"][0][0] is calls["rows"][1][0] is out["x_q"][0]
    assert calls["rows"][0][1] is calls["rows"][1][1] is out["x_q"][1]
    layer.forward(x[:2], out=layer.alloc_outputs(2) | {"x_q": out["x_q"]})  # of another length: new ones
    assert calls["rows"][2][0].shape == (2, 64) and calls["rows"][2][1].shape == (2, 4)
    mine = layer.alloc_rows(3)
    layer.forward(x, out=out, x_q=mine)
    assert calls["rows"][3][0] is mine[0] and out["x_q"][0] is calls["rows"][0][0]


@pytest.mark.parametrize("stream", [None, 5])
def test_buffers_are_allocated_for_the_stream(calls, stream):
    layer, x = calls["layer"], torch.zeros(3, 64, dtype=torch.bfloat16)
    layer.forward(x, stream=stream)
    layer.forward_norm(x, None, None, 1e-6, stream=stream)
    assert len(calls["alloc"]) == 9 + 11 and set(calls["alloc"]) == {stream}
