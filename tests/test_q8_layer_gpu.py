"""The 8-bit layer (binding.DSMoEQ8) on a caller's stream."""
import pytest
import torch

import mixture_experts_layer_score_b200 as M
import workloads as W
from tests.gpu_cases import make_case

pytestmark = pytest.mark.gpu


def busy(ms=20):
    """About `ms` of work queued on the current stream."""
    torch.cuda._sleep(int(ms * 1.5e6))


@pytest.fixture(scope="module")
def case():
    cfg, T = W.get_config("tiny"), 512
    gpu, _ = make_case(cfg, T)
    layer = M.DSMoEQ8(M.cfg_from(cfg, T), gpu)
    xs = [torch.randn(T, cfg.d_model, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(3)]
    want = [layer.forward(x)["h"].clone() for x in xs]
    torch.cuda.synchronize()
    yield layer, xs, want
    assert M.dsmoe_get_status(layer.handle) == M.DSMOE_OK
    layer.close()


def test_outputs_reused_on_a_side_stream(case):
    """Calls with one `out` on a side stream, which is behind; the current stream allocates and writes
    tensors of every buffer's size in between."""
    layer, xs, want = case
    side = torch.cuda.Stream()
    out = layer.alloc_outputs(xs[0].shape[0])
    torch.cuda.synchronize()
    got = []
    for x in xs:
        with torch.cuda.stream(side):
            busy()
        layer.forward(x, out=out, stream=side)
        with torch.cuda.stream(side):
            got.append(out["h"].clone())
        for t in (out["x_q"][0], out["x_q"][1]):
            for _ in range(4):
                torch.empty(t.shape, dtype=torch.uint8, device="cuda").fill_(77)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_what_the_current_stream_still_reads_is_not_taken(case):
    """Tensors of every buffer's size that were just freed on the current stream, whose reads are
    still to come there: a call on a side stream that allocates its outputs does not write to them."""
    layer, xs, want = case
    side = torch.cuda.Stream()
    T, d = xs[0].shape
    o = layer.forward(xs[0])
    sizes = [t.numel() * t.element_size() for k, t in o.items() if t is not None and k != "x_q"]
    sizes += [t.numel() for t in o["x_q"]] + [2 * T * d] * 2
    del o
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    kept = [torch.empty_like(t) for t in old]
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    busy()
    for a, b in zip(kept, old):
        a.copy_(b)
    del old, a, b
    first = layer.forward(xs[0], stream=side)
    second = layer.forward_norm(xs[1], xs[2], w, 1e-6, stream=side)
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in kept)
    assert torch.equal(first["h"], want[0])
    again = layer.forward_norm(xs[1], xs[2], w, 1e-6)
    assert torch.equal(second["h"], again["h"])


def test_outputs_freed_while_the_current_stream_reads_them(case):
    """Outputs made on a side stream, read on the current one after waiting for it and then dropped:
    the next call on the side stream does not overwrite what is still being read."""
    layer, xs, want = case
    side = torch.cuda.Stream()
    kept = []
    for x in xs:
        o = layer.forward(x, stream=side.cuda_stream)
        torch.cuda.current_stream().wait_stream(side)
        busy()
        kept.append(o["h"].clone())
        del o
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))
