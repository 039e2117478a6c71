"""The layer on 8-bit rows and weights (dsmoe_forward_q8, binding.DSMoEQ8) against the float64
layer of the same 8-bit operands.

The reference dequantises the kernel's own 8-bit rows and weights and quantises each SwiGLU row
by the definition. What separates the kernel from it: fp32 sums, a bf16 rounding of each
expert row and one of h (the layer's own bound of 2e-2 of the RMS of h, tests/parity.py), and
SwiGLU values that the fp32 sums carry across an e4m3 border, each moving one of F terms of a
row by 2^-3: below 1% of an expert row's RMS from F = 128 on."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_score_b200 as M
import workloads as W
from oracle import dsmoe_q8 as Q
from tests import parity as PAR
from tests.gpu_cases import make_case, sample_rows

pytestmark = pytest.mark.gpu
NP = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
BYTES = lambda t: t.detach().cpu().view(torch.uint8).numpy()  # noqa: E731

CASES = [("tiny", 1), ("tiny", 300), ("gshard_c", 200), ("ds2b", 520), ("v4_decode_slice", 16), ("v4_hash_t16", 16)]


class Weights:
    """Dequantised experts of a DSMoEQ8, fetched on first use."""

    def __init__(self, layer):
        self.layer, self.seen = layer, {}

    def __call__(self, name, e):
        if (name, e) not in self.seen:
            q, s = self.layer.q[name]
            self.seen[name, e] = Q.dequantize_weights(BYTES(q[e:e + 1]), BYTES(s[e:e + 1]))[0]
        return self.seen[name, e]


def ffn(w, prefix, e, u):
    m = Q.silu(u @ w(prefix + "_gate", e).T) * (u @ w(prefix + "_up", e).T)
    return Q.dequantize_rows(*Q.quantize_rows(m)) @ w(prefix + "_down", e).T


def reference(layer, u, base, idx, gates, n_shared, rows, experts=None):
    """h at `rows`: u the dequantised 8-bit rows, idx and gates the layer's routing."""
    w = Weights(layer)
    out = base[rows].copy()
    for i in range(n_shared):
        out += ffn(w, "Ws", i, u[rows])
    lo = 0 if experts is None else experts[0]
    for e in np.unique(idx[rows]):
        if experts is not None and not experts[0] <= e < experts[1]:
            continue
        t, k = np.nonzero(idx[rows] == e)
        out[t] += gates[rows][t, k][:, None] * ffn(w, "W", int(e) - lo, u[rows][t])
    return out


def near(h, ref):
    return np.abs(h - ref).max() / np.sqrt(np.mean(ref ** 2)) <= PAR.H_TOL


@pytest.mark.parametrize("name,T", CASES)
def test_layer(name, T):
    cfg = W.get_config(name)
    gpu, _ = make_case(cfg, T)
    ids = gpu.get("token_ids")
    wide = M.DSMoE(M.cfg_from(cfg, T), gpu)
    o16 = wide.forward(gpu["x"], token_ids=ids, with_scores=True)
    layer = M.DSMoEQ8(M.cfg_from(cfg, T), gpu)
    out = layer.forward(gpu["x"], token_ids=ids, with_scores=True)
    torch.cuda.synchronize()
    for k in ("topk_idx", "gates", "counts", "f", "P", "P_sum", "scores"):  # the routing is the bf16 layer's
        assert (o16[k] is None) == (out[k] is None) and (out[k] is None or torch.equal(o16[k], out[k])), k
    rows = sample_rows(T, 24)
    u = Q.dequantize_rows(*Q.quantize_rows(NP(gpu["x"])))
    idx, gates = out["topk_idx"].cpu().numpy(), NP(out["gates"])
    assert near(NP(out["h"])[rows], reference(layer, u, NP(gpu["x"]), idx, gates, cfg.n_shared, rows))
    # the 8-bit operands themselves: three roundings of at most 2^-4 in each expert term
    part = NP(o16["h"]) - NP(gpu["x"])
    off = np.linalg.norm(NP(out["h"]) - NP(o16["h"]))
    assert off <= 3 * 2.0 ** -4 * np.linalg.norm(part) + 2.0 ** -8 * np.linalg.norm(NP(o16["h"]))
    # rows that the caller has quantised, and a base that is not x
    x_q = layer.alloc_rows(T)
    M.dsmoe_q8_quantize(layer.handle, T, cfg.d_model, gpu["x"], *x_q)
    assert torch.equal(layer.forward(gpu["x"], token_ids=ids, x_q=x_q)["h"], out["h"])
    base = torch.randn(T, cfg.d_model, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    o = layer.forward(gpu["x"], token_ids=ids, x_q=x_q, residual=base)
    assert near(NP(o["h"])[rows], reference(layer, u, NP(base), idx, gates, cfg.n_shared, rows))
    assert M.dsmoe_get_status(layer.handle) == M.DSMOE_OK
    wide.close()
    layer.close()


def test_block_with_norm_selection_and_a_graph():
    """norm -> layer as a block, under a selection variant, eager and as a replayed graph on new
    input values."""
    cfg, T = W.get_config("tiny"), 137
    gpu, _ = make_case(cfg, T)
    layer = M.DSMoEQ8(M.cfg_from(cfg, T), gpu)
    layer.set_selection(mask_top=1, k_active=5)
    d = cfg.d_model
    g = torch.Generator().manual_seed(1)
    res = torch.randn(T, d, generator=g).bfloat16().cuda()
    w = (1 + 0.2 * torch.randn(d, generator=g)).bfloat16().cuda()
    o = layer.forward_norm(gpu["x"], res, w, 1e-6)
    r = Q.add_residual(NP(gpu["x"]), NP(res))
    np.testing.assert_array_equal(NP(o["r"]), r)
    u = Q.dequantize_rows(*Q.quantize_rows(NP(o["u"])))
    rows = sample_rows(T, 16)
    idx = o["topk_idx"].cpu().numpy()
    assert idx.shape == (T, 5)
    assert near(NP(o["h"])[rows], reference(layer, u, r, idx, NP(o["gates"]), cfg.n_shared, rows))

    x = gpu["x"].clone()
    bufs = [torch.empty_like(x), torch.empty_like(x), *layer.alloc_rows(T)]
    out = layer.alloc_outputs(T)

    def block():
        M.dsmoe_norm_q8(layer.handle, T, x, res, w, 1e-6, *bufs)
        layer.forward(bufs[1], out=out, residual=bufs[0], x_q=bufs[2:])

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        block()
    torch.cuda.synchronize()
    assert torch.equal(out["h"], o["h"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        block()
    x.copy_(torch.randn(T, d, generator=g).bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    replayed = out["h"].clone()
    block()
    torch.cuda.synchronize()
    assert torch.equal(replayed, out["h"]) and not torch.equal(replayed, o["h"])
    assert M.dsmoe_get_status(layer.handle) == M.DSMOE_OK
    del graph
    layer.close()


def test_expert_ranges_add_up():
    """fp32 partial sums of two blocks of experts, the first with the shared expert and the base."""
    cfg, T = W.get_config("tiny"), 90
    gpu, _ = make_case(cfg, T)
    N, total = cfg.n_routed, 0
    for e0, e1 in ((0, 20), (20, N)):
        part = {k: (v[e0:e1] if k in ("W_gate", "W_up", "W_down") else v) for k, v in gpu.items()}
        layer = M.DSMoEQ8(M.cfg_from(cfg, T), part)
        layer.set_expert_range(e0, e1, partial=True, add_shared=e0 == 0)
        out = layer.forward(gpu["x"])
        assert out["h"].dtype == torch.float32
        u = Q.dequantize_rows(*Q.quantize_rows(NP(gpu["x"])))
        idx, gates = out["topk_idx"].cpu().numpy(), NP(out["gates"])
        base = NP(gpu["x"]) if e0 == 0 else np.zeros((T, cfg.d_model))
        ref = reference(layer, u, base, idx, gates, cfg.n_shared if e0 == 0 else 0, np.arange(T), (e0, e1))
        assert np.abs(NP(out["h"]) - ref).max() / np.sqrt(np.mean(NP(gpu["x"]) ** 2)) <= PAR.H_TOL
        total = total + out["h"]
        layer.close()
    layer = M.DSMoEQ8(M.cfg_from(cfg, T), gpu)
    whole = layer.forward(gpu["x"])["h"]
    # the same terms added in another order, then rounded to bf16
    assert (np.abs(NP(total) - NP(whole)) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(NP(total)) + 2.0 ** -18).all()
    layer.close()


def test_a_training_forward_is_forgotten_and_no_tokens():
    cfg, T = W.get_config("tiny"), 64
    gpu, _ = make_case(cfg, T)
    layer = M.DSMoEQ8(M.cfg_from(cfg, T), gpu)
    M.dsmoe_set_training(layer.handle, True)
    out = layer.alloc_outputs(T)
    M.dsmoe_forward(layer.handle, T, gpu["x"], None, gpu["W_router"], None, gpu["W_gate"], gpu["W_up"], gpu["W_down"],
                    gpu["Ws_gate"], gpu["Ws_up"], gpu["Ws_down"], out["h"], out["topk_idx"], out["gates"],
                    out["counts"], out["f"], out["P"])
    layer.forward(gpu["x"])
    dh, dY = torch.zeros_like(gpu["x"]), torch.zeros(T * cfg.top_k, cfg.d_model, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(M.DsmoeError) as e:
        M.dsmoe_backward_experts(layer.handle, T, dh, dY, gpu["W_gate"], gpu["W_up"], gpu["W_down"], gpu["Ws_gate"],
                                 gpu["Ws_up"], gpu["Ws_down"], None, torch.empty(T, cfg.d_model, device="cuda"))
    assert e.value.status == M.DSMOE_ERR_INVALID_ARG
    empty = layer.forward(gpu["x"][:0])
    torch.cuda.synchronize()
    assert empty["h"].shape == (0, cfg.d_model) and not empty["counts"].any() and not empty["P"].any()
    for bad in (dict(x_q=(None, None)), dict(residual=gpu["x"].view(-1)[1:1 + 63 * cfg.d_model])):
        with pytest.raises((M.DsmoeError, TypeError)):
            layer.forward(gpu["x"], **bad)
    torch.cuda.synchronize()
    layer.close()


def test_training_with_a_norm_in_front():
    """A training step of norm -> layer: the layer's dx is the norm's dy; the norm's gradients against
    the float64 formula fed the kernel's dx (dx: half a bf16 step, and fp32 sums)."""
    cfg, T = W.get_config("tiny"), 96
    gpu, _ = make_case(cfg, T)
    d, K = cfg.d_model, cfg.top_k
    g = torch.Generator().manual_seed(5)
    r = torch.randn(T, d, generator=g).bfloat16().cuda()
    w = (1 + 0.2 * torch.randn(d, generator=g)).bfloat16().cuda()
    dh = torch.randn(T, d, generator=g).bfloat16().cuda()
    layer = M.DSMoE(M.cfg_from(cfg, T), gpu)
    M.dsmoe_set_training(layer.handle, True)
    u = torch.empty_like(r)
    M.dsmoe_norm_q8(layer.handle, T, r, None, w, 1e-6, None, u, None, None)
    out = layer.forward(u, with_scores=True)
    f32 = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    dg, dY = f32(T, K), torch.empty(T * K, d, dtype=torch.bfloat16, device="cuda")
    M.dsmoe_backward_gates(layer.handle, T, dh, out["gates"], dg, dY)
    dxr, du = f32(T, d), f32(T, d)
    M.dsmoe_backward_router(layer.handle, T, u, gpu["W_router"], out["topk_idx"], out["gates"], out["scores"], dg, None,
                            0.0, f32(T, cfg.n_routed), dxr, f32(cfg.n_routed, d))
    M.dsmoe_backward_experts(layer.handle, T, dh, dY, gpu["W_gate"], gpu["W_up"], gpu["W_down"], gpu["Ws_gate"],
                             gpu["Ws_up"], gpu["Ws_down"], dxr, du)
    dx, dw = torch.empty_like(r), f32(d)
    M.dsmoe_norm_backward(layer.handle, T, du, None, r, w, 1e-6, dx, dw)
    ex, ew = Q.norm_backward(NP(du), None, NP(r), NP(w), 1e-6)
    assert np.abs(NP(dx) - ex).max() <= 2.0 ** -8 * np.abs(ex).max() + 1e-4 * np.sqrt(np.mean(ex ** 2))
    assert np.linalg.norm(NP(dw) - ew) <= 1e-5 * np.linalg.norm(ew) + 1e-6
    assert M.dsmoe_get_status(layer.handle) == M.DSMOE_OK
    layer.close()


def test_weights_are_ready_for_any_stream():
    """Constructing from bf16 weights waits for their quantisation, queued behind earlier work of
    the current stream: a forward on another stream follows without an event."""
    cfg, T = W.get_config("tiny"), 64
    gpu, _ = make_case(cfg, T)
    ref = M.DSMoEQ8(M.cfg_from(cfg, T), gpu)
    want = ref.forward(gpu["x"])["h"]
    busy = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    out, side = torch.empty_like(busy), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        torch.mm(busy, busy, out=out)
    layer = M.DSMoEQ8(M.cfg_from(cfg, T), gpu)
    assert torch.cuda.current_stream().query()
    o = layer.forward(gpu["x"], stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(o["h"], want)
    ref.close()
    layer.close()
