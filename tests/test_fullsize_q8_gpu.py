"""The 8-bit layer at full size (V3-shaped prefill: T = 8192, d = 7168, 256 routed + 1 shared experts
of d_ff = 2048, top-8; V4-shaped decode of 256 tokens; the 2B-shaped layer), stage by stage from what
the stage before left in the workspace.

The routing is the bf16 layer's over every token. For whole experts, the highest-numbered ones that
received rows and the most loaded one: the gathered 8-bit rows byte by byte, the gate/up product's
8-bit rows from them and the down product's bf16 rows from those, against float64 with the
tolerances of tests/q8_cases.py. On sampled token rows, the last ones included: the shared experts'
fp32 rows from their own 8-bit rows (one shared expert), and h from all of it: h is the bf16 rounding
(half a step, 2^-8) of at most 1 + K' fp32 terms."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_score_b200 as M
import workloads as W
from tests import q8_cases as C
from tests.gpu_cases import make_case, sample_rows
from tests.q8_cases import E8, F8, F64, values

pytestmark = pytest.mark.gpu

CASES = [("v3_prefill", 6), ("v4_decode_t256", 24), ("ds2b", 6)]


def rows_of(view, R, n):
    """8-bit rows [R, n] and their scales out of a workspace buffer that holds [values | scales]."""
    raw, S = view.reshape(-1).view(torch.uint8), M.dsmoe_q8_scale_cols(n)
    return raw[:R * n].view(R, n).view(F8), raw[R * n:R * (n + S)].view(R, S).view(E8)


@pytest.mark.parametrize("name,n_experts", CASES)
def test_full_size(name, n_experts):
    cfg = W.get_config(name)
    T, d, F, K = cfg.T, cfg.d_model, cfg.d_ff, cfg.top_k
    gpu, _ = make_case(cfg, T, gen_device="cuda")
    wide = M.DSMoE(M.cfg_from(cfg, T), gpu)
    o16 = wide.forward(gpu["x"], with_scores=True)
    torch.cuda.synchronize()
    wide.close()
    layer = M.DSMoEQ8(M.cfg_from(cfg, T), gpu)
    g = torch.Generator(device="cuda").manual_seed(1)
    base = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    out = layer.forward(gpu["x"], with_scores=True, residual=base)
    torch.cuda.synchronize()
    assert M.dsmoe_get_status(layer.handle) == M.DSMOE_OK
    for k in ("topk_idx", "gates", "counts", "f", "P", "P_sum", "scores"):
        assert torch.equal(o16[k], out[k]), k
    ws = lambda n: M.workspace_view(layer.handle, n)  # noqa: E731
    R = T * K
    off, slot = ws("offsets")[0].long(), ws("slot_of")[:T].long()
    assert torch.equal(off, torch.cat([off.new_zeros(1), out["counts"].long().cumsum(0)]))
    assert torch.equal(slot.reshape(-1).sort().values, torch.arange(R, device="cuda"))
    xp, a1, y = rows_of(ws("Xp"), R, d), rows_of(ws("A1"), R, F), ws("Y")
    expert = torch.searchsorted(off[1:].contiguous(), slot.reshape(-1), right=True)
    assert torch.equal(expert.view(T, K), out["topk_idx"].long())
    at = torch.empty(R, dtype=torch.long, device="cuda")  # the token of each slot
    at[slot.reshape(-1)] = torch.arange(T, device="cuda").repeat_interleave(K)
    for mine, rows in zip(xp, out["x_q"]):  # the gathered rows, all of them
        assert torch.equal(mine.view(torch.uint8), rows.view(torch.uint8)[at])
    used = torch.nonzero(out["counts"]).view(-1).tolist()
    for e in sorted({*used[-(n_experts - 1):], int(out["counts"].argmax())}):
        s = slice(int(off[e]), int(off[e + 1]))
        w = [values(layer.q[n][0][e], layer.q[n][1][e]) for n in ("W_gate", "W_up", "W_down")]
        C.check_gated(values(xp[0][s], xp[1][s]), w[0], w[1], a1[0][s], a1[1][s])
        C.check_plain(values(a1[0][s], a1[1][s]), w[2], y[s])
    rows = torch.from_numpy(np.union1d(sample_rows(T, 256), np.arange(max(0, T - 40), T))).cuda()
    total = base[rows].to(F64)
    if cfg.n_shared:
        hs = ws("Hs")[rows].to(F64)
        if cfg.n_shared == 1:
            m = rows_of(ws("A1s"), T, cfg.d_ff_shared)
            ref, err = C.sums(values(m[0][rows], m[1][rows]), values(layer.q["Ws_down"][0][0], layer.q["Ws_down"][1][0]))
            assert bool(((hs - total - ref).abs() <= err + 2.0 ** -23 * (total + ref).abs()).all())
        total = hs
    terms = out["gates"][rows].to(F64)[..., None] * y[slot[rows]].to(F64)
    total, mag = total + terms.sum(1), total.abs() + terms.abs().sum(1)
    assert bool(((out["h"][rows].to(F64) - total).abs() <= 2.0 ** -8 * total.abs() + (K + 2) * 2.0 ** -23 * mag).all())
    layer.close()
