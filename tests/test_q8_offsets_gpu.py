"""Offsets that decrease: the grouped products read them as their running maximum, so they give the
bits of a call with that maximum (whose values tests/test_q8_gpu.py checks), leave the other rows
as they were, and no role of the kernel waits for a tile that no other role works on."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_score_b200 as M

from tests.test_q8_gpu import BYTES, q8_empty, rows

pytestmark = pytest.mark.gpu

CASES = [  # offsets, R, N, K
    ([0, 500] * 16 + [0], 500, 256, 1024),               # a cluster per tile, more groups than tiles
    ([0, 500] * 16 + [0], 500, 256, 128),                # 32-token tiles
    ([-5, 300, 100, 200, 400, 390, 900, 10, 600], 600, 1024, 1280),
    ([0, 2000] * 40 + [7], 2000, 2048, 256),             # more than 32 groups
    ([1999, 5, 1500, -1, 2100, 1800], 1900, 1280, 2048),  # the first is the largest but one
    ([700, 100, 1200, 300, 1500], 1500, 2048, 5120),     # gated: chains, 160-token tiles; plain: 240
    ([700, 100, 1200, 300, 1500], 1500, 2048, 1408),     # 240-token tiles
    (list(range(0, 640, 10)) + [320] + list(range(650, 1280, 10)), 1300, 384, 640),
]


@pytest.mark.parametrize("off,R,N,K", CASES)
def test_decreasing_offsets_are_their_running_maximum(off, R, N, K):
    h = M.dsmoe_create(M.make_cfg(d_model=64, n_routed=1, top_k=1, d_ff=64, max_tokens=1))
    E = len(off) - 1
    x = rows(R, K, 1)
    W = [(rows(N, K, 2 + i, 0.3) * (K ** -0.5)).view(1, N, K).expand(E, N, K) * 2.0 ** (torch.arange(E) % 3 - 1)
         .to("cuda", torch.bfloat16)[:, None, None] for i in range(2)]
    a = q8_empty(R, K)
    M.dsmoe_q8_quantize(h, R, K, x, *a)
    w = []
    for t in W:
        q = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
        s = torch.empty(E, -(-N // 128), M.dsmoe_q8_scale_cols(K), dtype=torch.uint8, device="cuda")
        M.dsmoe_q8_quantize_weights(h, E, N, K, t.contiguous(), q, s)
        w += [q, s]
    top = np.maximum.accumulate(np.clip(off, 0, R))
    got = []
    for o in (off, top.tolist()):
        o = torch.tensor(o, dtype=torch.int32, device="cuda")
        y, (q, s) = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda"), q8_empty(R, N)
        q.view(torch.uint8).fill_(9)
        s.view(torch.uint8).fill_(9)
        M.dsmoe_q8_matmul(h, E, R, N, K, o, *a, *w[:2], y)
        M.dsmoe_q8_gated_matmul(h, E, R, N, K, o, *a, *w, q, s)
        torch.cuda.synchronize()
        assert M.dsmoe_get_status(h) == M.DSMOE_OK
        got.append((y.view(torch.int16).cpu().numpy(), BYTES(q), BYTES(s)))
    for mine, want in zip(*got):
        np.testing.assert_array_equal(mine, want)
    out = np.r_[0:top[0], top[-1]:R]
    y, q, s = got[0]
    seven = int(torch.tensor(7.0, dtype=torch.bfloat16).view(torch.int16))
    assert (y[out] == seven).all() and (q[out] == 9).all() and (s[out] == 9).all()
    if top[-1] > top[0]:
        inside = slice(top[0], top[-1])
        assert not (y[inside] == seven).all(axis=1).any() and not (s[inside] == 9).any()
    M.dsmoe_destroy(h)
