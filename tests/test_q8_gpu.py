"""The 8-bit path's operators on the GPU against the float64 definitions (oracle/dsmoe_q8.py).

Tolerances, from the arithmetic: quantisation is exact; a bf16 output is within half a step
(2^-8 of its value) of a value that carries the error of an fp32 sum, at most (number of
additions) 2^-24 of the sum of magnitudes (2^-23 where the tensor core may truncate); an 8-bit
output within half an e4m3 step (2^-4 of its value, or 2^-10 of its block's scale)."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_score_b200 as M
from oracle import dsmoe_q8 as Q

pytestmark = pytest.mark.gpu
EPS = 1e-6
NP = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
BYTES = lambda t: t.detach().cpu().view(torch.uint8).numpy()  # noqa: E731


@pytest.fixture(scope="module")
def handle():
    h = M.dsmoe_create(M.make_cfg(d_model=64, n_routed=1, top_k=1, d_ff=64, max_tokens=1))
    yield h
    assert M.dsmoe_get_status(h) == M.DSMOE_OK
    M.dsmoe_destroy(h)


def rows(R, C, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, C, generator=g) * torch.exp(spread * torch.randn(R, 1, generator=g))
    return x.bfloat16().cuda()


def q8_empty(R, C):
    return (torch.empty(R, C, dtype=torch.float8_e4m3fn, device="cuda"),
            torch.empty(R, M.dsmoe_q8_scale_cols(C), dtype=torch.float8_e8m0fnu, device="cuda"))


def q8_rows(x):
    """8-bit rows of a CPU/GPU bf16 tensor by the definition, on the GPU; and their values."""
    q, s = Q.quantize_rows(NP(x))
    return torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), Q.dequantize_rows(q, s)


def q8_weights(W):
    q, s = Q.quantize_weights(NP(W))
    return torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), Q.dequantize_weights(q, s)


# ------------------------------------------------------------------------- quantisation
@pytest.mark.parametrize("R,C", [(1, 16), (1, 128), (3, 144), (33, 704), (512, 256), (130, 1280), (7, 7168),
                                 (2, 32768)])
def test_quantize_rows(handle, R, C):
    x = rows(R, C, seed=R + C, spread=8.0)
    if R > 2:
        x[2] = 0
        x[0, :2] = torch.tensor([448.0, -448.0])
        x[1, 0] = 3.3e38
    q, s = q8_empty(R, C)
    M.dsmoe_q8_quantize(handle, R, C, x, q, s)
    eq, es = Q.quantize_rows(NP(x))
    np.testing.assert_array_equal(BYTES(s), es)
    np.testing.assert_array_equal(BYTES(q), eq)


def test_quantize_rows_not_finite(handle):
    x = rows(4, 300 // 16 * 16)
    x[0, 5], x[1, 200], x[2, 130] = float("inf"), float("nan"), float("-inf")
    q, s = q8_empty(*x.shape)
    M.dsmoe_q8_quantize(handle, *x.shape, x, q, s)
    eq, es = Q.quantize_rows(NP(x))
    np.testing.assert_array_equal(BYTES(s), es)
    np.testing.assert_array_equal(BYTES(q), eq)


@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (2, 128, 128), (3, 200, 144), (2, 72, 704), (1, 896, 1280)])
def test_quantize_weights(handle, E, N, K):
    W = (rows(E * N, K, seed=N)).view(E, N, K)
    q = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, -(-N // 128), M.dsmoe_q8_scale_cols(K), dtype=torch.uint8, device="cuda")
    M.dsmoe_q8_quantize_weights(handle, E, N, K, W, q, s)
    eq, es = Q.quantize_weights(NP(W))
    np.testing.assert_array_equal(BYTES(s), es)
    np.testing.assert_array_equal(BYTES(q), eq)


# --------------------------------------------------------------------------------- norm
NORM = [(1, 64), (3, 192), (16, 7168), (33, 1280), (257, 256), (5, 8192), (4, 8256), (3, 16448), (2, 32768)]


@pytest.mark.parametrize("T,d", NORM)
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm(T, d, with_residual):
    h = M.dsmoe_create(M.make_cfg(d_model=d, n_routed=1, top_k=1, d_ff=64, max_tokens=T))
    x, res = rows(T, d, 1), rows(T, d, 2) if with_residual else None
    w = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(5))).bfloat16().cuda()
    if T > 2:
        x[1] = 0
        if with_residual:
            res[1] = 0
    r, u = torch.empty_like(x), torch.empty_like(x)
    q, s = q8_empty(T, d)
    M.dsmoe_norm_q8(h, T, x, res, w, EPS, r, u, q, s)
    er = Q.add_residual(NP(x), None if res is None else NP(res))
    np.testing.assert_array_equal(NP(r), er)
    eu, _ = Q.norm(er, NP(w), EPS)
    # rounding, and the fp32 sum of d squares (at most 8 * 4 + 5 + 32 additions in a row), its
    # root and two products
    assert (np.abs(NP(u) - eu) <= (2.0 ** -8 + 80 * 2.0 ** -24) * np.abs(eu)).all()
    eq, es = Q.quantize_rows(NP(u))
    np.testing.assert_array_equal(BYTES(s), es)
    np.testing.assert_array_equal(BYTES(q), eq)
    # each output alone, and r in the place of the residual or x
    u2, (q2, s2) = torch.empty_like(x), q8_empty(T, d)
    M.dsmoe_norm_q8(h, T, x, res, w, EPS, None, u2, None, None)
    into = (x if res is None else res).clone()
    M.dsmoe_norm_q8(h, T, into if res is None else x, None if res is None else into, w, EPS, into, None, q2, s2)
    assert torch.equal(u, u2) and torch.equal(into, r)
    assert (BYTES(q2) == BYTES(q)).all() and (BYTES(s2) == BYTES(s)).all()
    M.dsmoe_destroy(h)


# (up to four rows one block adds dw itself, beyond that a second kernel does)
@pytest.mark.parametrize("T,d", NORM + [(1500, 128), (4, 1024), (5, 1024), (2, 7168), (20, 64)])
@pytest.mark.parametrize("with_dres", [False, True])
def test_norm_backward(T, d, with_dres):
    h = M.dsmoe_create(M.make_cfg(d_model=d, n_routed=1, top_k=1, d_ff=64, max_tokens=T + 3))
    g = torch.Generator().manual_seed(7)
    r, dres = rows(T, d, 3), rows(T, d, 4) if with_dres else None
    w = (1 + 0.3 * torch.randn(d, generator=g)).bfloat16().cuda()
    dy = torch.randn(T, d, generator=g).cuda()
    dx, dw = torch.empty_like(r), torch.empty(d, device="cuda")
    M.dsmoe_norm_backward(h, T, dy, dres, r, w, EPS, dx, dw)
    ex, ew = Q.norm_backward(NP(dy), None if dres is None else NP(dres), NP(r), NP(w), EPS)
    _, rstd = Q.norm(NP(r), NP(w), EPS)
    a1 = np.abs(rstd * NP(w) * NP(dy))
    a2 = np.abs(NP(r)) * rstd ** 3 * np.abs(NP(dy) * NP(w) * NP(r)).mean(axis=1, keepdims=True)
    a3 = 0 if dres is None else np.abs(NP(dres))
    assert (np.abs(NP(dx) - ex) <= 2.0 ** -8 * np.abs(ex) + 320 * 2.0 ** -24 * (a1 + a2 + a3)).all()
    assert (np.abs(NP(dw) - ew) <= (T + 160) * 2.0 ** -24 * np.abs(NP(dy) * NP(r) * rstd).sum(axis=0)).all()
    if dres is not None:  # in place, and again: the same bits
        again = dres.clone()
        dw2 = torch.empty_like(dw)
        M.dsmoe_norm_backward(h, T, dy, again, r, w, EPS, again, dw2)
        assert torch.equal(again, dx) and torch.equal(dw, dw2)
    M.dsmoe_norm_backward(h, 0, None, None, None, w, EPS, None, dw)
    assert (dw == 0).all()
    M.dsmoe_destroy(h)


# ----------------------------------------------------------------------------- products
def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32).cuda()


PRODUCTS = [  # counts of each expert, first row, rows behind the last, N, K
    ([1], 0, 0, 8, 16),
    ([1], 0, 0, 128, 128),
    ([3, 0, 1], 0, 0, 136, 144),
    ([0, 0], 0, 5, 64, 64),
    ([17, 5, 0, 130, 1], 3, 4, 264, 704),
    ([2, 1, 0, 3], 0, 0, 1000, 2048),
    ([250], 0, 1, 1280, 896),
    ([511, 240, 241, 16], 0, 0, 256, 528),
    ([300, 20], 0, 0, 512, 1296),
    ([600], 1, 0, 2304, 256),
    # few tiles: the CTAs of a cluster share one along K (8, 4 and 2 of them, uneven ranges)
    ([5], 0, 0, 1024, 7168),
    ([1], 1, 1, 776, 4624),
    ([32], 0, 0, 2048, 2064),
    ([0, 40, 3], 0, 2, 520, 1552),
    # ... of 112-token tiles
    ([128], 0, 0, 2048, 7168),
    ([111, 113, 160, 224], 1, 3, 600, 3968),
]


def check_product(handle, counts, first, behind, N, K, seed=0):
    E, R = len(counts), first + sum(counts) + behind
    x, W = rows(R, K, seed + 1), (rows(E * N, K, seed + 2, 0.3)).view(E, N, K)
    qa, sa, a = q8_rows(x)
    qw, sw, w = q8_weights(W)
    off = offsets_of(counts, first)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    M.dsmoe_q8_matmul(handle, E, R, N, K, off, qa, sa, qw, sw, out)
    o = [int(v) for v in off.cpu()]
    y, mag = Q.grouped(a, w, o), Q.grouped(np.abs(a), np.abs(w), o)
    got = NP(out)
    assert (got[:o[0]] == 7).all() and (got[o[-1]:] == 7).all()
    s = slice(o[0], o[-1])
    assert (np.abs(got - y)[s] <= (2.0 ** -8 * np.abs(y) + (K + 2) * 2.0 ** -23 * mag)[s]).all()
    return out


@pytest.mark.parametrize("counts,first,behind,N,K", PRODUCTS)
def test_product(handle, counts, first, behind, N, K):
    check_product(handle, counts, first, behind, N, K)


def check_gated(handle, counts, first, behind, N, K, seed=0, amp=1.0):
    E, R = len(counts), first + sum(counts) + behind
    x = rows(R, K, seed + 1)
    Wg, Wu = ((rows(E * N, K, seed + i, 0.3) * (amp / K ** 0.5)).view(E, N, K) for i in (2, 3))
    qa, sa, a = q8_rows(x)
    qg, sg, wg = q8_weights(Wg)
    qu, su, wu = q8_weights(Wu)
    off = offsets_of(counts, first)
    q, s = q8_empty(R, N)
    q.view(torch.uint8).fill_(9)
    s.view(torch.uint8).fill_(9)
    M.dsmoe_q8_gated_matmul(handle, E, R, N, K, off, qa, sa, qg, sg, qu, su, q, s)
    o = [int(v) for v in off.cpu()]
    sl = slice(o[0], o[-1])
    bq, bs = BYTES(q), BYTES(s)
    assert (bq[:o[0]] == 9).all() and (bq[o[-1]:] == 9).all() and (bs[:o[0]] == 9).all() and (bs[o[-1]:] == 9).all()
    if o[0] == o[-1]:
        return q, s
    g, u = Q.grouped(a, wg, o)[sl], Q.grouped(a, wu, o)[sl]
    eg, eu = ((K + 2) * 2.0 ** -23 * Q.grouped(np.abs(a), np.abs(v), o)[sl] for v in (wg, wu))
    m = Q.silu(g) * u
    # |SiLU'| <= 1.1; exp, the division and the product in fp32 at a few steps each
    em = 1.1 * eg * np.abs(u) + (np.abs(Q.silu(g)) + 1.1 * eg) * eu + 2.0 ** -18 * np.abs(m)
    nb = -(-N // 128)
    assert (bs[sl][:, nb:] == 127).all()
    step = np.repeat(Q.decode_scale(bs[sl][:, :nb]), 128, axis=1)[:, :N]
    v = Q.decode_e4m3(bq[sl]) * step
    assert (np.abs(v - m) <= np.maximum(2.0 ** -4 * np.abs(m), 2.0 ** -10 * step) * (1 + 2.0 ** -4) + em).all()
    for b in range(nb):  # the scale is the definition's, unless the maximum is within its error of a border
        part, err = np.abs(m[:, 128 * b:128 * b + 128]), em[:, 128 * b:128 * b + 128].max(axis=1)
        lo, hi = Q.scale_byte(np.maximum(part.max(axis=1) - err, 0)), Q.scale_byte(part.max(axis=1) + err)
        assert ((bs[sl][:, b] >= lo) & (bs[sl][:, b] <= hi)).all()
    return q, s


@pytest.mark.parametrize("counts,first,behind,N,K",
                         [(c, f, b, -(-N // 16) * 16, K) for c, f, b, N, K in PRODUCTS])
def test_gated(handle, counts, first, behind, N, K):
    check_gated(handle, counts, first, behind, N, K)


def test_gated_large_arguments(handle):
    """Gates far from zero (|g| of a few hundred): SiLU saturates, nothing overflows to NaN."""
    check_gated(handle, [20, 3], 0, 0, 144, 256, amp=200.0)


@pytest.mark.parametrize("T_exp", [-60, 50])
def test_product_far_scales(handle, T_exp):
    """Scales far from one: rows of 2^T_exp against weights of 2^-T_exp."""
    K, N, R = 256, 128, 5
    x = (rows(R, K).float() * 2.0 ** T_exp).bfloat16()
    W = (rows(N, K, 3, 0.1).float() * 2.0 ** -T_exp).bfloat16().view(1, N, K)
    qa, sa, a = q8_rows(x)
    qw, sw, w = q8_weights(W)
    out = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    M.dsmoe_q8_matmul(handle, 1, R, N, K, offsets_of([R]), qa, sa, qw, sw, out)
    y, mag = a @ w[0].T, np.abs(a) @ np.abs(w[0]).T
    assert (np.abs(NP(out) - y) <= 2.0 ** -8 * np.abs(y) + (K + 2) * 2.0 ** -23 * mag).all()


def test_product_nan_stays_in_its_row(handle):
    """A NaN block of one row makes that row NaN and no other, one of the weights its 128 features."""
    K, N, R = 384, 256, 40
    x, W = rows(R, K), rows(2 * N, K, 4, 0.2).view(2, N, K)
    x[7, 130] = float("inf")
    W[1, 200, 5] = float("nan")
    (qa, sa, _), (qw, sw, _) = q8_rows(x), q8_weights(W)
    out = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    M.dsmoe_q8_matmul(handle, 2, R, N, K, offsets_of([30, 10]), qa, sa, qw, sw, out)
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros((R, N), bool)
    want[7] = True
    want[30:, 128:] = True
    np.testing.assert_array_equal(nan, want)


def test_offsets_out_of_range_touch_nothing_else(handle):
    """Offsets are clipped to [0, R], a group that would end before it starts is empty, and rows
    that decreasing offsets give to two groups are one of the two's."""
    K, N, R = 128, 128, 40
    x, W = rows(R, K), rows(3 * N, K, 4, 0.2).view(3, N, K)
    (qa, sa, a), (qw, sw, w) = q8_rows(x), q8_weights(W)
    for off, owner in (([-5, 10, 8, 30], {0: range(0, 8), 2: range(10, 30)}), ([0, 50, 60, 70], {0: range(40)}),
                       ([60, 50, 90, 41], {})):
        out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
        M.dsmoe_q8_matmul(handle, 3, R, N, K, torch.tensor(off, dtype=torch.int32, device="cuda"), qa, sa, qw, sw, out)
        got = NP(out)
        for e, rs in owner.items():
            rs = list(rs)
            y, mag = a[rs] @ w[e].T, np.abs(a[rs]) @ np.abs(w[e]).T
            assert (np.abs(got[rs] - y) <= 2.0 ** -8 * np.abs(y) + (K + 2) * 2.0 ** -23 * mag).all()
        assert (got[min(30, off[-1]) if owner.get(2) else 40:] == 7).all() and (bool(owner) or (got == 7).all())
    assert M.dsmoe_get_status(handle) == M.DSMOE_OK


# ------------------------------------------------------------------------------ together
def test_norm_then_gated_then_product_on_a_stream_and_in_a_graph():
    """The operators as a program chains them, on a stream that is not the default one, then
    captured and replayed on new input values: the replay gives the eager call's bits."""
    T, d, F, E = 37, 256, 192, 1
    h = M.dsmoe_create(M.make_cfg(d_model=d, n_routed=1, top_k=1, d_ff=64, max_tokens=T))
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    Wg, Wu, Wd = (rows(o, i, k, 0.2).view(1, o, i) / 16 for k, (o, i) in enumerate(((F, d), (F, d), (d, F))))
    (qg, sg, wg), (qu, su, wu), (qd, sd, wd) = (q8_weights(W) for W in (Wg, Wu, Wd))
    off = offsets_of([T])
    x, res = rows(T, d, 1), rows(T, d, 2)
    r, u = torch.empty_like(x), torch.empty_like(x)
    q, s = q8_empty(T, d)
    mq, ms = q8_empty(T, F)
    y = torch.empty_like(x)

    def chain(stream):
        M.dsmoe_norm_q8(h, T, x, res, w, EPS, r, u, q, s, stream)
        M.dsmoe_q8_gated_matmul(h, E, T, F, d, off, q, s, qg, sg, qu, su, mq, ms, stream)
        M.dsmoe_q8_matmul(h, E, T, d, F, off, mq, ms, qd, sd, y, stream)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    chain(st)
    torch.cuda.synchronize()
    a = Q.dequantize_rows(BYTES(q), BYTES(s))
    m = Q.silu(a @ wg[0].T) * (a @ wu[0].T)
    got = Q.dequantize_rows(BYTES(mq), BYTES(ms))
    assert np.linalg.norm(got - m) <= 2.0 ** -4 * np.linalg.norm(m)
    ey = got @ wd[0].T
    assert (np.abs(NP(y) - ey) <= 2.0 ** -8 * np.abs(ey) + (F + 2) * 2.0 ** -23 * (np.abs(got) @ np.abs(wd[0]).T)).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        chain(st)
    x.copy_(rows(T, d, 11))
    chain(None)
    torch.cuda.synchronize()
    eager = y.clone()
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(eager, y) and float(y.float().abs().sum()) > 0
    assert M.dsmoe_get_status(h) == M.DSMOE_OK
    del graph
    M.dsmoe_destroy(h)


@pytest.mark.parametrize("counts,N,K", [([300, 41, 7], 256, 1024), ([3], 256, 7168)])  # persistent; a cluster per tile
def test_wait_limit_runs_out_then_the_handle_recovers(counts, N, K):
    """With a limit of 1 ns some role gives up, the kernel drains what it started and returns, the
    status says so once; with the default limit the same handle's products are right again."""
    h = M.dsmoe_create(M.make_cfg(d_model=64, n_routed=1, top_k=1, d_ff=64, max_tokens=1))
    M.dsmoe_set_wait_limit(h, 1)
    E, R = len(counts), sum(counts)
    q = torch.zeros(R, K, dtype=torch.uint8, device="cuda")
    s = torch.full((R, M.dsmoe_q8_scale_cols(K)), 127, dtype=torch.uint8, device="cuda")
    W = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    ws = torch.full((E, N // 128, M.dsmoe_q8_scale_cols(K)), 127, dtype=torch.uint8, device="cuda")
    out = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    M.dsmoe_q8_matmul(h, E, R, N, K, offsets_of(counts), q, s, W, ws, out)
    M.dsmoe_q8_gated_matmul(h, E, R, N, K, offsets_of(counts), q, s, W, ws, W, ws, *q8_empty(R, N))
    torch.cuda.synchronize()
    assert M.dsmoe_get_status(h) == M.DSMOE_ERR_DEVICE_TIMEOUT
    assert M.dsmoe_get_status(h) == M.DSMOE_OK
    M.dsmoe_set_wait_limit(h, 2_000_000_000)
    check_product(h, counts, 0, 0, N, K)
    check_gated(h, counts, 0, 0, N, K)
    assert M.dsmoe_get_status(h) == M.DSMOE_OK
    M.dsmoe_destroy(h)


# ------------------------------------------------------------------- beyond 32-bit addresses
LAST = 21  # rows of the end that are checked


def test_rows_past_2_31_values():
    """Rows whose first value lies past 2^31: quantisation, the norm and its backward pass, and a
    product, each checked at the last rows (the others are zeros)."""
    d = 8192
    T = (1 << 31) // d + 5000
    h = M.dsmoe_create(M.make_cfg(d_model=d, n_routed=1, top_k=1, d_ff=64, max_tokens=T))
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    x[-LAST:] = rows(LAST, d, 3)
    q, s = q8_empty(T, d)
    M.dsmoe_q8_quantize(h, T, d, x, q, s)
    eq, es = Q.quantize_rows(NP(x[-LAST:]))
    np.testing.assert_array_equal(BYTES(q[-LAST:]), eq)
    np.testing.assert_array_equal(BYTES(s[-LAST:]), es)
    W = rows(64, d, 4, 0.2).view(1, 64, d)
    qw, sw, w = q8_weights(W)
    out = torch.empty(T, 64, dtype=torch.bfloat16, device="cuda")
    M.dsmoe_q8_matmul(h, 1, T, 64, d, None, q, s, qw, sw, out)
    a = Q.dequantize_rows(eq, es)
    y, mag = a @ w[0].T, np.abs(a) @ np.abs(w[0]).T
    assert (np.abs(NP(out[-LAST:]) - y) <= 2.0 ** -8 * np.abs(y) + (d + 2) * 2.0 ** -23 * mag).all()
    assert not out[:-LAST].any()
    wn = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(5))).bfloat16().cuda()
    u = torch.empty_like(x)
    M.dsmoe_norm_q8(h, T, x, None, wn, EPS, None, u, None, None)
    eu, rstd = Q.norm(NP(x[-LAST:]), NP(wn), EPS)
    assert (np.abs(NP(u[-LAST:]) - eu) <= (2.0 ** -8 + 80 * 2.0 ** -24) * np.abs(eu)).all()
    dy = torch.zeros(T, d, device="cuda")
    dy[-LAST:] = torch.randn(LAST, d, generator=torch.Generator().manual_seed(6)).cuda()
    dw = torch.empty(d, device="cuda")
    M.dsmoe_norm_backward(h, T, dy, None, x, wn, EPS, u, dw)
    ey, r = NP(dy[-LAST:]), NP(x[-LAST:])
    ex, ew = Q.norm_backward(ey, None, r, NP(wn), EPS)
    mag = np.abs(rstd * NP(wn) * ey) + np.abs(r) * rstd ** 3 * np.abs(ey * NP(wn) * r).mean(axis=1, keepdims=True)
    assert (np.abs(NP(u[-LAST:]) - ex) <= 2.0 ** -8 * np.abs(ex) + 320 * 2.0 ** -24 * mag).all()
    assert (np.abs(NP(dw) - ew) <= (LAST + 160) * 2.0 ** -24 * np.abs(ey * r * rstd).sum(axis=0)).all()
    assert M.dsmoe_get_status(h) == M.DSMOE_OK
    M.dsmoe_destroy(h)


def test_weights_past_2_31_values(handle):
    """The last expert of a weight tensor of more than 2^31 values, plain and gated."""
    E, N, K, R = 41, 7168, 7424, 40
    W = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    W[-1] = rows(N, K, 9, 0.2) / 64
    q = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, N // 128, M.dsmoe_q8_scale_cols(K), dtype=torch.uint8, device="cuda")
    M.dsmoe_q8_quantize_weights(handle, E, N, K, W, q, s)
    eq, es = Q.quantize_weights(NP(W[-1:, -128:]))
    np.testing.assert_array_equal(BYTES(q[-1:, -128:]), eq)
    np.testing.assert_array_equal(BYTES(s[-1:, -1:]), es)
    qa, sa, a = q8_rows(rows(R, K, 2))
    w = Q.dequantize_weights(eq, es)[0]
    off = offsets_of([0] * (E - 1) + [R])
    out = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    M.dsmoe_q8_matmul(handle, E, R, N, K, off, qa, sa, q, s, out)
    y, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    err = (K + 2) * 2.0 ** -23 * mag
    assert (np.abs(NP(out)[:, -128:] - y) <= 2.0 ** -8 * np.abs(y) + err).all()
    gq, gs = q8_empty(R, N)
    M.dsmoe_q8_gated_matmul(handle, E, R, N, K, off, qa, sa, q, s, q, s, gq, gs)
    m = Q.silu(y) * y
    step = Q.decode_scale(BYTES(gs))[:, N // 128 - 1][:, None]
    got = Q.decode_e4m3(BYTES(gq)[:, -128:]) * step
    em = 1.1 * err * np.abs(y) + (np.abs(Q.silu(y)) + 1.1 * err) * err + 2.0 ** -18 * np.abs(m)
    assert (np.abs(got - m) <= np.maximum(2.0 ** -4 * np.abs(m), 2.0 ** -10 * step) * (1 + 2.0 ** -4) + em).all()


def test_slices_of_rows_and_experts(handle):
    """Slices as they come: rows from the third on and experts from the second on, whose scales are
    only 4-byte aligned (one word of scales per row), and 8-bit rows written into a slice."""
    E, N, K, R = 3, 48, 144, 30
    qa, sa, a = q8_rows(rows(R, K, 1))
    qw, sw, w = q8_weights(rows(E * N, K, 2, 0.2).view(E, N, K))
    assert sa.shape[1] == 4 and sw[1:].data_ptr() % 16 == 4
    out = torch.empty(R - 3, N, dtype=torch.bfloat16, device="cuda")
    off = offsets_of([20, 7])
    M.dsmoe_q8_matmul(handle, E - 1, R - 3, N, K, off, qa[3:], sa[3:], qw[1:], sw[1:], out)
    o = [0, 20, 27]
    y, mag = Q.grouped(a[3:], w[1:], o), Q.grouped(np.abs(a[3:]), np.abs(w[1:]), o)
    assert (np.abs(NP(out) - y) <= 2.0 ** -8 * np.abs(y) + (K + 2) * 2.0 ** -23 * mag).all()
    q, s = q8_empty(R, N)
    q.view(torch.uint8).fill_(9)
    s.view(torch.uint8).fill_(9)
    M.dsmoe_q8_gated_matmul(handle, E - 1, R - 3, N, K, off, qa[3:], sa[3:], qw[1:], sw[1:], qw[1:], sw[1:], q[3:],
                            s[3:])
    assert (BYTES(q)[:3] == 9).all() and (BYTES(s)[:3] == 9).all()
    m = Q.silu(y) * y
    assert np.linalg.norm(Q.dequantize_rows(BYTES(q)[3:], BYTES(s)[3:]) - m) <= 2.0 ** -4 * np.linalg.norm(m)
    x = rows(R, K, 5)
    M.dsmoe_q8_quantize(handle, R - 3, K, x[3:], qa[3:], sa[3:])
    eq, es = Q.quantize_rows(NP(x[3:]))
    np.testing.assert_array_equal(BYTES(qa[3:]), eq)
    np.testing.assert_array_equal(BYTES(sa[3:]), es)


# ----------------------------------------------------------------------- two calls at once
def test_two_handles_on_two_streams():
    """Products of two handles in flight together give the bits of each alone."""
    cases = []
    for i, (counts, N, K) in enumerate((([200, 3, 90], 512, 1040), ([7], 256, 4096), ([30, 300], 384, 704))):
        h = M.dsmoe_create(M.make_cfg(d_model=64, n_routed=1, top_k=1, d_ff=64, max_tokens=1))
        E, R = len(counts), sum(counts)
        qa, sa, _ = q8_rows(rows(R, K, i))
        qw, sw, _ = q8_weights(rows(E * N, K, i + 9, 0.2).view(E, N, K))
        out = [torch.empty(R, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        cases.append((h, (E, R, N, K, offsets_of(counts), qa, sa, qw, sw), out))
    torch.cuda.synchronize()
    for h, a, out in cases:
        M.dsmoe_q8_matmul(h, *a, out[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for (h, a, out), st in zip(cases, streams):
            M.dsmoe_q8_matmul(h, *a, out[1], st)
    torch.cuda.synchronize()
    for h, a, out in cases:
        assert torch.equal(out[0], out[1])
        assert M.dsmoe_get_status(h) == M.DSMOE_OK
        M.dsmoe_destroy(h)
