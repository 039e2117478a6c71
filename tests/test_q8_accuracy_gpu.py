"""The accuracy of the 8-bit rows of a gate/up product with a long K, where the accumulation shows.

SwiGLU's fp32 value reaches an e4m3 border with a probability in proportion to its error, so the
values whose e4m3 byte differs from the float64 definition's measure the error of the sums. The
limit: an fp32 sum of the plain form (a torch fp32 product of the same operands, its elementwise
SiLU and product) may be at most one bit finer, i.e. twice its count n, and four standard
deviations of the two counts, sqrt(2 n) and sqrt(n), on top."""
import math

import pytest
import torch

import mixture_experts_layer_score_b200 as M

pytestmark = pytest.mark.gpu
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def values(q, s, dtype):
    """Rows [R, C] of 8-bit values and their scales, dequantised."""
    C = q.shape[-1]
    return q.to(dtype) * s.to(dtype)[..., :-(-C // 128)].repeat_interleave(128, -1)[..., :C]


def scale_of(m):
    """2^k of each row's blocks of 128: the smallest with max <= 448 2^k, k >= -126."""
    amax = m.abs().unflatten(-1, (-1, 128)).amax(-1).double()
    f, e = torch.frexp(amax)  # f 2^e, 0.5 <= f < 1; 448 = 0.875 2^9
    k = (e - 9 + (f > 0.875)).clamp(min=-126)
    return torch.ldexp(torch.ones_like(amax), k)


def encode(m):
    """e4m3 values (as float64) of m's rows and their scales, by the definition."""
    s = scale_of(m)
    v = m.double() / s.repeat_interleave(128, -1)
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step, s


# counts of each expert, N, K, repetitions: 160-token tiles, 32-token tiles, clusters of two CTAs; the
# longest sum of one chain (240-token tiles); 112-token tiles
CASES = [([2048, 2100, 1996, 2048], 2048, 7168, 1), ([16] * 64, 2048, 32768, 1), ([32], 9472, 32768, 8),
         ([2048, 2100, 1996, 2048], 2048, 2048, 2), ([80, 90, 108, 100] * 8, 2048, 8192, 2)]


@pytest.mark.parametrize("counts,N,K,times", CASES)
def test_gated_sums_are_as_good_as_fp32(counts, N, K, times):
    h = M.dsmoe_create(M.make_cfg(d_model=64, n_routed=1, top_k=1, d_ff=64, max_tokens=1))
    E, R, S = len(counts), sum(counts), M.dsmoe_q8_scale_cols(K)
    g = torch.Generator(device="cuda").manual_seed(11)
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    own = plain = 0
    tf32 = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    for _ in range(times):
        x = torch.randn(R, K, generator=g, device="cuda").bfloat16()
        a, sa = torch.empty(R, K, dtype=F8, device="cuda"), torch.empty(R, S, dtype=E8, device="cuda")
        M.dsmoe_q8_quantize(h, R, K, x, a, sa)
        w = []
        for _ in range(2):
            W = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda").normal_(0, K ** -0.5, generator=g)
            q = torch.empty(E, N, K, dtype=F8, device="cuda")
            s = torch.empty(E, N // 128, S, dtype=E8, device="cuda")
            M.dsmoe_q8_quantize_weights(h, E, N, K, W, q, s)
            w += [q, s]
            del W
        q, s = torch.empty(R, N, dtype=F8, device="cuda"), torch.empty(R, M.dsmoe_q8_scale_cols(N), dtype=E8,
                                                                       device="cuda")
        M.dsmoe_q8_gated_matmul(h, E, R, N, K, off, a, sa, *w, q, s)
        for e in range(E):
            rows = slice(int(off[e]), int(off[e + 1]))
            exact, rounded = ([values(a[rows], sa[rows], t) @ values(w[i][e], w[i + 1][e].repeat_interleave(128, 0),
                                                                     t).T for i in (0, 2)]
                              for t in (torch.float64, torch.float32))
            m, m32 = (v[0] / (1 + torch.exp(-v[0])) * v[1] for v in (exact, rounded))
            want, ws = encode(m)
            own += int((values(q[rows], s[rows], torch.float64) != want * ws.repeat_interleave(128, -1)).sum())
            v32, s32 = encode(m32)
            plain += int((v32 * s32.repeat_interleave(128, -1) != want * ws.repeat_interleave(128, -1)).sum())
        del w
    torch.backends.cuda.matmul.allow_tf32 = tf32
    print("values across a border: %d, of an fp32 product %d, of %d" % (own, plain, times * R * N))
    assert own <= 2 * plain + 4 * math.sqrt(3 * plain)
    assert M.dsmoe_get_status(h) == M.DSMOE_OK
    M.dsmoe_destroy(h)
