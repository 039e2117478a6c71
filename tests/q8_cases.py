"""Cases of the 8-bit products, one or more for every way in which dsmoe_q8_tiling cuts them up:
(tokens of a tile, shared by a cluster, summed in several chains); and their checks against float64.

Tolerances as in tests/test_q8_gpu.py: an fp32 sum of K terms that the tensor core may truncate,
K 2^-23 of the sum of magnitudes; bf16 half a step, 2^-8; e4m3 half a step, 2^-4 of the value or 2^-10 of
its block's scale."""
import torch

import mixture_experts_layer_score_b200 as M

BF16, GATED, FP32 = M.DSMOE_Q8_BF16, M.DSMOE_Q8_GATED, M.DSMOE_Q8_FP32
EIGHT = [3, 0, 16, 11, 1, 20, 5, 8] * 8                  # 8 rows an expert
SIXTY = [60, 1, 113, 0, 112, 111, 58, 25] * 2            # 60
LARGE = [300, 100, 0, 511, 240, 241, 130, 161]           # 210, on the borders of 160 and 240

GROUPED = [  # output, variant, rows of each expert, N, K; where not clustered more tiles than SMs
    (BF16, (32, False, False), EIGHT, 1288, 704),
    (BF16, (32, True, False), [5, 9], 520, 4624),
    (BF16, (112, False, False), SIXTY, 2568, 1296),
    (BF16, (112, True, False), [250, 260, 240, 258], 72, 4608),
    (BF16, (240, False, False), LARGE, 5128, 4112),
    (BF16, (240, False, False), [511, 240, 241, 16], 5640, 1424),
    (GATED, (32, False, False), EIGHT, 400, 704),
    (GATED, (32, False, True), EIGHT, 400, 5136),
    (GATED, (32, True, False), [5, 9], 272, 4624),
    (GATED, (32, True, True), [7, 9], 144, 32768),
    (GATED, (112, False, False), SIXTY, 1296, 704),
    (GATED, (112, False, True), SIXTY, 1296, 2832),
    (GATED, (112, True, False), [250, 260, 240, 258], 80, 4608),
    (GATED, (112, True, True), [47, 90, 3, 48] * 8, 64, 7168),
    (GATED, (160, False, True), LARGE, 2064, 2064),
    (GATED, (160, False, True), LARGE, 1936, 7168),
    (GATED, (240, False, False), [511, 240, 241, 16], 2832, 1296),
    (GATED, (240, False, False), LARGE, 2064, 2048),
]

SHARED = [  # variant of the fp32 product, tokens, d, F_s, shared experts
    ((32, False, False), 16, 4096, 448, 1),
    ((32, True, False), 40, 512, 1536, 1),
    ((32, True, False), 40, 512, 1536, 3),
    ((112, False, False), 1000, 2560, 704, 1),
    ((112, False, False), 1000, 2560, 704, 2),
    ((112, True, False), 1500, 64, 4608, 1),
]


def variant(output, E, R, N, K, num_sms=148):
    t = M.dsmoe_q8_tiling(E, R, N, K, output, num_sms=num_sms)
    return t["tokens"], t["splits"] > 1, t["chains"] > 1


def tiles(counts, tok, N, output):
    return sum(-(-c // tok) for c in counts) * -(-N // (128 if output == GATED else 256))


# ------------------------------------------------------------------------ float64 checks
F8, E8, F64 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.float64


def values(q, s):
    """Rows [R, C] or one expert's weights [N, K] (scales of 128 rows) in float64."""
    s = s.to(F64)
    if s.shape[0] != q.shape[0]:
        s = s.repeat_interleave(128, 0)[:q.shape[0]]
    C = q.shape[1]
    return q.to(F64) * s[:, :-(-C // 128)].repeat_interleave(128, 1)[:, :C]


def sums(a, w):
    """a w^T in float64, and the error of an fp32 sum of its terms."""
    return a @ w.T, (a.shape[1] + 2) * 2.0 ** -23 * (a.abs() @ w.abs().T)


def check_plain(a, w, out):
    """bf16 rows of a w^T."""
    y, err = sums(a, w)
    assert bool(((out.to(F64) - y).abs() <= 2.0 ** -8 * y.abs() + err).all())


def check_gated(a, w_gate, w_up, q, s):
    """8-bit rows of SiLU(a w_gate^T) (a w_up^T)."""
    (g, eg), (u, eu) = sums(a, w_gate), sums(a, w_up)
    silu = g / (1 + torch.exp(-g))
    m = silu * u
    # |SiLU'| <= 1.1; exp, the division and the product in fp32 at a few steps each
    em = 1.1 * eg * u.abs() + (silu.abs() + 1.1 * eg) * eu + 2.0 ** -18 * m.abs()
    N = m.shape[1]
    nb = -(-N // 128)
    assert bool((s.view(torch.uint8)[:, nb:] == 127).all())
    step = s[:, :nb].to(F64).repeat_interleave(128, 1)[:, :N]
    half = torch.maximum(2.0 ** -4 * m.abs(), 2.0 ** -10 * step)
    assert bool(((q.to(F64) * step - m).abs() <= half * (1 + 2.0 ** -4) + em).all())
    for b in range(nb):  # the smallest power that holds the block, or within the error of it
        part = slice(128 * b, 128 * b + 128)
        top, off, p = m[:, part].abs().amax(1), em[:, part].amax(1), s[:, b].to(F64)
        assert bool((448 * p >= top - off).all() and (448 * (p / 2) <= top + off).all()), b
