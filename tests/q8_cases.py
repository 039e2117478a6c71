"""Cases of the 8-bit products, one or more for every way in which dsmoe_q8_tiling cuts them up:
(tokens of a tile, shared by a cluster, summed in several chains)."""
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
    (GATED, (160, False, True), LARGE, 2064, 2832),
    (GATED, (160, False, True), LARGE, 1936, 7168),
    (GATED, (240, False, False), [511, 240, 241, 16], 2832, 1296),
    (GATED, (240, False, False), LARGE, 2064, 2560),
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
