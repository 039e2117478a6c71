"""How the 8-bit products are cut up (dsmoe_q8_tiling, no GPU): by the rows of an expert, also where
only a range of the experts is here."""
import pytest

import mixture_experts_layer_score_b200 as M
from tests import q8_cases as C

OUT = (M.DSMOE_Q8_BF16, M.DSMOE_Q8_GATED, M.DSMOE_Q8_FP32)


@pytest.mark.parametrize("output", OUT[:2])
@pytest.mark.parametrize("ranks", [2, 8])
@pytest.mark.parametrize("per", [1, 16, 24, 100, 128, 300])
@pytest.mark.parametrize("N,K", [(2048, 7168), (7168, 2048), (896, 1280)])
def test_an_expert_range_takes_the_tile_of_its_own_rows(output, ranks, per, N, K):
    """`per` rows for each expert: a rank's tile is that of a call with its own rows alone."""
    E = 256
    part = M.dsmoe_q8_tiling(E // ranks, E * per, N, K, output, E_all=E)
    alone = M.dsmoe_q8_tiling(E // ranks, E // ranks * per, N, K, output)
    assert part["tokens"] == alone["tokens"] and part["grid"] >= alone["grid"]


def test_sixteen_rows_an_expert():
    """A rank's 32 of 256 experts with 16 rows each: 32-token tiles, as on a GPU that holds all."""
    assert M.dsmoe_q8_tiling(32, 4096, 2048, 7168, M.DSMOE_Q8_GATED, E_all=256)["tokens"] == 32
    assert M.dsmoe_q8_tiling(32, 4096, 7168, 2048, M.DSMOE_Q8_BF16, E_all=256)["tokens"] == 32


@pytest.mark.parametrize("output", OUT)
def test_every_row_has_a_tile(output):
    """The clusters of a launch are as many as its tiles can be, for the worst split of the rows."""
    for E in (1, 3, 32, 256):
        for R in (1, 7, 31, 128, 600, 5000):
            for K in (128, 1024, 4608, 7168, 32768):
                for N in (128, 640, 2048):
                    t = M.dsmoe_q8_tiling(E, R, N, K, output)
                    n = -(-N // (128 if output == M.DSMOE_Q8_GATED else 256))
                    groups = min(E, R)
                    # one row in all groups but one
                    worst = (groups - 1 + -(-(R - groups + 1) // t["tokens"])) * n
                    if t["splits"] > 1:
                        assert t["grid"] >= worst * t["splits"] and t["grid"] <= 148
                        assert -(-K // 512) >= t["splits"]
                    else:
                        assert t["grid"] >= min(worst, 148)
                    assert t["tokens"] <= (240, 240, 112)[output]


@pytest.mark.parametrize("K", [128, 2048, 2560, 2561 + 15, 4096, 7168, 16384, 32768])
@pytest.mark.parametrize("E,R", [(1, 1), (1, 128), (4, 676), (32, 600), (32, 3300), (32, 8192)])
def test_chains_of_a_gated_sum_are_short(K, E, R):
    """At most 2048 values in one accumulator, whatever shares K (a group of 512 more where it does
    not divide: 32 tokens in clusters of two and K = 32768)."""
    K = K // 16 * 16
    for N in (128, 512, 2048, 9472):
        t = M.dsmoe_q8_tiling(E, R, N, K, M.DSMOE_Q8_GATED)
        groups = -(-(-(-K // 512)) // t["splits"])
        assert -(-groups // t["chains"]) <= (5 if (K, t["tokens"], t["splits"]) == (32768, 32, 2) else 4), t
        assert t["tokens"] != 240 or t["chains"] == 1
        assert M.dsmoe_q8_tiling(E, R, N, K, M.DSMOE_Q8_BF16)["chains"] == 1


def test_refusals():
    ok = dict(E=1, R=1, N=16, K=16, output=0)
    M.dsmoe_q8_tiling(**ok)
    for bad in (dict(R=0), dict(E=0), dict(E=2, E_all=1), dict(N=12), dict(K=8), dict(output=3), dict(output=-1),
                dict(num_sms=0), dict(output=1, N=8)):
        with pytest.raises(M.DsmoeError):
            M.dsmoe_q8_tiling(**(ok | bad))


# ------------------------------------------------------------- what the GPU cases go through
def test_the_cases_are_the_variants_that_they_name():
    for output, want, counts, N, K in C.GROUPED:
        assert C.variant(output, len(counts), sum(counts), N, K) == want, (output, want, N, K)
        assert want[1] or C.tiles(counts, want[0], N, output) > 148, (output, want, N, K)
    for want, T, d, Fs, _ in C.SHARED:
        assert C.variant(C.FP32, 1, T, d, Fs) == want, (want, T, d, Fs)


def test_every_variant_has_a_case():
    """The variants that any sizes lead to, over a grid of them, each have a case on the GPU."""
    reached = set()
    for output in OUT:
        for E in (1,) if output == M.DSMOE_Q8_FP32 else (1, 2, 4, 8, 16, 32, 64, 256, 512):
            for R in (1, 5, 16, 17, 32, 64, 128, 256, 512, 640, 1008, 1500, 3000, 8192, 65536):
                for N in (64, 128, 512, 1024, 1280, 2048, 4096, 7168, 9472, 16384):
                    for K in (16, 128, 512, 704, 1024, 1536, 2048, 2560, 2576, 4096, 4608, 7168, 14336, 32768):
                        reached.add((output, C.variant(output, E, R, N, K)))
    cases = {(c[0], c[1]) for c in C.GROUPED} | {(C.FP32, c[0]) for c in C.SHARED}
    assert reached == cases
