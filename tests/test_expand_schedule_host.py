"""CPU-only checks of how the gated block's products and the weight gradient are divided: every
division is whole and within the kernel's limits, and the shapes of the GPU tests take the paths that
they are there for (another cost estimate could otherwise silently lead them elsewhere)."""
import random

from bit_gemm_wise_b200 import w4

SMS = 148
NULL, SHAPE, GROUP, ARG = 1, 2, 3, 5
COUNTERS = 4096 * 4 * 4


def check(s, lanes_per_tile, lanes, cols, red, sources, widest, sum_stages, sms):
    pair = s["ctas_per_tile"]
    assert pair in (1, 2)
    lane_tiles = -(-(-(-lanes // lanes_per_tile)) // pair)
    col_tiles = -(-cols // s["columns"])
    tiles = s["units"] // s["parts"]
    assert s["units"] == s["parts"] * tiles and tiles == lane_tiles * col_tiles
    assert s["columns"] % (16 * pair) == 0 and s["columns"] <= widest[pair - 1] and pair * (sms // pair) >= s["ctas"] > 0
    assert s["ctas"] == pair * min(s["units"], sms // pair)
    assert s["stages"] == sources * -(-red // 64)
    assert s["parts"] == 1 or 4 * s["parts"] <= s["stages"]
    longest = -(-s["stages"] // s["parts"])
    assert s["stages_per_sum"] == (s["stages"] if longest <= sum_stages else sum_stages)
    if s["parts"] > 1:
        assert pair * tiles <= 4096 and s["sums_bytes"] == COUNTERS + s["units"] * pair * s["columns"] * 512
    return longest, s


def places(s):
    """Workspace of a product without parts, whose tiles take several accumulators in 16 bits."""
    return COUNTERS + s["ctas"] * s["columns"] * 512


def test_divisions_over_many_shapes():
    rng = random.Random(1)
    size = lambda lo, hi: int(lo * (hi / lo) ** rng.random())
    for _ in range(3000):
        M, K, sms = size(17, 1 << 22), 32 * size(1, 1 << 15), rng.choice([1, 2, 3, 36, 132, SMS, SMS, SMS])
        H = 8 * size(1, 1 << 15)
        if M * K > 1 << 40 or M * H > 1 << 40 or H * K > 1 << 40:
            continue
        s = w4.w4a16_gated_schedule(M, H, K, 32, sms)
        long, _ = check(s, 64, H, M, K, 1, (256, 256), 512, sms)
        if s["parts"] == 1:
            assert s["sums_bytes"] == (places(s) if long > 512 else 0)
        g, d = w4.w4a16_gated_bwd_schedule(M, H, K, 32, sms)
        check(g, 64, H, M, K, 1, (256, 256), 512, sms)
        check(d, 128, K, M, H, 2, (256, 256), 512, sms)
        s = w4.w4a16_dgrad_schedule(M, H, K, 32, sms)
        check(s, 128, K, M, H, 1, (256, 256), 512, sms)
        need = []
        for flags in (0, w4.W4_OUT_FP32):
            s = w4.fp8_ckpt_wgrad_schedule(M, H, K, flags, sms)
            check(s, 128, K, H, M, 1, (192, 256), 32 if flags else 512, sms)
            need.append(s["sums_bytes"])
            if flags and s["parts"] == 1:
                assert s["sums_bytes"] == 0     # fp32 results are added up where they stand
        assert need[0] >= need[1]               # one query serves both


def test_few_rows_divide_nothing_and_refusals():
    assert set(w4.w4a16_gated_schedule(16, 4096, 4096, 128, SMS).values()) == {0}
    L, P = w4.lib(), 0x1000
    assert L.w4a16_gated_schedule(32, 64, 128, 128, SMS, None) == NULL
    assert L.fp8_ckpt_wgrad_schedule(32, 64, 128, 0, SMS, None) == NULL
    for fn in (L.w4a16_gated_schedule, L.w4a16_gated_bwd_schedule, L.w4a16_dgrad_schedule):
        assert fn(0, 64, 128, 128, SMS, P) == SHAPE and fn(32, 64, 128, 48, SMS, P) == GROUP
        assert fn(32, 64, 128, 128, 0, P) == SHAPE and fn(32, 64, 128, 128, 4097, P) == SHAPE
    assert L.w4a16_gated_bwd_schedule(32, 12, 128, 128, SMS, P) == SHAPE
    assert L.w4a16_dgrad_schedule(32, 12, 128, 128, SMS, P) == SHAPE
    assert L.fp8_ckpt_wgrad_schedule(32, 12, 128, 0, SMS, P) == SHAPE
    assert L.fp8_ckpt_wgrad_schedule(32, 64, 128, 2, SMS, P) == ARG


PAIRS = SMS // 2


def test_shapes_of_pairs_with_several_tiles():
    s = w4.w4a16_gated_schedule(1030, 3000, 768, 128, SMS)
    assert s["ctas_per_tile"] == 2 and s["units"] > PAIRS and s["parts"] == 1
    g, d = w4.w4a16_gated_bwd_schedule(1030, 3000, 768, 128, SMS)
    assert g["ctas_per_tile"] == 2 and g["units"] > PAIRS and d["ctas_per_tile"] == 2 and d["parts"] > 1
    g, d = w4.w4a16_gated_bwd_schedule(600, 2056, 640, 32, SMS)
    assert d["ctas_per_tile"] == 2 and d["parts"] > 1 and d["stages"] // 2 % (d["stages"] // d["parts"]) != 0
    s = w4.w4a16_dgrad_schedule(1100, 1000, 4224, 64, SMS)
    assert s["ctas_per_tile"] == 2 and s["units"] > PAIRS
    s = w4.w4a16_dgrad_schedule(300, 4096, 2112, 32, SMS)
    assert s["ctas_per_tile"] == 2 and s["parts"] > 1
    s = w4.fp8_ckpt_wgrad_schedule(8000, 520, 1056, 0, SMS)
    assert s["ctas_per_tile"] == 2 and s["parts"] > 1
    s = w4.fp8_ckpt_wgrad_schedule(700, 1544, 4160, 0, SMS)
    assert s["ctas_per_tile"] == 2 and s["units"] > PAIRS
    s = w4.fp8_ckpt_wgrad_schedule(5000, 1544, 4160, w4.W4_OUT_FP32, SMS)
    assert s["ctas_per_tile"] == 2 and s["units"] > PAIRS and s["stages_per_sum"] < s["stages"]


def test_shapes_of_long_reductions():
    for s in (w4.w4a16_dgrad_schedule(512, 1 << 20, 9472, 128, SMS), w4.w4a16_gated_schedule(512, 4736, 1 << 20, 128, SMS),
              w4.fp8_ckpt_wgrad_schedule(1 << 21, 512, 9472, 0, SMS)):
        assert s["parts"] == 1 and s["stages_per_sum"] == 512 and s["sums_bytes"] == places(s)
    s = w4.fp8_ckpt_wgrad_schedule(1 << 22, 512, 64, 0, SMS)
    assert s["parts"] > 1 and s["stages"] // s["parts"] > s["stages_per_sum"]


def test_shapes_of_the_edges():
    """One CTA a tile, and pairs."""
    assert w4.w4a16_gated_schedule(300, 520, 1088, 64, SMS)["ctas_per_tile"] == 1
    assert w4.w4a16_gated_schedule(600, 2056, 640, 32, SMS)["ctas_per_tile"] == 2
    assert [s["ctas_per_tile"] for s in w4.w4a16_gated_bwd_schedule(600, 2056, 640, 32, SMS)] == [2, 2]
    assert w4.w4a16_dgrad_schedule(300, 520, 1088, 64, SMS)["ctas_per_tile"] == 1
    assert w4.w4a16_dgrad_schedule(300, 4096, 2112, 32, SMS)["ctas_per_tile"] == 2
