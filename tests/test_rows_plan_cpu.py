"""CPU: the plan queries of include/w4a8_rows.h, and that every kernel the expert
MLP and the adapter linear can take is taken by some GPU test's sizes."""
import ctypes

import pytest

pytest.importorskip("torch")

import bit_quantized_amd as w4
import test_gpu_rows
import test_gpu_rows_long
import test_gpu_rows_paths as paths
from bit_quantized_amd import _lib

TOKEN, STREAM, RUN, TILE = w4.ROWS_TOKEN, w4.ROWS_STREAM, w4.ROWS_RUN, w4.ROWS_TILE


def moe_plans():
    cases = [c[:5] for c in test_gpu_rows.MOE + test_gpu_rows_long.MOE + paths.MOE_TILE + paths.MOE_COLUMNS]
    return [(c, w4.moe_mlp_plan(*c)) for c in cases]


def test_gpu_tests_reach_every_expert_kernel():
    plans = moe_plans()
    up = {(p.tile_rows, p.up_path) for _, p in plans}
    assert up == {(1, TOKEN), (16, STREAM), (16, RUN), (32, STREAM), (32, RUN), (64, STREAM), (64, RUN), (256, TILE)}
    down = {(p.tile_rows, p.down_path, p.down_columns > 1) for _, p in plans}
    one = {(r, s, False) for r, s in up}
    # (16 rows: past 32 groups a column is a run of its own)
    assert down == one | {(16, STREAM, True), (32, STREAM, True), (64, STREAM, True), (32, RUN, True), (64, RUN, True)}
    # 256-row tiles: the groups' two buffers change places, several strips, a last strip of half a tile
    tiles = [c for c, p in plans if p.up_path == TILE]
    assert {c[4] // 128 % 2 for c in tiles} == {0, 1} and {c[3] // 128 % 2 for c in tiles} == {0, 1}
    assert all(min(c[3], c[4]) // 128 >= 3 for c in tiles) and any(c[4] // 16 % 16 for c in tiles)


def test_gpu_tests_reach_every_adapter_kernel():
    cases = [c[:5] for c in test_gpu_rows.LORA + test_gpu_rows_long.LORA + paths.LORA_PATHS]
    plans = [(c, w4.lora_linear_plan(c[0], c[2], c[1], c[3], c[4])) for c in cases]
    reached = {(p.path, (c[0] + 15) // 16 if p.path in (STREAM, RUN) else 0, p.in_epilogue) for c, p in plans}
    want = {(TOKEN, 0, 1), (TOKEN, 0, 0), (STREAM, 1, 1), (TILE, 0, 0), (TILE, 0, 1)}
    assert reached == want | {(s, n, 0) for s in (STREAM, RUN) for n in (1, 2, 3, 4)}
    assert {-(-c[4] // 32) for c, p in plans if p.path == TILE and p.in_epilogue} == {1, 2, 3, 4}  # steps of 32 ranks
    assert {p.sorted for c, p in plans if c[0] <= 64} == {0, 1}
    assert any(p.ksplit > 1 for c, p in plans if p.path == TILE)


def test_plan_queries_refuse():
    lib = _lib.load()
    moe, lora = _lib.MoeMlpPlan(), _lib.LoraLinearPlan()
    assert lib.w4a8_moe_mlp_plan(4, 2, 8, 256, 384, None) == -1
    assert lib.w4a8_lora_linear_plan(4, 256, 384, 3, 16, None) == -1
    for args, status in (((0, 2, 8, 256, 384), -1), ((4, 0, 8, 256, 384), -1), ((4, 2, 8, 200, 384), -2)):
        assert lib.w4a8_moe_mlp_plan(*args, ctypes.byref(moe)) == status
    for args, status in (((0, 256, 384, 3, 16), -1), ((4, 256, 384, 3, 7), -2), ((4, 256, 200, 3, 16), -2)):
        assert lib.w4a8_lora_linear_plan(*args, ctypes.byref(lora)) == status
    with pytest.raises(w4._lib.W4A8Error):
        w4.moe_mlp_plan(4, 2, 8, 200, 384)
    with pytest.raises(w4._lib.W4A8Error):
        w4.lora_linear_plan(4, 256, 384, 3, 7)
    assert w4.moe_mlp_plan(1 << 20, 8, 8, 256, 4096).tokens < 1 << 20  # several passes
