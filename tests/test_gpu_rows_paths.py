"""GPU: the kernels of the expert MLP and the adapter linear that only larger
batches take, each case with the kernel that it has to reach (the plan queries
of include/w4a8_rows.h), so that a change of the rules that choose cannot
leave one of them without a test.

Definitions, checks and tolerances are those of test_gpu_rows.py.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_rows import (acts, check_lora, check_moe, gen, lora_case, moe_case, moe_ref, pack, randn, w4,  # noqa: E402, F401
                           weight)

STREAM, RUN, TILE = 2, 3, 4

# 256-row tiles, at least three groups of inputs (odd and even numbers), several strips of channels,
# a last strip of half a tile: M, k, E, I, K
MOE_TILE = [(4500, 3, 5, 384, 640), (1700, 6, 6, 640, 1152), (3001, 3, 3, 640, 1280), (12000, 1, 7, 512, 640)]


@pytest.mark.parametrize("M,k,E,I,K", MOE_TILE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("skew", [False, True], ids=["even", "skewed"])
def test_moe_tiles(w4, M, k, E, I, K, dtype, skew):  # noqa: F811
    p = w4.moe_mlp_plan(M, k, E, I, K)
    assert (p.tile_rows, p.up_path, p.down_path) == (256, TILE, TILE)
    x, up, down, ids, wt = moe_case(M + K, M, k, E, I, K, dtype, drop=0.3 if skew else 0.0, skew=skew)
    y = w4.moe_mlp(x, *pack(w4, up, down, E), ids, wt)
    check_moe(y, *moe_ref(x, up, down, ids, wt, E))


# rows of each expert: whole tiles, last tiles of up to 64, 128 and more rows, and an expert without any
ENDS = [2048, 1, 2 * 256 + 63, 3 * 256 + 64, 256 + 65, 0, 5 * 256 + 127, 4 * 256 + 128, 1024 + 129, 6 * 256 + 200, 3 * 256 + 255]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_moe_tile_ends(w4, dtype):  # noqa: F811
    """Every kind of last tile, slots of other experts between them, repeated
    calls with the same bits, and nothing written outside."""
    k, E, I, K = 3, len(ENDS), 384, 896
    g = gen(99)
    flat = torch.cat([torch.full((n,), e, dtype=torch.int32) for e, n in enumerate(ENDS)] +
                     [torch.full((998,), -1, dtype=torch.int32), torch.full((500,), E, dtype=torch.int32)])
    flat = flat[: flat.numel() // k * k]
    ids = flat[torch.randperm(flat.numel(), generator=torch.Generator().manual_seed(5))].view(-1, k).cuda().contiguous()
    M = ids.shape[0]
    p = w4.moe_mlp_plan(M, k, E, I, K)
    assert (p.tile_rows, p.up_path, p.down_path) == (256, TILE, TILE)
    x = acts(g, M, K, dtype)
    up, down = weight(g, E * 2 * I, K), weight(g, E * K, I)
    wt = torch.softmax(randn(g, M, k), dim=1).contiguous()
    ups = pack(w4, up, down, E)
    y = w4.moe_mlp(x, *ups, ids, wt)
    check_moe(y, *moe_ref(x, up, down, ids, wt, E))
    need = w4.moe_mlp_workspace_bytes(M, k, E, I, K)
    buf = torch.randint(0, 256, (need + 8192,), generator=g, device="cuda", dtype=torch.uint8)
    guard = buf.clone()
    band = torch.full((M * K + 4096,), 7.0, device="cuda", dtype=torch.bfloat16)
    for _ in range(3):
        out = w4.moe_mlp(x, *ups, ids, wt, out=band[2048: 2048 + M * K].view(M, K), workspace=buf[4096: 4096 + need])
        assert torch.equal(out, y)
    assert torch.equal(buf[:4096], guard[:4096]) and torch.equal(buf[4096 + need:], guard[4096 + need:])
    assert (band[:2048] == 7).all() and (band[2048 + M * K:] == 7).all()


# several columns to a wavefront of the down product, with columns that end inside a strip and inside
# a wavefront's share: M, k, E, I, K, tile rows, kernel, columns
MOE_COLUMNS = [
    (60, 3, 40, 128, 4224, 16, STREAM, 4), (40, 4, 32, 256, 4096, 16, STREAM, 3), (100, 4, 32, 128, 4096, 32, STREAM, 3),
    (300, 5, 32, 128, 4224, 64, STREAM, 5), (300, 6, 24, 512, 4096, 64, STREAM, 5), (120, 4, 32, 2176, 2432, 32, RUN, 2),
    (300, 5, 24, 1152, 4096, 64, RUN, 3), (300, 5, 24, 2176, 2176, 64, RUN, 2),
]


@pytest.mark.parametrize("M,k,E,I,K,rows,path,columns", MOE_COLUMNS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_moe_columns(w4, M, k, E, I, K, rows, path, columns, dtype):  # noqa: F811
    p = w4.moe_mlp_plan(M, k, E, I, K)
    assert (p.tile_rows, p.down_path, p.down_columns) == (rows, path, columns)
    x, up, down, ids, wt = moe_case(M + K, M, k, E, I, K, dtype, drop=0.2, skew=E % 3 == 0)
    y = w4.moe_mlp(x, *pack(w4, up, down, E), ids, wt)
    check_moe(y, *moe_ref(x, up, down, ids, wt, E))


# the adapters added by the 256-row tiles, ranks in one and in several steps of 32, whole and half tiles,
# and a few rows over many channels and groups: M, K, N, L, R, seg, kernel, in the epilogue
LORA_PATHS = [
    (300, 384, 33040, 3, 72, 1, TILE, 1), (300, 384, 33040, 3, 128, 7, TILE, 1), (1030, 256, 17424, 6, 96, 5, TILE, 1),
    (1000, 384, 17424, 6, 128, 1, TILE, 1), (1000, 256, 25504, 5, 104, 300, TILE, 1), (257, 256, 33040, 200, 64, 1, TILE, 1),
    (10, 4224, 32784, 3, 16, 1, RUN, 0), (16, 4608, 32784, 20, 104, 1, RUN, 0),
]


@pytest.mark.parametrize("M,K,N,L,R,seg,path,epilogue", LORA_PATHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_lora_paths(w4, M, K, N, L, R, seg, path, epilogue, dtype):  # noqa: F811
    p = w4.lora_linear_plan(M, N, K, L, R)
    assert (p.path, p.in_epilogue) == (path, epilogue)
    x, w, A, B, sc, ids = lora_case(M + N, M, K, N, L, R, dtype, seg)
    y = w4.lora_linear(x, w4.pack_weights(*w), w4.LoraAdapters(A, B, sc), ids)
    check_lora(y, x, w, A, B, sc, ids)
