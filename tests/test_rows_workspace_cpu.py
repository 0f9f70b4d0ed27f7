"""CPU: a workspace of the size asked for M rows serves every smaller number of
rows too.  The calls here lack their output pointer, which is refused only
after the workspace was found large enough, so nothing is enqueued."""
import pytest

from test_rows_abi_cpu import _lora, _moe, lib  # noqa: F401

TOO_SMALL, INVALID = -4, -1


def fewer(M):
    """Row counts up to M: all of the small ones, the edges of the tiles, a spread of the rest."""
    some = set(range(1, min(M, 530) + 1)) | {M}
    for t in range(256, M + 1, 256):
        some |= {t - 1, t, min(t + 1, M)}
    v = 1.0
    while v < M:
        some.add(int(v))
        v *= 1.07
    return sorted(some)


@pytest.mark.parametrize("N,K,L,R", [(18944, 3584, 16, 16), (3584, 18944, 32, 64), (3584, 3584, 64, 32), (256, 384, 3, 16),
                                     (16, 128, 1, 8), (16, 65536, 2, 128), (65536, 256, 4, 128), (4096, 4096, 65536, 128),
                                     (1040, 131072, 5, 8)])
@pytest.mark.parametrize("M", [2, 16, 17, 64, 65, 256, 257, 2048, 33000])
def test_lora_workspace_serves_fewer_rows(lib, M, N, K, L, R):  # noqa: F811
    have = lib.w4a8_lora_linear_workspace_bytes(M, N, K, L, R)
    assert have
    for m in fewer(M):
        got = _lora(lib, M=m, N=N, K=K, L=L, R=R, wsb=have, wb=1 << 34, y=None)
        assert got == INVALID, f"{m} rows: status {got}, {have} bytes asked for {M}"
    assert _lora(lib, M=M, N=N, K=K, L=L, R=R, wsb=64, y=None) == TOO_SMALL


@pytest.mark.parametrize("k,E,I,K", [(8, 128, 768, 2048), (4, 32, 1280, 3584), (1, 1, 128, 128), (1, 1024, 128, 128),
                                     (64, 64, 128, 128), (2, 5, 256, 3200), (7, 15, 384, 128)])
@pytest.mark.parametrize("M", [2, 17, 300, 5000, 33000, 90000])
def test_moe_workspace_serves_fewer_rows(lib, M, k, E, I, K):  # noqa: F811
    have = lib.w4a8_moe_mlp_workspace_bytes(M, k, E, I, K)
    assert have
    for m in fewer(M):
        got = _moe(lib, M=m, k=k, E=E, I=I, K=K, wsb=have, upb=1 << 40, downb=1 << 40, y=None)
        assert got == INVALID, f"{m} rows: status {got}, {have} bytes asked for {M}"
    assert _moe(lib, M=M, k=k, E=E, I=I, K=K, wsb=have - 1, upb=1 << 40, downb=1 << 40, y=None) == TOO_SMALL


@pytest.mark.parametrize("k,E,I,K", [(1, 1, 128, 128), (2, 5, 256, 3200), (8, 128, 128, 128), (1, 1024, 128, 128),
                                     (6, 64, 1280, 3584)])
def test_moe_query_never_falls(lib, k, E, I, K):  # noqa: F811
    ask = [lib.w4a8_moe_mlp_workspace_bytes(m, k, E, I, K) for m in range(1, 70000)]
    assert all(a <= b for a, b in zip(ask, ask[1:]))


@pytest.mark.parametrize("N,K,L,R", [(18944, 3584, 16, 16), (3584, 18944, 32, 64), (16, 128, 1, 8), (1040, 131072, 5, 8)])
def test_lora_query_never_falls(lib, N, K, L, R):  # noqa: F811
    ask = [lib.w4a8_lora_linear_workspace_bytes(m, N, K, L, R) for m in range(1, 70000)]
    assert all(a <= b for a, b in zip(ask, ask[1:]))
