"""Into how many parts the keys of attention over the 8-bit cache are split, from the workspace asked for."""
import pytest

from tests.test_heads_host import cache, cached
from tests.test_layers_host import sc  # noqa: F401  (a fixture)


def parts(sc, B, T, Hkv, D, H, Lq=1, kind=1, **opt):
    N = -(-T // 64)
    c = cache(sc, B=B, N=N, P=B * N, Hkv=Hkv, D=D)
    need = sc.sc_cached_attn_workspace_bytes(kind, c, cached(sc, Lq=Lq, H=H, **opt))
    one = B * H * Lq * (D + 1) * 4
    assert need % one == 0 and need // one != 1
    return max(1, need // one)


def test_long_caches_are_split_whatever_the_number_of_sequences(sc):
    # 4 key heads over 65536 tokens: from one sequence to the 96 whose workgroups half fill the GPU
    for D in (64, 128):
        got = [parts(sc, B, 65536, 4, D, 16) for B in (1, 8, 40, 47, 48, 64, 80, 96, 97)]
        assert got == [128, 24, 5, 5, 4, 3, 3, 2, 1], got


def test_short_caches_are_split_where_it_pays(sc):
    # a few parts of short caches cost a launch more than they save, whatever limits them
    assert [parts(sc, 1, T, 4, 64, 16) for T in (64, 1000, 2500, 3000, 3100, 3584, 10240)] == [1, 1, 1, 5, 6, 7, 20]
    for D in (64, 128):
        assert [parts(sc, B, 4096, 4, D, 16) for B in (8, 38, 39, 47, 48, 64, 96)] == [8, 6, 1, 1, 1, 1, 1]
        assert [parts(sc, B, 8192, 4, D, 16) for B in (8, 38, 39, 47, 48, 64, 96)] == [16, 6, 5, 5, 1, 1, 1]
        assert [parts(sc, B, 16384, 4, D, 16) for B in (8, 38, 39, 47, 48, 64, 96)] == [24, 6, 5, 5, 4, 3, 2]
    # a window's keys count, not the cache's
    assert parts(sc, 64, 65536, 4, 128, 16, window=256) == 1
    assert parts(sc, 1, 65536, 4, 64, 16, window=3500, sinks=4) == 6


@pytest.mark.parametrize("Lq", [5, 16, 17, 64])
def test_more_rows_are_split_from_two_parts_on(sc, Lq):
    # 17 packed rows and more: workgroups of 64 rows
    assert [parts(sc, 1, T, 1, 64, 4, Lq=Lq) for T in (960, 1024, 4096)] == [1, 2, 8]
