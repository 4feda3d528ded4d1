"""GPU parity of the eviction, every byte, where its kernel divides the cells otherwise than for short
tables: keys that do not fit shared memory, runs of more than 1024 cells per warp (their masks are
formed twice), one CTA per sequence and KV head of a long sequence, clusters of which most CTAs hold
no cell."""
import pytest

from test_gpu_evict import Cache, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["exp", "ties", "equal", "odd"])
def test_keys_that_do_not_fit_one_cta(fp8, kind):
    """80 (sequence, KV head) pairs have one CTA of 32 warps each: the keys of 60000 cells are read from
    the weights again in every round, and a warp's run is two blocks of 1024 cells."""
    lens = [60000, 300, 17, 5000, 0, 1, 2000, 33, 1025, 16]
    c = Cache(20, 8, lens, fp8, kind=kind)
    check(c, 1000, 4, 130)
    check(c, 16000, 5, 37)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["exp", "ties", "equal"])
def test_long_runs_of_small_ctas(fp8, kind):
    """160 pairs and more have CTAs of 16 warps: 20500 cells are runs of 1312, held in shared memory;
    50000 are not held."""
    lens = [20500, 300] + [40 + i for i in range(16)] + [16385, 19999]
    check(Cache(21, 8, lens, fp8, kind=kind), 700, 4, 65)
    if kind != "equal":
        check(Cache(22, 8, [50000] + lens[1:], fp8, kind=kind), 9000, 0, 4001)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,Hkv,width", [(1, 1, 8192), (2, 2, 8192), (3, 2, 4096), (5, 3, 1024), (2, 8, 16384)])
def test_short_sequences_behind_a_wide_table(fp8, B, Hkv, width):
    """The clusters are made for the longest sequence the table could hold; most of their CTAs, or all
    but one, hold no cell of these."""
    lens = [300, 9001, 33, 0, 5000][:B]
    for kind in ("exp", "ties"):
        c = Cache(23 + B, Hkv, lens, fp8, width=width, kind=kind)
        check(c, 200, 4, 57)
        check(c, 32, 0, 32)
        check(c, 299, 0, 0)


def test_clusters_whose_keys_do_not_fit():
    """60 pairs have clusters of two: 100001 cells are 50016 keys per CTA, more than it holds."""
    c = Cache(24, 12, [100001, 70, 33, 3, 1200], True, kind="ties")
    check(c, 3000, 4, 200)
