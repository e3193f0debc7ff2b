"""Every form of the 8-bit linear and every shape of its tiles.  The rules by
which the host chooses (csrc/int8.cu) are restated here for the 148 SMs of a
B200, and the sizes are searched for by them, so that each form is run whichever
sizes reach it.  Tolerances as in test_linear_int8.py."""
import pytest
import torch

from tests.test_linear_int8 import check, operands

gpu = pytest.mark.gpu
SMS = 148


def ceil(a, b):
    return -(-a // b)


def tile_cost(pair, bn):
    if bn == 64:
        return 88 if pair else 92
    return 30 + bn * 83 // 100 if pair else bn + 47


def tiles(M, N):
    """(pair, width, width of the narrower tiles behind or 0) of the tiled form."""
    best, plan = 0, None
    for pair in (True, False):
        rows, units = (256, SMS // 2) if pair else (128, SMS)
        mt = ceil(M, rows)
        tried = [(bn, ceil(N, bn), 64, 0) for bn in (256, 192, 128, 64)]
        waves = mt * ceil(N, 256) // units
        for w in range(max(1, waves - 1), waves + 1):
            nt = min(w * units // mt, N // 256)
            rest = N - nt * 256
            if nt > 0 and rest > 0:
                tried += [(256, nt, bn, ceil(rest, bn)) for bn in (192, 128, 64)]
        for bn, nt, bn2, nt2 in tried:
            wide, every = mt * nt, mt * (nt + nt2)
            cost = 0
            for c in (0, wide % units):
                n1, n = ceil(wide - c, units), ceil(every - c, units)
                cost = max(cost, n1 * tile_cost(pair, bn) + (n - n1) * tile_cost(pair, bn2))
            if not best or cost < best:
                best, plan = cost, (pair, bn, bn2 if nt2 else 0)
    return plan


def split(N, K):
    """Blocks that share a tile's K in the swapped form."""
    nk, mt, places = ceil(K, 128), ceil(N, 128), SMS * 7 // 8
    best, least = 1, 2 * nk
    for s in range(2, min(8, nk // 4) + 1):
        if mt * s > 2 * places:
            break
        cost = 2 * (1 if mt * s <= places else 2) * ceil(nk, s) + 6 + s
        if cost < least:
            best, least = s, cost
    return best


def form(M, N, K):
    if K <= 8192 and M <= 2 and N * K <= (64 << 20 if M == 1 else 24 << 20):
        return "dot", M, 4 if N > 8192 else 2
    if K > 1024 and M <= (128 if K >= 8192 and N <= 64 * SMS // 2 else 64):
        return "swapped", ceil(M, 16), split(N, K)
    return ("tiled", *tiles(M, N))


def first_of_each():
    """The first size of a grid that reaches each form, for every form it reaches."""
    found = {}
    for M, N, K in ([(M, N, K) for N in (7, 1000, 8200, 12288, 14340) for K in (16, 1040, 2864, 4096) for M in (1, 2)]
                    + [(M, N, K) for N in (8, 130, 1000, 2100, 4096, 4736, 6152, 9000, 37000)
                       for K in (1040, 1296, 2064, 2608, 3056, 4112, 8208, 14336)
                       for M in (1, 2, 3, 17, 33, 49, 64, 65, 80, 81, 100, 112, 127, 128)]
                    + [(M, N, K) for N in (8, 72, 5000, 6152, 8200, 9480, 18952, 20000, 28680, 37896) for K in (144, 1008)
                       for M in (3, 65, 129, 257, 385, 513, 700, 1500, 2300)]):
        found.setdefault(form(M, N, K), (M, N, K))
    return found


def test_the_sizes_reach_every_form():
    f = set(first_of_each())
    assert {x[1:] for x in f if x[0] == "dot"} == {(1, 2), (1, 4), (2, 2), (2, 4)}
    assert {x[1] for x in f if x[0] == "swapped"} == set(range(1, 9))
    assert {x[2] for x in f if x[0] == "swapped"} >= {1, 2, 3, 4, 5, 6, 7, 8}
    shapes = {x[1:] for x in f if x[0] == "tiled"}
    for pair in (True, False):
        assert shapes >= {(pair, bn, 0) for bn in (64, 128, 192, 256)}
        assert shapes >= {(pair, 256, 64), (pair, 256, 192)}
    assert (True, 256, 128) in shapes


@gpu
@pytest.mark.parametrize("M,N,K", sorted(first_of_each().values()))
def test_each_form(M, N, K):
    x, w = operands(M + N + K, M, N, K, full=True)
    check(x, w, bias=torch.randn(N, device="cuda"))


@gpu
@pytest.mark.parametrize("M", [65, 80, 81, 100, 127, 128])
@pytest.mark.parametrize("N,K", [(4096, 14336), (1000, 8208), (130, 65536), (4736, 8192), (4737, 8192)])
def test_more_tokens_over_a_narrow_long_layer(M, N, K):
    check(*operands(M + N, M, N, K, full=True))


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 8193, 1040), (1, 12288, 2064), (1, 14336, 4096), (1, 8192, 8192), (1, 8193, 8176), (2, 8200, 2864),
                                   (2, 12290, 2032), (2, 8192, 3056), (2, 8192, 3088), (2, 515, 8192)])
def test_one_and_two_tokens_around_the_bounds_of_the_dot_form(M, N, K):
    check(*operands(M + N, M, N, K, full=True))
