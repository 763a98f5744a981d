"""Head norms on the GPU with so many rows that a group of lanes takes several
heads of a position in turn (two from 32768 rows on 256 CUs, eight from 131072),
the last one fewer, and goes on to further positions in the backward pass.

Tolerances are those of tests/test_gpu_headnorm.py.  Weight gradients are sums
of up to 16 rows a group, 16 groups, 64 workgroups' parts and 16 of those, 112
additions in a chain, each off by at most 2^-24 of a partial sum with a sign of
its own: sqrt(112) 2^-24 = 6.3e-7, of which SUM_TOL is six times (longer rows of
positions have 11 rounds of 2 rows in a group's part: the same)."""
import pytest
import torch

from tests.test_gpu_headnorm import TYPES, check, make

pytestmark = pytest.mark.gpu

# heads of 2, 3 and 8 in turn, neither tensor's heads a multiple of them
MANY = [(2, 1050, 11, 7), (2, 1600, 11, 5), (4, 2100, 11, 5)]
# vectors of one and two a lane, single elements, no rotation, part of it, all of it
WIDTHS = [(32, 16), (128, 128), (64, 0), (80, 32), (10, 6)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,R", WIDTHS)
@pytest.mark.parametrize("B,L,Hq,Hk", MANY)
@pytest.mark.parametrize("kind,interleaved", [("rms", False), ("l2", True)])
def test_several_heads_in_turn(B, L, Hq, Hk, d, R, kind, interleaved, dtype):
    T, tol = TYPES[dtype]
    check(*make(B, L, Hq, Hk, d, R, T, seed=d + L), tol, kind, interleaved)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,Hq,Hk,d,R", [(2, 45000, 2, 1, 8, 8), (2, 45000, 2, 1, 16, 16), (3, 6000, 2, 1, 16, 0), (1, 20000, 1, 1, 33, 12)])
def test_many_short_rows(B, L, Hq, Hk, d, R, dtype):
    T, tol = TYPES[dtype]
    x, dy, w, tab, pos = make(B, L, Hq, Hk, d, R, T, seed=d + R)
    check(x, dy, w, tab, pos, tol, "rms", False)
    check(x, dy, [None, w[1]], tab, None, tol, "l2", False)
