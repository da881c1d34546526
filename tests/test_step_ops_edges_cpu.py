"""Refusals of routing by scores, the dense product and the AdamW step at the
ends of their arguments' ranges (CPU only: no call here reaches a launch)."""
import ctypes
import os
import types

import pytest
import torch

from mixture_experts_layer_17_amd import binding as B

OK, EINVAL, EUNSUP = 0, 1, 2
FAKE = ctypes.c_void_p(0x10000)
BIG = 1 << 60
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        pytest.fail("libmoe.so not built: run __graft_entry__.build()")
    return B.lib()


def adamw(L, n=64, length=1 << 20, offset=0, eps=1e-8, bits=32, dtype=0):
    t = (B._AdamwTensor * 1)(B._AdamwTensor(0x10000, 0x20000, 0x10000, n, offset, 0.1, 1.0))
    scale = FAKE if bits == 8 else None
    return L.moe_adamw_step(t, 1, dtype, bits, length, FAKE, FAKE, scale, scale, None, 1e-3, 0.9, 0.999, eps, 1, None, None, 7,
                            FAKE, FAKE, scale, scale, None, None)


def test_route_scored_bwd_refusals_one_by_one(L):
    def bwd(T=10, E=16, k=2, score=0, scale=1.0):
        return L.moe_route_scored_bwd(FAKE, FAKE, FAKE, T, E, k, score, 1, scale, 0, FAKE, None)

    for bad in (dict(T=-1), dict(score=7), dict(score=-1), dict(scale=NAN), dict(scale=float("inf")), dict(k=0), dict(E=0),
                dict(k=5, E=4)):
        assert bwd(**bad) == EINVAL, bad
    for bad in (dict(k=9), dict(k=17), dict(E=257), dict(T=1 << 28)):
        assert bwd(**bad) == EUNSUP, bad


def test_adamw_sizes_at_the_end_of_64_bits(L):
    top = (1 << 63) - 1
    for n in (top, top - 31, top - 30, top - 63):
        for length in (top, 1 << 40):
            assert adamw(L, n=n, length=length) in (EINVAL, EUNSUP), (n, length)
    assert adamw(L, n=top, length=top) == EINVAL                      # its last block passes the states' end
    assert adamw(L, n=top - 31, length=top) == EUNSUP
    assert adamw(L, n=top - 63, length=top - 31, offset=64) == EINVAL
    assert adamw(L, n=0, length=0) == OK
    for n in (top - 31, top - 63, 1 << 62):
        assert L.moe_adamw_state_values(FAKE, FAKE, FAKE, FAKE, n, FAKE, FAKE, None) == EUNSUP, n


def test_adamw_eps_outside_what_the_reciprocal_takes(L):
    """The hardware's reciprocal takes subnormal values for zero and gives zero for a subnormal result: a positive eps lies
    in 2^-126 .. 2^100."""
    for bits in (32, 8):
        for bad in (1e-39, 1e-50, 5e-324, 2.0 ** -127, 1e38, 1.01 * 2.0 ** 100):
            assert adamw(L, eps=bad, bits=bits) == EINVAL, bad
        for good in (0.0, 2.0 ** -126, 1e-12, 2.0 ** 100):
            assert adamw(L, eps=good, n=0, bits=bits) == OK, good


@pytest.mark.parametrize("dtype", [0, 1])
def test_linear_sizes_whose_launch_would_pass_its_limit(L, dtype):
    """A launch holds fewer than 2^32 threads: what would take more is refused, not left to fail."""
    def fwd(M, K, N):
        return L.moe_linear(FAKE, FAKE, None, None, dtype, M, K, N, 0, FAKE, None, FAKE, BIG, None)

    def bwd(M, K, N):
        return L.moe_linear_bwd(FAKE, FAKE, FAKE, None, dtype, M, K, N, 0, None, 0, None, FAKE, FAKE, None, FAKE, BIG, None)

    top = (1 << 31) - 1
    for M in (top, top - 126):
        assert fwd(M, 8, 1) == EUNSUP and L.moe_linear_workspace(dtype, M, 8, 1, 0) == 0, M
        assert bwd(M, 1, 8) == EUNSUP and L.moe_linear_workspace(dtype, M, 1, 8, 1) == 0, M
    # what fits stays: 64-row tiles of fp32 take four threads a row, the bf16 ones two
    M = (1 << 30) - 512
    assert L.moe_linear_workspace(dtype, M, 8, 1, 0) > 0 and L.moe_linear_workspace(dtype, M, 1, 8, 1) > 0
    if dtype == 1:
        assert L.moe_linear_workspace(dtype, (1 << 31) - (1 << 16), 8, 1, 0) > 0


def test_binding_refuses_numbers_of_more_than_32_bits():
    """The C ABI takes these in 32 bits: a larger one would be cut, and 2^32 + 4 groups taken for 4."""
    lg = torch.zeros(4, 8)
    for name in ("groups", "top_groups", "group_best"):
        for bad in ((1 << 32) + 1, 1 << 31, -(1 << 32) + 1):
            with pytest.raises(B.MoeError, match=name):
                B.moe_route_scored(lg, 2, **{name: bad})
    plan = types.SimpleNamespace(tensors=[], at=[], device=torch.device("cpu"))
    for bad in ((1 << 64) + 1, 1 << 63, -(1 << 64) + 1):
        with pytest.raises(B.MoeError, match="step ="):
            B.moe_adamw_step(plan, 0.1, bad)
