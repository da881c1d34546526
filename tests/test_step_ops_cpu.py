"""Host-side validation of routing by scores, the dense product and the AdamW
step, and the oracle against differences and hand values (CPU only: no call here
reaches a launch)."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from mixture_experts_layer_17_amd import binding as B
from oracle import step_ops_oracle as so

EINVAL, EUNSUP, EWS = 1, 2, 3
FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10004)
BIG = 1 << 50
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        pytest.fail("libmoe.so not built: run __graft_entry__.build()")
    return B.lib()


def test_route_scored_validation(L):
    def fwd(lg=FAKE, b=FAKE, T=10, E=16, k=2, score=1, groups=4, top=2, best=2, renorm=1, scale=1.0, idx=FAKE, g=FAKE,
            c=FAKE, off=FAKE, src=FAKE, dst=FAKE, mxb=FAKE, ws=FAKE, n=BIG):
        return L.moe_route_scored(lg, b, T, E, k, score, groups, top, best, renorm, scale, idx, g, c, off, src, dst, mxb,
                                  ws, n, None)

    for name in ("lg", "idx", "g", "c", "off", "src", "dst", "ws"):
        assert fwd(**{name: None}) == EINVAL, name
    for name in ("lg", "b", "idx", "g", "c", "off", "src", "dst", "mxb", "ws"):
        assert fwd(**{name: ODD}) == EINVAL, name
    assert fwd(T=-1) == fwd(k=0) == fwd(E=0) == fwd(k=8, E=4, groups=1, top=1) == EINVAL
    assert fwd(E=257) == fwd(k=9) == EUNSUP
    assert fwd(score=2) == fwd(score=-1) == EINVAL
    assert fwd(scale=NAN) == fwd(scale=INF) == EINVAL
    assert fwd(groups=0) == fwd(groups=3) == fwd(groups=17) == EINVAL      # do not divide E
    assert fwd(top=0) == fwd(top=5) == EINVAL
    assert fwd(best=0) == fwd(best=3) == EINVAL
    assert fwd(groups=16, top=2, best=2) == EINVAL                        # two best of groups of one
    assert fwd(k=5, top=1) == EINVAL                                      # four experts stay
    assert fwd(E=256, groups=128, top=64, best=1) == EUNSUP
    need = L.moe_route_scored_workspace(10, 16, 2)
    assert need > 0 and fwd(n=need - 1) == EWS
    assert L.moe_route_scored_workspace(10, 300, 2) == L.moe_route_scored_workspace(10, 2, 3) == 0
    assert L.moe_route_scored_workspace(1 << 31, 8, 1) == L.moe_route_scored_workspace(1 << 28, 8, 1) == 0
    assert fwd(T=1 << 28) == fwd(T=1 << 40) == EUNSUP and L.moe_route_scored_workspace((1 << 28) - 64, 8, 1) > 0

    def bwd(lg=FAKE, idx=FAKE, dg=FAKE, T=10, E=16, k=2, score=0, renorm=1, scale=1.0, acc=0, out=FAKE):
        return L.moe_route_scored_bwd(lg, idx, dg, T, E, k, score, renorm, scale, acc, out, None)

    for name in ("lg", "idx", "dg", "out"):
        assert bwd(**{name: None}) == bwd(**{name: ODD}) == EINVAL, name
    assert bwd(T=0, lg=None, out=None) == 0
    assert bwd(T=-1) == bwd(score=7) == bwd(scale=NAN) == bwd(k=17, E=16, T=1) == EINVAL or bwd(k=17) == EUNSUP
    assert bwd(E=300) == bwd(T=1 << 28) == EUNSUP

    def upd(c=FAKE, S=1, E=8, rate=0.1, b=FAKE, out=FAKE):
        return L.moe_route_bias_update(c, S, E, rate, b, out, None)

    for name in ("c", "b", "out"):
        assert upd(**{name: None}) == upd(**{name: ODD}) == EINVAL, name
    assert upd(S=0) == upd(E=0) == upd(E=257) == upd(rate=NAN) == EINVAL


def test_linear_validation(L):
    def fwd(x=FAKE, w=FAKE, b=FAKE, res=FAKE, dt=1, M=4, K=64, N=32, act=2, y=FAKE, z=FAKE, ws=FAKE, n=BIG):
        return L.moe_linear(x, w, b, res, dt, M, K, N, act, y, z, ws, n, None)

    assert fwd(M=0, x=None, y=None) == 0
    for name in ("x", "w", "y", "ws"):
        assert fwd(**{name: None}) == EINVAL, name
    for name in ("x", "w", "b", "res", "y", "z", "ws"):
        assert fwd(**{name: ODD}) == EINVAL, name
    assert fwd(dt=2) == fwd(M=-1) == fwd(K=0) == fwd(N=0) == fwd(act=4) == fwd(act=-1) == EINVAL
    assert fwd(K=(1 << 20) + 1) == fwd(N=(1 << 20) + 1) == fwd(M=1 << 31) == fwd(M=1 << 30, K=1024) == EUNSUP
    need = L.moe_linear_workspace(1, 4, 64, 32, 0)
    assert need > 0 and fwd(n=need - 1) == EWS
    assert L.moe_linear_workspace(1, 4, 0, 32, 0) == L.moe_linear_workspace(2, 4, 64, 32, 0) == 0
    assert L.moe_linear_workspace(1, 0, 64, 32, 0) > 0 and L.moe_linear_workspace(0, 0, 64, 32, 1) > 0
    # odd rows of bf16 are copied, fp32 ones are not
    assert L.moe_linear_workspace(1, 1000, 63, 65, 0) >= 1000 * 64 * 2 + 63 * 72 * 2

    def bwd(dy=FAKE, x=FAKE, w=FAKE, z=FAKE, dt=0, M=4, K=64, N=32, act=1, iz=FAKE, ia=3, dres=FAKE, dx=FAKE, dw=FAKE,
            db=FAKE, ws=FAKE, n=BIG):
        return L.moe_linear_bwd(dy, x, w, z, dt, M, K, N, act, iz, ia, dres, dx, dw, db, ws, n, None)

    for name in ("dy", "x", "w", "z", "iz", "ws"):
        assert bwd(**{name: None}) == EINVAL, name
    for name in ("dy", "x", "w", "z", "iz", "dres", "dx", "dw", "db", "ws"):
        assert bwd(**{name: ODD}) == EINVAL, name
    assert bwd(dx=None) == EINVAL                      # dres and in_act without a dx
    assert bwd(act=9) == bwd(ia=9) == bwd(K=-1) == EINVAL
    assert bwd(n=L.moe_linear_workspace(0, 4, 64, 32, 1) - 1) == EWS


def _tensors(*rows):
    arr = (B._AdamwTensor * len(rows))()
    for a, r in zip(arr, rows):
        base = dict(w=0x10000, g=0x20000, w_out=0x10000, n=100, offset=0, weight_decay=0.1, lr_scale=1.0)
        base.update(r)
        for k, v in base.items():
            setattr(a, k, v)
    return arr


def test_adamw_validation(L):
    def step(rows=({},), dt=0, bits=32, length=1 << 20, m=FAKE, v=FAKE, ms=None, vs=None, master=None, lr=1e-3, b1=0.9,
             b2=0.999, eps=1e-8, t=1, tdev=None, gs=None, mo=FAKE, vo=FAKE, mso=None, vso=None, mastero=None, count=None):
        arr = _tensors(*rows)
        return L.moe_adamw_step(arr, len(rows) if count is None else count, dt, bits, length, m, v, ms, vs, master, lr, b1,
                                b2, eps, t, tdev, gs, 7, mo, vo, mso, vso, mastero, None)

    assert step(count=0, m=None) == 0
    assert step(rows=({"n": 0, "w": 0},)) == 0                            # an empty tensor is skipped
    for name in ("m", "v", "mo", "vo"):
        assert step(**{name: None}) == step(**{name: ODD}) == EINVAL, name
    for name in ("tdev", "gs"):
        assert step(**{name: ODD}) == EINVAL, name
    assert step(dt=2) == step(bits=16) == step(count=-1) == step(length=-1) == EINVAL
    assert step(b1=1.0) == step(b1=-0.1) == step(b2=1.0) == step(b2=NAN) == step(eps=-1.0) == step(eps=INF) == EINVAL
    assert step(lr=NAN) == step(lr=1e300) == step(t=0) == EINVAL
    assert step(dt=0, master=FAKE, mastero=FAKE) == EINVAL                # an fp32 weight is its own master
    assert step(dt=1, master=FAKE) == step(dt=1, mastero=FAKE) == EINVAL
    ok8 = dict(bits=8, ms=FAKE, vs=FAKE, mso=FAKE, vso=FAKE)
    for name in ("ms", "vs", "mso", "vso"):
        assert step(**{**ok8, name: None}) == step(**{**ok8, name: ODD}) == EINVAL, name
    for name in ("w", "g", "w_out"):
        assert step(rows=({name: 0},)) == step(rows=({name: 0x10004},)) == EINVAL, name
    assert step(rows=({"n": -1},)) == step(rows=({"offset": 16},)) == step(rows=({"offset": -32},)) == EINVAL
    assert step(length=127) == EINVAL                                     # 100 values take 128
    assert step(rows=({}, {"offset": 96})) == step(rows=({"offset": 128}, {"offset": 0})) == EINVAL
    assert step(rows=({"weight_decay": NAN},)) == step(rows=({"lr_scale": INF},)) == EINVAL
    assert step(rows=({"lr_scale": 3e38},), lr=1e30) == EINVAL
    assert step(rows=({"weight_decay": 3e38, "lr_scale": 1e30},), lr=1.0) == EINVAL
    assert step(rows=({"n": 1 << 37},), length=1 << 40) == EUNSUP

    def values(m=FAKE, ms=FAKE, v=FAKE, vs=FAKE, n=64, mo=FAKE, vo=FAKE):
        return L.moe_adamw_state_values(m, ms, v, vs, n, mo, vo, None)

    assert values(n=0, m=None) == 0
    assert values(n=-32) == values(n=33) == EINVAL
    for name in ("m", "ms", "v", "vs", "mo", "vo"):
        assert values(**{name: None}) == values(**{name: ODD}) == EINVAL, name
    assert values(n=1 << 40) == EUNSUP


def test_binding_refuses_names_and_lists():
    lg = torch.zeros(4, 8)
    with pytest.raises(B.MoeError, match="score"):
        B.moe_route_scored(lg, 2, score="tanh")
    with pytest.raises(B.MoeError, match="k = 9"):
        B.moe_route_scored(lg, 9)
    with pytest.raises(B.MoeError, match="act"):
        B.moe_linear(lg, torch.zeros(8, 8), act="tanh")
    with pytest.raises(B.MoeError, match="not on the current GPU"):
        B.moe_linear(lg, torch.zeros(8, 8))
    with pytest.raises(B.MoeError, match="expected"):
        B.moe_linear(lg, torch.zeros(7, 8))
    w = [torch.zeros(3, 5), torch.zeros(7)]
    state = B.moe_adamw_state(w, bits=8)
    assert state["offsets"] == [0, 32] and state["m"].numel() == 64 and state["m_scale"].numel() == 2
    for bad in (lambda: B.moe_adamw_state([], 32), lambda: B.moe_adamw_state(w, 16), lambda: B.moe_adamw_plan(w, w[:1], state),
                lambda: B.moe_adamw_plan(w, w, B.moe_adamw_state(w[:1])), lambda: B.moe_adamw_plan(w, w, state, weight_decay=[0.1]),
                lambda: B.moe_adamw_plan(w, w[::-1], state), lambda: B.moe_adamw_plan(w, w, state)):
        with pytest.raises(B.MoeError):
            bad()
    with pytest.raises(B.MoeError, match="8 bits"):
        B.moe_adamw_state_values(B.moe_adamw_state(w))


# ------------------------------------------------------------------- the oracle

@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_oracle_gate_gradient_against_differences(kind, renorm):
    rng = np.random.default_rng(1)
    lg, idx = rng.standard_normal((3, 7)), np.array([[1, 4, 0], [2, 3, 6], [5, 0, 1]])
    dg = rng.standard_normal((3, 3))
    got = so.route_scored_bwd(lg, idx, dg, kind, renorm, 1.7)
    h = 1e-6
    for t in range(3):
        for e in range(7):
            up, dn = lg.copy(), lg.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = ((so.gates(up, idx, kind, renorm, 1.7) - so.gates(dn, idx, kind, renorm, 1.7)) * dg).sum() / (2 * h)
            assert abs(got[t, e] - d) < 1e-8  # central differences: h^2 / 6 of third derivatives, 2^-53 / h of rounding


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu"])
def test_oracle_linear_gradient_against_differences(name):
    rng = np.random.default_rng(2)
    in_z, w, b, dy = rng.standard_normal((4, 5)), rng.standard_normal((5, 3)), rng.standard_normal(3), rng.standard_normal((4, 3))

    def f(in_z_, w_, b_):
        return (so.linear(so.act(in_z_, "silu"), w_, b_, name)[0] * dy).sum()

    x = so.act(in_z, "silu")
    z = so.linear(x, w, b, name)[1]
    dx, dw, db = so.linear_bwd(dy, x, w, z, name, in_z, "silu")[:3]
    h = 1e-6
    for got, at, arg in ((dx, in_z, 0), (dw, w, 1), (db, b, 2)):
        for i in np.ndindex(at.shape):
            up, dn = at.copy(), at.copy()
            up[i] += h
            dn[i] -= h
            args = [in_z, w, b]
            args[arg] = up
            d = f(*args)
            args[arg] = dn
            d = (d - f(*args)) / (2 * h)
            assert abs(got[i] - d) < 2e-8


def test_oracle_route_by_hand():
    # groups {0, 1}, {2, 3}; worth by the best one: 0.9 and 0.8; by the best two: 1.0 and 1.5
    s = np.array([[0.9, 0.1, 0.8, 0.7]])
    lg = np.log(s / (1 - s))
    one = so.route_scored(lg, 1, "sigmoid", groups=2, top_groups=1, group_best=1)
    two = so.route_scored(lg, 2, "sigmoid", groups=2, top_groups=1, group_best=2, scale=2.0)
    assert one["topk_idx"].tolist() == [[0]] and two["topk_idx"].tolist() == [[2, 3]]
    assert np.allclose(two["gates"], [[2 * 0.8 / 1.5, 2 * 0.7 / 1.5]])
    biased = so.route_scored(lg, 2, "sigmoid", bias=[0, 5, 0, 0], renorm=False)
    assert biased["topk_idx"].tolist() == [[1, 0]] and np.allclose(biased["gates"], [[0.1, 0.9]])
    assert so.bias_update([3, 1, 2], [0.0, 0.0, 0.5], 0.1).tolist() == [-0.1, 0.1, 0.5]


def test_oracle_codes_by_hand():
    assert so.e4m3([0x00, 0x01, 0x08, 0x38, 0x7E, 0xBC]).tolist() == [0.0, 2.0 ** -9, 2.0 ** -6, 1.0, 448.0, -1.5]
    x = np.zeros(32)
    x[:3] = 448.0, -1.0625, 2.0 ** -20
    low, byte = so.encode(x, np.zeros(32))
    high, _ = so.encode(x, np.full(32, 65535))
    assert byte.tolist() == [127] and low[:3].tolist() == [0x7E, 0xB8, 0] and high[:3].tolist() == [0x7E, 0xB9, 1]
    assert so.encode(x, np.zeros(32), root=True)[0][2] == 1
    assert so.encode(np.full(32, 449.0), np.zeros(32))[1].tolist() == [128]
    assert so.encode(np.full(32, NAN), np.zeros(32))[1].tolist() == [255]


def test_random_halves_are_even_and_apart():
    """Means over n draws of a uniform variable lie within 5 standard deviations of 1/2, and so do products of pairs of
    halves, neighbours, tensors and steps of 1/4."""
    n = 1 << 16
    draws = [h / 65536 for t, step in ((0, 1), (1, 1), (0, 2)) for h in so.random_halves(3, t, step, n)]
    sd = math.sqrt(1 / 12 / n)
    for a in draws:
        assert abs(a.mean() - 0.5) < 5 * sd and abs(a.var() - 1 / 12) < 5 * math.sqrt(1 / 180 / n)
        assert abs(((a[1:] - 0.5) * (a[:-1] - 0.5)).mean()) < 5 / 12 / math.sqrt(n)
    for i in range(len(draws)):
        for j in range(i):
            assert abs(((draws[i] - 0.5) * (draws[j] - 0.5)).mean()) < 5 / 12 / math.sqrt(n)
