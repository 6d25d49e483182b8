"""The few-token layer and the linear layer refuse bad calls on the host, before any device work (no GPU needed)."""
import ctypes
from dataclasses import replace

import pytest
import torch

import sparse_mixture_experts_rms_b200 as moe
from sparse_mixture_experts_rms_b200 import build as moe_build

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe._lib()


CFG = moe.MoEConfig(T=8, d_model=256, E=8, k=2, ffn_offsets=[128 * i for i in range(9)])


def few(lib, cfg, ws=1 << 20, n=None, **at):
    """Status of a call with fake, aligned pointers that nothing may read."""
    names = ["x", "gamma", "Wr", "bias", "W1", "W3", "W2", "residual", "out", "expert_idx", "gate", "r", "counts"]
    ptr = {k: 4096 * (i + 1) for i, k in enumerate(names)}
    ptr.update(at)
    n = moe.moe_few_workspace_size(cfg) if n is None else n
    return lib.moe_layer_fwd_few(ctypes.byref(cfg.c()), *[P(ptr[k]) for k in names], P(ws), n, P(0))


def test_few_limits(lib):
    assert moe.MOE_FEW_MAX_TOKENS == 64
    assert moe.moe_few_workspace_size(replace(CFG, T=64)) > moe.moe_few_workspace_size(CFG) > 256
    assert moe.moe_few_workspace_size(replace(CFG, T=65)) == 0
    assert few(lib, replace(CFG, T=65), n=1 << 30) == moe.MOE_ERR_UNSUPPORTED
    for bad in (dict(T=-1), dict(k=9), dict(d_model=100), dict(eps=float("nan"))):
        assert moe.moe_few_workspace_size(replace(CFG, **bad)) == 0
        assert few(lib, replace(CFG, **bad), n=1 << 30) == moe.MOE_ERR_INVALID_ARG
    assert few(lib, replace(CFG, T=0), counts=0) == moe.MOE_OK


def test_few_workspace_of_more_tokens_serves_fewer(lib):
    sizes = [moe.moe_few_workspace_size(replace(CFG, T=t)) for t in range(65)]
    assert sizes == sorted(sizes) and sizes[0] > 0


@pytest.mark.parametrize("name", ["x", "gamma", "Wr", "W1", "W3", "W2", "out"])
def test_few_refuses_missing_tensors(lib, name):
    assert few(lib, CFG, **{name: 0}) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name,off", [("x", 8), ("gamma", 2), ("Wr", 1), ("bias", 2), ("W1", 8), ("W3", 8), ("W2", 8),
                                      ("residual", 8), ("out", 8), ("expert_idx", 2), ("gate", 1), ("r", 2),
                                      ("counts", 2)])
def test_few_refuses_misaligned_tensors(lib, name, off):
    assert few(lib, CFG, **{name: (1 << 24) + off}) == moe.MOE_ERR_ALIGNMENT


def test_few_refuses_bad_workspaces(lib):
    n = moe.moe_few_workspace_size(CFG)
    assert few(lib, CFG, n=n - 1) == moe.MOE_ERR_WORKSPACE
    assert few(lib, CFG, ws=0) == moe.MOE_ERR_WORKSPACE
    assert few(lib, CFG, ws=(1 << 20) + 16) == moe.MOE_ERR_ALIGNMENT


LIN = moe.MoELinearConfig(T=5, K=64, N=128, activation="gelu")


def fwd(lib, c, ws=1 << 20, n=1 << 30, **at):
    names = ["x", "W", "bias", "residual", "y", "z"]
    ptr = {k: 4096 * (i + 1) for i, k in enumerate(names)}
    ptr.update(at)
    return lib.moe_linear_fwd(ctypes.byref(c), *[P(ptr[k]) for k in names], P(ws), n, P(0))


def bwd(lib, c, ws=1 << 20, n=1 << 30, **at):
    names = ["x", "W", "z", "dy", "dx", "dW", "dbias"]
    ptr = {k: 4096 * (i + 1) for i, k in enumerate(names)}
    ptr.update(at)
    return lib.moe_linear_bwd(ctypes.byref(c), *[P(ptr[k]) for k in names], P(ws), n, P(0))


@pytest.mark.parametrize("bad", [dict(T=-1), dict(K=0), dict(K=12), dict(N=0), dict(N=4), dict(N=-8),
                                 dict(activation=-1), dict(activation=5), dict(ldx=56), dict(ldx=68), dict(ldw=120),
                                 dict(ldr=1), dict(ldy=-8), dict(ldz=132), dict(lddy=64), dict(lddx=60),
                                 dict(lddw=64)])
def test_linear_refuses_bad_shapes(lib, bad):
    c = LIN.c()
    for k, v in bad.items():
        setattr(c, k, v)
    assert fwd(lib, c) == moe.MOE_ERR_INVALID_ARG
    assert bwd(lib, c) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_linear_workspace_size(ctypes.byref(c)) == 0


def test_linear_refuses_what_its_arithmetic_cannot_hold(lib):
    assert fwd(lib, LIN.c((1 << 38) + 8)) == moe.MOE_ERR_UNSUPPORTED      # the copy engine's row distance
    for big in (dict(T=(1 << 30) + 1), dict(K=(1 << 30) + 8), dict(N=(1 << 30) + 8)):
        c = replace(LIN, **big).c()
        assert fwd(lib, c, n=1 << 50) == bwd(lib, c, n=1 << 50) == moe.MOE_ERR_UNSUPPORTED
        assert lib.moe_linear_workspace_size(ctypes.byref(c)) == 0
    assert moe.moe_linear_workspace_size(replace(LIN, T=1 << 30)) > (1 << 30) * 128 * 2


def test_linear_refuses_missing_and_misaligned_tensors(lib):
    c = LIN.c()
    for name in ("x", "W", "y"):
        assert fwd(lib, c, **{name: 0}) == moe.MOE_ERR_INVALID_ARG
    for name, off in (("x", 8), ("W", 2), ("bias", 2), ("residual", 8), ("y", 8), ("z", 8)):
        assert fwd(lib, c, **{name: (1 << 24) + off}) == moe.MOE_ERR_ALIGNMENT
    for name in ("dy", "z", "x", "W"):
        assert bwd(lib, c, **{name: 0}) == moe.MOE_ERR_INVALID_ARG
    for name, off in (("x", 8), ("W", 2), ("z", 8), ("dy", 8), ("dx", 8), ("dW", 8), ("dbias", 2)):
        assert bwd(lib, c, **{name: (1 << 24) + off}) == moe.MOE_ERR_ALIGNMENT
    assert bwd(lib, c, dx=0, dW=0, dbias=0) == moe.MOE_OK      # nothing wanted


def test_linear_workspace(lib):
    n = moe.moe_linear_workspace_size(LIN)
    assert n >= 256 + 5 * 128 * 2
    c = LIN.c()
    for call in (fwd, bwd):
        assert call(lib, c, n=n - 1) == moe.MOE_ERR_WORKSPACE
        assert call(lib, c, ws=0) == moe.MOE_ERR_WORKSPACE
        assert call(lib, c, ws=(1 << 20) + 16) == moe.MOE_ERR_ALIGNMENT
    sizes = [moe.moe_linear_workspace_size(replace(LIN, T=t)) for t in (0, 1, 2, 64, 65, 128, 129, 1000, 4096, 70000)]
    assert sizes == sorted(sizes)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_a_device_say_so(lib):
    assert few(lib, CFG) == moe.MOE_ERR_NO_DEVICE
    assert fwd(lib, LIN.c()) == moe.MOE_ERR_NO_DEVICE
    assert bwd(lib, LIN.c()) == moe.MOE_ERR_NO_DEVICE


def test_binding_refuses_host_tensors_and_unknown_activations(lib):
    with pytest.raises(ValueError, match="unknown activation"):
        moe.moe_linear_workspace_size(replace(LIN, activation="tanh"))
    t = torch.zeros((5, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        moe.moe_linear_fwd(LIN, t, t, None, None, t, t)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        moe.moe_layer_fwd_few(CFG, t, t, t, None, t, t, t, t, t)
    with pytest.raises(TypeError):
        moe.moe_linear_fwd(LIN, 5, t, None, None, t, t)


def test_linear_refuses_outputs_in_the_place_of_others(lib):
    at = {k: 4096 * (i + 1) for i, k in enumerate(["x", "W", "bias", "residual", "y", "z"])}
    for out, other in [("y", "x"), ("y", "W"), ("y", "z"), ("z", "x"), ("z", "W"), ("z", "residual")]:
        assert fwd(lib, LIN.c(), **{out: at[other]}) == moe.MOE_ERR_INVALID_ARG, (out, other)
    # the residual in y's place: with another row distance a row would be read after its place was written
    assert fwd(lib, LIN.c(0, 0, 136, 128), residual=at["y"]) == moe.MOE_ERR_INVALID_ARG
    assert fwd(lib, LIN.c(0, 0, 136, 0), residual=at["y"]) == moe.MOE_ERR_INVALID_ARG
    assert fwd(lib, LIN.c(0, 0, 128, 0), residual=at["y"], n=0) == moe.MOE_ERR_WORKSPACE  # allowed, as far as this goes
    at = {k: 4096 * (i + 1) for i, k in enumerate(["x", "W", "z", "dy", "dx", "dW", "dbias"])}
    for out in ["dx", "dW", "dbias"]:
        for other in at:
            if other != out:
                assert bwd(lib, LIN.c(), **{out: at[other]}) == moe.MOE_ERR_INVALID_ARG, (out, other)


def test_linear_config_copies_and_follows_its_fields():
    import copy
    import pickle
    c = replace(LIN)
    first = c._arg(8, 0)._obj
    assert c._arg(8, 0)._obj is first and (first.T, first.ldx) == (5, 8)  # the same call keeps its struct
    c.T = 6
    assert c._arg(8, 0)._obj.T == 6 and c._arg(0, 0)._obj.ldx == 0
    for d in (copy.copy(c), copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        d.T = 7
        assert d._arg(0, 0)._obj.T == 7 and c._arg(0, 0)._obj.T == 6


def test_linear_plan_checks_its_arguments(lib):
    p = moe._LinearPlan()

    def plan(cfg, product=0, out=ctypes.byref(p)):
        return lib.moe_linear_plan(ctypes.byref(cfg.c()), product, 0, 0, out)

    assert plan(replace(LIN, K=12)) == plan(LIN, 3) == plan(LIN, -1) == moe.MOE_ERR_INVALID_ARG
    assert plan(LIN, 0, None) == plan(replace(LIN, T=0)) == moe.MOE_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="unknown product"):
        moe.moe_linear_plan(LIN, "dz")
    if not torch.cuda.is_available():
        assert [plan(LIN, i) for i in range(3)] == [moe.MOE_ERR_NO_DEVICE] * 3


def test_few_layer_keeps_its_own_configuration(monkeypatch):
    """cfg is read when the layer is made: what its owner does to it (or to its list of offsets) later reaches no call."""
    monkeypatch.setattr(moe, "alloc_few_workspace", lambda cfg, device=None, stream=None: None)
    t = torch.zeros(1)
    cfg = replace(CFG, T=8, ffn_offsets=list(CFG.ffn_offsets))
    layer = moe.MoEFewLayer(cfg, t, t, None, t, t, t)
    before = list(layer._config(3).ffn_offsets[0:9])
    cfg.ffn_offsets[1:8] = [256, 384, 512, 640, 768, 896, 960]
    cfg.T, cfg.k = 1, 1
    assert list(layer._config(3).ffn_offsets[0:9]) == before
    assert list(layer._config(7).ffn_offsets[0:9]) == before and layer._config(7).k == 2


def test_linear_forward_asks_for_a_workspace_without_the_backwards_scratch(lib):
    big = moe.MoELinearConfig(T=16384, K=4096, N=14336, activation="silu")
    n = moe.moe_linear_fwd_workspace_size(big)
    assert n == moe.moe_linear_fwd_workspace_size(LIN) == 4096
    assert moe.moe_linear_workspace_size(big) > 16384 * 14336 * 2
    assert moe.moe_linear_workspace_size(LIN) >= n            # a workspace of the layer serves its forward
    bad = LIN.c()
    bad.K = 12
    assert lib.moe_linear_fwd_workspace_size(ctypes.byref(bad)) == 0
    fine = moe.MOE_OK if torch.cuda.is_available() else moe.MOE_ERR_NO_DEVICE
    if fine != moe.MOE_OK:                                    # (with a device the call would run, on these pointers)
        assert fwd(lib, big.c(), n=n) == fine
    assert fwd(lib, big.c(), n=n - 1) == moe.MOE_ERR_WORKSPACE
    assert bwd(lib, big.c(), n=n) == moe.MOE_ERR_WORKSPACE
