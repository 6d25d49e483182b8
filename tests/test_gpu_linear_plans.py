"""Every kernel of the linear layer, for every product that takes it, against the formulas in 64 bits.

A product's kernel, tile and split follow from a cost model, so each case names the plan it is there for and the test
asserts it (moe_linear_plan): a refit of the model that moves a product elsewhere fails here and does not pass
untested.  The cases cover, for the forward and both gradients, every split of every tile width of the three kernels,
pairs that work through three and more tiles (both accumulators in turn), the blocked tile order (an M panel above
48 MB), ragged ends in every extent, padded rows, and operands copied by 3-D boxes (extents that are multiples of 64).
Bounds as in test_gpu_linear.py.
"""
import pytest
import torch

import sparse_mixture_experts_rms_b200 as moe
from tests.test_gpu_linear import BF, Buf, act, act_grad, gam, grad_error, randn, rounded, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_rms_b200 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def ids(c):
    return "-".join(str(v) for v in c)


# T, K, N, residual, z, kernel, tile, split
FWD = [
    (9, 72, 8, 1, 1, "split", 16, 2),
    (65, 456, 8, 1, 1, "split", 32, 8),
    (778, 224, 4888, 1, 1, "split", 112, 1),
    (303, 464, 1288, 1, 1, "split", 80, 3),
    (157, 2344, 1064, 1, 1, "split", 80, 8),
    (768, 2816, 1408, 1, 1, "split", 128, 4),
    (560, 1216, 6216, 0, 0, "split", 192, 1),
    (267, 1800, 3256, 1, 1, "split", 144, 2),
    (523, 1912, 1704, 1, 0, "split", 176, 3),
    (270, 1488, 1960, 0, 1, "split", 144, 4),
    (265, 328, 14384, 0, 0, "pair", 256, 1),
    (2309, 520, 6664, 1, 1, "pair", 256, 1),   # 270 tiles for the pairs of 148 SMs
    (2309, 520, 6664, 1, 0, "pair", 256, 1),
    (2309, 520, 6664, 0, 1, "pair", 256, 1),
    (2304, 512, 6656, 0, 0, "pair", 256, 1),
    (9513, 136, 264, 1, 1, "pair", 128, 1),
    (8200, 4096, 1032, 1, 1, "pair", 256, 1),  # x: 67 MB
    (6362, 2600, 8, 1, 1, "pair_split", 128, 2),
    (466, 5600, 1304, 1, 1, "pair_split", 128, 3),
    (1178, 7800, 136, 1, 0, "pair_split", 128, 4),
    (789, 2824, 1432, 1, 1, "pair_split", 256, 2),
    (789, 2816, 1472, 0, 0, "pair_split", 256, 2),
    (1531, 2800, 664, 0, 1, "pair_split", 256, 3),
    (3308, 3800, 136, 1, 1, "pair_split", 256, 4),
]

# product, T, K, N, kernel, tile, split
BWD = [
    ("dx", 65, 8, 456, "split", 32, 8),
    ("dx", 783, 5120, 224, "split", 112, 1),
    ("dx", 313, 1296, 464, "split", 80, 3),
    ("dx", 157, 1056, 2328, "split", 80, 8),
    ("dx", 768, 1408, 2816, "split", 128, 4),
    ("dx", 530, 6240, 1296, "split", 192, 1),
    ("dx", 270, 3168, 1624, "split", 144, 2),
    ("dx", 523, 1744, 1456, "split", 176, 3),
    ("dx", 282, 1984, 1504, "split", 144, 4),
    ("dx", 2309, 6664, 520, "pair", 256, 1),
    ("dx", 2304, 6656, 512, "pair", 256, 1),
    ("dx", 9513, 264, 136, "pair", 128, 1),
    ("dx", 8200, 1032, 4096, "pair", 256, 1),
    ("dx", 6306, 8, 2600, "pair_split", 128, 2),
    ("dx", 455, 1336, 5600, "pair_split", 128, 3),
    ("dx", 1210, 160, 7400, "pair_split", 128, 4),
    ("dx", 799, 1456, 2864, "pair_split", 256, 2),
    ("dx", 1157, 904, 2800, "pair_split", 256, 3),
    ("dx", 962, 672, 5800, "pair_split", 256, 4),
    ("dW", 333, 584, 520, "split", 64, 2),
    ("dW", 449, 8, 8, "split", 64, 8),
    ("dW", 266, 264, 9736, "split", 128, 1),
    ("dW", 2215, 1136, 920, "split", 128, 2),
    ("dW", 930, 968, 656, "split", 128, 3),
    ("dW", 2816, 896, 1408, "split", 128, 3),
    ("dW", 1929, 720, 664, "split", 128, 4),
    ("dW", 4993, 720, 272, "split", 128, 8),
    ("dW", 1200, 568, 6264, "split", 192, 1),
    ("dW", 3674, 528, 2976, "split", 192, 2),
    ("dW", 2241, 520, 1880, "split", 192, 3),
    ("dW", 2060, 552, 1288, "split", 192, 4),
    ("dW", 5444, 328, 792, "split", 192, 8),
    ("dW", 6000, 3088, 1328, "split", 256, 1),
    ("dW", 521, 2312, 6664, "pair", 256, 1),
    ("dW", 512, 2304, 6656, "pair", 256, 1),
    ("dW", 130, 9520, 264, "pair", 128, 1),
    ("dW", 4100, 8200, 1032, "pair", 256, 1),
    ("dW", 2600, 6336, 8, "pair_split", 128, 2),
    ("dW", 5500, 496, 1296, "pair_split", 128, 3),
    ("dW", 7700, 1176, 136, "pair_split", 128, 4),
    ("dW", 2815, 912, 1416, "pair_split", 256, 2),
    ("dW", 2815, 960, 1472, "pair_split", 256, 2),
    ("dW", 2500, 1672, 648, "pair_split", 256, 3),
    ("dW", 4001, 3120, 136, "pair_split", 256, 4),
]


def pad_of(N):
    """Rows apart by more than their length, but dense where the extents are there for the 3-D copies."""
    return 0 if N % 64 == 0 else 24


def no_error(ws):
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(ws, raise_on_error=False) == 0


@pytest.mark.parametrize("case", FWD, ids=ids)
def test_forward(case):
    T, K, N, has_r, save, *plan = case
    cfg = moe.MoELinearConfig(T, K, N, "gelu")
    assert moe.moe_linear_plan(cfg, "fwd", residual=bool(has_r), z=bool(save)) == tuple(plan)
    g = torch.Generator(device="cuda").manual_seed(T + K)
    pad = pad_of(N)
    x, W = Buf(T, K, pad, randn(g, T, K)), Buf(K, N, pad, randn(g, K, N, std=K ** -0.5))
    b = torch.randn(N, generator=g, device="cuda")
    r = Buf(T, N, pad, randn(g, T, N)) if has_r else None
    y, z = Buf(T, N, pad), Buf(T, N, pad) if save else None
    ws = moe.alloc_linear_workspace(cfg)

    def call():
        moe.moe_linear_fwd(cfg, x.view, W.view, b, r.view if r else None, y.view, ws, z=z.view if z else None)
        no_error(ws)

    call()
    X, Wd = x.view.double(), W.view.double()
    zr = X @ Wd + b.double()
    dz = gam(K) * (X.abs() @ Wd.abs()) + 2.0 ** -23 * zr.abs()
    a = act(zr, "gelu")
    ref = a + (r.view.double() if has_r else 0)
    within(y.view, ref, rounded(1.13 * dz + 2.0 ** -20 * a.abs() + 2.0 ** -23 * ref.abs(), ref), "y")
    assert y.clean()
    if save:
        within(z.view, zr, rounded(dz, zr), "z")
        assert z.clean()
    first = y.view.clone()
    call()
    assert torch.equal(y.view, first)


@pytest.mark.parametrize("case", BWD, ids=ids)
def test_gradients(case):
    product, T, K, N, *plan = case
    kind = "silu" if T % 2 else "none"   # dz from the workspace, dense, or dy itself with its padded rows
    cfg = moe.MoELinearConfig(T, K, N, kind)
    assert moe.moe_linear_plan(cfg, product) == tuple(plan)
    g = torch.Generator(device="cuda").manual_seed(T + N)
    pad = pad_of(N)
    x, W = Buf(T, K, pad, randn(g, T, K)), Buf(K, N, pad, randn(g, K, N, std=K ** -0.5))
    z, dy = Buf(T, N, pad, randn(g, T, N, std=2.0)), Buf(T, N, pad, randn(g, T, N))
    out = Buf(T, K, pad) if product == "dx" else Buf(K, N, pad)
    ws = moe.alloc_linear_workspace(cfg)

    def call():
        dx, dW = (out.view, None) if product == "dx" else (None, out.view)
        moe.moe_linear_bwd(cfg, x.view, W.view, z.view, dy.view, dx, dW, None, ws)
        no_error(ws)

    call()
    dz = dy.view.double() * act_grad(z.view.double(), kind)
    err = dy.view.double().abs() * grad_error(z.view, kind)
    operand = 0.0 if kind == "none" else err * (1 + 2.0 ** -8) + 2.0 ** -8 * dz.abs()
    if product == "dx":
        Wd = W.view.double()
        ref, b = dz @ Wd.T, (operand + gam(N) * dz.abs()) @ Wd.abs().T
    else:
        X = x.view.double()
        ref, b = X.T @ dz, X.abs().T @ (operand + gam(T) * dz.abs())
    within(out.view, ref, rounded(b, ref), product)
    assert out.clean()
    first = out.view.clone()
    call()
    assert torch.equal(out.view, first)


def product(kind, T, K, N, g):
    """A product's call, its output and its workspace."""
    cfg = moe.MoELinearConfig(T, K, N)
    ws = moe.alloc_linear_workspace(cfg)
    x, W, dy = randn(g, T, K), randn(g, K, N, std=K ** -0.5), randn(g, T, N)
    out = torch.empty({"fwd": (T, N), "dx": (T, K), "dW": (K, N)}[kind], dtype=BF, device="cuda")

    def call():
        if kind == "fwd":
            moe.moe_linear_fwd(cfg, x, W, None, None, out, ws)
        else:
            moe.moe_linear_bwd(cfg, x, W, None, dy, out if kind == "dx" else None, out if kind == "dW" else None, None,
                               ws)
    return cfg, call, out, ws


# one of each kernel for each product
EACH = [("fwd", 157, 2344, 1064, "split"), ("fwd", 2309, 520, 6664, "pair"), ("fwd", 3308, 3800, 136, "pair_split"),
        ("dx", 157, 1056, 2328, "split"), ("dx", 2309, 6664, 520, "pair"), ("dx", 962, 672, 5800, "pair_split"),
        ("dW", 5444, 328, 792, "split"), ("dW", 521, 2312, 6664, "pair"), ("dW", 4001, 3120, 136, "pair_split")]


@pytest.mark.parametrize("case", EACH, ids=ids)
def test_waits_run_out_then_recover(case):
    kind, T, K, N, kernel = case
    cfg, call, out, ws = product(kind, T, K, N, torch.Generator(device="cuda").manual_seed(7))
    assert moe.moe_linear_plan(cfg, kind)[0] == kernel
    call()
    no_error(ws)
    want = out.clone()
    moe.moe_set_wait_limit(ws, 1)
    call()
    torch.cuda.synchronize()
    code = moe.moe_get_device_error(ws, raise_on_error=False)
    # a wait may also complete within its first polls: then nothing ran out and the result stands
    assert code & moe.MOE_DEVERR_TIMEOUT or (code == 0 and torch.equal(out, want)), f"device error word 0x{code:x}"
    moe.moe_set_wait_limit(ws, 0)
    for _ in range(2):
        out.zero_()
        call()
        no_error(ws)
        assert torch.equal(out, want)


def test_every_kernel_at_once_on_its_own_stream():
    g = torch.Generator(device="cuda").manual_seed(5)
    runs = []
    for kind, T, K, N, kernel in EACH:
        cfg, call, out, ws = product(kind, T, K, N, g)
        assert moe.moe_linear_plan(cfg, kind)[0] == kernel
        call()
        runs.append((call, out, out.clone(), ws))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(20):
        for (call, *_), s in zip(runs, streams):
            with torch.cuda.stream(s):
                call()
    torch.cuda.synchronize()
    for _, out, want, ws in runs:
        assert moe.moe_get_device_error(ws) == 0
        assert torch.equal(out, want)
