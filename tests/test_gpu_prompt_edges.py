"""Ends of the prompt-side operators' ranges on the GPU: arguments, magnitudes and orders of calls at which a form
that is right elsewhere can be wrong."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from prompt_common import U, check_near, check_q8, offsets_of, products, quantize, value_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    import bitplane_mixed_precision_b200 as pm
    return pm


def empty(*shape, dtype=torch.uint8):
    return torch.empty(*shape, dtype=dtype, device="cuda")


# ---------------------------------------------------------------- SwiGLU

@pytest.mark.parametrize("rows", [3, 200])
@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("out", ["bf16", "q8"])
def test_swiglu_of_large_gates(pm, rows, kind, out):
    """One product a sum, all of them exact, so that SwiGLU's own error is what is seen: 17 + |g| / 20 roundings, and,
    where exp(-|g|) is subnormal, a step of the subnormals in it. Up values near 2^100 bring what is left into range."""
    K, I = 128, 64
    gates = [-104.0, -96.0, -88.0, -80.0, -30.0, -0.5, 0.0, 0.5, 30.0, 88.0, 104.0]
    g = torch.tensor((gates * 6)[:I], device="cuda")
    u = torch.where(g < -60, 2.0 ** 100, 1.5)
    x, w = torch.zeros(rows, K, device="cuda"), torch.zeros(1, 2 * I, K, device="cuda")
    x[:, 0], w[0, :I, 0], w[0, I:, 0] = 1.0, g, u
    t = pm.Q8 if kind == "q8" else pm.BF16
    (xc, xs), (wc, ws) = (quantize(x), quantize(w)) if kind == "q8" else ((x.bfloat16(), None), (w.bfloat16(), None))
    h = empty(rows, I, dtype=torch.uint8 if out == "q8" else torch.bfloat16)
    hs = empty(rows, I // 32) if out == "q8" else None
    pm.grouped_swiglu(pm.make_dense(t, wc, ws, 1, 2 * I, K), pm.make_rows(t, xc, xs, rows), offsets_of([rows]), rows,
                      pm.Q8 if out == "q8" else pm.BF16, h, hs)
    torch.cuda.synchronize()
    g, u = g.double().expand(rows, I), u.double().expand(rows, I)
    v = g * torch.sigmoid(g) * u
    dv = (17 + g.abs() / 20) * U * v.abs() + (g.abs() + 1) * 2.0 ** -149 * u
    if out == "q8":
        check_q8(h, hs, v, dv)
    else:
        check_near(h, v, dv, 2.0 ** -8)


@pytest.mark.parametrize("rows", [3, 200])
def test_swiglu_of_gates_that_are_not_finite(pm, rows):
    """The formula's values: inf * u for a gate of +inf, and NaN for -inf (-inf * 0) and NaN; zeros far below zero."""
    K, I = 64, 64
    gates = [float("inf"), float("-inf"), float("nan"), 3e38, -3e38, -1000.0, 1.0, 0.0]
    g = torch.tensor(gates * (I // 8), device="cuda").bfloat16()
    x, w = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((rows, K), (1, 2 * I, K)))
    x[:, 0], w[0, :I, 0], w[0, I:, 0] = 1.0, g, 0.5
    h = empty(rows, I, dtype=torch.bfloat16)
    pm.grouped_swiglu(pm.make_dense(pm.BF16, w, None, 1, 2 * I, K), pm.make_rows(pm.BF16, x, None, rows),
                      offsets_of([rows]), rows, pm.BF16, h, None)
    torch.cuda.synchronize()
    h = h.view(rows, I // 8, 8).float()
    assert bool((h[..., 0] == float("inf")).all()) and bool(h[..., 1:3].isnan().all())
    assert bool((h[..., 3] == 0.5 * g[3].float()).all()) and not h[..., [4, 5, 7]].any()
    assert bool(((h[..., 6] - 0.5 * torch.sigmoid(torch.tensor(1.0))).abs() <= 2.0 ** -9 * 0.5).all())


# ---------------------------------------------------------------- pairs by expert

COUNTERS = """
import sys
import numpy as np
import torch
import bitplane_mixed_precision_b200 as pm
E, T, k = int(sys.argv[1]), 300, 3
ids = np.random.default_rng(E).integers(0, E, (T, k)).astype(np.int32)
o, r, t = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * k, T * k))
pm.group_pairs(torch.from_numpy(ids).cuda(), T, k, E, o, r, t)
order = np.argsort(ids.reshape(-1), kind="stable")
assert np.array_equal(t.cpu().numpy(), order // k)
assert np.array_equal(o.cpu().numpy()[1:], np.cumsum(np.bincount(ids.reshape(-1), minlength=E)))
"""


@pytest.mark.parametrize("E", [767, 768, 769])
def test_group_pairs_where_its_counters_fill_48_kb(E):
    """16 counters an expert are 48 KB at 768 experts, what a block has without asking for more. In a process of its
    own: once a call has asked for more, the next ones have it."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", COUNTERS, str(E)], cwd=root, capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr


# ---------------------------------------------------------------- norm

def norm_formula(r, gain, eps):
    """(v, bound) in 64 bits: as test_gpu_prompt's, and a step of the subnormals, to which small values are rounded."""
    r64 = r.double()
    ms = r64.pow(2).mean(1, keepdim=True) + eps
    v = torch.where(ms == 0, 0.0, r64 / ms.sqrt()) * gain.double()
    return v, 30 * U * v.abs() + 2.0 ** -149 * (1 + gain.double().abs())


@pytest.mark.parametrize("H", [128, 4096, 12800])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-20, 1e-6])
@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-25, 1e-21, 1e-16, 1e-10, 1e10, 1e17, 1e18, 1e25, 5e37])
def test_residual_norm_q8_over_the_floats(pm, scale, eps, H):
    """Rows whose squares leave the floats at either end, one with a single large value, one of zeros; an eps that
    counts beside them or does not."""
    T = 4
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    r = torch.randn(T, H, generator=g, device="cuda").clamp(-6, 6) * scale
    r[1, 1:] *= 1e-3
    r[2] = 0.0
    gain = 1 + 0.2 * torch.randn(H, generator=g, device="cuda")
    eps = float(np.float32(eps))
    v, dv = norm_formula(r, gain, eps)
    before = r.clone()
    codes, scales, x = empty(T, H), empty(T, H // 32), empty(T, H, dtype=torch.bfloat16)
    pm.residual_norm_q8(r, None, gain, eps, T, H, codes, scales, x)
    torch.cuda.synchronize()
    assert torch.equal(r, before)
    check_q8(codes, scales, v, dv)
    check_near(x, v, dv, 2.0 ** -8)


def test_residual_norm_q8_adds_before_it_scales(pm):
    """The stored sum is r + y at both ends, and the norm is of that."""
    T, H = 3, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    scale = torch.tensor([[1e-30], [1.0], [1e30]], device="cuda")
    r, y = (torch.randn(T, H, generator=g, device="cuda") * scale for _ in range(2))
    want = r + y
    x = empty(T, H, dtype=torch.bfloat16)
    pm.residual_norm_q8(r, y, None, 0.0, T, H, None, None, x)
    torch.cuda.synchronize()
    assert torch.equal(r, want)
    v, dv = norm_formula(want, torch.ones(H, device="cuda"), 0.0)
    check_near(x, v, dv, 2.0 ** -8)


def test_residual_norm_q8_of_infinities(pm):
    """As the formula has it in floats: the mean is infinite, its inverse root 0, so that finite values are zeros and
    the infinite ones NaN."""
    T, H = 2, 256
    r = torch.ones(T, H, device="cuda")
    r[0, 5], r[1, 200] = float("inf"), float("-inf")
    codes, scales, x = empty(T, H), empty(T, H // 32), empty(T, H, dtype=torch.bfloat16)
    pm.residual_norm_q8(r, None, None, 0.0, T, H, codes, scales, x)
    torch.cuda.synchronize()
    bad = r.isinf()
    assert torch.equal(x.isnan(), bad) and not x[~bad].any()
    blocks = bad.view(T, -1, 32).any(2)
    assert torch.equal(scales == 255, blocks) and not scales[~blocks].any()


@pytest.mark.parametrize("T,H", [(1, 8), (5, 72), (3, 136), (700, 1000), (2, 4104), (2, 32760)])
def test_residual_norm_in_bf16_alone_takes_multiples_of_8(pm, T, H):
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    r, y = (torch.randn(T, H, generator=g, device="cuda") for _ in range(2))
    gain = 1 + 0.2 * torch.randn(H, generator=g, device="cuda")
    want = r + y
    x = torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device="cuda")
    pm.residual_norm_q8(r, y, gain, 1e-6, T, H, None, None, x)
    torch.cuda.synchronize()
    assert torch.equal(r, want) and bool((x[T] == 7.0).all())
    v, dv = norm_formula(want, gain, 1e-6)
    check_near(x[:T], v, dv, 2.0 ** -8)


def test_a_bf16_layer_of_a_width_of_8s(pm):
    """DenseExperts takes bf16 matrices in multiples of 8, and so does every step of their layer."""
    from bitplane_mixed_precision_b200.prompt import DenseExperts, PromptLayer
    E, H, I, k, T = 5, 136, 72, 2, 30
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    X = DenseExperts(E, H, I, lambda e, m, w: w.copy_(0.1 * torch.randn(w.numel(), generator=g, device="cuda")), pm.BF16)
    L = PromptLayer(X, k, T)
    r = torch.randn(T, H, generator=g, device="cuda")
    L.norm(r, None, T, eps=1e-6)
    L.route(torch.randn(T, E, generator=g, device="cuda"), T)
    y = L.forward(T)
    torch.cuda.synchronize()
    check_near(L.x[:T], *norm_formula(r, torch.ones(H, device="cuda"), 1e-6), 2.0 ** -8)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    x, up, down = L.x.double(), X.up.double(), X.down.double()
    for t in range(T):
        for i in range(k):
            e = int(L.ids[t, i])
            p = up[e] @ x[t]
            want[t] += float(L.w[t, i]) * (down[e] @ (p[:I] * torch.sigmoid(p[:I]) * p[I:]).bfloat16().double())
    # two roundings to bf16 on the way (h, nearly always the same one, and the rows): 2^-8 each of what they carry
    assert float((y - want).norm() / want.norm()) <= 2.0 ** -7


# ---------------------------------------------------------------- products

@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("K,N", [(256, 1096), (1152, 776), (640, 2048)])
def test_down_products_of_many_ragged_experts(pm, kind, out, K, N):
    """Rows in place (no index), enough row tiles for 256 matrix rows a tile and several tiles for every SM: boxes of 32
    and of 128 rows in turn, ragged last columns, rows behind the last expert left alone."""
    rng = np.random.default_rng(K + N)
    counts = [int(n) for n in rng.integers(0, 260, 90)]
    counts[0], counts[7], counts[20], counts[50], counts[89] = 1, 0, 128, 1025, 64
    M, extra = sum(counts), 5
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    x = torch.randn(M + extra, K, generator=g, device="cuda") * torch.exp(torch.randn(M + extra, 1, generator=g,
                                                                                      device="cuda"))
    w = torch.randn(len(counts), N, K, generator=g, device="cuda") * K ** -0.5
    t, xs, ws = pm.BF16, None, None
    if kind == "q8":
        t, (x, xs), (w, ws) = pm.Q8, quantize(x), quantize(w)
        x64, w64 = value_of(x, xs)[:M], value_of(w, ws)
    else:
        x, w = x.bfloat16(), w.bfloat16()
        x64, w64 = x.double()[:M], w.double()
    o = torch.full((M + extra, N), 7.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    pm.grouped_matmul(pm.make_dense(t, w, ws, len(counts), N, K), pm.make_rows(t, x, xs, M + extra), offsets_of(counts),
                      M + extra, pm.F32 if out == "f32" else pm.BF16, o)
    torch.cuda.synchronize()
    check_near(o[:M], *products(x64, w64, counts), U if out == "f32" else 2.0 ** -8)
    assert bool((o[M:] == 7.0).all())
