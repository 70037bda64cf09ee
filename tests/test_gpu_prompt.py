"""The prompt-side operators on the GPU against plain 64-bit forms: conversion to q8, residual norm with an
8-bit output, pairs by expert, grouped products with and without SwiGLU, combination."""
import numpy as np
import pytest
import torch

from prompt_common import (U, bytes_of, check_near, check_q8, offsets_of, products, quantize, swiglu, value_of)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    import bitplane_mixed_precision_b200 as pm
    return pm


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def empty(*shape, dtype=torch.uint8):
    return torch.empty(*shape, dtype=dtype, device="cuda")


# ---------------------------------------------------------------- q8

def q8_inputs(kind, rows, K):
    v = randn(gen(rows * 7 + K), rows, K)
    if kind == "wide":
        v = v * torch.exp2(torch.randint(-140, 120, (rows, K), generator=gen(3), device="cuda").float())
    elif kind == "edges":  # block maxima on both sides of 448 * 2^e, at it, and zero blocks
        top = torch.tensor([448.0, 448.00003, 447.99997, 1.75, 1.7500001, 3.5, 0.0, 2.0 ** -126, 2.0 ** -140],
                           device="cuda")
        v = v.clamp(-1, 1) * 0.5
        v.view(-1, 32)[:, 5] = 1.0
        n = v.numel() // 32
        v = (v.view(-1, 32) * top.repeat(n // 9 + 1)[:n, None]).view(rows, K)
    return v


@pytest.mark.parametrize("kind", ["normal", "wide", "edges"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (17, 4096), (1000, 160)])
@pytest.mark.parametrize("bf16", [False, True])
def test_quantize_q8_is_exact(pm, kind, rows, K, bf16):
    v = q8_inputs(kind, rows, K)
    if bf16:
        v = v.bfloat16()
    codes, scales = empty(rows, K), empty(rows, K // 32)
    pm.quantize_q8(v, bf16, rows, K, codes, scales)
    rc, rs = quantize(v)
    torch.cuda.synchronize()
    assert torch.equal(scales, rs)
    assert torch.equal(codes, rc)


def test_quantize_q8_blocks_that_are_not_finite(pm):
    v = randn(gen(1), 4, 128)
    v[0, 3], v[1, 40], v[2, 127] = float("nan"), float("inf"), float("-inf")
    codes, scales = empty(4, 128), empty(4, 4)
    pm.quantize_q8(v, False, 4, 128, codes, scales)
    torch.cuda.synchronize()
    bad = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[1, 1] = bad[2, 3] = True
    assert torch.equal(scales == 255, bad)
    wide = bad.repeat_interleave(32, 1)
    assert bool((codes[wide] == 0x7f).all())
    assert torch.equal(value_of(codes, scales).isnan(), wide)


# ---------------------------------------------------------------- norm

def norm_reference(r, y, gain, eps):
    """The formula in 64 bits from the float r + y, and the float form's bound: at most 45 roundings in the
    sum of squares (halved by the root), 4 in the root and its inverse, 2 in the products."""
    r2 = r if y is None else r + y
    v = r2.double()
    ms = v.pow(2).mean(1, keepdim=True) + eps
    v = torch.where(ms == 0, 0.0, v / ms.sqrt())
    if gain is not None:
        v = v * gain.double()
    return r2, v, 30 * U * v.abs()


@pytest.mark.parametrize("T,H", [(1, 128), (3, 256), (5, 384), (149, 1024), (2, 4096), (1025, 4096), (33, 5120),
                                 (7, 8192), (4, 12800), (2, 32768)])
@pytest.mark.parametrize("with_y,with_gain,outs", [(True, True, "q"), (True, False, "qx"), (False, True, "x"),
                                                   (False, False, "q")])
def test_residual_norm_q8(pm, T, H, with_y, with_gain, outs):
    g = gen(T + H)
    r = randn(g, T, H) * torch.exp(randn(g, 1, H))
    y = randn(g, T, H) if with_y else None
    gain = 1 + 0.3 * randn(g, H) if with_gain else None
    r2, v, dv = norm_reference(r, y, gain, 1e-6)
    codes, scales = (empty(T, H), empty(T, H // 32)) if "q" in outs else (None, None)
    x = empty(T, H, dtype=torch.bfloat16) if "x" in outs else None
    pm.residual_norm_q8(r, y, gain, 1e-6, T, H, codes, scales, x)
    torch.cuda.synchronize()
    assert torch.equal(r, r2)
    if codes is not None:
        check_q8(codes, scales, v, dv)
    if x is not None:
        check_near(x, v, dv, 2.0 ** -8)


@pytest.mark.parametrize("scale", [1e-18, 1e-3, 1e15])
def test_residual_norm_q8_magnitudes(pm, scale):
    T, H = 3, 512
    r = randn(gen(4), T, H) * scale
    r2, v, dv = norm_reference(r, None, None, 0.0)
    codes, scales = empty(T, H), empty(T, H // 32)
    pm.residual_norm_q8(r, None, None, 0.0, T, H, codes, scales)
    torch.cuda.synchronize()
    check_q8(codes, scales, v, dv)


def test_residual_norm_q8_rows_of_zeros_and_not_finite(pm):
    T, H = 5, 256
    r = randn(gen(5), T, H)
    r[1] = 0.0
    r[3, 77] = float("nan")
    codes, scales = empty(T, H), empty(T, H // 32)
    x = empty(T, H, dtype=torch.bfloat16)
    pm.residual_norm_q8(r, None, None, 0.0, T, H, codes, scales, x)
    torch.cuda.synchronize()
    assert not codes[1].any() and not scales[1].any() and not x[1].any()
    assert bool((scales[3] == 255).all()) and bool((codes[3] == 0x7f).all()) and bool(x[3].isnan().all())
    keep = [0, 2, 4]
    _, v, dv = norm_reference(r[keep], None, None, 0.0)
    check_q8(codes[keep], scales[keep], v, dv)


def test_residual_norm_q8_follows_residual_norm(pm):
    """Without a gain and with eps 0 the bf16 output is pmoe_residual_norm's up to the order of the sum."""
    T, H = 9, 2048
    r = randn(gen(6), T, H)
    y = randn(gen(7), T, H)
    r1, r2 = r.clone(), r.clone()
    x1, x2 = empty(T, H, dtype=torch.bfloat16), empty(T, H, dtype=torch.bfloat16)
    pm.residual_norm(r1, y, T, H, x1)
    pm.residual_norm_q8(r2, y, None, 0.0, T, H, None, None, x2)
    torch.cuda.synchronize()
    assert torch.equal(r1, r2)
    assert float((x1.float() - x2.float()).abs().max() / x1.float().abs().max()) <= 2.0 ** -7


# ---------------------------------------------------------------- pairs by expert

def group_reference(ids, E):
    flat = ids.reshape(-1).astype(np.int64)
    live = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(live, flat, E), kind="stable")[: int(live.sum())]
    row_of = np.full(flat.size, -1, np.int32)
    row_of[order] = np.arange(order.size)
    offsets = np.zeros(E + 1, np.int32)
    offsets[1:] = np.cumsum(np.bincount(flat[live], minlength=E))
    return offsets, row_of, (order // ids.shape[1]).astype(np.int32)


@pytest.mark.parametrize("kind", ["random", "padded", "one", "none", "skewed"])
@pytest.mark.parametrize("T,k,E", [(0, 4, 8), (1, 1, 1), (1, 10, 512), (7, 3, 5), (129, 8, 64), (512, 8, 64),
                                   (513, 8, 64), (333, 32, 33), (3000, 10, 512), (16384, 10, 512), (5000, 4, 2048),
                                   (70001, 10, 700)])
def test_group_pairs(pm, T, k, E, kind):
    rng = np.random.default_rng(T + k + E)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)  # an id may come twice in a token
    if kind == "padded":
        ids[rng.random((T, k)) < 0.3] = -1
        ids[rng.random((T, k)) < 0.1] = E
        ids[rng.random((T, k)) < 0.1] = 2 ** 31 - 1
        ids[rng.random((T, k)) < 0.1] = -2 ** 31
    elif kind == "one":
        ids[:] = E - 1
    elif kind == "none":
        ids[:] = -1
    elif kind == "skewed":
        ids = np.minimum((E * rng.random((T, k)) ** 6).astype(np.int32), E - 1)
    offsets, row_of, token_of = group_reference(ids, E)
    P = T * k
    d = torch.from_numpy(ids).cuda()
    o, r, t = (torch.full((n,), -7, dtype=torch.int32, device="cuda") for n in (E + 1, P + 3, P + 3))
    n = pm.group_workspace_bytes(T, k, E)
    assert n <= 148 * E * 4
    ws = torch.full((n + 16,), 0xAB, dtype=torch.uint8, device="cuda")
    pm.group_pairs(d, T, k, E, o, r, t, ws if n else None, n)
    torch.cuda.synchronize()
    assert np.array_equal(o.cpu().numpy(), offsets)
    assert np.array_equal(r.cpu().numpy()[:P], row_of)
    got = t.cpu().numpy()
    assert np.array_equal(got[: token_of.size], token_of)
    assert (got[token_of.size:] == -7).all() and (r.cpu().numpy()[P:] == -7).all()
    assert bool((ws[n:] == 0xAB).all())


# ---------------------------------------------------------------- combination

@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (1, 10, 4096), (33, 8, 2048), (5, 3, 1032), (700, 10, 264), (2, 32, 16)])
@pytest.mark.parametrize("bf16", [False, True])
def test_combine_rows(pm, T, k, H, bf16):
    g = gen(T * k + H)
    P = T * k
    rows = randn(g, P, H)
    rows = rows.bfloat16() if bf16 else rows
    w = randn(g, T, k)
    row_of = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    dead = torch.rand(P, generator=g, device="cuda") < 0.2
    row_of[dead] = torch.tensor([-1, P, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda").repeat(P)[:P][dead]
    w.view(-1)[dead] = float("nan")  # the weight of a pair without a row is not read
    y = torch.full((T, H), float("nan"), device="cuda")
    pm.combine_rows(rows, bf16, row_of, w, T, k, H, y)
    torch.cuda.synchronize()
    w64 = torch.where(dead.view(T, k), 0.0, w).double()
    v = rows.double()[torch.where(dead, 0, row_of).long()].view(T, k, H)
    ref = (v * w64[..., None]).sum(1)
    check_near(y, ref, k * U * (v.abs() * w64.abs()[..., None]).sum(1), U)


# ---------------------------------------------------------------- grouped products

COUNTS = {
    "ragged": [1, 0, 127, 128, 0, 129, 5, 0, 300, 64],
    "single": [0, 0, 1, 0],
    "one": [77],
    "large": [700, 3, 0, 513],
    "many": [n % 4 for n in range(600)],
}


def case(kind, counts, K, N, n=None, seed=0, extra=0):
    """Weights and rows: (W args, X args, sorted x in 64 bits, w in 64 bits). n: gather from n tokens."""
    g = gen(seed + K + N + len(counts))
    M, E = sum(counts), len(counts)
    index = None
    src = M + extra
    if n is not None:
        src = n
        index = torch.randint(0, n, (M + extra,), generator=g, device="cuda").to(torch.int32)
    x, w = randn(g, src, K), randn(g, E, N, K) * K ** -0.5
    if kind == "q8":
        x = x * torch.exp2(torch.randint(-6, 7, (src, 1), generator=g, device="cuda").float())
        xc, xs = quantize(x)
        wc, wscale = quantize(w * torch.exp(randn(g, E, N, 1)))
        x64, w64 = value_of(xc, xs), value_of(wc, wscale)
        W, X = (wc, wscale), (xc, xs)
    else:
        x, w = x.bfloat16(), w.bfloat16()
        x64, w64 = x.double(), w.double()
        W, X = (w, None), (x, None)
    x64 = x64[:M] if index is None else x64[index[:M].long()]
    return W, X, src, index, x64, w64


def run_matmul(pm, kind, W, X, n, index, offsets, rows, N, K, out_type, out, stream=None):
    t = pm.Q8 if kind == "q8" else pm.BF16
    pm.grouped_matmul(pm.make_dense(t, W[0], W[1], W[0].shape[0], N, K), pm.make_rows(t, X[0], X[1], n, index),
                      offsets, rows, out_type, out, stream)


SHAPES = {"bf16": [(64, 128), (8, 8), (72, 40), (1000, 264), (1024, 512), (2056, 136)],
          "q8": [(128, 128), (256, 8), (384, 264), (1024, 512), (2176, 136)]}


@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("kind,K,N", [(t, K, N) for t in SHAPES for K, N in SHAPES[t]])
def test_grouped_matmul(pm, kind, K, N, out, gather, counts):
    c = COUNTS[counts]
    if counts == "many" and K * N > 1 << 18:
        K, N = (256 if kind == "q8" else 136), 72
    M = sum(c)
    extra = 5
    W, X, n, index, x64, w64 = case(kind, c, K, N, 50 if gather else None, extra=extra)
    o = torch.full((M + extra, N), 7.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    run_matmul(pm, kind, W, X, n, index, offsets_of(c), M + extra, N, K, pm.F32 if out == "f32" else pm.BF16, o)
    torch.cuda.synchronize()
    p, d = products(x64, w64, c)
    check_near(o[:M], p, d, U if out == "f32" else 2.0 ** -8)
    assert bool((o[M:] == 7.0).all())  # rows behind the last expert


def run_swiglu(pm, kind, W, X, n, index, offsets, rows, I, K, out_type, h, hs, stream=None):
    t = pm.Q8 if kind == "q8" else pm.BF16
    pm.grouped_swiglu(pm.make_dense(t, W[0], W[1], W[0].shape[0], 2 * I, K), pm.make_rows(t, X[0], X[1], n, index),
                      offsets, rows, out_type, h, hs, stream)


SW_SHAPES = {"bf16": [(64, 64), (8, 32), (136, 96), (1000, 160), (1024, 256)],
             "q8": [(128, 32), (256, 64), (384, 160), (1024, 256)]}


@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", ["q8", "bf16"])
@pytest.mark.parametrize("kind,K,I", [(t, K, I) for t in SW_SHAPES for K, I in SW_SHAPES[t]])
def test_grouped_swiglu(pm, kind, K, I, out, gather, counts):
    c = COUNTS[counts]
    if counts == "many" and K * I > 1 << 16:
        K, I = (256 if kind == "q8" else 136), 32
    M = sum(c)
    extra = 3
    W, X, n, index, x64, w64 = case(kind, c, K, 2 * I, 50 if gather else None, seed=1, extra=extra)
    h = empty(M + extra, I, dtype=torch.uint8 if out == "q8" else torch.bfloat16).fill_(7)
    hs = empty(M + extra, I // 32).fill_(9) if out == "q8" else None
    run_swiglu(pm, kind, W, X, n, index, offsets_of(c), M + extra, I, K, pm.Q8 if out == "q8" else pm.BF16, h, hs)
    torch.cuda.synchronize()
    v, dv = swiglu(*products(x64, w64, c))
    if out == "q8":
        check_q8(h[:M], hs[:M], v, dv)
        assert bool((hs[M:] == 9).all())
    else:
        check_near(h[:M], v, dv, 2.0 ** -8)
    assert bool((h[M:] == 7).all())


def test_grouped_swiglu_bf16_widths_of_8(pm):
    c = [3, 130, 0, 20]
    for I in (8, 24, 200):
        W, X, n, index, x64, w64 = case("bf16", c, 72, 2 * I, 11, seed=2)
        h = empty(sum(c), I, dtype=torch.bfloat16)
        run_swiglu(pm, "bf16", W, X, n, index, offsets_of(c), sum(c), I, 72, pm.BF16, h, None)
        torch.cuda.synchronize()
        check_near(h, *swiglu(*products(x64, w64, c)), 2.0 ** -8)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_grouped_rows_outside_x_read_zeros(pm, kind):
    c, K, N = [4, 140], 256, 64
    W, X, n, index, x64, w64 = case(kind, c, K, N, 20, seed=3)
    bad = torch.zeros(sum(c), dtype=torch.bool, device="cuda")
    bad[[1, 3, 9, 100, 143]] = True
    index[bad] = torch.tensor([-1, 20, 2 ** 31 - 1, -2 ** 31, 21], dtype=torch.int32, device="cuda")
    x64[bad] = 0.0
    o = torch.full((sum(c), N), 7.0, device="cuda")
    run_matmul(pm, kind, W, X, n, index, offsets_of(c), sum(c), N, K, pm.F32, o)
    torch.cuda.synchronize()
    check_near(o, *products(x64, w64, c), U)
    assert bool((o[bad] == 0).all())


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_grouped_values_stay_with_their_rows_and_experts(pm, kind):
    """NaN in one row, in another expert and in unused rows of x shows nowhere else."""
    c, K, N = [130, 0, 70], 256, 72
    W, X, n, index, x64, w64 = case(kind, c, K, N, seed=4, extra=9)
    if kind == "q8":
        X[1][60], X[1][205:], W[1][1] = 255, 255, 255
    else:
        X[0][60], X[0][205:], W[0][1] = float("nan"), float("nan"), float("nan")
    o = torch.full((209, N), 7.0, device="cuda")
    run_matmul(pm, kind, W, X, n, index, offsets_of(c), 209, N, K, pm.F32, o)
    torch.cuda.synchronize()
    assert bool(o[60].isnan().all())
    live = torch.arange(200, device="cuda") != 60
    p, d = products(x64, w64, c)
    check_near(o[:200][live], p[live], d[live], U)
    assert bool((o[200:] == 7.0).all())


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_grouped_offsets_that_make_no_sense_stay_in_bounds(pm, kind):
    """Offsets that fall, start below zero or end behind the rows: nothing outside out is touched, and an
    expert whose own range is sound has its rows."""
    c, K, N, M = [50, 30, 20], 128, 64, 100
    W, X, n, index, x64, w64 = case(kind, c, K, N, seed=5)
    for off in ([-5, 40, 30, 900], [0, 2 ** 31 - 1, -2 ** 31, 0], [100, 100, 50, 2 ** 31 - 1]):
        o = torch.full((M + 40, N), 7.0, device="cuda")
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        run_matmul(pm, kind, W, X, n, index, offsets, M, N, K, pm.F32, o)
        torch.cuda.synchronize()
        assert bool((o[M:] == 7.0).all())
        for e in range(3):
            a, b = max(off[e], 0), min(off[e + 1], M)
            others = [i for f in range(3) if f != e for i in range(max(off[f], 0), min(off[f + 1], M))]
            mine = [i for i in range(a, b) if i not in set(others)]
            if mine:
                p, d = products(x64[mine], w64[e:e + 1], [len(mine)])
                check_near(o[mine], p, d, U)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_grouped_products_on_two_streams_and_in_a_graph(pm, kind):
    """Two calls at once, and a captured call replayed on new inputs, give what single calls give."""
    c, K, I = [40, 0, 200, 7], 256, 64
    W, X, n, index, x64, w64 = case(kind, c, K, 2 * I, 30, seed=6)
    M, off = sum(c), offsets_of(c)
    outs = [(empty(M, I), empty(M, I // 32)) for _ in range(4)]
    run_swiglu(pm, kind, W, X, n, index, off, M, I, K, pm.Q8, *outs[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in (0, 1):
        run_swiglu(pm, kind, W, X, n, index, off, M, I, K, pm.Q8, *outs[1 + i], stream=streams[i])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_swiglu(pm, kind, W, X, n, index, off, M, I, K, pm.Q8, *outs[3], stream=torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    for h, s in outs[1:]:
        assert torch.equal(h, outs[0][0]) and torch.equal(s, outs[0][1])
    off.copy_(offsets_of([7, 200, 0, 40]))
    graph.replay()
    run_swiglu(pm, kind, W, X, n, index, off, M, I, K, pm.Q8, *outs[0])
    torch.cuda.synchronize()
    assert torch.equal(outs[3][0], outs[0][0]) and torch.equal(outs[3][1], outs[0][1])


def test_pointers_that_are_not_device_memory_are_refused(pm):
    """Host tensors are refused before a launch; so are views with gaps."""
    r, codes, scales = torch.randn(2, 128), torch.empty(2, 128, dtype=torch.uint8), torch.empty(2, 4, dtype=torch.uint8)
    with pytest.raises(pm.PmoeError) as ei:
        pm.residual_norm_q8(r, None, None, 0.0, 2, 128, codes, scales)
    assert ei.value.code == 1
    with pytest.raises(pm.PmoeError) as ei:
        pm.residual_norm_q8(r.cuda(), None, None, 0.0, 2, 128, codes.cuda(), scales)
    assert ei.value.code == 1
    with pytest.raises(ValueError):
        pm.residual_norm_q8(randn(gen(1), 2, 256)[:, :128], None, None, 0.0, 2, 128, codes.cuda(), scales.cuda())


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("what", ["f32", "bf16", "swiglu q8", "swiglu bf16"])
@pytest.mark.parametrize("K,N", [(256, 1088), (1152, 576)])
def test_grouped_products_with_many_tiles_per_sm(pm, kind, what, K, N):
    """Enough row tiles for the wide weight tiles, several for every SM, with ragged last columns: both
    accumulators in turn, the columns that they share, stages that wrap."""
    rng = np.random.default_rng(K + N)
    c = [int(n) for n in rng.integers(0, 200, 150)]
    c[3], c[77] = 1300, 0
    M = sum(c)
    W, X, n, index, x64, w64 = case(kind, c, K, N, 999, seed=8)
    p, d = products(x64, w64, c)
    off = offsets_of(c)
    if what in ("f32", "bf16"):
        o = empty(M, N, dtype=torch.float32 if what == "f32" else torch.bfloat16)
        run_matmul(pm, kind, W, X, n, index, off, M, N, K, pm.F32 if what == "f32" else pm.BF16, o)
        torch.cuda.synchronize()
        check_near(o, p, d, U if what == "f32" else 2.0 ** -8)
        return
    I = N // 2
    v, dv = swiglu(p, d)
    h = empty(M, I, dtype=torch.uint8 if what == "swiglu q8" else torch.bfloat16)
    hs = empty(M, I // 32) if what == "swiglu q8" else None
    run_swiglu(pm, kind, W, X, n, index, off, M, I, K, pm.Q8 if hs is not None else pm.BF16, h, hs)
    torch.cuda.synchronize()
    if hs is not None:
        check_q8(h, hs, v, dv)
    else:
        check_near(h, v, dv, 2.0 ** -8)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_grouped_wait_that_runs_out_is_reported_and_the_next_call_is_exact(pm, kind):
    """With the wait limit at 1 ns the roles give up, after what they issued has landed; the record names
    it, and the next call with the default limit is the same as before, bit for bit."""
    c, K, N = [300, 0, 200, 700], 4096, 512
    W, X, n, index, x64, w64 = case(kind, c, K, N, 64, seed=9)
    M, off = sum(c), offsets_of(c)
    outs = [torch.full((M, N), float("nan"), device="cuda") for _ in range(3)]
    assert pm.grouped_error() == (0, 0)
    run_matmul(pm, kind, W, X, n, index, off, M, N, K, pm.F32, outs[0])
    assert pm.grouped_error() == (0, 0)
    pm.set_wait_limit_ns(1)
    try:
        run_matmul(pm, kind, W, X, n, index, off, M, N, K, pm.F32, outs[1])
        torch.cuda.synchronize()
    finally:
        pm.set_wait_limit_ns(0)
    assert pm.grouped_error()[0] == 3
    assert pm.grouped_error() == (0, 0)  # read once
    run_matmul(pm, kind, W, X, n, index, off, M, N, K, pm.F32, outs[2])
    assert pm.grouped_error() == (0, 0)
    assert torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("rows", [5, 100])
def test_grouped_q8_scales_at_both_ends(pm, rows):
    """Scales far from one that cancel in the products, the smallest scale among them."""
    K, N = 256, 136
    g = gen(10)
    xc, xs = quantize(randn(g, rows, K))
    wc, ws = quantize(randn(g, 1, N, K))
    down = torch.randint(0, 20, xs.shape, generator=g, device="cuda").to(torch.uint8)
    xs = down                                    # 2^-127 .. 2^-108
    ws = (254 - 20 + torch.randint(0, 20, ws.shape, generator=g, device="cuda")).to(torch.uint8) - 7  # 2^100 .. 2^119
    x64, w64 = value_of(xc, xs), value_of(wc, ws)
    o = empty(rows, N, dtype=torch.float32)
    run_matmul(pm, "q8", (wc, ws), (xc, xs), rows, None, offsets_of([rows]), rows, N, K, pm.F32, o)
    torch.cuda.synchronize()
    check_near(o, *products(x64, w64, [rows]), U)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_grouped_matmul_one_crowded_expert_among_many(pm, kind):
    """Tiles for few rows, most of them of one expert; as many experts as the products take."""
    for c in ([0] * 100 + [1000] + [1] * 200, [i % 3 for i in range(2048)]):
        K, N = 256, 72
        M = sum(c)
        W, X, n, index, x64, w64 = case(kind, c, K, N, 77, seed=11)
        o = empty(M, N, dtype=torch.float32)
        run_matmul(pm, kind, W, X, n, index, offsets_of(c), M, N, K, pm.F32, o)
        torch.cuda.synchronize()
        check_near(o, *products(x64, w64, c), U)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_grouped_matmul_past_2_31_elements(pm, kind):
    """Rows of out, and rows of x, behind 2^31 elements."""
    K, N, M = 4096, 4096, 540_000
    g = gen(12)
    free = torch.cuda.mem_get_info()[0]
    if free < 24 << 30:
        pytest.skip("needs 24 GB")
    w = randn(g, 1, N, K) * K ** -0.5
    if kind == "bf16":
        x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        W, X = (w.bfloat16(), None), (x, None)
        w64 = W[0].double()
    else:
        x = torch.randint(0, 0x70, (M, K), dtype=torch.uint8, generator=g, device="cuda")
        xs = torch.full((M, K // 32), 120, dtype=torch.uint8, device="cuda")
        W, X = quantize(w), (x, xs)
        w64 = value_of(*W)
    o = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    run_matmul(pm, kind, W, X, M, None, offsets_of([M]), M, N, K, pm.BF16, o)
    torch.cuda.synchronize()
    at = torch.tensor([0, 1, 129, 262_143, 262_144, 300_001, 524_287, 524_288, 539_000, M - 1], device="cuda")
    x64 = x[at].double() if kind == "bf16" else value_of(x[at], X[1][at])
    p, d = products(x64, w64, [len(at)])
    check_near(o[at], p, d, 2.0 ** -8)


def test_grouped_matmul_experts_past_2_31_elements(pm):
    K, N, E = 1024, 4096, 600
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    g = gen(13)
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    c = [0] * E
    c[0], c[511], c[512], c[599] = 2, 3, 4, 5
    x = randn(g, 14, K).bfloat16()
    o = empty(14, N, dtype=torch.float32)
    run_matmul(pm, "bf16", (w, None), (x, None), 14, None, offsets_of(c), 14, N, K, pm.F32, o)
    torch.cuda.synchronize()
    live = [0, 511, 512, 599]
    p, d = products(x.double(), w[live].double(), [c[e] for e in live])
    check_near(o, p, d, U)


def test_rows_past_2_31_elements(pm):
    """Norm and combination on rows behind 2^31 elements."""
    T, H = 600_000, 4096
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    r = torch.empty(T, H, device="cuda").normal_(generator=gen(14))
    codes, scales = empty(T, H), empty(T, H // 32)
    pm.residual_norm_q8(r, None, None, 0.0, T, H, codes, scales)
    torch.cuda.synchronize()
    at = torch.tensor([0, 524_287, 524_288, T - 1], device="cuda")
    _, v, dv = norm_reference(r[at], None, None, 0.0)
    check_q8(codes[at], scales[at], v, dv)
    w = torch.full((T, 1), 0.5, device="cuda")
    row_of = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    y = torch.empty(T, H, device="cuda")
    pm.combine_rows(r, False, row_of, w, T, 1, H, y)
    torch.cuda.synchronize()
    assert torch.equal(y[at], 0.5 * r[T - 1 - at])


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_grouped_rows_of_an_empty_x_are_zeros(pm, kind):
    """No input rows at all: every index names a row outside."""
    K, N = 256, 64
    W, X, *_ = case(kind, [5, 40], K, N, 3, seed=15)
    index = torch.tensor([0, 1, -1, 7, 2 ** 31 - 1] * 9, dtype=torch.int32, device="cuda")
    o = torch.full((45, N), 7.0, device="cuda")
    run_matmul(pm, kind, W, (None, None), 0, index, offsets_of([5, 40]), 45, N, K, pm.F32, o)
    torch.cuda.synchronize()
    assert not o.any()


def test_calls_from_several_host_threads(pm):
    """Different sizes at once from threads with streams of their own: the results of each call alone."""
    import threading
    jobs = []
    for i, E in enumerate((8, 700, 2048, 33)):
        ids = torch.randint(-1, E + 1, (900, 7), dtype=torch.int32, generator=gen(20 + i), device="cuda")
        W, X, n, index, _, _ = case("q8", [30 + i, 0, 200 * i, 5], 256, 128, 60, seed=20 + i)
        jobs.append((E, ids, W, X, n, index, [30 + i, 0, 200 * i, 5]))

    def run(job, st):
        E, ids, W, X, n, index, c = job
        P, M = ids.numel(), sum(c)
        o, r, t = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (E + 1, P, P))
        ws = empty(pm.group_workspace_bytes(900, 7, E) + 16)
        off = offsets_of(c)
        h = torch.zeros(M, 128, device="cuda")
        torch.cuda.synchronize()
        for _ in range(20):
            pm.group_pairs(ids, 900, 7, E, o, r, t, ws, ws.numel(), st)
            run_matmul(pm, "q8", W, X, n, index, off, M, 128, 256, pm.F32, h, stream=st)
        st.synchronize()
        return o, r, t, h

    want = [run(j, torch.cuda.current_stream()) for j in jobs]
    got = [None] * len(jobs)

    def work(i):
        got[i] = run(jobs[i], torch.cuda.Stream())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
