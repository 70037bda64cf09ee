"""Arguments of the prompt-side operators that are refused on the host, before anything is enqueued."""
import pytest


@pytest.fixture(scope="module")
def pm():
    import bitplane_mixed_precision_b200 as pm
    return pm


A = 1 << 20  # an address with every alignment that a call asks for; refused calls never follow it


def refused(pm, code, f, *a):
    with pytest.raises(pm.PmoeError) as ei:
        f(*a)
    assert ei.value.code == code


def test_quantize_q8_refusals(pm):
    good = [A, False, 4, 64, A, A]
    for at, v in ((0, None), (4, None), (5, None), (2, -1), (3, 0), (3, 48), (0, A + 8), (4, A + 2), (2, 1 << 60)):
        a = list(good)
        a[at] = v
        refused(pm, 1, pm.quantize_q8, *a)
    pm.quantize_q8(A, False, 0, 64, A, A)  # no rows: nothing to do


def test_residual_norm_q8_refusals(pm):
    good = [A, A, A, 1e-6, 4, 256, A, A, A]
    for at, v in ((0, None), (3, -1.0), (3, float("nan")), (4, -1), (5, 0), (5, 64), (5, 132), (6, None), (7, None),
                  (0, A + 4), (1, A + 4), (2, A + 8), (6, A + 4), (7, A + 2), (8, A + 8)):
        a = list(good)
        a[at] = v
        refused(pm, 1, pm.residual_norm_q8, *a)
    refused(pm, 1, pm.residual_norm_q8, A, A, A, 0.0, 4, 256, None, None, None)
    refused(pm, 7, pm.residual_norm_q8, A, A, A, 0.0, 4, 32768 + 128, A, A, A)
    pm.residual_norm_q8(A, None, None, 0.0, 0, 256, A, A)


def test_group_pairs_refusals(pm):
    good = [A, 4, 3, 8, A, A, A, None, 0]
    for at, v in ((0, None), (1, -1), (2, 0), (2, 33), (3, 0), (4, None), (5, None), (6, None), (1, 1 << 30),
                  (0, A + 2), (4, A + 1)):
        a = list(good)
        a[at] = v
        refused(pm, 1, pm.group_pairs, *a)
    refused(pm, 7, pm.group_pairs, A, 4, 3, 2049, A, A, A)
    n = pm.group_workspace_bytes(4096, 10, 512)
    assert 0 < n <= 148 * 512 * 4
    assert pm.group_workspace_bytes(1, 10, 512) == 0
    refused(pm, 5, pm.group_pairs, A, 4096, 10, 512, A, A, A, A, n - 1)
    refused(pm, 5, pm.group_pairs, A, 4096, 10, 512, A, A, A, None, n)


def test_combine_rows_refusals(pm):
    good = [A, True, A, A, 4, 3, 64, A]
    for at, v in ((0, None), (2, None), (3, None), (4, -1), (5, 0), (5, 33), (6, 0), (6, 12), (7, None), (0, A + 8),
                  (7, A + 8)):
        a = list(good)
        a[at] = v
        refused(pm, 1, pm.combine_rows, *a)
    pm.combine_rows(None, True, None, None, 0, 3, 64, None)


def dense(pm, type=1, w=A, scales=A, E=4, N=64, K=256):
    return pm.make_dense(type, w, scales, E, N, K)


def rows(pm, type=1, x=A, scales=A, n=10, index=None):
    return pm.make_rows(type, x, scales, n, index)


@pytest.mark.parametrize("W,X,call", [
    (dict(w=None), {}, {}), (dict(scales=None), {}, {}), (dict(E=0), {}, {}), (dict(N=0), {}, {}),
    (dict(N=60), {}, {}), (dict(K=0), {}, {}), (dict(K=192), {}, {}), (dict(type=2), dict(type=2), {}),
    (dict(w=A + 8), {}, {}), (dict(scales=A + 8), {}, {}),
    (dict(type=0, scales=None), {}, {}),                       # types differ
    (dict(type=0, K=260, scales=None), dict(type=0, scales=None), {}),
    (dict(type=0), dict(type=0, scales=None), {}),             # bf16 with scales
    ({}, dict(x=None), {}), ({}, dict(scales=None), {}), ({}, dict(n=-1), {}), ({}, dict(n=9), {}),
    ({}, dict(x=A + 8), {}), ({}, dict(scales=A + 8), {}), ({}, dict(index=A + 2), {}),
    ({}, {}, dict(offsets=None)), ({}, {}, dict(out=None)), ({}, {}, dict(out=A + 8)), ({}, {}, dict(rows=-1)),
    ({}, {}, dict(out_type=1)), ({}, {}, dict(out_type=3)),
])
def test_grouped_matmul_refusals(pm, W, X, call):
    c = dict(offsets=A, rows=10, out_type=2, out=A)
    c.update(call)
    refused(pm, 1, pm.grouped_matmul, dense(pm, **W), rows(pm, **X), c["offsets"], c["rows"], c["out_type"], c["out"])


@pytest.mark.parametrize("W,call", [
    (dict(N=72), {}), (dict(N=96), dict(out_type=1)), ({}, dict(out_type=2)), ({}, dict(out_type=1, hs=None)),
    ({}, dict(out_type=0)), ({}, dict(h=None)),
])
def test_grouped_swiglu_refusals(pm, W, call):
    c = dict(out_type=1, h=A, hs=A)
    c.update(call)
    refused(pm, 1, pm.grouped_swiglu, dense(pm, **W), rows(pm), A, 10, c["out_type"], c["h"], c["hs"])


def test_grouped_products_take_at_most_2048_experts(pm):
    refused(pm, 7, pm.grouped_matmul, dense(pm, E=2049), rows(pm), A, 10, 2, A)
    pm.grouped_matmul(dense(pm), rows(pm), A, 0, 2, A)  # no rows: nothing to do


def test_views_with_gaps_are_refused(pm):
    torch = pytest.importorskip("torch")
    gaps = torch.zeros(4, 512)[:, :256]
    with pytest.raises(ValueError):
        pm.residual_norm_q8(gaps, None, None, 0.0, 4, 256, A, A)
    with pytest.raises(ValueError):
        pm.combine_rows(gaps, False, A, A, 2, 2, 256, A)
    with pytest.raises(ValueError):
        pm.make_dense(pm.BF16, gaps, None, 1, 4, 256)
