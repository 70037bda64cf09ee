"""The prompt-side operators run together, as a layer uses them: every step against the 64-bit form of what
the step before it left, captured and replayed, on two streams at once, and against the plane store's own
layer on the same experts."""
import numpy as np
import pytest
import torch

from bitplane_mixed_precision_b200.prompt import DenseExperts, PromptLayer
from bitplane_mixed_precision_b200.store import ResidentLayer
from gpu_common import device_fill, tokens
from prompt_common import U, check_near, check_q8, products, swiglu, value_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    import bitplane_mixed_precision_b200 as pm
    return pm


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def experts(pm, kind, E, H, I, seed):
    g = gen(seed)

    def fill(e, m, w):
        w.copy_(torch.randn(w.numel(), generator=g, device="cuda") * 0.05)

    return DenseExperts(E, H, I, fill, pm.Q8 if kind == "q8" else pm.BF16)


def values(codes, scales):
    return codes.double() if scales is None else value_of(codes, scales)


def inputs(E, H, T, seed):
    g = gen(seed)
    return (torch.randn(T, H, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda"),
            torch.randn(T, E, generator=g, device="cuda"), 1 + 0.2 * torch.randn(H, generator=g, device="cuda"))


@pytest.mark.parametrize("kind", ["q8", "bf16"])
@pytest.mark.parametrize("T", [1, 37, 700])
def test_every_step_of_a_prompt(pm, kind, T):
    E, H, I, k = 12, 384, 256, 3
    X = experts(pm, kind, E, H, I, 1)
    L = PromptLayer(X, k, 800)
    r, y, logits, gain = inputs(E, H, T, 2)
    r0 = r.clone()
    L.norm(r, y, T, gain, 1e-6)
    L.route(logits, T)
    ids = L.ids[:T]
    if T > 1:
        ids[T // 3] = -1  # a padded token
        ids[T // 2, 1] = E
    out = L.forward(T)
    torch.cuda.synchronize()
    assert pm.grouped_error() == (0, 0)
    # norm
    v = (r0 + y).double()
    assert torch.equal(r, r0 + y)
    v = v / (v.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * gain.double()
    if kind == "q8":
        check_q8(L.x[:T], L.x_scales[:T], v, 30 * U * v.abs())
    else:
        check_near(L.x[:T], v, 30 * U * v.abs(), 2.0 ** -8)
    # pairs by expert
    flat = ids.reshape(-1).cpu().numpy().astype(np.int64)
    live = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(live, flat, E), kind="stable")[: int(live.sum())]
    M = order.size
    counts = [int(n) for n in np.bincount(flat[live], minlength=E)]
    assert L.offsets.cpu().tolist() == [0] + list(np.cumsum(counts))
    assert np.array_equal(L.token_of[:M].cpu().numpy(), order // k)
    # gate, up and SwiGLU on the rows of x that the norm left
    x64 = values(L.x[:T], None if kind == "bf16" else L.x_scales[:T])[torch.from_numpy(order // k).cuda()]
    h, dh = swiglu(*products(x64, values(X.up, X.up_scales), counts))
    if kind == "q8":
        check_q8(L.h[:M], L.h_scales[:M], h, dh)
    else:
        check_near(L.h[:M], h, dh, 2.0 ** -8)
    # down on the rows that SwiGLU left
    h64 = values(L.h[:M], None if kind == "bf16" else L.h_scales[:M])
    check_near(L.out[:M], *products(h64, values(X.down, X.down_scales), counts), 2.0 ** -8)
    # combination of the rows that the down products left
    row_of = np.full(flat.size, -1)
    row_of[order] = np.arange(M)
    at = torch.from_numpy(row_of).cuda().view(T, k)
    w = torch.where(at < 0, 0.0, L.w[:T]).double()
    rows = L.out.double()[at.clamp(min=0)]
    check_near(out, (rows * w[..., None]).sum(1), k * U * (rows.abs() * w.abs()[..., None]).sum(1), U)


@pytest.mark.parametrize("kind", ["q8", "bf16"])
def test_a_captured_prompt_replays_on_new_inputs(pm, kind):
    E, H, I, k, T = 9, 256, 128, 2, 300
    X = experts(pm, kind, E, H, I, 3)
    L, L2 = PromptLayer(X, k, T), PromptLayer(X, k, T)
    r, y, logits, gain = inputs(E, H, T, 4)

    def run(layer, st=None):
        layer.norm(r, y, T, gain, 1e-6, st)
        layer.route(logits, T, st)
        return layer.forward(T, st)

    run(L)  # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(L, torch.cuda.current_stream())
    for seed in (5, 6):
        fresh = inputs(E, H, T, seed)
        for a, b in zip((r, y, logits, gain), fresh):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        r.copy_(fresh[0])
        want = run(L2)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_two_prompts_at_once(pm):
    """Two layers' buffers over the same experts, on two streams, give what each gives alone."""
    E, H, I, k, T = 16, 512, 256, 4, 500
    X = experts(pm, "q8", E, H, I, 7)
    runs = []
    for seed in (8, 9):
        r, y, logits, gain = inputs(E, H, T, seed)
        L = PromptLayer(X, k, T)
        L.norm(r.clone(), y, T, gain)
        L.route(logits, T)
        alone = L.forward(T).clone()
        runs.append((PromptLayer(X, k, T), r, y, logits, gain, alone, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for L, r, y, logits, gain, alone, st in runs:
            with torch.cuda.stream(st):
                r2 = r.clone()
                L.norm(r2, y, T, gain, 0.0, st)
                L.route(logits, T, st)
                L.forward(T, st)
    torch.cuda.synchronize()
    for L, *_, alone, st in runs:
        assert torch.equal(L.y, alone)


def test_dense_experts_of_a_stored_layer(pm):
    """bf16 experts decoded from the plane store at 8 bits against the store's own layer on the same tokens.
    The roundings that differ (weights, h and the rows in bf16, at most 2^-8 each and of both signs) come to
    about 2^-8 of the output's norm; 2^-6 is four times that. q8 rounds weights and h to e4m3 (at most 2^-4,
    about 2.5 % in the mean): three of them in a row, of both signs, stay below 2^-3."""
    seed, E, H, I, G, k, T = 21, 16, 1024, 256, 128, 4, 24
    R = ResidentLayer(E, H, I, G, device_fill(seed))
    logits, xb = tokens(seed, T, E, H)
    logits = torch.from_numpy(logits).cuda()
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    pm.route(logits, T, E, k, ids, w)
    depth = torch.full((T, k), 8, dtype=torch.uint8, device="cuda")
    ws_bytes = pm.layer_workspace_bytes(T, k, E, H, I)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    ref = torch.empty(T, H, device="cuda")
    x = torch.from_numpy(xb.view(np.int16)).cuda()
    pm.moe_layer_fwd(R.layer, x, ids, w, depth, T, k, ref, ws, ws_bytes)
    for kind, most in ((pm.BF16, 2.0 ** -6), (pm.Q8, 2.0 ** -3)):
        L = PromptLayer(DenseExperts.from_layer(R, kind), k, T)
        if kind == pm.Q8:
            pm.quantize_q8(x, True, T, H, L.x, L.x_scales)
        else:
            L.x.copy_(x.view(torch.bfloat16))
        L.ids.copy_(ids)
        L.w.copy_(w)
        y = L.forward(T)
        torch.cuda.synchronize()
        err = float((y - ref).norm() / ref.norm())
        assert err <= most, err


def test_a_prompt_longer_than_its_buffers_is_refused(pm):
    L = PromptLayer(experts(pm, "bf16", 4, 64, 64, 11), 2, 10)
    with pytest.raises(ValueError):
        L.forward(11)
    assert L.forward(0).shape == (0, 64)
