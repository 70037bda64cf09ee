"""The prompt-side operators in the order in which a program enqueues them: on torch's current stream, behind what
writes their inputs, and one call after another on the same buffers."""
import pytest
import torch

from bitplane_mixed_precision_b200.prompt import DenseExperts, PromptLayer
from prompt_common import quantize

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    import bitplane_mixed_precision_b200 as pm
    return pm


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def experts(kind, E, H, I, seed):
    g = gen(seed)

    def fill(e, m, w):
        w.copy_(torch.randn(w.numel(), generator=g, device="cuda") * 0.05)

    return DenseExperts(E, H, I, fill, kind)


def inputs(E, H, T, seed):
    g = gen(seed)
    return (torch.randn(T, H, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda"),
            torch.randn(T, E, generator=g, device="cuda"))


@pytest.mark.parametrize("kind", [0, 1])
def test_a_layer_follows_the_current_stream(pm, kind):
    """Without a stream, behind a long pause and the copies that bring the inputs: on a side stream, and captured."""
    E, H, I, k, T = 9, 256, 128, 2, 200
    X = experts(kind, E, H, I, 1)
    first, second = inputs(E, H, T, 2), inputs(E, H, T, 3)
    r, y, logits = (torch.zeros_like(a) for a in first)
    L = PromptLayer(X, k, T)

    def run():
        L.norm(r, y, T)
        L.route(logits, T)
        return L.forward(T)

    def load(values):
        for to, a in zip((r, y, logits), values):
            to.copy_(a)

    want = []
    for values in (first, second):
        load(values)
        want.append(run().clone())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
        load(first)
        got = run().clone()
    side.synchronize()
    assert torch.equal(got, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for values, w in zip((second, first), (want[1], want[0])):
        load(values)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


# ---------------------------------------------------------------- records of a wait that ran out

@pytest.fixture
def short_waits(pm):
    """A wait limit of 1 ns while the context is open: the accumulators of a 8192-deep product take longer."""
    class Limit:
        def __enter__(self):
            pm.set_wait_limit_ns(1)

        def __exit__(self, *_):
            torch.cuda.synchronize()
            pm.set_wait_limit_ns(0)

    yield Limit()
    pm.set_wait_limit_ns(0)


class Product:
    """One expert's product, 700 x 8192 x 512."""
    def __init__(self, pm, seed):
        g = gen(seed)
        M, K, N = 700, 8192, 512
        self.x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
        self.w = torch.randn(1, N, K, generator=g, device="cuda").bfloat16()
        self.offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        self.out = torch.empty(M, N, device="cuda")
        self.error = torch.zeros(2, dtype=torch.int32, device="cuda")
        self.dense, self.M = pm.make_dense(pm.BF16, self.w, None, 1, N, K), M

    def __call__(self, pm, own, stream=None):
        rows = pm.make_rows(pm.BF16, self.x, None, self.M, None, self.error if own else None)
        pm.grouped_matmul(self.dense, rows, self.offsets, self.M, pm.F32, self.out, stream)


def test_calls_with_a_record_of_their_own(pm, short_waits):
    """A call's failure shows in its own record alone, and another caller's check does not clear it."""
    a, b = Product(pm, 1), Product(pm, 2)
    a(pm, True)
    b(pm, True)
    torch.cuda.synchronize()
    want = a.out.clone()
    assert pm.grouped_error() == (0, 0) and a.error.tolist() == [0, 0]
    side = torch.cuda.Stream()
    with short_waits:
        a(pm, True, side)
    b(pm, True)
    assert pm.grouped_error() == (0, 0)
    assert a.error.tolist()[0] == 3 and b.error.tolist() == [0, 0]
    first = a.error.tolist()
    with short_waits:
        a(pm, True)
    assert a.error.tolist() == first  # the first one stays until it is cleared
    a.error.zero_()
    a(pm, True)
    torch.cuda.synchronize()
    assert a.error.tolist() == [0, 0] and torch.equal(a.out, want)


def test_the_device_s_record_is_taken_once_from_any_stream(pm, short_waits):
    a = Product(pm, 3)
    a(pm, False)
    assert pm.grouped_error() == (0, 0)
    side = torch.cuda.Stream()
    with short_waits:
        a(pm, False)
    code, detail = pm.grouped_error(side)
    assert code == 3 and detail > 0
    assert pm.grouped_error() == (0, 0) and a.error.tolist() == [0, 0]


def test_a_record_that_is_not_device_memory_is_refused(pm):
    a = Product(pm, 4)
    a.error = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(pm.PmoeError) as ei:
        a(pm, True)
    assert ei.value.code == 1


@pytest.mark.parametrize("kind", [0, 1])
def test_a_layer_reports_a_wait_that_ran_out(pm, short_waits, kind):
    E, H, I, k, T = 4, 8192, 512, 2, 600
    X = experts(kind, E, H, I, 5)
    L, other = PromptLayer(X, k, T), PromptLayer(X, k, T)
    r, y, logits = inputs(E, H, T, 6)
    L.norm(r, y, T)
    L.route(logits, T)
    want = L.forward(T).clone()
    assert L.error() == (0, 0)
    with short_waits:
        L.forward(T)
    assert other.error() == (0, 0) and pm.grouped_error() == (0, 0)
    assert L.error()[0] == 3
    assert L.error() == (0, 0)
    assert torch.equal(L.forward(T), want) and L.error() == (0, 0)


def test_a_product_that_gives_up_ends_once_its_own_copies_have_landed(pm, short_waits):
    """No fixed pause is put in their place: a call that gives up in its first tile takes less than a complete one and
    2 ms beside."""
    a = Product(pm, 7)

    def timed():
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        start.record(torch.cuda.default_stream())
        a(pm, True)
        end.record(torch.cuda.default_stream())
        torch.cuda.synchronize()
        return start.elapsed_time(end)

    timed()
    full = min(timed() for _ in range(3))
    with short_waits:
        short = min(timed() for _ in range(3))
    assert a.error.tolist()[0] == 3
    assert short <= full + 2.0, (short, full)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("rows", [5, 20, 700])
def test_products_that_give_up_at_different_places(pm, kind, gather, rows):
    """Limits from 1 ns to some 50 us stop the roles at different stages; calls follow one another at once on the same
    SMs, and the first call with the default limit is exact again."""
    g = gen(8)
    E, K, N = 3, 4096, 1024
    M, n = E * rows, 100 if gather else E * rows
    t = pm.Q8 if kind == "q8" else pm.BF16
    x, w = torch.randn(n, K, generator=g, device="cuda"), torch.randn(E, N, K, generator=g, device="cuda")
    xs = ws = None
    if kind == "q8":
        (x, xs), (w, ws) = quantize(x), quantize(w)
    else:
        x, w = x.bfloat16(), w.bfloat16()
    index = torch.randint(0, n, (M,), generator=g, device="cuda").to(torch.int32) if gather else None
    offsets = torch.tensor([0, rows, 2 * rows, M], dtype=torch.int32, device="cuda")
    error = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = torch.empty(M, N, device="cuda")
    dense, x_rows = pm.make_dense(t, w, ws, E, N, K), pm.make_rows(t, x, xs, n, index, error)

    def call():
        pm.grouped_matmul(dense, x_rows, offsets, M, pm.F32, out)

    call()
    torch.cuda.synchronize()
    want = out.clone()
    assert error.tolist() == [0, 0]
    try:
        for ns in (1, 600, 2000, 5000, 10000, 20000, 50000):
            pm.set_wait_limit_ns(ns)
            for _ in range(20):
                call()
    finally:
        torch.cuda.synchronize()
        pm.set_wait_limit_ns(0)
    error.zero_()
    out.zero_()
    call()
    torch.cuda.synchronize()
    assert error.tolist() == [0, 0] and torch.equal(out, want)


# ---------------------------------------------------------------- one launch behind another

def test_pairs_again_in_one_workspace(pm):
    """Calls at once behind one another, with other ids and outputs but the same workspace, captured too: a call's
    histograms are not written before the sort in front has read its own."""
    T, k, E, n = 2000, 5, 300, 12
    P = T * k
    sets = [torch.randint(-1, E, (T, k), dtype=torch.int32, generator=gen(30 + i), device="cuda") for i in range(n)]
    size = pm.group_workspace_bytes(T, k, E)
    assert size > 0  # several blocks
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def outputs():
        return [[torch.full((m,), -7, dtype=torch.int32, device="cuda") for m in (E + 1, P, P)] for _ in range(n)]

    def run(outs, pause):
        for ids, o in zip(sets, outs):
            pm.group_pairs(ids, T, k, E, *o, ws, size, torch.cuda.current_stream())
            if pause:
                torch.cuda.synchronize()

    want, got, replayed = outputs(), outputs(), outputs()
    run(want, True)
    for ids, (offsets, row_of, _) in zip(sets, want):
        flat = torch.where(ids.reshape(-1) < 0, E, ids.reshape(-1)).long()
        assert torch.equal(offsets[1:], torch.bincount(flat, minlength=E + 1)[:E].cumsum(0).int())
        order = torch.argsort(flat, stable=True)[: int(offsets[-1])]
        assert torch.equal(row_of[order], torch.arange(order.numel(), dtype=torch.int32, device="cuda"))
    for _ in range(3):
        run(got, False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(replayed, False)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for w, a, b in zip(want, got, replayed):
        assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(w, a, b))


@pytest.mark.parametrize("T", [3, 600])
@pytest.mark.parametrize("kind", [0, 1])
def test_a_layer_again_and_again_in_the_same_buffers(pm, kind, T):
    """Nothing but the layer's own launches, each of which may start while the one in front still writes what it reads;
    two sets of ids take turns, so that every buffer holds another call's values first."""
    E, H, I, k, n = 40, 512, 256, 4, 16
    X = experts(kind, E, H, I, 9)
    L, P = PromptLayer(X, k, T), T * k
    ids = [torch.randint(-1, E, (T, k), dtype=torch.int32, generator=gen(40 + i), device="cuda") for i in range(2)]
    r0 = torch.randn(T, H, generator=gen(42), device="cuda")
    L.w.copy_(torch.rand(T, k, generator=gen(43), device="cuda"))
    sums = [torch.empty(T, H, device="cuda") for _ in range(n)]

    def run(pause):
        r, y = r0.clone(), None
        steps = []
        for i in range(n):
            steps += [lambda y=y: L.norm(r, y, T), lambda i=i: pm.group_pairs(
                          ids[i % 2], T, k, E, L.offsets, L.row_of, L.token_of, L.ws, L.ws.numel(), st),
                      lambda: pm.grouped_swiglu(X.up_dense, pm.make_rows(kind, L.x, L.x_scales, T, L.token_of),
                                                L.offsets, P, kind, L.h, L.h_scales, st),
                      lambda: pm.grouped_matmul(X.down_dense, pm.make_rows(kind, L.h, L.h_scales, P), L.offsets, P,
                                                pm.BF16, L.out, st),
                      lambda i=i: pm.combine_rows(L.out, True, L.row_of, L.w, T, k, H, sums[i], st)]
            y = sums[i]
        st = torch.cuda.current_stream()
        for s in steps:
            s()
            if pause:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [r] + [s.clone() for s in sums]

    want = run(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))
    assert float(want[0].abs().max()) < float("inf") and pm.grouped_error() == (0, 0)


def test_a_captured_layer_behind_copies_and_a_join(pm):
    """In a graph the launch in front may be a copy, or two branches that join: the early launch waits for those too."""
    E, H, I, k, T = 9, 256, 128, 2, 200
    X = experts(1, E, H, I, 11)
    L, alone = PromptLayer(X, k, T), PromptLayer(X, k, T)
    given = inputs(E, H, T, 12)
    r, y, logits = (torch.zeros_like(a) for a in given)
    staged = [a.clone() for a in given]
    side = torch.cuda.Stream()
    out = torch.empty(T, H, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000)
            logits.copy_(staged[2])
        r.copy_(staged[0])
        y.copy_(staged[1])
        L.norm(r, y, T)
        main.wait_stream(side)
        L.route(logits, T)
        out.copy_(L.forward(T))
    for seed in (13, 14, 15):
        for to, a in zip(staged, inputs(E, H, T, seed)):
            to.copy_(a)
        graph.replay()
        torch.cuda.synchronize()
        alone.norm(staged[0].clone(), staged[1], T)
        alone.route(staged[2], T)
        want = alone.forward(T)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
