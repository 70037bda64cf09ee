"""The prompt-side operators in the order in which a program enqueues them: on torch's current stream, behind what
writes their inputs, and one call after another on the same buffers."""
import pytest
import torch

from bitplane_mixed_precision_b200.prompt import DenseExperts, PromptLayer

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
