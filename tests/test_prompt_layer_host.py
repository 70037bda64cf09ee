"""What a prompt's layer hands to the library, seen on the host: the library's calls are replaced by records."""
import contextlib
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

CALLS = ("residual_norm_q8", "route", "group_pairs", "grouped_swiglu", "grouped_matmul", "combine_rows")


@pytest.fixture
def calls(monkeypatch):
    """[(name, arguments)] of the library calls made, which do nothing."""
    from bitplane_mixed_precision_b200 import prompt
    made = []
    for name in CALLS:
        monkeypatch.setattr(prompt, name, lambda *a, name=name: made.append((name, a)))
    return made


def layer(kind, T=10, k=2, E=4, H=256, I=128):
    from bitplane_mixed_precision_b200 import prompt
    experts = SimpleNamespace(E=E, H=H, I=I, kind=kind, up=torch.empty(1), up_dense=None, down_dense=None)
    return prompt.PromptLayer(experts, k, T)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("given", [False, True])
def test_calls_run_on_the_current_stream_or_the_given_one(monkeypatch, calls, kind, given):
    """torch's side streams do not wait for the default stream: a layer on that one would race with its inputs."""
    L = layer(kind)
    asked = []

    def current(device=None):
        asked.append(torch.device(device))
        return "the current stream"

    monkeypatch.setattr(torch.cuda, "current_stream", current)
    stream = ("the given stream",) if given else ()
    L.norm(torch.zeros(5, 256), None, 5, None, 0.0, *stream)
    L.route(torch.zeros(5, 4), 5, *stream)
    L.forward(5, *stream)
    assert [n for n, _ in calls] == list(CALLS)
    assert all(a[-1] == ("the given stream" if given else "the current stream") for _, a in calls)
    assert all(d == L.y.device for d in asked)
