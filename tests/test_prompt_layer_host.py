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


def test_decoding_a_stored_layer_allocates_on_its_own_stream(monkeypatch):
    """torch gives memory freed on the host to later work of the stream that it was allocated on: a buffer of
    another stream could be written again while the decoding still reads it."""
    from bitplane_mixed_precision_b200 import prompt
    from bitplane_mixed_precision_b200.store import ResidentLayer
    now = ["the current stream"]

    @contextlib.contextmanager
    def on(stream):
        before, now[0] = now[0], stream
        yield
        now[0] = before

    new, made = torch.empty, []

    def empty(*a, **kw):
        made.append(now[0])
        return new(*a, **kw).zero_()

    E, H, I, G = 2, 128, 128, 128
    R = ResidentLayer.__new__(ResidentLayer)
    R.E, R.H, R.I, R.G, R.mat_words = E, H, I, G, H * I // 32
    R.slot_words, R.scale_len = 3 * R.mat_words, 2 * I * (H // G) + H * (I // G)
    R.pool = torch.zeros(E * 8 * R.slot_words, dtype=torch.int32)
    R.scales, R.codebooks = torch.ones(E * R.scale_len), torch.zeros(E * 3 * 510)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch, "empty", empty)
    streams = []
    monkeypatch.setattr(prompt, "extract_prefix", lambda *a: streams.append(a[-1]))
    X = prompt.DenseExperts.from_layer(R, prompt.BF16, stream="the given stream")
    assert X.up.shape == (E, 2 * I, H)
    assert set(streams) == {"the given stream"} and len(streams) == 3 * E
    assert len(made) >= 4 and set(made) == {"the given stream"}


def test_a_layer_has_a_record_of_its_own(calls, monkeypatch):
    """Both products of a layer record a wait that ran out in the layer's own words, not in the device's that every
    caller clears; the words are taken once."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    L, other = layer(1), layer(1)
    L.forward(5)
    made = {n: a for n, a in calls}
    for name in ("grouped_swiglu", "grouped_matmul"):
        assert made[name][1].error == L.errors.data_ptr() != other.errors.data_ptr()
    assert L.error() == (0, 0)
    L.errors[0], L.errors[1] = 3, 10
    assert L.error() == (3, 10) and L.error() == (0, 0)


def test_a_record_that_is_not_aligned_is_refused():
    import bitplane_mixed_precision_b200 as pm
    A = 1 << 20  # refused calls never follow it
    with pytest.raises(pm.PmoeError) as ei:
        pm.grouped_matmul(pm.make_dense(1, A, A, 4, 64, 256), pm.make_rows(1, A, A, 10, None, A + 4), A, 10, 2, A)
    assert ei.value.code == 1


def test_logits_with_gaps_are_refused(calls, monkeypatch):
    """The router reads rows of E values one after another: columns of a wider tensor would be read as other tokens'."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    L = layer(0)
    wide = torch.zeros(5, 8)
    with pytest.raises(ValueError):
        L.route(wide[:, :4], 5)
    assert not calls
    logits = wide[:, :4].contiguous()
    L.route(logits, 5)
    assert calls[0][1][0] == logits.data_ptr()


def test_tensors_that_are_too_short_or_of_another_type_are_refused(calls, monkeypatch):
    """The library takes addresses: a bf16 residual stream, or fewer rows than tokens, would be read past its end."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    L = layer(1)
    r, y, gain, logits = torch.zeros(5, 256), torch.zeros(5, 256), torch.zeros(256), torch.zeros(5, 4)
    for bad in (dict(r=r.bfloat16()), dict(r=r[:4]), dict(y=y.half()), dict(y=y[:4]), dict(gain=gain.double()),
                dict(gain=gain[:255])):
        with pytest.raises(ValueError):
            L.norm(bad.get("r", r), bad.get("y", y), 5, bad.get("gain", gain))
    for bad in (logits.bfloat16(), logits[:4], logits.long()):
        with pytest.raises(ValueError):
            L.route(bad, 5)
    assert not calls
    L.norm(r, None, 5)
    L.norm(r.data_ptr(), y, 4, gain)
    L.route(logits, 5)
    assert len(calls) == 3


@pytest.mark.parametrize("kind,E,H,I", [(1, 4, 192, 128), (1, 4, 128, 64), (0, 4, 132, 64), (0, 4, 64, 12), (2, 4, 128, 128),
                                        (0, 0, 64, 64), (1, 2049, 128, 128), (1, 4, 0, 128)])
def test_experts_that_no_product_would_take_are_refused(kind, E, H, I):
    """Before they are filled: every product would refuse them, after minutes of filling."""
    from bitplane_mixed_precision_b200.prompt import DenseExperts
    with pytest.raises(ValueError):
        DenseExperts(E, H, I, lambda e, m, w: None, kind, device="cpu")
