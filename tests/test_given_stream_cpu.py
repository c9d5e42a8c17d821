"""Memory that the bindings make for a call on a given stream, without a GPU: it is that stream's."""
import contextlib

import pytest

torch = pytest.importorskip("torch")


class Stream:
    device, device_index, cuda_stream = torch.device("cuda", 0), 0, 7


@pytest.fixture
def streams(monkeypatch):
    """(the stream given, what was made under which stream, the streams recorded)."""
    given, here, inside, made, recorded = Stream(), Stream(), [], [], []

    @contextlib.contextmanager
    def on(s):
        inside.append(s)
        yield
        inside.pop()

    empty = torch.empty

    def make(*args, device=None, **kw):
        made.append(inside[-1] if inside else here)
        return empty(*args, **kw)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: here)
    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append(s))
    return given, here, made, recorded


def test_scratch_is_the_streams(streams):
    from rwkv_linear_attention_wkv_b200 import gdr
    given, here, made, recorded = streams
    gdr._scratch(64, 0, given)
    assert made == [given] and recorded == [here]
    gdr._scratch(64, 0, None)
    gdr._scratch(64, 0, here)
    assert made == [given, here, here] and recorded == [here]


def test_a_stream_of_another_device_is_refused():
    from rwkv_linear_attention_wkv_b200 import gdr
    with pytest.raises(ValueError, match="stream must be of cuda:1"):
        gdr._run(None, 1, Stream())


@pytest.mark.parametrize("name", ["wkv_forward", "wkv_forward_bf16", "wkv_forward_state", "wkv_decode_step",
                                  "wkv_decode_steps", "wkv_backward", "wkv_backward_state",
                                  "wkv_forward_checkpointed", "wkv_backward_checkpointed",
                                  "wkv7_forward", "wkv_mstate_forward"])
def test_results_are_the_streams(streams, monkeypatch, name):
    import rwkv_linear_attention_wkv_b200 as W
    given, _, made, _ = streams
    called = []
    monkeypatch.setattr(W, "_need", lambda *a: None)
    monkeypatch.setattr(W, "_call", lambda *a: called.append(a[0]))
    monkeypatch.setattr(W, "wkv_backward_workspace_bytes", lambda *a: 0)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    x = torch.zeros(2, 3, 4)
    rows, vector = torch.zeros(2, 3, 4, 4), torch.zeros(4)
    args = {"wkv_decode_step": [x] * 8, "wkv_decode_steps": [x[0], x[0]] + [rows] * 3 + [x] * 3,
            "wkv_backward": [vector] * 2 + [x] * 4, "wkv_backward_state": [vector] * 2 + [x] * 4,
            "wkv_backward_checkpointed": [vector] * 2 + [x] * 5, "wkv7_forward": [rows] * 6,
            "wkv_mstate_forward": [rows] * 4}.get(name, [vector] * 2 + [x] * 3)
    getattr(W, name)(*args, stream=given)
    assert called == [name] and made and all(s is given for s in made)
