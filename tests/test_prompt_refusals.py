"""Every tensor of a prompt-side call is one of the current device: a host tensor, or another device's,
is refused by its name before anything is launched (no GPU needed: the library's entry points are
replaced, and tensors say where they are)."""
import pytest

torch = pytest.importorskip("torch")


class On:
    """A host tensor that says it is on device `dev`."""

    def __init__(self, x, dev=0):
        self.x, self.dev = x, dev

    def __getattr__(self, name):
        return getattr(self.x, name)

    is_cuda = True

    def get_device(self):
        return self.dev


def half(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def ints(*values):
    return torch.tensor(values, dtype=torch.int32)


def arguments():
    """name -> (entry point, all tensors of a call, other arguments, shape of the call)."""
    T, H, Hk, D, N = 4, 4, 2, 128, 16
    quant = dict(k_cache=torch.zeros(N, Hk, D, dtype=torch.int8), v_cache=torch.zeros(N, Hk, D // 2, dtype=torch.uint8),
                 k_scales=half(N, Hk, D // 32), v_scales=half(N, Hk, D // 32))
    rows = dict(k=half(T, Hk, D), v=half(T, Hk, D))
    f32 = torch.zeros(T, H, dtype=torch.float32)
    ws = torch.zeros(512, dtype=torch.uint8)
    status = ints(0)
    return {
        "rope": (dict(q=half(T, H, D), k=half(T, Hk, D), positions=ints(0, 1, 2, 3), table=torch.zeros(D // 2, dtype=torch.int64),
                      q_out=half(T, H, D), k_out=half(T, Hk, D)), {}),
        "cache_write": (dict(**rows, slots=ints(3, 2, 1, 0), **quant, status=status), {}),
        "cache_read": (dict(slots=ints(3, 2, 1, 0), **quant, k_out=half(T, Hk, D), v_out=half(T, Hk, D), status=status),
                       dict(head_dim=D)),
        "prefill": (dict(q=half(T, H, D), **rows, offsets=ints(0, 1, 4), out=half(T, H, D), lse=f32, ws=ws), {}),
        "prefill_chunk": (dict(q=half(T, H, D), offsets=ints(0, 1, 4), **quant, seq_lens=ints(5, 16),
                               cell_plan=torch.zeros(2, 16, dtype=torch.int32), out=half(T, H, D), lse=f32, ws=ws), {}),
    }


@pytest.fixture
def calls(kvattn, monkeypatch):
    """call(name, replaced tensors) -> launches made."""
    launched = []
    monkeypatch.setattr(kvattn, "_current_device", lambda: 0)
    for name in ("rope", "cache_write", "cache_read", "prefill", "prefill_chunk"):
        monkeypatch.setattr(kvattn.lib, f"kvattn_{name}", lambda *a, name=name: launched.append(name) or 0)

    def call(name, **over):
        tensors, rest = arguments()[name]
        tensors = {k: On(x) for k, x in tensors.items()} | over
        if "table" in tensors:
            tensors["table"] = kvattn.RopeTable(tensors["table"], 1.0, 128)
        launched.clear()
        getattr(kvattn, name)(**tensors, **rest, stream=77)
        return list(launched)
    return call


NAMES = [(name, arg) for name, (tensors, _) in arguments().items() for arg in tensors]


@pytest.mark.parametrize("name", list(arguments()))
def test_a_whole_call_passes(calls, name):
    assert calls(name) == [name]


@pytest.mark.parametrize("place", ["host", "device 1"])
@pytest.mark.parametrize("name,arg", NAMES)
def test_each_tensor_of_a_call(calls, name, arg, place):
    x = arguments()[name][0][arg]
    with pytest.raises(ValueError, match=rf"^{arg}: a tensor of the current CUDA device"):
        calls(name, **{arg: x if place == "host" else On(x, 1)})


def test_rope_of_one_tensor(calls):
    k = arguments()["rope"][0]["k"]
    assert calls("rope", q=None, q_out=None) == ["rope"]
    with pytest.raises(ValueError, match="^k: a tensor of the current CUDA device"):
        calls("rope", q=None, q_out=None, k=k)


@pytest.mark.parametrize("name,over", [
    ("rope", dict(table=torch.zeros(63, dtype=torch.int64))),          # fewer angles than n_rot says
    ("rope", dict(table=torch.zeros(64, dtype=torch.int32))),
    ("rope", dict(table=torch.zeros(128, dtype=torch.int64)[::2])),
    ("cache_write", dict(status=torch.zeros(3, dtype=torch.uint8))),   # no whole word
    ("cache_read", dict(status=torch.zeros(0, dtype=torch.int32))),
    ("prefill", dict(ws=torch.zeros(1, dtype=torch.uint8).expand(512))),
    ("prefill_chunk", dict(ws=torch.zeros(1024, dtype=torch.uint8)[::2])),
])
def test_tables_words_and_workspaces_that_are_too_small(calls, name, over):
    with pytest.raises(ValueError):
        calls(name, **{k: On(x) for k, x in over.items()})
