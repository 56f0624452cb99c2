"""Every tensor of a serving step's calls is one of the current device and of the layout that the call
names: refused by its name before anything is launched (no GPU needed: the library's entry points are
replaced, and tensors say where they are)."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_prompt_refusals import On, half, ints  # noqa: E402


def arguments():
    """name -> (all tensors of a call, other arguments, the entry point that it ends in)."""
    T, H, Hk, D, N = 4, 4, 2, 128, 16
    cache = dict(k_cache=half(N, Hk, D), v_cache=half(N, Hk, D))
    f32, ws = torch.zeros(T, H, dtype=torch.float32), torch.zeros(512, dtype=torch.uint8)
    rows = dict(q=half(T, H, D), offsets=ints(0, 1, 4), **cache, seq_lens=ints(5, 16), cell_plan=torch.zeros(2, 16, dtype=torch.int32),
                out=half(T, H, D), lse=f32, ws=ws)
    turned = dict(q=half(T, H, D), k=half(T, Hk, D), positions=torch.zeros(2, T, dtype=torch.int32),
                  table=torch.zeros(D // 2, dtype=torch.int64), axis=torch.zeros(D // 2, dtype=torch.uint8), q_out=half(T, H, D),
                  k_out=half(T, Hk, D))
    return {
        "norm_rope": (dict(**turned, q_weight=half(D), k_weight=half(D)), {}, "norm_rope"),
        "rope": (turned, {}, "norm_rope"),
        "step_maps": (dict(lens=ints(1, 2), n_new=ints(1, 1), tables=torch.zeros(2, 4, dtype=torch.int32), free_blocks=ints(3, 4, 5),
                           n_free=ints(3), plan=torch.zeros(2, 64, dtype=torch.int32), status=ints(0)),
                      dict(block_cells=16, n_cells=256), "step_maps"),
        "prefill": (dict(q=half(T, H, D), k=half(T, Hk, D), v=half(T, Hk, D), offsets=ints(0, 1, 4), out=half(T, H, D), lse=f32, ws=ws),
                    dict(window=3, sinks=1), "prefill_window"),
        "prefill_chunk window": (rows, dict(window=3, sinks=1), "prefill_chunk_window"),
        "prefill_chunk shared": (rows, dict(shared=8), "prefill_chunk_shared"),
    }


@pytest.fixture
def calls(kvattn, monkeypatch):
    """call(name, replaced tensors) -> launches made."""
    launched = []
    monkeypatch.setattr(kvattn, "_current_device", lambda: 0)
    for name in ("rope", "norm_rope", "step_maps", "prefill", "prefill_window", "prefill_chunk", "prefill_chunk_window",
                 "prefill_chunk_shared"):
        monkeypatch.setattr(kvattn.lib, f"kvattn_{name}", lambda *a, name=name: launched.append(name) or 0)

    def call(name, rest=(), **over):
        tensors, more, _ = arguments()[name]
        tensors = {k: On(x) for k, x in tensors.items()} | over
        if "table" in tensors:
            tensors["table"] = kvattn.RopeTable(tensors["table"], 1.0, 128, tensors.pop("axis"), 2)
        out = {}
        if name == "step_maps":
            made = kvattn.step_maps_buffers(2, 8, device="cpu")
            made._at = made._at[:2] + (0,) + made._at[3:]
            out = {"out": made}
        launched.clear()
        getattr(kvattn, name.split()[0])(**tensors, **more | dict(rest), **out, stream=77)
        return list(launched)
    return call


NAMES = [(name, arg) for name, (tensors, _, _) in arguments().items() for arg in tensors]


@pytest.mark.parametrize("name", list(arguments()))
def test_a_whole_call_passes(calls, name):
    assert calls(name) == [arguments()[name][2]]


@pytest.mark.parametrize("place", ["host", "device 1"])
@pytest.mark.parametrize("name,arg", NAMES)
def test_each_tensor_of_a_call(calls, name, arg, place):
    x = arguments()[name][0][arg]
    with pytest.raises(ValueError, match=rf"^{arg}: a tensor of the current CUDA device"):
        calls(name, **{arg: x if place == "host" else On(x, 1)})


@pytest.mark.parametrize("name,over", [
    ("norm_rope", dict(table=torch.zeros(63, dtype=torch.int64))), ("norm_rope", dict(table=torch.zeros(64, dtype=torch.int32))),
    ("norm_rope", dict(axis=torch.zeros(63, dtype=torch.uint8))), ("norm_rope", dict(axis=torch.zeros(64, dtype=torch.int32))),
    ("norm_rope", dict(axis=torch.zeros(128, dtype=torch.uint8)[::2])), ("norm_rope", dict(q_weight=torch.zeros(128))),
    ("norm_rope", dict(k_weight=half(127))), ("norm_rope", dict(k_weight=half(256)[::2])),
    ("norm_rope", dict(positions=torch.zeros(4, dtype=torch.int32))), ("norm_rope", dict(positions=torch.zeros(2, 4))),
    ("norm_rope", dict(q_out=half(4, 4, 256))), ("norm_rope", dict(k=half(3, 2, 128))), ("norm_rope", dict(q=half(4, 4, 128).float())),
    ("step_maps", dict(lens=ints(1))), ("step_maps", dict(n_new=ints(1, 2, 3))), ("step_maps", dict(lens=torch.zeros(2, dtype=torch.int64))),
    ("step_maps", dict(tables=torch.zeros(3, 4, dtype=torch.int32))), ("step_maps", dict(tables=torch.zeros(8, dtype=torch.int32))),
    ("step_maps", dict(tables=torch.zeros(2, 8, dtype=torch.int32)[:, ::2])), ("step_maps", dict(plan=torch.zeros(1, 64, dtype=torch.int32))),
    ("step_maps", dict(plan=torch.zeros(2, 64))), ("step_maps", dict(n_free=ints(1, 2))),
    ("step_maps", dict(status=torch.zeros(3, dtype=torch.uint8))),
    ("prefill", dict(ws=torch.zeros(1, dtype=torch.uint8).expand(512))), ("prefill_chunk shared", dict(ws=torch.zeros(1024, dtype=torch.uint8)[::2])),
])
def test_shapes_types_and_layouts(calls, name, over):
    with pytest.raises(ValueError):
        calls(name, **{k: On(x) for k, x in over.items()})


def test_free_blocks_go_with_their_count(calls):
    for gone in ("free_blocks", "n_free"):
        with pytest.raises(ValueError, match="go together"):
            calls("step_maps", **{gone: None})
    assert calls("step_maps", free_blocks=None, n_free=None) == ["step_maps"]


@pytest.mark.parametrize("name,rest", [("prefill", dict(window=None, sinks=2)), ("prefill_chunk window", dict(window=None, sinks=2)),
                                       ("prefill_chunk window", dict(shared=4)), ("prefill_chunk shared", dict(sinks=1))])
def test_windows_first_tokens_and_prefixes_that_do_not_go_together(calls, name, rest):
    with pytest.raises(ValueError):
        calls(name, rest=rest)


def test_without_window_or_prefix_the_plain_forms(calls):
    assert calls("prefill", rest=dict(window=None, sinks=0)) == ["prefill"]
    assert calls("prefill_chunk window", rest=dict(window=None, sinks=0)) == ["prefill_chunk"]
    assert calls("prefill_chunk shared", rest=dict(shared=0)) == ["prefill_chunk"]
