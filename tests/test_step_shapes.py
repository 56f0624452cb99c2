"""Shapes that a serving step's calls want where a count alone would let another layout through (no GPU
needed: the library's entry points are replaced, as in test_step_refusals.py)."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_prompt_refusals import On  # noqa: E402
from tests.test_step_refusals import arguments, calls  # noqa: E402,F401


@pytest.mark.parametrize("name", ["norm_rope", "rope"])
@pytest.mark.parametrize("shape", [(4, 2), (8,), (1, 8), (8, 1), (2, 2, 2), (2, 4, 1), (1, 2, 4)])
def test_positions_of_several_axes_are_rows_of_tokens(calls, name, shape):  # noqa: F811
    """[axes][T]: [T][axes] holds as many values, and would turn heads by other tokens' positions."""
    with pytest.raises(ValueError, match="^positions: "):
        calls(name, positions=On(torch.zeros(shape, dtype=torch.int32)))
    assert calls(name, positions=On(torch.zeros(2, 4, dtype=torch.int32))) == ["norm_rope"]


def test_without_a_free_list_nothing_is_said_to_be_left(calls, kvattn, monkeypatch):  # noqa: F811
    """What step_maps makes for itself holds no count then: it would be whatever the memory held."""
    tensors, more, _ = arguments()["step_maps"]
    tensors = {k: On(x) for k, x in tensors.items()}
    made = kvattn.StepMaps

    def here(n_seq, n_tok, device):
        m = made(n_seq, n_tok, "cpu")
        m._at = m._at[:2] + (0,) + m._at[3:]
        return m
    monkeypatch.setattr(kvattn, "StepMaps", here)
    monkeypatch.setattr(kvattn, "_other_stream", lambda s: False)
    m = kvattn.step_maps(**tensors | dict(free_blocks=None, n_free=None), **more, n_tok=8, stream=77)
    assert m.n_free is None and m.slots.numel() == 8
    assert kvattn.step_maps(**tensors, **more, out=m, stream=77).n_free.numel() == 1   # (counted now)
    assert kvattn.step_maps(**tensors, **more, n_tok=8, stream=77).n_free.numel() == 1
    b = kvattn.step_maps_buffers(2, 8, device="cpu")
    assert kvattn.step_maps(**tensors | dict(free_blocks=None, n_free=None), **more, out=b, stream=77).n_free.tolist() == [0]


def test_buffers_hold_no_rubbish(kvattn, monkeypatch):
    """A count that no step has written is 0, not what the memory held."""
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).fill_(-77))
    m = kvattn.step_maps_buffers(3, 9, device="cpu")
    assert m.n_free.tolist() == [0]
    assert [x.numel() for x in (m.offsets, m.seq_lens, m.positions, m.slots)] == [4, 3, 9, 9]
    assert all(x.data_ptr() % 16 == 0 for x in (m.offsets, m.seq_lens, m.positions, m.slots, m.n_free))
