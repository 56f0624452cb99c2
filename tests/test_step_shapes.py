"""Shapes that a serving step's calls want where a count alone would let another layout through (no GPU
needed: the library's entry points are replaced, as in test_step_refusals.py)."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_prompt_refusals import On  # noqa: E402
from tests.test_step_refusals import calls  # noqa: E402,F401


@pytest.mark.parametrize("name", ["norm_rope", "rope"])
@pytest.mark.parametrize("shape", [(4, 2), (8,), (1, 8), (8, 1), (2, 2, 2), (2, 4, 1), (1, 2, 4)])
def test_positions_of_several_axes_are_rows_of_tokens(calls, name, shape):  # noqa: F811
    """[axes][T]: [T][axes] holds as many values, and would turn heads by other tokens' positions."""
    with pytest.raises(ValueError, match="^positions: "):
        calls(name, positions=On(torch.zeros(shape, dtype=torch.int32)))
    assert calls(name, positions=On(torch.zeros(2, 4, dtype=torch.int32))) == ["norm_rope"]
