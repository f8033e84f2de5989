"""The state that ``GatedDeltaMixer`` hands out."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_mixer_gpu import mixer  # noqa: E402
from test_sequence_gpu import randn  # noqa: E402


@pytest.mark.parametrize("b", [1, 2])
def test_mixer_state_is_its_own(b):
    """The state of a prompt holds the last tokens, not the whole prompt."""
    m = mixer().eval()
    with torch.no_grad():
        y, state = m(randn(11, b, 50, 64))
    assert state.taps.untyped_storage().nbytes() == state.taps.numel() * 4
