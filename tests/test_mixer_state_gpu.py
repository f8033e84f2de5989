"""The state that ``GatedDeltaMixer`` hands out, and what it makes of places
past a sequence's length."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import sync  # noqa: E402
from test_mixer_gpu import mixer  # noqa: E402
from test_sequence_gpu import randn  # noqa: E402


@pytest.mark.parametrize("b", [1, 2])
def test_mixer_state_is_its_own(b):
    """The state of a prompt holds the last tokens, not the whole prompt."""
    m = mixer().eval()
    with torch.no_grad():
        y, state = m(randn(11, b, 50, 64))
    assert state.taps.untyped_storage().nbytes() == state.taps.numel() * 4


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_mixer_gradients_past_a_length(bad):
    """What stands past a sequence's length reaches no gradient."""
    m = mixer()
    x = randn(12, 3, 40, 64)
    lengths = torch.tensor([0, 17, 40], dtype=torch.int32, device="cuda")
    live = (torch.arange(40, device="cuda") < lengths[:, None])[..., None]
    gy = randn(13, 3, 40, 64)
    want = None
    for fill in (0.0, bad):
        z = torch.where(live, x, fill).requires_grad_()
        y, state = m(z, lengths=lengths)
        assert torch.equal(torch.nan_to_num(y)[~live.expand_as(y)],
                           torch.nan_to_num(z)[~live.expand_as(y)])
        got = torch.autograd.grad([torch.where(live, y, 0.0), state.states],
                                  (z,) + tuple(m.parameters()), [gy, state.states.detach()])
        sync()
        got = (y.detach()[live.expand_as(y)], state.taps, state.states) + got
        for s, t in zip(got, want or got):
            assert torch.isfinite(s).all() and torch.equal(s, t)
        want = got
