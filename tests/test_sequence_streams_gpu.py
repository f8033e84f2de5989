"""The sequence operators on a stream that is not the current one: what a
call allocates is not memory that the current stream still works on, and
what it returns is not handed out again while the current stream reads it."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402
from test_sequence_gpu import BF16, delta_inputs, randn  # noqa: E402


def calls():
    """Each call, as a function of its stream, and what it allocates."""
    x, dy = randn(1, 2000, 512, dtype=BF16), randn(2, 2000, 512, dtype=BF16)
    y, mean, rstd = dwc.layer_norm(x)
    a = delta_inputs(3, 2, 150, 2, 2, 64, 64, BF16)
    token = [t[:, :1] for t in a[:5]]
    return {"layer_norm": lambda s: dwc.layer_norm(x, stream=s),
            "layer_norm_bwd": lambda s: dwc.layer_norm_bwd(dy, x, mean, rstd, stream=s),
            "dropout": lambda s: (dwc.dropout(x, 0.5, 3, stream=s),),
            "delta_rule": lambda s: dwc.delta_rule(*a, stream=s),
            "delta_rule_bwd": lambda s: dwc.delta_rule_bwd(a[2], None, *a, stream=s),
            "delta_rule_step": lambda s: dwc.delta_rule_step(*token, a[5], stream=s)}


NAMES = ["layer_norm", "layer_norm_bwd", "dropout", "delta_rule", "delta_rule_bwd",
         "delta_rule_step"]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_the_current_stream_is_left_alone(name, handle):
    log(f"case stream {name} {handle}")
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    sync()
    here = torch.cuda.current_stream()
    held = [torch.full((1 << n,), 7.0, device="cuda") for n in range(10, 23)]
    copies = [torch.empty_like(t) for t in held]
    sync()
    torch.cuda._sleep(20_000_000)  # some milliseconds, then the blocks are read
    for c, t in zip(copies, held):
        c.copy_(t)
    del held, t  # free for the current stream, which has yet to read them
    got = call(side.cuda_stream if handle else side)
    here.wait_stream(side)
    sync()
    for c in copies:
        assert (c == 7.0).all()
    for s, t in zip(got, want):
        assert torch.equal(s, t)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_outlive_their_readers(name):
    log(f"case stream outputs {name}")
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    sync()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)
    copies = [t.clone() for t in got]
    del got  # the current stream has yet to read them
    with torch.cuda.stream(side):
        over = [torch.full_like(t, 3.0) for t in want for _ in range(3)]
    sync()
    for s, t in zip(copies, want):
        assert torch.equal(s, t)
    del over


def test_workspace_is_not_shared_between_streams():
    """Calls under way on two streams at once."""
    a = delta_inputs(5, 4, 600, 4, 4, 64, 64, BF16)
    want = dwc.delta_rule_bwd(a[2], None, *a)
    sync()
    sides = [torch.cuda.Stream() for _ in range(3)]
    got = [dwc.delta_rule_bwd(a[2], None, *a, stream=s) for _ in range(3) for s in sides]
    for s in sides:
        torch.cuda.current_stream().wait_stream(s)
    sync()
    for g in got:
        for s, t in zip(g, want):
            assert s is t is None or torch.equal(s, t)
