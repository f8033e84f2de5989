"""The forms that the selective scan chooses by size: one pass with two or four
states a wave, chunks with 4, 8 or 16 states a lane, several blocks of states,
many sequences, and lengths around the ends of stages, chunks and eights."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_helpers import dwc, log, sync  # noqa: E402
from test_sequence_gpu import BF16, F16, F32, randn  # noqa: E402
from test_scan_gpu import NAMES, check, inputs, reference, run_case  # noqa: E402


# long sequences of few channels go in chunks
@pytest.mark.parametrize("b,l,d,n,g,lens", [
    (1, 500, 10, 3, 1, None), (1, 450, 20, 8, 2, None), (2, 600, 30, 16, 1, [600, 333]),
    (1, 900, 66, 12, 1, [899]), (1, 450, 24, 40, 1, None), (1, 400, 12, 100, 2, None),
    (2, 420, 9, 17, 3, [1, 420])])
def test_chunks(b, l, d, n, g, lens):
    log(f"case scan in chunks {b} {l} {d} {n} {g} {lens}")
    run_case(b, l, d, n, g, lens, True, True, True, BF16)


# many sequences of few tokens in one pass, four states a wave
@pytest.mark.parametrize("b,l,d,n,gate", [(300, 5, 3, 16, True), (129, 17, 130, 9, False),
                                          (40, 3, 450, 16, True)])
def test_many_sequences(b, l, d, n, gate):
    log(f"case scan of many sequences {b} {l} {d} {n}")
    lens = [(7 * i) % (l + 1) for i in range(b)]
    run_case(b, l, d, n, 1, lens, gate, True, True, F16)


# each count of workgroups and of states a wave
@pytest.mark.parametrize("b", [9, 70, 130, 260])
@pytest.mark.parametrize("n", [8, 12, 20, 28, 40])
def test_counts_of_workgroups(b, n):
    log(f"case scan of {b} sequences, {n} states")
    lens = [(11 * i) % 40 for i in range(b)]
    run_case(b, 37, 5, n, 1, lens, True, True, True, F16)


@pytest.mark.parametrize("d,n", [(17, 20), (33, 16), (15, 40), (47, 32), (65, 12)])
def test_channels_of_narrow_workgroups(d, n):
    """Channels that end inside workgroups of 16 and 32 of them, two groups."""
    log(f"case scan of {d} channels, {n} states")
    run_case(2, 50, 2 * d, n, 2, [50, 21], True, True, False, F32)


@pytest.mark.parametrize("l", [1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129])
def test_lengths_at_the_ends(l):
    """One sequence of each length, beside a longer one."""
    log(f"case scan length {l}")
    run_case(2, 140, 34, 16, 1, [l, 140], True, True, True, F32)
    run_case(1, l, 34, 33, 1, None, False, True, True, F32)


def test_forms_agree():
    """One channel block alone goes in chunks, beside 300 more in one pass: the
    same sequence gives the same values to the bounds of both."""
    a = inputs(21, 1, 600, 64, 16, 1, F32)
    alone = dwc.selective_scan(*a, softplus=True)
    ref = reference(a, None, True)
    for name, got in zip(("y", "s1"), alone):
        check(name + " in chunks", got, ref[name])
    many = [t.expand(300, *t.shape[1:]) if t is not None and i in (0, 1, 3, 4, 6) else t
            for i, t in enumerate(a)]
    many[8] = a[8].repeat(300, 1, 1)
    y, s1 = dwc.selective_scan(*many, softplus=True)
    sync()
    for i in (0, 137, 299):
        check("y in one pass", y[i:i + 1], ref["y"])
        check("s1 in one pass", s1[i:i + 1], ref["s1"])
    assert (y == y[:1]).all() and (s1 == s1[:1]).all()


def test_converted_module():
    """A mixer converted to bf16 as a whole still runs, its vectors in fp32."""
    from depthwise_convolution_dwc_amd.nn import SelectiveScanMixer

    torch.manual_seed(0)
    m = SelectiveScanMixer(32, states=8, device="cuda").to(torch.bfloat16)
    x = randn(1, 2, 9, 32, dtype=BF16)
    y, state = m(x)
    y.float().sum().backward()
    assert all(torch.isfinite(p.grad).all() and p.grad.dtype == BF16 for p in m.parameters())
    with torch.no_grad():
        assert m.step(x[:, :1], type(state)(*(t.detach() for t in state))).dtype == BF16


def test_gradients_alone_of_broadcast_sequences():
    """Operands with batch stride 0 are read in place."""
    a = inputs(22, 1, 40, 20, 16, 2, BF16)
    many = [t.expand(3, *t.shape[1:]) if t is not None and i in (0, 1, 3, 4, 6) else t
            for i, t in enumerate(a)]
    many[8] = a[8].repeat(3, 1, 1)
    dy = randn(1, 1, 40, 20, dtype=BF16)
    one = dwc.selective_scan_bwd(dy, None, *a, softplus=True)
    got = dwc.selective_scan_bwd(dy.expand(3, 40, 20), None, *many, softplus=True)
    for name, s, t in zip(NAMES[2:], got, one):
        if t.dim() > 2 and name != "dA":
            assert (s == t).all(), name


@pytest.mark.parametrize("b,l,d,n", [(2, 150, 70, 16), (1, 600, 20, 5), (3, 40, 66, 33), (1, 600, 9, 70)])
def test_infinite_rates(b, l, d, n):
    """States whose decay is 0 at every token, sequences that end inside a
    stage, an eight and a chunk."""
    log(f"case scan with infinite rates {b} {l} {d} {n}")
    a = inputs(23, b, l, d, n, 1, F32)
    lens = [l - 3 - 8 * i for i in range(b)]
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dy, ds1 = randn(24, b, l, d), randn(25, b, d, n)
    a[2][:, n // 2] = -1e30  # exp(dt A) is 0 in 64 bits too
    ref = reference(a, lens, True)
    large = dwc.selective_scan(*a, lengths=lengths, softplus=True)
    for name, got in zip(("y", "s1"), large):
        check(name, got, ref[name])
    large += dwc.selective_scan_bwd(dy, ds1, *a, lengths=lengths, softplus=True)
    large += dwc.selective_scan_step(*a, lengths=lengths, softplus=True)
    a[2][:, n // 2] = -float("inf")
    got = dwc.selective_scan(*a, lengths=lengths, softplus=True)
    got += dwc.selective_scan_bwd(dy, ds1, *a, lengths=lengths, softplus=True)
    got += dwc.selective_scan_step(*a, lengths=lengths, softplus=True)
    for s, t in zip(got, large):
        assert torch.isfinite(s).all() and (s == t).all()


def test_two_streams_at_once():
    """Calls that run side by side have workspaces of their own."""
    cases = [inputs(26 + i, 2, 300, 96, n, 1, BF16) for i, n in enumerate((16, 40))]
    dys = [randn(30 + i, 2, 300, 96, dtype=BF16) for i in range(2)]
    want = [dwc.selective_scan(*a, softplus=True) + dwc.selective_scan_bwd(dy, None, *a, softplus=True)
            for a, dy in zip(cases, dys)]
    streams = [torch.cuda.Stream() for _ in cases]
    sync()
    got = [[], []]
    for _ in range(5):
        for i, (s, a, dy) in enumerate(zip(streams, cases, dys)):
            with torch.cuda.stream(s):
                got[i].append(dwc.selective_scan(*a, softplus=True)
                              + dwc.selective_scan_bwd(dy, None, *a, softplus=True))
    sync()
    for runs, ref in zip(got, want):
        for run in runs:
            assert all((s == t).all() for s, t in zip(run, ref))
