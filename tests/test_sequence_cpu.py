"""The sequence-layer entry points without a GPU: struct layouts, and every
refusal of a bad call, which happens before anything is launched."""

import ctypes
import os

import pytest

import depthwise_convolution_dwc_amd as dwc
from depthwise_convolution_dwc_amd import sequence as seq

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.skipif(not os.path.exists(dwc.LIB_PATH), reason="libdwc.so not built")

BAD, UNSUPPORTED, MISALIGNED, WORKSPACE, ALIAS = 1, 2, 3, 4, 5
A = 1 << 20  # made-up device addresses, far apart: no call below launches
NAN, INF = float("nan"), float("inf")


def at(i, off=0):
    return (i + 1) * (1 << 32) + off


def test_struct_sizes():
    assert ctypes.sizeof(seq.NormProblem) == 48
    assert ctypes.sizeof(seq.DropoutProblem) == 40
    assert ctypes.sizeof(seq.DeltaProblem) == 16 + 6 * 24 + 24


def norm(rows=4, c=8, xs=8, ds=8, x=0, y=0, w=0, eps=1e-5):
    return seq.NormProblem(rows, c, xs, ds, x, y, w, eps)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), BAD), (dict(c=0), BAD), (dict(xs=7), BAD), (dict(x=3), BAD), (dict(y=5), BAD),
    (dict(w=-1), BAD), (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD), (dict(eps=INF), BAD),
    (dict(rows=1 << 40), UNSUPPORTED), (dict(c=1 << 33, xs=1 << 33), UNSUPPORTED),
    (dict(rows=1 << 31, xs=1 << 36), UNSUPPORTED)])
def test_norm_problem_refused(change, status):
    p = norm(**change)
    st = dwc.lib().dwc_layer_norm(ctypes.byref(p), at(0), at(1), at(2), at(3), at(4), at(5), None)
    assert st == status and dwc.last_error()


def test_norm_pointers_refused():
    f, p = dwc.lib().dwc_layer_norm, ctypes.byref(norm())
    assert f(None, at(0), None, None, at(3), None, None, None) == BAD
    assert f(p, None, None, None, at(3), None, None, None) == BAD
    assert f(p, at(0), None, None, None, None, None, None) == BAD
    assert f(p, at(0), None, None, at(3), at(4), None, None) == BAD  # mean without rstd
    assert f(p, at(0, 2), None, None, at(3), None, None, None) == MISALIGNED
    assert f(p, at(0), None, None, at(3, 1), None, None, None) == MISALIGNED
    assert f(p, at(0), None, None, at(0, 64), None, None, None) == ALIAS
    assert f(p, at(0), at(1), None, at(1, -16), None, None, None) == ALIAS
    assert f(p, at(0), None, None, at(3), at(3, 16), at(5), None) == ALIAS
    assert f(ctypes.byref(norm(rows=0)), None, None, None, None, None, None, None) == 0


def test_norm_bwd_refused():
    p, need = norm(), ctypes.c_size_t()
    f = dwc.lib().dwc_layer_norm_bwd
    assert dwc.lib().dwc_layer_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(need)) == 0
    assert need.value > 0
    a = [at(i) for i in range(9)]

    def call(p=p, ws=at(9), n=need.value, **ch):
        b = list(a)
        for k, v in ch.items():
            b[int(k[1:])] = v
        return f(ctypes.byref(p), b[0], b[1], b[2], b[3], b[4], b[5], b[6], b[7], ws, n, None)

    assert call(n=need.value - 1) == WORKSPACE
    assert call(ws=None) == WORKSPACE
    assert call(a0=None) == BAD and call(a2=None) == BAD and call(a5=None) == BAD
    assert call(a5=a[0]) == ALIAS and call(a6=a[7]) == ALIAS
    assert call(ws=a[1]) == ALIAS
    assert call(p=norm(ds=3)) == BAD


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), BAD), (dict(p=-0.1), BAD), (dict(p=1.01), BAD), (dict(p=NAN), BAD),
    (dict(dtype=3), BAD), (dict(n=1 << 34), UNSUPPORTED)])
def test_dropout_problem_refused(change, status):
    kw = dict(n=16, p=0.5, seed=1, offset=0, dtype=0, reserved=0)
    kw.update(change)
    p = seq.DropoutProblem(*kw.values())
    assert dwc.lib().dwc_dropout(ctypes.byref(p), at(0), None, at(1), None) == status


def test_dropout_pointers_refused():
    p, f = seq.DropoutProblem(16, 0.5, 1, 0, 0, 0), dwc.lib().dwc_dropout
    assert f(None, at(0), None, at(1), None) == BAD
    assert f(ctypes.byref(p), None, None, at(1), None) == BAD
    assert f(ctypes.byref(p), at(0, 2), None, at(1), None) == MISALIGNED
    assert f(ctypes.byref(p), at(0), None, at(0), None) == ALIAS
    assert f(ctypes.byref(p), at(0), at(1, 60), at(1), None) == ALIAS
    assert f(ctypes.byref(seq.DropoutProblem(0, 0.5, 1, 0, 0, 0)), None, None, None, None) == 0


def delta(b=2, l=5, hk=2, hv=4, dk=16, dv=8, dtype=0, scale=0.25, **st):
    I = ctypes.c_int64 * 3
    d = dict(q=I(l * hk * dk, hk * dk, dk), k=I(l * hk * dk, hk * dk, dk),
             v=I(l * hv * dv, hv * dv, dv), g=I(l * hv, hv, 1), beta=I(l * hv, hv, 1),
             do=I(l * hv * dv, hv * dv, dv))
    for k, v in st.items():
        d[k] = I(*v)
    return seq.DeltaProblem(b, l, d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], hk, hv, dk,
                            dv, dtype, scale)


def delta_step(p, **ch):
    a = dict(q=at(0), k=at(1), v=at(2), g=at(3), beta=at(4), s0=at(5), lengths=None, o=at(6),
             s1=at(7))
    a.update(ch)
    return dwc.lib().dwc_delta_step(ctypes.byref(p), *a.values(), None)


BAD_DELTA = [
    (dict(b=-1), BAD), (dict(l=-1), BAD), (dict(hk=0), BAD), (dict(hk=3), BAD), (dict(dk=0), BAD),
    (dict(dv=0), BAD), (dict(dtype=4), BAD), (dict(scale=NAN), BAD), (dict(scale=INF), BAD),
    (dict(q=(-1, 32, 16)), BAD), (dict(v=(1 << 60, 1, 1)), BAD), (dict(dk=257), UNSUPPORTED),
    (dict(dv=4097), UNSUPPORTED), (dict(b=70000), UNSUPPORTED), (dict(l=1 << 31), UNSUPPORTED)]


@pytest.mark.parametrize("change,status", BAD_DELTA)
def test_delta_problem_refused(change, status):
    assert delta_step(delta(**change)) == status and dwc.last_error()
    need = ctypes.c_size_t()
    if "q" not in change and "v" not in change:
        for op in (0, 1):
            assert dwc.lib().dwc_delta_workspace_size(ctypes.byref(delta(**change)), op,
                                                      ctypes.byref(need)) == status


def test_delta_step_pointers_refused():
    p = delta()
    for name in ("q", "k", "v", "g", "beta", "o", "s1"):
        assert delta_step(p, **{name: None}) == BAD, name
    for name in ("q", "g", "s0", "o", "s1"):
        assert delta_step(p, **{name: at(30, 2)}) == MISALIGNED, name
    assert delta_step(p, o=at(2)) == ALIAS
    assert delta_step(p, s1=at(5, 4)) == ALIAS  # partly over s0: only the whole state in place
    assert delta_step(delta(b=0)) == 0


def test_delta_chunked_limits():
    need = ctypes.c_size_t()
    f = dwc.lib().dwc_delta_workspace_size
    assert f(ctypes.byref(delta(dk=129)), 0, ctypes.byref(need)) == UNSUPPORTED
    assert f(ctypes.byref(delta()), 2, ctypes.byref(need)) == BAD
    assert f(ctypes.byref(delta()), 0, None) == BAD
    assert f(None, 0, ctypes.byref(need)) == BAD


def test_tensor_calls_refuse_host_tensors_and_wrong_types():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        dwc.layer_norm(x)
    with pytest.raises(TypeError):
        dwc.layer_norm([1.0])
    with pytest.raises(ValueError):
        dwc.dropout(x, 0.5, 1)
    q = torch.zeros(1, 2, 1, 4)
    with pytest.raises(ValueError):
        dwc.delta_rule(q, q, q, q[..., 0], q[..., 0])


def test_delta_chunked_pointers_refused():
    p, need = delta(), ctypes.c_size_t()
    lib = dwc.lib()
    for op in (0, 1):
        assert lib.dwc_delta_workspace_size(ctypes.byref(p), op, ctypes.byref(need)) == 0
        assert need.value > 0
        names = (["q", "k", "v", "g", "beta", "s0", "lengths", "o", "s1"] if op == 0 else
                 ["dout", "ds1", "q", "k", "v", "g", "beta", "s0", "lengths", "dq", "dk", "dv",
                  "dg", "dbeta", "ds0"])
        f = lib.dwc_delta_fwd if op == 0 else lib.dwc_delta_bwd

        def call(p=p, ws=at(40), n=need.value, **ch):
            a = {name: at(i) for i, name in enumerate(names)}
            a["lengths"] = None
            a.update(ch)
            return f(ctypes.byref(p) if p else None, *a.values(), ws, n, None)

        assert call(p=None) == BAD
        assert call(n=need.value - 1) == WORKSPACE and call(ws=None) == WORKSPACE
        assert call(ws=at(40, 64)) == MISALIGNED
        for name in names:
            if name not in ("lengths", "s0", "ds1", "ds0"):
                assert call(**{name: None}) == BAD, name
            if name != "lengths":
                assert call(**{name: at(30, 1)}) == MISALIGNED, name
        out = names[7] if op == 0 else "dq"
        assert call(**{out: at(names.index("v"))}) == ALIAS
        assert call(ws=at(names.index("q"))) == ALIAS
        if op == 0:
            assert call(s1=at(names.index("s0"))) == ALIAS
        assert call(p=delta(q=(-4, 1, 1))) == BAD
        assert call(p=delta(b=0)) == 0


@pytest.mark.parametrize("change", [dict(b=4096, hk=16, hv=16, l=64 * 128),
                                    dict(b=65535, hk=2, hv=2, dv=4096)])
def test_delta_chunked_launch_range(change):
    need = ctypes.c_size_t()
    p = delta(**change)
    f = dwc.lib().dwc_delta_workspace_size
    assert [f(ctypes.byref(p), op, ctypes.byref(need)) for op in (0, 1)] == [UNSUPPORTED] * 2


def test_dropout_position_refused():
    p, f = seq.DropoutProblem(16, 0.5, 1, 0, 0, 0), dwc.lib().dwc_dropout_at
    a = (ctypes.byref(p), at(0), None, at(1))
    assert f(*a, None, None) == BAD
    assert f(*a, at(2, 4), None) == MISALIGNED
    assert f(*a, at(1, 56), None) == ALIAS
    assert f(None, at(0), None, at(1), at(2), None) == BAD


def test_norm_bwd_columns_past_the_launch_range():
    """The columns' sums take 64 threads each of a launch's 2^32."""
    need, f = ctypes.c_size_t(), dwc.lib().dwc_layer_norm_bwd
    size = dwc.lib().dwc_layer_norm_bwd_workspace_size
    for c, status in (((1 << 25) - 1, 0), (1 << 25, UNSUPPORTED), (1 << 30, UNSUPPORTED)):
        p = ctypes.byref(norm(rows=2, c=c, xs=c, ds=c))
        assert size(p, ctypes.byref(need)) == status
        if status:
            far = [i << 40 for i in range(1, 10)]
            assert f(p, *far[:8], far[8], 1 << 40, None) == status and dwc.last_error()
