"""Host-side checks of the gated delta rule: refusals before any HIP call, and the tests' own tolerances."""
import ctypes
import os

import pytest
import torch

import device_wide_prefix_amd as dws
from delta_reference import close, inputs, reference

FAKE = 0x100000      # never dereferenced: every call here fails its checks, or passes a null one
NAMES = ("q", "k", "v", "g", "beta")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dws.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dws.load_library()


def arguments(**more):
    """Arguments that pass every check but the last, a workspace."""
    a = dws.DeltaRuleArgs()
    a.tokens, a.n_seqs, a.heads_qk, a.heads_v, a.dim_k, a.dim_v = 128, 2, 2, 4, 64, 32
    a.dtype, a.g_dtype, a.beta_dtype, a.scale = dws.BFLOAT16, dws.FLOAT32, dws.BFLOAT16, 1.0
    at = FAKE

    def rows(heads, dim, size):
        nonlocal at
        r = dws.Rows(at, heads * dim, dim)
        at += (128 * heads * dim * size + 4095) // 4096 * 4096
        return r

    a.q, a.k, a.v = rows(2, 64, 2), rows(2, 64, 2), rows(4, 32, 2)
    a.g, a.beta, a.out = rows(4, 1, 4), rows(4, 1, 2), rows(4, 32, 2)
    a.out_grad, a.q_grad, a.k_grad = rows(4, 32, 2), rows(2, 64, 2), rows(2, 64, 2)
    a.v_grad, a.g_grad, a.beta_grad = rows(4, 32, 2), rows(4, 1, 2), rows(4, 1, 2)
    a.d_final_state = at
    at += 2 * 4 * 64 * 32 * 4 * 8
    for k, v in more.items():
        setattr(a, k, v)
    a.end = at
    return a


def call(lib, name, a):
    return getattr(lib, name)(ctypes.byref(a), None)


CALLS = ("dws_delta_rule", "dws_delta_rule_backward", "dws_delta_rule_step")


@pytest.mark.parametrize("name", CALLS)
def test_refusals(lib, name):
    bad, unsupported = dws.ERR_INVALID_ARG, dws.ERR_UNSUPPORTED
    assert getattr(lib, name)(None, None) == bad
    for more, status in (
            ({"dtype": dws.INT32}, bad), ({"dtype": 7}, bad), ({"dtype": -1}, bad), ({"beta_dtype": dws.UINT32}, bad),
            ({"g_dtype": dws.PAIR_U32}, bad), ({"tokens": -1}, bad), ({"n_seqs": 0}, bad), ({"n_seqs": 3}, bad),
            ({"heads_qk": 0}, bad), ({"heads_v": 3}, bad), ({"heads_v": -2}, bad), ({"dim_k": 0}, bad),
            ({"dim_v": -1}, bad), ({"dim_k": 257}, unsupported), ({"dim_v": 1 << 20}, unsupported),
            ({"heads_v": 65536}, unsupported), ({"tokens": 1 << 31, "n_seqs": 1}, unsupported),
            ({"tokens": 1 << 30, "n_seqs": 1 << 30}, unsupported),
            ({"q": dws.Rows(None, 128, 64)}, bad), ({"q": dws.Rows(FAKE, -1, 64)}, bad),
            ({"v": dws.Rows(FAKE, 1 << 41, 64)}, bad), ({"k": dws.Rows(FAKE + 1, 128, 64)}, dws.ERR_MISALIGNED),
            ({"g": dws.Rows(FAKE + 2, 4, 1)}, dws.ERR_MISALIGNED), ({"beta": dws.Rows(2**64 - 16, 4, 1)}, bad),
            ({"d_offsets": FAKE + 4}, dws.ERR_MISALIGNED)):
        assert call(lib, name, arguments(**more)) == status, more


def test_refusals_of_outputs(lib):
    bad = dws.ERR_INVALID_ARG
    for name in ("dws_delta_rule", "dws_delta_rule_step"):
        extra = {} if name == "dws_delta_rule" else {"d_initial_state": arguments().d_final_state}
        # an output that names an element twice
        for rows in (dws.Rows(1 << 40, 0, 32), dws.Rows(1 << 40, 127, 32), dws.Rows(1 << 40, 128, 31), dws.Rows(1 << 40, 16, 32)):
            assert call(lib, name, arguments(out=rows, **extra)) == bad
        assert call(lib, name, arguments(out=dws.Rows(None, 128, 32), **extra)) == bad
        # the slots' states
        assert call(lib, name, arguments(d_slots=1 << 41, n_states=0, **extra)) == bad
        assert call(lib, name, arguments(d_slots=(1 << 41) + 2, n_states=4, **extra)) == dws.ERR_MISALIGNED
        assert call(lib, name, arguments(d_slots=1 << 41, n_states=1 << 40, **extra)) == dws.ERR_UNSUPPORTED
    assert call(lib, "dws_delta_rule", arguments(d_final_state=FAKE + 2)) == dws.ERR_MISALIGNED
    # step: one state array, in place
    assert call(lib, "dws_delta_rule_step", arguments()) == bad
    assert call(lib, "dws_delta_rule_step", arguments(d_final_state=None)) == bad
    a = arguments()
    assert call(lib, "dws_delta_rule_step", arguments(d_initial_state=a.d_final_state, out=a.v)) == dws.ERR_OVERLAP
    assert call(lib, "dws_delta_rule_backward", arguments(d_slots=FAKE, n_states=4)) == dws.ERR_UNSUPPORTED
    assert call(lib, "dws_delta_rule_backward", arguments(g=dws.Rows(None, 4, 1))) == bad     # dg of no g
    assert call(lib, "dws_delta_rule_backward", arguments(q_grad=dws.Rows(1 << 40, 64, 64))) == bad


@pytest.mark.parametrize("name,backward", [("dws_delta_rule", 0), ("dws_delta_rule_backward", 1)])
def test_workspace(lib, name, backward):
    need = ctypes.c_size_t(0)
    a = arguments()
    size = lib.dws_delta_rule_workspace
    assert size(ctypes.byref(a), backward, None) == dws.ERR_INVALID_ARG
    assert size(None, backward, ctypes.byref(need)) == dws.ERR_INVALID_ARG
    assert size(ctypes.byref(arguments(dim_k=300)), backward, ctypes.byref(need)) == dws.ERR_UNSUPPORTED
    assert size(ctypes.byref(a), backward, ctypes.byref(need)) == dws.OK and need.value > 0
    far = 1 << 44
    assert call(lib, name, a) == dws.ERR_INVALID_ARG                                                # none
    assert call(lib, name, arguments(d_workspace=far, workspace_bytes=need.value - 1)) == dws.ERR_INVALID_ARG
    assert call(lib, name, arguments(d_workspace=far + 16, workspace_bytes=need.value)) == dws.ERR_MISALIGNED
    # every overlap of an output or of the workspace with another operand
    fits = {"workspace_bytes": need.value, "d_workspace": far}
    q = a.q.data
    outs = ("out",) if not backward else ("q_grad", "k_grad", "v_grad", "g_grad", "beta_grad")
    assert call(lib, name, arguments(d_workspace=q, workspace_bytes=need.value)) == dws.ERR_OVERLAP
    for o in outs:
        r = getattr(a, o)
        for other in ("q", "k", "v", "g", "beta") + (("out_grad",) if backward else ()):
            moved = dws.Rows(getattr(a, other).data, r.token_stride, r.head_stride)
            assert call(lib, name, arguments(**fits, **{o: moved})) == dws.ERR_OVERLAP, (o, other)
    if not backward:
        assert call(lib, name, arguments(**fits, d_initial_state=a.d_final_state + 4)) == dws.ERR_OVERLAP
        assert call(lib, name, arguments(**fits, d_final_state=q)) == dws.ERR_OVERLAP


def test_workspace_grows_with_the_call(lib):
    def need(backward=0, **more):
        n = ctypes.c_size_t(0)
        assert lib.dws_delta_rule_workspace(ctypes.byref(arguments(**more)), backward, ctypes.byref(n)) == dws.OK
        return n.value

    assert need(d_final_state=None) < need() < need(1)
    assert need(tokens=1 << 20) > 1000 * need()


def test_packed_arguments_are_the_structure():
    """The binding packs dws_delta_rule_args: every member of the structure where the packed value goes."""
    assert dws._DELTA.size == ctypes.sizeof(dws.DeltaRuleArgs)
    a = [0] * 56
    places = {"n_seqs": dws._N_SEQS, "d_offsets": dws._OFFSETS, "g_dtype": dws._G_DTYPE, "d_initial_state": dws._INITIAL,
              "d_final_state": dws._FINAL, "d_slots": dws._SLOTS, "n_states": dws._N_STATES, "d_final_grad": dws._FINAL_GRAD,
              "d_initial_grad": dws._INITIAL_GRAD, "zero_rest": dws._ZERO_REST, "d_workspace": dws._WORKSPACE,
              "workspace_bytes": dws._WORKSPACE + 1, "tokens": 0, "heads_qk": 3, "heads_v": 4, "dim_k": 5, "dim_v": 6,
              "dtype": 7, "beta_dtype": 9, "scale": 10}
    rows = {"q": dws._Q, "k": dws._K, "v": dws._V, "g": dws._G, "beta": dws._BETA, "out": dws._OUT, "out_grad": dws._OUT_GRAD,
            "q_grad": dws._Q_GRAD, "k_grad": dws._K_GRAD, "v_grad": dws._V_GRAD, "g_grad": dws._G_GRAD, "beta_grad": dws._BETA_GRAD}
    for i in range(56):
        a[i] = i + 1
    s = dws.DeltaRuleArgs.from_buffer_copy(dws._DELTA.pack(*a))
    assert len(places) + 3 * len(rows) == 56
    for name, at in places.items():
        assert getattr(s, name) == at + 1, name
    for name, at in rows.items():
        r = getattr(s, name)
        assert (r.data, r.token_stride, r.head_stride) == (at + 1, at + 2, at + 3), name


def test_options(lib):
    """Unknown ones are refused; fp32 gates' gradients take fp32's alignment and room."""
    wide = dws.DELTA_FP32_GRADS
    for name in CALLS:
        for unknown in (1 << 30, -1, 1 << 8):
            assert call(lib, name, arguments(options=unknown)) == dws.ERR_INVALID_ARG
    need = ctypes.c_size_t(0)
    assert lib.dws_delta_rule_workspace(ctypes.byref(arguments(options=1 << 30)), 1, ctypes.byref(need)) == dws.ERR_INVALID_ARG
    assert lib.dws_delta_rule_workspace(ctypes.byref(arguments(options=wide)), 1, ctypes.byref(need)) == dws.OK
    name, fits = "dws_delta_rule_backward", {"workspace_bytes": need.value, "d_workspace": 1 << 44}
    for grad in ("g_grad", "beta_grad"):
        assert call(lib, name, arguments(**fits, options=wide, **{grad: dws.Rows((1 << 40) + 2, 4, 1)})) == dws.ERR_MISALIGNED
        # 512 elements that end where beta begins in 16 bits, and lie over it in 32
        before = dws.Rows(arguments().beta.data - 128 * 4 * 2, 4, 1)
        moved = dict(fits, g=dws.Rows(1 << 41, 4, 1), options=wide)
        assert call(lib, name, arguments(**moved, **{grad: before})) == dws.ERR_OVERLAP
    assert call(lib, name, arguments(**fits, options=wide, d_initial_grad=(1 << 42) + 2)) == dws.ERR_MISALIGNED


def test_workspace_of_precise_outputs(lib):
    """What a call with a final state needs, for the 16-bit types; more for gradients up to 128 key columns."""
    def need(backward=0, **more):
        n = ctypes.c_size_t(0)
        assert lib.dws_delta_rule_workspace(ctypes.byref(arguments(**more)), backward, ctypes.byref(n)) == dws.OK
        return n.value

    assert need(d_final_state=None) < need(d_final_state=None, options=dws.DELTA_PRECISE) == need()
    assert need(options=dws.DELTA_PRECISE) == need()
    assert need(dtype=dws.FLOAT32, d_final_state=None, options=dws.DELTA_PRECISE) == need(dtype=dws.FLOAT32)
    assert need(1, options=dws.DELTA_PRECISE) > need(1)
    for more in ({"dim_k": 200}, {"dtype": dws.FLOAT32}):
        assert need(1, options=dws.DELTA_PRECISE, **more) == need(1, **more)


def test_packed_options_are_the_structure():
    s = dws.DeltaRuleArgs.from_buffer_copy(dws._delta_packed([i + 1 for i in range(56)], 77))
    assert (s.options, s.zero_rest, s.d_workspace, s.workspace_bytes, s.tokens) == (77, 54, 55, 56, 1)
    s = dws.DeltaRuleArgs.from_buffer_copy(dws._delta_packed([i + 1 for i in range(56)], 0))
    assert (s.options, s.zero_rest, s.d_workspace) == (0, 54, 55)


def test_binding_refuses_cpu_tensors():
    x, offsets, initial = inputs(1, [8], 1, 1, 16, 16, torch.float32, device="cpu")
    args = [x[a] for a in NAMES]
    with pytest.raises(TypeError):
        dws.delta_rule(*args)
    with pytest.raises(TypeError):
        dws.delta_rule_backward(x["v"], *args)
    with pytest.raises(TypeError):
        dws.delta_rule_step(*args, initial)
    with pytest.raises(ValueError):
        dws.delta_rule_step(*args, initial[0])


@pytest.mark.parametrize("name", ["delta_rule", "delta_rule_step"])
@pytest.mark.parametrize("which", NAMES + ("state", "out"))
def test_tensors_that_require_gradients_are_refused(name, which):
    """A result without a graph would train nothing and say nothing. (Without the refusal these fail as CPU tensors.)"""
    x, _, initial = inputs(1, [8], 1, 1, 16, 16, torch.float32, device="cpu")
    x.update(state=initial, out=torch.empty_like(x["v"]))
    x[which].requires_grad_()

    def call():
        more = {"initial_state": x["state"]} if name == "delta_rule" else {"state": x["state"]}
        return getattr(dws, name)(*(x[a] for a in NAMES), out=x["out"], **more)

    with pytest.raises(RuntimeError, match="no graph"):
        call()
    with torch.no_grad(), pytest.raises(TypeError):
        call()


def test_tolerances_see_a_mistake():
    """The oracle with a mistake planted (a decay applied one token late) is far outside the tolerances."""
    x, offsets, initial = inputs(19, [100], 1, 2, 32, 16, torch.float32, device="cpu")
    want, final = reference(*(x[a] for a in NAMES), offsets.tolist(), initial.double(), 0.2)
    late = dict(x, g=torch.cat([x["g"][:1] * 0, x["g"][:-1]]))
    got, state = reference(*(late[a] for a in NAMES), offsets.tolist(), initial.double(), 0.2)
    for a, b, what in ((got, want, "out"), (state, final, "state")):
        with pytest.raises(AssertionError):
            close(a, b, torch.bfloat16, what)
